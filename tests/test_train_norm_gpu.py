"""The gradient norm over the whole range of float32: sums that overflow or vanish in float32 although the norm does
not, and what makes it infinite or NaN."""
import math

import numpy as np
import pytest
import torch

from cross_vendor_gradient_gb300 import Context
from tests import train_ref as ref
from tests.test_train_gpu import DTYPES, gen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    with Context([1]) as c:
        yield c


def norm_of(ctx, tensors, max_norm=0.0):
    out = torch.full((2,), -1.0, device="cuda")
    ctx.grad_norm(tensors, out, max_norm=max_norm)
    return out.cpu().double().tolist()


def check(ctx, tensors):
    want = math.sqrt(sum(float(t.double().square().sum()) for t in tensors))
    max_norm = float(np.float32(want / 2))
    norm, factor = norm_of(ctx, tensors, max_norm=max_norm)
    # a sum of positive terms: 10 roundings of each within a tile, 3 of the compensated sum, 2^-28 of what vanishes
    # next to the least sum that is taken as it is; halved by the root, and the result's own rounding.  A subnormal
    # result has that of 2^-149.
    assert abs(norm - want) <= 9 * ref.U * want + 2.0 ** -149, (norm, want)
    clip = min(1.0, max_norm / (norm + 1e-6)) if max_norm > 0 else 1.0
    assert abs(factor - clip) <= 4 * ref.U * clip + 2.0 ** -149


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [1e18, 3e16, 1e10, 1e-10, 1e-15, 1e-19, 1e-21, 1e-24, 1e-30, 1e-37])
@pytest.mark.parametrize("n", [1, 33, 5000, 3_000_000])
def test_norm_of_large_and_small_gradients(ctx, n, scale, dtype):
    t = (torch.randn(n, generator=gen(n)).clamp(-9, 9) * scale).to(DTYPES[dtype]).cuda()
    check(ctx, [t])
    check(ctx, [t[1:], t[:1]])  # off the vectors


def test_norm_of_subnormal_gradients(ctx):
    check(ctx, [torch.full((100_000,), 2.0 ** -149, device="cuda")])
    check(ctx, [torch.full((77,), 2.0 ** -140, device="cuda")])
    check(ctx, [torch.full((4099,), 2.0 ** -133, device="cuda", dtype=torch.bfloat16)])
    for mantissa_bit in (1, 15, 16, 22):  # a single bit of float32's
        check(ctx, [torch.full((2000,), 2.0 ** (mantissa_bit - 149), device="cuda")])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_norm_of_gradients_of_many_sizes(ctx, dtype):
    """Large, ordinary, tiny and zero tensors together, and sizes that change within a tensor."""
    g, dt = gen(9), DTYPES[dtype]
    parts = [torch.randn(n, generator=g) * s for n, s in ((5000, 1e-25), (40_000, 1e-22), (3, 1e-19), (9000, 0.0))]
    tiny = [p.to(dt).cuda() for p in parts]
    check(ctx, tiny)
    check(ctx, [torch.cat(tiny)])
    check(ctx, tiny + [torch.full((2,), 1e-20, device="cuda", dtype=dt)])
    check(ctx, tiny + [torch.ones(1, device="cuda", dtype=dt)])
    large = (torch.randn(70_000, generator=g).clamp(-6, 6) * 2e18).to(dt).cuda()
    check(ctx, tiny + [large])
    check(ctx, [torch.cat(tiny + [large])])
    check(ctx, [(torch.exp(torch.randn(300_000, generator=g) * 15)).clamp(max=1e18).to(dt).cuda()])
    check(ctx, [torch.full((3,), 1e-24, device="cuda", dtype=dt)] * 1500)  # more tensors than one launch takes


@pytest.mark.parametrize("dtype", DTYPES)
def test_norm_is_infinite_or_nan_as_the_gradients_are(ctx, dtype):
    dt = DTYPES[dtype]
    for n in (1, 5000, 600_000):
        for bad in (float("inf"), float("-inf")):
            t = torch.ones(n, device="cuda", dtype=dt)
            t[n // 2] = bad
            norm, factor = norm_of(ctx, [t], max_norm=1.0)
            assert norm == float("inf") and math.isnan(factor)
        t[n // 3] = float("nan")  # beside the infinite one, or in its place
        norm, factor = norm_of(ctx, [t], max_norm=1.0)
        assert math.isnan(norm) and math.isnan(factor)
    t = torch.ones(64, device="cuda", dtype=dt)
    t[1], t[3] = float("inf"), float("nan")
    assert math.isnan(norm_of(ctx, [t])[0])
    assert norm_of(ctx, [torch.zeros(100_000, device="cuda", dtype=dt)], 1.0) == [0.0, 1.0]
    assert norm_of(ctx, [-torch.zeros(100_000, device="cuda", dtype=dt)], 1.0) == [0.0, 1.0]


def test_norm_refuses_what_has_no_square_in_float32(ctx):
    ok, beyond = 1.84e19, 1.85e19  # the root of the largest float32 is 1.8447e19
    t = torch.ones(10_000, device="cuda")
    t[77] = ok
    check(ctx, [t])
    t[78:100] = ok
    check(ctx, [t])
    t[77] = beyond
    norm, factor = norm_of(ctx, [t], max_norm=1.0)
    assert norm == float("inf") and math.isnan(factor)


def test_norm_of_float16_at_its_ends(ctx):
    check(ctx, [torch.full((3_000_000,), 65504.0, device="cuda", dtype=torch.float16)])
    check(ctx, [torch.full((3_000_000,), 2.0 ** -24, device="cuda", dtype=torch.float16)])
