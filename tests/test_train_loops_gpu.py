"""The training-step operators where a team of threads walks over many rows, a warp over many tiles, a block over whole
spans, and a table over many tensors; and that no element of a long row is left out of its sums."""
import pytest
import torch

from cross_vendor_gradient_gb300 import Context, payload_bytes, rms_norm_payload_bytes
from tests import train_ref as ref
from tests.test_train_gpu import BETAS, DTYPES, EPS, LR, WD, Guarded, adamw_case, adamw_check, cpu64, gen, snapshot

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    with Context([1]) as c:
        yield c


def cuda_gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


# ------------------------------------------------------------- many rows

def rows_of(cols):
    """More than there are teams: narrow rows have up to 32 teams a block."""
    return 100_003 if cols < 64 else 20_003


PIECE = 304  # rows of a call in which every team has one row; a multiple of 8, so that rows keep their alignment
CODECS = [("none", 256), ("e4m3", 128), ("e5m2", 256)]


def sampled(rows):
    """Rows from both ends and between."""
    return torch.cat([torch.arange(40), torch.randint(40, rows - 40, (300,), generator=gen(1)), torch.arange(rows - 40, rows)])


class Norm:
    """x + residual to out, sum and rstd, of any rows."""

    def __init__(self, ctx, codec, block):
        self.ctx, self.codec, self.block = ctx, codec, block

    def __call__(self, x, residual, w, out=None, total=None):
        rows, cols = x.shape
        if out is None:
            out = torch.empty_like(x) if self.codec == "none" else torch.zeros(
                rms_norm_payload_bytes(self.codec, self.block, rows, cols), dtype=torch.uint8, device="cuda")
        total = torch.empty_like(x) if total is None else total
        rstd = torch.empty(rows, device="cuda")
        self.ctx.rms_norm(x, w, out, residual=residual, sum_out=total, rstd=rstd, codec=self.codec, block=self.block)
        if self.codec == "none":
            return out, total, rstd
        nb = -(-cols // self.block)
        codes, scales = ref.payload_parts(out, rows * cols, self.block, self.codec, rows * nb)
        return codes.view(torch.uint8).view(rows, cols), scales.view(rows, nb), total, rstd


def rows_case(cols, dt):
    g, rows = cuda_gen(cols), rows_of(cols)
    x, res = (torch.randn(rows, cols, device="cuda", generator=g).mul_(s).to(dt) for s in (1.0, 3.0))
    x[:, ::13] *= 8
    return x, res, (1 + 0.2 * torch.randn(cols, device="cuda", generator=g)).to(dt)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("codec,block", CODECS)
@pytest.mark.parametrize("cols", [40, 257, 768, 2047, 2048])
def test_rms_norm_of_many_rows(ctx, cols, codec, block, dtype):
    dt, norm = DTYPES[dtype], Norm(ctx, codec, block)
    x, res, w = rows_case(cols, dt)
    rows = len(x)
    got = norm(x, res, w)
    # the bits of the same rows in calls with one row a team
    for at in range(0, rows, PIECE if rows < 50_000 else 8 * PIECE):
        if at + PIECE > rows:
            at = (rows - PIECE) // 8 * 8
        n = min(PIECE, rows - at)
        for a, b in zip(got, norm(x[at:at + n].clone(), res[at:at + n].clone(), w)):
            assert torch.equal(a[at:at + n], b), at
    # and the definition
    pick = sampled(rows)
    h, rstd, y, err = ref.rms_forward(x[pick].cpu(), res[pick].cpu(), w.cpu(), 1e-5, dt)
    assert torch.equal(got[-2][pick].cpu(), h)
    assert bool(((cpu64(got[-1][pick]) - rstd).abs() <= rstd * err).all())
    bound = y.abs() * (err + 3 * ref.U) + 2.0 ** -149
    if codec == "none":
        assert bool(((cpu64(got[0][pick]) - y).abs() <= bound + ref.rounding(y, dt)).all())
    else:
        few = torch.zeros(rms_norm_payload_bytes(codec, block, len(pick), cols), dtype=torch.uint8)
        codes, scales = ref.payload_parts(few, len(pick) * cols, block, codec, got[1][pick].numel())
        codes.view(torch.uint8).copy_(got[0][pick].cpu().flatten())
        scales.copy_(got[1][pick].cpu().flatten())
        ref.check_fp8(few, y, bound, len(pick), cols, block, codec, "%d columns" % cols)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("cols", [40, 257, 2047, 2048])
def test_rms_norm_of_many_rows_in_place(ctx, cols, dtype):
    """Outputs on the inputs, while later rows are loaded ahead: the bits of separate buffers."""
    norm = Norm(ctx, "none", 256)
    x, res, w = rows_case(cols, DTYPES[dtype])
    out, total, rstd = norm(x, res, w)
    for swap in (False, True):
        a, b = x.clone(), res.clone()
        got = norm(a, b, w, out=b if swap else a, total=a if swap else b)
        assert torch.equal(got[0], out) and torch.equal(got[1], total) and torch.equal(got[2], rstd)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("cols", [40, 257, 1001, 2047, 2048, 4096])
def test_rms_norm_gradient_of_many_rows(ctx, cols, dtype):
    dt = DTYPES[dtype]
    h, dsum, w = rows_case(cols, dt)
    g, rows = cuda_gen(cols + 1), len(h)
    dy = (torch.randn(rows, cols, device="cuda", generator=g) * 0.1).to(dt)
    rstd = torch.rand(rows, device="cuda", generator=g) + 0.1
    for ds in (dsum, None):
        dx, dw = torch.empty_like(h), torch.empty_like(w)
        ctx.rms_norm_backward(dy, h, w, rstd, dx, dw, dsum=ds)
        few, dw_few = torch.empty(PIECE, cols, device="cuda", dtype=dt), torch.empty_like(w)
        for at in list(range(0, rows - PIECE, 8 * PIECE)) + [(rows - PIECE) // 8 * 8]:
            part = slice(at, at + PIECE)
            ctx.rms_norm_backward(dy[part].clone(), h[part].clone(), w, rstd[part].clone(), few, dw_few,
                                  dsum=None if ds is None else ds[part].clone())
            assert torch.equal(dx[part], few), at
        pick = sampled(rows)
        want, _, err, _ = ref.rms_backward(dy[pick].cpu(), h[pick].cpu(), w.cpu(), rstd[pick].cpu(),
                                           None if ds is None else ds[pick].cpu(), dt)
        assert bool(((cpu64(dx[pick]) - want).abs() <= err).all())
        # dweight: a thread adds its rows one by one, at least 152 / 8 teams share them, then the partial sums
        terms = (dy.double() * h.double() * rstd.double()[:, None])
        want_dw = terms.sum(0)
        err = (rows / 19 + 200) * ref.U * terms.abs().sum(0) + ref.rounding(want_dw, dt)
        assert bool(((dw.double() - want_dw).abs() <= err).all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", [(20_003, 257), (9001, 2047), (20_000, 768), (3000, 9000), (700, 20_001)])
def test_rms_norm_weight_gradient_counts_every_row_in_every_type(ctx, rows, cols, dtype):
    """Small whole numbers: every partial sum is exact, so dweight is the sum, rounded once."""
    g, dt = cuda_gen(rows), DTYPES[dtype]
    dy, h = (torch.randint(-4, 5, (rows, cols), device="cuda", generator=g).to(dt) for _ in range(2))
    dx, dw = torch.empty_like(h), torch.empty(cols, device="cuda", dtype=dt)
    ctx.rms_norm_backward(dy, h, torch.ones(cols, device="cuda", dtype=dt), torch.ones(rows, device="cuda"), dx, dw)
    assert torch.equal(dw, (dy.double() * h.double()).sum(0).to(dt))


# ------------------------------------------------- every element of a row

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("cols", [129, 1001, 2048, 8200, 16_383, 16_384, 16_385, 20_001, 65_536])
def test_no_element_of_a_row_is_left_out(ctx, cols, dtype):
    """Rows with a single element that is not zero: rstd, and the mean in dx, show whether it was counted."""
    dt = DTYPES[dtype]
    at = sorted({c for p in (0, 1, 7, 8, 31, 32, 255, 256, 2047, 2048, 4095, 8191, 16_383, 16_384, cols // 2, cols - 257, cols - 9,
                             cols - 2, cols - 1) for c in (p,) if 0 <= c < cols})
    rows = len(at)
    x = torch.zeros(rows, cols, device="cuda", dtype=dt)
    index = torch.arange(rows, device="cuda"), torch.tensor(at, device="cuda")
    x[index] = 8.0
    w, out, rstd = torch.ones(cols, device="cuda", dtype=dt), torch.empty_like(x), torch.empty(rows, device="cuda")
    ctx.rms_norm(x, w, out, eps=1e-5, rstd=rstd)
    want = 1 / (64 / cols + 1e-5) ** 0.5  # 64 is exact; 1 / cols, eps, a product-sum, a root, a division
    assert bool(((rstd.double() - want).abs() <= 5 * ref.U * want).all())
    y = torch.zeros(rows, cols, device="cuda", dtype=torch.float64)
    y[index] = 8 * rstd.double()
    assert bool(((out.double() - y).abs() <= y * ref.U + ref.rounding(y, dt) * (y != 0)).all())
    # dy likewise, next to h of ones: every dx of the row has the mean, dweight every row's
    h, scale = torch.ones(rows, cols, device="cuda", dtype=dt), torch.full((rows,), 2.0, device="cuda")
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    ctx.rms_norm_backward(x, h, w, scale, dx, dw)
    mean = 8 * 2 / cols
    want = 2 * (x.double() - 2 * mean)
    assert bool(((dx.double() - want).abs() <= 4 * ref.U * (2 * x.double() + 4 * mean) + ref.rounding(want, dt)).all())
    want = torch.zeros(cols, device="cuda", dtype=torch.float64)
    want[index[1]] = 16.0
    assert torch.equal(dw.double(), want)


# ------------------------------------------------------- AdamW over much

@pytest.mark.parametrize("block", [128, 256])
@pytest.mark.parametrize("shift", [0, 3])
def test_adamw_in_whole_spans(ctx, block, shift):
    """Over 10 M elements: blocks take spans of 32 tiles, whose scales pass through shared memory."""
    ns = [6_000_001, 4_300_000, 65] if shift else [6_000_000, 4_300_000, 64]
    hold = Guarded()
    tensors = adamw_case(ns, "bf16", "e4m3", block, True, shift, 17, hold)
    before = snapshot(tensors)
    ctx.adamw_step(*tensors[:4], step=5, lr=LR, betas=BETAS, eps=EPS, weight_decay=WD, copies=tensors[4], states="e4m3",
                   block=block, seed=99)
    adamw_check(before, snapshot(tensors), ns, "e4m3", block, 1.0, 5, 99, "bf16")
    hold.check()


def test_adamw_with_more_tiles_than_warps(ctx):
    """Over 80 M elements of float32 states: a warp goes from tile to tile, and from tensor to tensor."""
    ns, g = [40_000_003, 5, 44_000_000], cuda_gen(8)
    total = sum(ns)

    def flat(scale):
        return torch.randn(total, device="cuda", generator=g) * scale
    p, grad, m, v = flat(0.05), flat(1e-2), flat(1e-3), flat(1e-2).square()
    want, bounds = ref.adamw(p.double(), grad.double(), m.double(), v.double(), 1.0, LR, BETAS, EPS, WD, 4)
    ctx.adamw_step(*(list(t.split(ns)) for t in (p, grad, m, v)), step=4, lr=LR, betas=BETAS, eps=EPS, weight_decay=WD)
    for got, w, b in zip((p, m, v), want, bounds):
        assert bool(((got.double() - w).abs() <= b).all())


@pytest.mark.parametrize("count", [31, 32, 33, 512, 513])
@pytest.mark.parametrize("states", ["none", "e4m3"])
def test_adamw_and_norm_at_the_ends_of_the_tables(ctx, states, count):
    """As many tensors as a small table holds, a large one, and one more; some are empty."""
    ns = [0 if i % 10 == 9 else 3 + 37 * i % 300 for i in range(count + count // 9)]
    while sum(n > 0 for n in ns) != count:
        ns.pop() if sum(n > 0 for n in ns) > count else ns.append(5)
    hold = Guarded()
    tensors = adamw_case(ns, "bf16", states, 128, True, 0, count, hold)
    out = torch.zeros(2, device="cuda")
    ctx.grad_norm(tensors[1], out)
    want = float(sum(cpu64(t).square().sum() for t in tensors[1])) ** 0.5
    assert abs(out[0].item() - want) <= 9 * ref.U * want
    before = snapshot(tensors)
    ctx.adamw_step(*tensors[:4], step=2, lr=LR, betas=BETAS, eps=EPS, weight_decay=WD, copies=tensors[4], states=states,
                   block=128, seed=5)
    adamw_check(before, snapshot(tensors), ns, states, 128, 1.0, 2, 5, "bf16")
    hold.check()
    assert payload_bytes("e4m3", 128, 0) == 0


@pytest.mark.parametrize("count", [32, 33, 1024, 1025])
def test_norm_at_the_ends_of_the_tables(ctx, count):
    g = cuda_gen(count)
    tensors = [torch.randn(1 + 13 * i % 90, device="cuda", generator=g) for i in range(count)]
    out = torch.zeros(2, device="cuda")
    ctx.grad_norm(tensors, out)
    want = float(torch.cat(tensors).double().norm())
    assert abs(out[0].item() - want) <= 9 * ref.U * want
