"""The RMS norm and its gradient where rows are narrow, or many to a team of threads, against 64-bit references."""
import pytest
import torch

from cross_vendor_gradient_gb300 import Context, rms_norm_payload_bytes
from tests import train_ref as ref
from tests.test_train_gpu import DTYPES, Guarded, cpu64, gen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    with Context([1]) as c:
        yield c


# ------------------------------------------------------------- narrow rows

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("cols", [1, 2, 3, 5, 6, 7])
def test_rms_norm_and_gradient_of_narrow_rows(ctx, cols, dtype):
    """Rows of less than a vector: several of them end within the tensor's last vector.  Buffers at 16 bytes, float32
    not at 32."""
    dt = DTYPES[dtype]
    shift = 4 if dtype == "f32" else 8
    for rows in (1, 2, 3, 9, 65, 5000):
        hold, g = Guarded(), gen(100 * cols + rows)

        def normal(*shape, scale=1.0):
            return (torch.randn(*shape, generator=g) * scale).to(dt)
        x, res = (hold(normal(rows, cols, scale=s), shift) for s in (1.0, 3.0))
        w = hold(1 + normal(cols, scale=0.2))
        dy, dsum = hold(normal(rows, cols, scale=0.1), shift), hold(normal(rows, cols), shift)
        out, total, dx = (hold(torch.zeros(rows, cols, dtype=dt), shift) for _ in range(3))
        rstd, dw = hold(torch.zeros(rows)), hold(torch.zeros(cols, dtype=dt))
        h, want_rstd, y, err = ref.rms_forward(x.cpu(), res.cpu(), w.cpu(), 1e-5, dt)
        bound = y.abs() * (err + 3 * ref.U) + 2.0 ** -149
        for codec, block in (("none", 256), ("e4m3", 128), ("e5m2", 256)):
            to = out if codec == "none" else hold(torch.zeros(rms_norm_payload_bytes(codec, block, rows, cols), dtype=torch.uint8))
            ctx.rms_norm(x, w, to, eps=1e-5, residual=res, sum_out=total, rstd=rstd, codec=codec, block=block)
            assert torch.equal(total.cpu(), h)
            assert bool(((cpu64(rstd) - want_rstd).abs() <= want_rstd * err).all())
            if codec == "none":
                assert bool(((cpu64(to) - y).abs() <= bound + ref.rounding(y, dt)).all())
            else:
                ref.check_fp8(to, y, bound, rows, cols, block, codec, "%d x %d" % (rows, cols))
        ctx.rms_norm_backward(dy, total, w, rstd, dx, dw, dsum=dsum)
        want_dx, want_dw, dx_err, dw_err = ref.rms_backward(dy.cpu(), h, w.cpu(), rstd.cpu(), dsum.cpu(), dt)
        assert bool(((cpu64(dx) - want_dx).abs() <= dx_err).all())
        assert bool(((cpu64(dw) - want_dw).abs() <= dw_err).all())
        hold.check()


@pytest.mark.parametrize("shape", [(5, 0), (2, 3, 0), (0, 8), (2, 0, 8), (0,), (8,)])
def test_rms_norm_of_shapes_without_elements(ctx, shape):
    """No columns, no rows, and a vector of one row: rstd has an entry for every row."""
    x = torch.ones(shape, device="cuda")
    w = torch.full(shape[-1:], 2.0, device="cuda")
    rows = x.shape[:-1].numel()
    rstd, out, total = torch.full((rows,), 7.0, device="cuda"), torch.zeros_like(x), torch.zeros_like(x)
    ctx.rms_norm(x, w, out, eps=0.0, residual=x, sum_out=total, rstd=rstd)
    payload = torch.zeros(rms_norm_payload_bytes("e4m3", 128, rows, shape[-1]), dtype=torch.uint8, device="cuda")
    ctx.rms_norm(x, w, payload, rstd=rstd, codec="e4m3", block=128)
    dx, dw = torch.zeros_like(x), torch.full_like(w, 7.0)
    ctx.rms_norm_backward(x, total, w, rstd, dx, dw)
    torch.cuda.synchronize()
    if x.numel():
        assert bool((out == 2).all()) and bool((total == 2).all()) and bool((rstd - 1 < 1e-5).all())
    elif shape[-1]:
        assert bool((dw == 0).all())
    else:
        assert bool((rstd == 7).all())  # nothing is written
