"""64-bit references of the training-step operators, and the error bounds of
their float32 arithmetic, shared by the tests.  Written from the formulas of
include/gb.h on CPU float64 tensors; U is float32's unit roundoff."""
import numpy as np
import torch

U = 2.0 ** -24
HALF_STEP = {d: torch.finfo(d).eps / 2 for d in (torch.float32, torch.bfloat16, torch.float16)}  # relative
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}      # absolute
TOP = {"e4m3": 448.0, "e5m2": 57344.0}
LEAST_EXP = {"e4m3": -6, "e5m2": -14}
FRACTION = {"e4m3": 3, "e5m2": 2}
FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


def rounding(x, dtype):
    """How far the nearest value of dtype may be from x."""
    return x.abs() * HALF_STEP[dtype] + TINY[dtype]


def payload_parts(payload, n, block, codec="e4m3", n_blocks=None):
    off = (n + 15) // 16 * 16
    nb = (n + block - 1) // block if n_blocks is None else n_blocks
    return payload[:n].view(FP8[codec]), payload[off:off + 4 * nb].view(torch.float32)


def decode(payload, n, block):
    codes, scales = payload_parts(payload.cpu(), n, block)
    return codes.double() * scales.double().repeat_interleave(block)[:n]


def block_top(x, block):
    """Largest magnitude of each block of the last dimension."""
    pad = -x.shape[-1] % block
    if pad:
        x = torch.cat([x, x.new_zeros(*x.shape[:-1], pad)], -1)
    return x.abs().reshape(*x.shape[:-1], -1, block).amax(-1)


def scale_rule(top, codec="e4m3"):
    k = torch.ceil(torch.log2(top.clamp(min=1e-300) / TOP[codec])).clamp(min=-126)
    return torch.where(top == 0, torch.ones_like(top), torch.pow(torch.tensor(2.0, dtype=torch.float64), k))


def quantum(y, codec="e4m3"):
    e = torch.frexp(y)[1] - 1
    return torch.pow(torch.tensor(2.0, dtype=torch.float64), (e.clamp(min=LEAST_EXP[codec]) - FRACTION[codec]).double())


# ---------------------------------------------------------- random numbers

def mix32(z):
    z = np.uint64(z) & np.uint64(0xFFFFFFFF)
    z ^= z >> np.uint64(16)
    z = z * np.uint64(0x85A308D3) & np.uint64(0xFFFFFFFF)
    z ^= z >> np.uint64(15)
    z = z * np.uint64(0xEC4E6C89) & np.uint64(0xFFFFFFFF)
    return z ^ (z >> np.uint64(16))


def random_16(seed, step, tensor, n, first=0):
    """(for m, for v): the random numbers, 0 .. 65535, of n elements from `first` on."""
    m32 = 0xFFFFFFFF
    key = mix32((seed & m32) + 0x9E3779B9)
    for word in (seed >> 32, step & m32, step >> 32, tensor):
        key = mix32(int(key) ^ int(word))
    i = np.arange(first, first + n, dtype=np.uint64)
    q = i >> np.uint64(3)
    low, high = q & np.uint64(m32), q >> np.uint64(32)
    z = mix32(np.uint64(key) + low * np.uint64(0x9E3779B1) % np.uint64(1 << 32) + high * np.uint64(0x85A308D3) % np.uint64(1 << 32))
    for j in range(1, 8):
        late = (i & np.uint64(7)) >= j
        z = np.where(late, (z * np.uint64(2891336453) + np.uint64(0x9E3779B9)) & np.uint64(m32), z)
    return torch.from_numpy((z >> np.uint64(16)).astype(np.float64)), torch.from_numpy((z & np.uint64(0xFFFF)).astype(np.float64))


# ------------------------------------------------------------------- AdamW

def adamw(p, g, m, v, scale, lr, betas, eps, wd, step):
    """(p, m, v) after the step, and the bounds of their float32 errors.

    m is one product added to another, each with a rounded factor: at most 4
    roundings of either term.  The gradient is squared: 6.  p's update has
    the relative error of the quotient (12 roundings at most, v's halved by
    the root), of m's terms and of the rate; p's own product two."""
    b1, b2 = betas
    g = g * scale
    m_terms, v_terms = b1 * m.abs() + (1 - b1) * g.abs(), b2 * v + (1 - b2) * g * g
    m, v = b1 * m + (1 - b1) * g, v_terms
    rate = lr / (1 - b1 ** step)
    den = torch.sqrt(v / (1 - b2 ** step)) + eps
    update = torch.where(m_terms == 0, torch.zeros_like(m), rate * m / den)
    size = torch.where(m_terms == 0, torch.zeros_like(m), rate * m_terms / den)
    p = p * (1 - lr * wd)
    bounds = (U * (4 * p.abs() + 24 * size + 2 * (p - update).abs()) + 2.0 ** -149, 5 * U * m_terms + 2.0 ** -149,
              7 * U * v_terms + 2.0 ** -149)
    return (p - update, m, v), bounds


def check_codes(codes, scales, x, bound, block, words, keep, what):
    """The codes (float8 tensor) and scales of an 8-bit state against x (64
    bits, within `bound` of what was encoded): the scale by the rule, and the
    code of floor(|y| / q + r), or a neighbour where x's bound reaches across."""
    codes, scales = codes.cpu().double(), scales.cpu().double()
    top, off = block_top(x, block), block_top(bound, block)
    lo, hi = scale_rule((top - off).clamp(min=0)), scale_rule(top + off)
    ok = (scales >= torch.minimum(lo, hi)) & (scales <= torch.maximum(lo, hi))
    assert bool(ok.all()), "%s: scale %r, rule %r" % (what, scales[~ok][0].item(), scale_rule(top)[~ok][0].item())
    s = scales.repeat_interleave(block)[:x.numel()]
    y, dy = x / s, bound / s
    # as the definition: magnitude q * floor(|y| / q + r)
    def at(mag):
        q = quantum(mag)
        z = torch.floor(mag / q + words / 65536) * q
        return torch.where(mag > 0, z.clamp(min=2.0 ** -9), z) if keep else z
    slack = dy + 2.0 ** -30
    least, most = at((y.abs() - slack).clamp(min=0)), at((y.abs() + slack).clamp(max=448.0))
    mag = codes.abs()
    bad = (mag < least) | (mag > most)
    if keep:
        bad &= ~((mag == 2.0 ** -9) & (least == 0))
    assert not bool(bad.any()), "%s: %d codes differ, first at %d: %r, y %r between %r and %r" % (
        what, int(bad.sum()), int(bad.nonzero()[0]), mag[bad][0].item(), y[bad][0].item(), least[bad][0].item(),
        most[bad][0].item())
    signs = (codes != 0) & (x.abs() > bound) & (torch.sign(codes) != torch.sign(x))
    assert not bool(signs.any()), "%s: sign" % what


# ---------------------------------------------------------------- RMS norm

def any_order(n):
    """Relative error bound of a float32 sum of n terms of one sign, whatever
    the order, with each term rounded once."""
    return (n + 1) * U


def rms_forward(x, residual, w, eps, dtype):
    """h (as held), rstd, y in 64 bits, and rstd's relative error."""
    h = x.float()
    if residual is not None:
        h = (h + residual.float()).to(dtype).float()  # one float32 addition, one rounding: exact to check
    h64 = h.double()
    rstd = 1 / torch.sqrt((h64 * h64).mean(-1) + eps)
    # the sum's error is halved by the root; eps and 1 / cols are rounded, then a product-sum, a root, a division
    err = any_order(x.shape[-1]) / 2 + 5 * U
    return h.to(dtype), rstd, h64 * rstd[:, None] * w.double(), err


def check_fp8(payload, y, bound, rows, cols, block, codec, what):
    nb = (cols + block - 1) // block
    codes, scales = payload_parts(payload.cpu(), rows * cols, block, codec, rows * nb)
    codes, scales = codes.double().view(rows, cols), scales.double().view(rows, nb)
    top, off = block_top(y, block), block_top(bound, block)
    lo, hi = scale_rule((top - off).clamp(min=0), codec), scale_rule(top + off, codec)
    ok = (scales >= torch.minimum(lo, hi)) & (scales <= torch.maximum(lo, hi))
    assert bool(ok.all()), "%s: scale" % what
    s = scales.repeat_interleave(block, 1)[:, :cols]
    z, dz = y / s, bound / s
    q = quantum(z, codec)
    bad = (codes - z).abs() > q / 2 + dz * (1 + 1e-9)
    # at a binade's edge the error may have crossed into the larger quantum
    edge = (codes - z).abs() <= quantum((z.abs() + dz).clamp(max=TOP[codec]), codec) / 2 + dz * (1 + 1e-9)
    bad &= ~edge
    assert not bool(bad.any()), "%s: %d codes, first %r for %r" % (what, int(bad.sum()), codes[bad][0].item(),
                                                                  z[bad][0].item())


def rms_backward(dy, h, w, rstd, dsum, dtype):
    """dx, dweight in 64 bits and their bounds (before rounding to dtype)."""
    dy, h, w, rstd = dy.double(), h.double(), w.double(), rstd.double()[:, None]
    cols, rows = h.shape[1], h.shape[0]
    xhat, a = h * rstd, dy * w
    c = (a * xhat).mean(-1, keepdim=True)
    c_err = (any_order(cols) + 4 * U) * (a * xhat).abs().mean(-1, keepdim=True)
    dx = rstd * (a - xhat * c)
    dx_err = rstd * (xhat.abs() * c_err + 6 * U * (a.abs() + (xhat * c).abs()))
    if dsum is not None:
        dx = dx + dsum.double()
        dx_err = dx_err + 2 * U * dx.abs()
    dw = (dy * xhat).sum(0)
    dw_err = (any_order(rows) + 3 * U) * (dy * xhat).abs().sum(0)
    return dx, dw, dx_err + rounding(dx, dtype), dw_err + rounding(dw, dtype)
