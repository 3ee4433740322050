"""Plain 64-bit forms of the microscaled operators, and the error bounds that their tests use.

Everything is written from the formats' definitions with torch double tensors (any
device).  Where an operator rounds to E4M3 between two steps, the reference also says how far
the rounded value may move when its input is off by a given amount, so that the
tolerances are bounds and not guesses.
"""
import torch

F64 = torch.float64
BF16_HALF_STEP = 2.0 ** -8   # torch.finfo(torch.bfloat16).eps / 2
# One fp32 addition, rounded or truncated, is off by at most 2^-23 of its result, so K of them by at
# most K 2^-23 of the sum of magnitudes.
FP32_STEP = 2.0 ** -23

E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
E4M3 = ([m * 2.0 ** -9 for m in range(8)]
        + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)])[:127]


def levels(fmt, device):
    return torch.tensor(E2M1 if fmt == "e2m1" else E4M3, dtype=F64, device=device)


def emax(fmt):
    return 2 if fmt == "e2m1" else 8


def scale_exponent(m, fmt):
    """Exponent of the scale of blocks whose largest magnitude is m (fp64)."""
    e = torch.frexp(m).exponent - 1 - emax(fmt)
    return torch.where(m > 0, e, torch.full_like(e, -127)).clamp(-127, 127)


def round_to(u, fmt):
    """(value, place) of the level nearest to |u|, ties to the even place, saturating."""
    lv = levels(fmt, u.device)
    mid = (lv[1:] + lv[:-1]) / 2
    a = u.abs()
    place = torch.bucketize(a, mid)                        # mid[i-1] < a <= mid[i]
    at = mid[place.clamp(max=len(mid) - 1)]
    place = place + ((a == at) & (place < len(mid)) & (place % 2 == 1)).to(place.dtype)
    return lv[place], place


def blocks(v):
    return v.reshape(*v.shape[:-1], -1, 32)


def quantize(v, fmt):
    """(codes uint8, scale codes uint8) of a finite fp64 matrix."""
    b = blocks(v)
    e = scale_exponent(b.abs().amax(-1), fmt)
    u = torch.ldexp(b, -e.unsqueeze(-1))
    _, place = round_to(u, fmt)
    place = place.to(torch.uint8).flatten(-2)
    sign = torch.signbit(v).to(torch.uint8)
    if fmt == "e4m3":
        codes = place | (sign << 7)
    else:
        n = place | (sign << 3)
        codes = n[..., 0::2] | (n[..., 1::2] << 4)
    return codes, (e + 127).to(torch.uint8)


def decode(codes, scales, fmt):
    """fp64 values; scale code 255 and E4M3 codes 0x7F / 0xFF are NaN."""
    lv = levels(fmt, codes.device)
    if fmt == "e4m3":
        lv = torch.cat([lv, lv.new_tensor([float("nan")])])
        v = lv[(codes & 127).long()] * torch.where(codes > 127, -1.0, 1.0).to(F64)
    else:
        n = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
        v = lv[(n & 7).long()] * torch.where(n > 7, -1.0, 1.0).to(F64)
    s = torch.ldexp(torch.ones_like(scales, dtype=F64), scales.int() - 127)
    s = torch.where(scales == 255, torch.full_like(s, float("nan")), s)
    return (blocks(v) * s.unsqueeze(-1)).flatten(-2)


def mx(v, fmt="e4m3"):
    return decode(*quantize(v, fmt), fmt)


def mx_shift(v, err, fmt="e4m3"):
    """How far mx(v) can move when each element of v is off by up to err: rounding is monotone
    for a fixed scale, so the ends of each element's interval under the smallest and the largest
    scale that the block can get bound every case."""
    q, b, d = blocks(mx(v, fmt)), blocks(v), blocks(err)
    a = b.abs()
    lo = scale_exponent((a - d).clamp(min=0).amax(-1), fmt)
    hi = scale_exponent((a + d).amax(-1), fmt)
    far = torch.zeros_like(q)
    for e in (lo, hi):
        for x in (b - d, b + d):
            u = torch.ldexp(x, -e.unsqueeze(-1))
            val = torch.ldexp(round_to(u, fmt)[0] * torch.sign(u), e.unsqueeze(-1))
            far = torch.maximum(far, (val - q).abs())
    return far.flatten(-2)


def grouped_mm(a, w_codes, w_scales, offsets, shift=None):
    """(y, tolerance) fp64 [R, N]: rows of a (fp64 [R, K]) by expert times w[e] transposed, and how
    far a result that is summed in fp32 and rounded once to bf16 may be off when each
    element of a may be off by `shift`.  Rows of no expert are NaN."""
    off = offsets.tolist()
    R, K = a.shape
    y = torch.full((R, w_codes.shape[1]), float("nan"), dtype=F64, device=a.device)
    tol = torch.zeros_like(y)
    for e in range(len(off) - 1):
        i, j = off[e], off[e + 1]
        if i == j:
            continue
        w = decode(w_codes[e], w_scales[e], "e2m1")
        y[i:j] = a[i:j] @ w.T
        mag = a[i:j].abs()
        if shift is not None:
            d = shift[i:j] @ w.abs().T
            tol[i:j] += d
            mag = mag + shift[i:j]
        sums = K * FP32_STEP * (mag @ w.abs().T)
        tol[i:j] += sums + BF16_HALF_STEP * (y[i:j].abs() + tol[i:j] + sums)
    return y, tol


def swiglu(h, h_err):
    """(act, error bound) of h [R, 2I] = gate | up that is off by up to h_err.  |silu'| < 1.1;
    the fast exponential is off by about |g| + 2 units of 2^-23 and the reciprocal and
    the products by a few more."""
    I = h.shape[1] // 2
    g, u = h[:, :I], h[:, I:]
    eg, eu = h_err[:, :I], h_err[:, I:]
    silu = g * torch.sigmoid(g)
    act = silu * u
    err = 1.1 * eg * (u.abs() + eu) + silu.abs() * eu + act.abs() * (8 + g.abs()) * FP32_STEP
    return act, err


def grouped_ffn(x, w13, s13, w2, s2, offsets, rows, k):
    """(y, tolerance) fp64 [R, H] in expanded order; x fp64 [T, H]."""
    xr = x[rows.long() // k]
    h, _ = grouped_mm(xr, w13, s13, offsets)
    h_err = torch.zeros_like(h)
    off = offsets.tolist()
    for e in range(len(off) - 1):
        i, j = off[e], off[e + 1]
        if i < j:
            w = decode(w13[e], s13[e], "e2m1").abs()
            h_err[i:j] = xr.shape[1] * FP32_STEP * (xr[i:j].abs() @ w.T)
    act, err = swiglu(h, h_err)
    yp, tolp = grouped_mm(mx(act), w2, s2, offsets, mx_shift(act, err))
    y, tol = torch.empty_like(yp), torch.empty_like(tolp)
    y[rows.long()], tol[rows.long()] = yp, tolp
    return y, tol


def rmsnorm(x, residual, weight, eps):
    """(h bf16, n fp64, error bound of an fp32 n): the sum of H squares is off by at most
    H 2^-24 of itself, the root by half of that; sqrt, reciprocal, mean and product add a
    handful of half steps."""
    h = x if residual is None else (x.float() + residual.float()).to(torch.bfloat16)
    v = h.to(F64)
    n = v / torch.sqrt(v.square().mean(-1, keepdim=True) + eps) * weight.to(F64)
    return h, n, n.abs() * (h.shape[-1] / 2 + 8) * 2.0 ** -24


def assert_within(got, want, tol, what):
    got = got.to(F64)
    bad = ~((got - want).abs() <= tol)
    assert not bool(bad.any()), (
        f"{what}: {int(bad.sum())} of {bad.numel()} outside their bound, worst "
        f"{float(((got - want).abs() - tol)[bad].max()):.3e} over at "
        f"{[int(i) for i in bad.nonzero()[0]]}")
