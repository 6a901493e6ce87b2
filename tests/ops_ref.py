"""Plain 64-bit implementations of the quantised norm, its backward pass and
the 4-bit linear, with bounds on how far a kernel that keeps its sums in 32
bits may be from them.

U = 2^-24 is half a step of fp32.  A sum of n terms in any order is off by at
most (n - 1) * U * sum |terms| (to first order); a sum of squares of N columns
goes through at most 8 * 4 terms in a thread, 5 shuffles and 16 warp totals,
so its relative error is below 64 * U, its square root's half of that, and
rsqrt adds 2 steps."""
import torch

U = 2.0 ** -24
EPS = 1e-6
REL_INV = 2.0 ** -18     # relative error of inv, and of a product with it, with room
BF16 = 2.0 ** -8         # half a step of bf16, relative
FP8 = 2.0 ** -4


def norm64(parts, res, gamma, eps=EPS):
    """h, inv [M, 1], y, and the bound of |y - y of a kernel|."""
    x = torch.stack([t.double() for t in parts])
    h, mag = x.sum(0), x.abs().sum(0)
    if res is not None:
        h, mag = h + res.double(), mag + res.double().abs()
    inv = 1 / torch.sqrt((h * h).mean(1, keepdim=True) + eps)
    y = h * inv * gamma.double()
    tol = REL_INV * y.abs() + (len(parts) + 2) * U * mag * inv * gamma.double().abs()
    return h, inv, y, tol


def grouped(t, group, fill=0.0):
    n = t.shape[-1]
    if n % group:
        t = torch.nn.functional.pad(t, (0, group - n % group), value=fill)
    return t.unflatten(-1, (-1, group))


def e8m0_value(b):
    return torch.where(b == 255, float("nan"), torch.exp2(b.double() - 127))


def pow2_byte(amax):
    """The E8M0 byte of the smallest power of two X >= 2^-127 with amax / X <= 448; 127 for zero."""
    m, e = torch.frexp(amax.double())
    b = (e - 9 + (m > 0.875)).clamp(min=-127) + 127
    return torch.where(amax > 0, b, 127).to(torch.int64)


def check_quant(q, scale, y, tol, group, pow2):
    """Codes and scales of a kernel against y (64 bits), whose own y is within tol."""
    yg, tg = grouped(y, group), grouped(tol, group)
    amax, slack = yg.abs().amax(-1), tg.amax(-1)
    lo, hi = (amax - slack).clamp(min=0), amax + slack
    if pow2:
        b = scale.to(torch.int64)
        ok = (b >= pow2_byte(lo)) & (b <= pow2_byte(hi)) | (b == pow2_byte(amax))
        s = e8m0_value(scale)
    else:
        s = scale.double()
        want = torch.where(amax > 0, (amax / 448).clamp(min=2.0 ** -126), 1.0)
        ok = (s - want).abs() <= slack / 448 + 2 * U * want
    assert ok.all(), f"{(~ok).sum()} scales, first at {torch.nonzero(~ok)[0].tolist()}"
    t = yg / s[..., None]
    d = tg / s[..., None] + 4 * U * t.abs()
    v = grouped(q.view(torch.float8_e4m3fn).float().double(), group)
    # rounding is monotone: the code of a t within d lies between those of t - d and t + d
    a = (t - d).clamp(-448, 448).float().to(torch.float8_e4m3fn).double()
    z = (t + d).clamp(-448, 448).float().to(torch.float8_e4m3fn).double()
    bad = ~((v >= a) & (v <= z))
    assert not bad.any(), f"{bad.sum()} codes, first at {torch.nonzero(bad)[0].tolist()}"
    # and a code stands for its value to half a step (2^-10 below the smallest normal step)
    assert ((v - t).abs() <= (FP8 * t.abs()).clamp(min=2.0 ** -10) + d).all()


def backward64(dys, h, gamma, dres, eps=EPS):
    """(dh, its bound, dgamma, its bound)."""
    x = torch.stack([t.double() for t in dys])
    dy, mag = x.sum(0), x.abs().sum(0)
    h, gm = h.double(), gamma.double()
    M, N = h.shape
    inv = 1 / torch.sqrt((h * h).mean(1, keepdim=True) + eps)
    g = dy * gm
    mean = (g * h).mean(1, keepdim=True)
    dh = inv * g - h * inv ** 3 * mean
    size = inv * mag * gm.abs() + h.abs() * inv ** 3 * mean.abs()
    # mean sums signed terms: its error is relative to their magnitudes
    err_mean = (len(dys) + 64) * U * (mag * gm.abs() * h.abs()).mean(1, keepdim=True)
    tol = REL_INV * size + len(dys) * U * inv * mag * gm.abs() + h.abs() * inv ** 3 * err_mean
    if dres is not None:
        dh = dh + dres.double()
    tol = tol + U * dh.abs()
    tol = tol + BF16 * (dh.abs() + tol) + 1e-38
    dg = (dy * h * inv).sum(0)
    tol_g = (REL_INV + (len(dys) + M + 64) * U) * (mag * h.abs() * inv).sum(0) + 1e-38
    return dh, tol, dg, tol_g


def dequant64(codes, scale, zero, group):
    c = codes.to(torch.int64)
    u = torch.stack((c & 15, c >> 4), -1).flatten(-2).double()
    K = u.shape[-1]
    z = 8.0 if zero is None else zero.double().repeat_interleave(group, -1)[..., :K]
    return (u - z) * scale.double().repeat_interleave(group, -1)[..., :K]


def linear64(xs, ws, group):
    """sum_r x_r @ w_r.T (x_r in 64 bits), and the bound: products are exact, a tensor instruction's sums
    are truncated (a step, 2U, for each of the K / 16 it runs through), a scale costs 2 roundings."""
    y = mag = 0
    for x, (codes, scale, zero) in zip(xs, ws):
        w = dequant64(codes, scale, zero, group)
        y, mag = y + x.double() @ w.T, mag + x.double().abs() @ w.abs().T
    K = xs[0].shape[1]
    tol = (K / 16 + 64) * 2 * U * mag
    return y, tol + BF16 * (y.abs() + tol) + 1e-38


def check(got, want, tol, what):
    got = got.double()
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.numel()} out of bounds, first at {torch.nonzero(bad)[0].tolist()}: "
                           f"{got[bad][0]} for {want[bad][0]} +- {tol[bad][0]}")
