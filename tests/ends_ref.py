"""Plain 64-bit implementations of LayerNorm, the vocabulary-parallel embedding and the
cross entropy, with bounds on how far a kernel that keeps its sums in 32 bits may be.

U = 2^-24 is half a step of fp32.  LayerNorm's mean: at most 8 * 4 terms in a thread, 5
shuffles and 16 warp totals, so it is off by less than 64 * U * mean|h|.  The squares
around it are as good as the mean is: c = h - mean carries that error and a rounding,
and var is off by less than 2 * err * mean|c| + err^2 (a warp's own mean, exact in the
join's formula, errs alike) + 64 * U * var; rsqrt halves the relative error and adds 2 steps."""
import torch

from tests.ops_ref import BF16, U, check  # noqa: F401

EPS = 1e-5
REL = 2.0 ** -18


def stats64(h, mag):
    """mean, inv, their bounds [M, 1], and xhat with its bound; h in 64 bits, mag >= |h|'s terms."""
    mean = h.mean(1, keepdim=True)
    c = h - mean
    var = (c * c).mean(1, keepdim=True)
    inv = 1 / torch.sqrt(var + EPS)
    err = 64 * U * mag.mean(1, keepdim=True) + U * mean.abs()
    rel = (2 * err * c.abs().mean(1, keepdim=True) + err * err + 64 * U * var) / (var + EPS) + REL
    xhat = c * inv
    tol = (err + U * (h.abs() + mean.abs())) * inv + rel * xhat.abs()
    return mean, inv, rel, xhat, tol


def layernorm64(parts, res, gamma, beta):
    """(y, its bound, h, its bound)."""
    x = torch.stack([t.double() for t in parts])
    h, mag = x.sum(0), x.abs().sum(0)
    if res is not None:
        h, mag = h + res.double(), mag + res.double().abs()
    _, inv, _, xhat, tol = stats64(h, mag)
    lost = (len(parts) + 1) * U * mag   # of h itself
    tol = (tol + (lost + lost.mean(1, keepdim=True)) * inv * 2) * gamma.double().abs()
    y = xhat * gamma.double()
    if beta is not None:
        y = y + beta.double()
        tol = tol + U * (y.abs() + beta.double().abs())
    return y, tol + BF16 * (y.abs() + tol) + 1e-38, h, BF16 * h.abs() + lost * 1.01 + 1e-38


def layernorm_backward64(dys, h, gamma, dres):
    """(dh, bound, dgamma, bound, dbeta, bound)."""
    x = torch.stack([t.double() for t in dys])
    dy, mag = x.sum(0), x.abs().sum(0)
    h, gm = h.double(), gamma.double()
    M = h.shape[0]
    _, inv, rel, xhat, tol_x = stats64(h, h.abs())
    g, gmag = dy * gm, mag * gm.abs()
    a, b = g.mean(1, keepdim=True), (g * xhat).mean(1, keepdim=True)
    dh = inv * (g - a - xhat * b)
    n = (len(dys) + 64) * U
    tol_a = n * gmag.mean(1, keepdim=True)
    tol_b = n * (gmag * xhat.abs()).mean(1, keepdim=True) + (gmag * tol_x).mean(1, keepdim=True) + rel * b.abs()
    tol = inv * (n * gmag + tol_a + xhat.abs() * tol_b + tol_x * b.abs()) + (rel + 8 * U) * inv * (
        gmag + a.abs() + xhat.abs() * b.abs())
    if dres is not None:
        dh = dh + dres.double()
    tol = tol + U * dh.abs()
    tol = tol + BF16 * (dh.abs() + tol) + 1e-38
    m = (len(dys) + M + 64) * U
    dgamma, dbeta = (dy * xhat).sum(0), dy.sum(0)
    return (dh, tol, dgamma, m * (mag * xhat.abs()).sum(0) + (mag * tol_x).sum(0) + 1e-38, dbeta, m * mag.sum(0) + 1e-38)
