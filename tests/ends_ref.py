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
    mean, inv, rel, xhat, tol_x = stats64(h, h.abs())
    g, gmag = dy * gm, mag * gm.abs()
    # a row with mean^2 <= 4 var has var = mean(h^2) - mean^2 and the products' sum less mean * sum g: the sums' errors are
    # relative to terms up to 5 var; mean(h^2) is off by 64 U of it, mean^2 by 2 |mean| * 64 U mean|h| and a rounding
    near = mean * mean <= 4.1 * (1 / (inv * inv) - EPS)
    lost = torch.where(near, 193 * U * (h * h).mean(1, keepdim=True) * inv * inv, 0.0)
    rel, tol_x = rel + lost, tol_x + lost * xhat.abs()
    a, b = g.mean(1, keepdim=True), (g * xhat).mean(1, keepdim=True)
    dh = inv * (g - a - xhat * b)
    n = (len(dys) + 64) * U
    tol_a = n * gmag.mean(1, keepdim=True)
    tol_b = n * (gmag * xhat.abs()).mean(1, keepdim=True) + (gmag * tol_x).mean(1, keepdim=True) + rel * b.abs()
    tol_b = tol_b + torch.where(near, inv * (n * (gmag * h.abs()).mean(1, keepdim=True) + n * mean.abs() * gmag.mean(1, keepdim=True)
                                             + 66 * U * a.abs() * h.abs().mean(1, keepdim=True)), 0.0)
    tol = inv * (n * gmag + tol_a + xhat.abs() * tol_b + tol_x * b.abs()) + (rel + 8 * U) * inv * (
        gmag + a.abs() + xhat.abs() * b.abs())
    if dres is not None:
        dh = dh + dres.double()
    tol = tol + U * dh.abs()
    tol = tol + BF16 * (dh.abs() + tol) + 1e-38
    m = (len(dys) + M + 64) * U
    dgamma, dbeta = (dy * xhat).sum(0), dy.sum(0)
    return (dh, tol, dgamma, m * (mag * xhat.abs()).sum(0) + (mag * tol_x).sum(0) + 1e-38, dbeta, m * mag.sum(0) + 1e-38)


def cross_entropy64(h, ws, targets, vocab, dloss=None):
    """loss, lse, dh, dw in 64 bits, each with its bound.

    A logit's products are summed by tensor instructions of 16 terms that cut their sums at one step, 64 of them at most
    before the sum goes on in rounded steps of half that, K / 256 at most; 16 more steps for what an instruction cuts from its
    terms: all relative to sum |h w|.  lse is off by no more than the worst logit of its row, by 2^-20 for exp and
    log (ex2 2^-22, 2^-21 for sums of up to 256 columns and joins) and by its rounding; d by its logit's error, lse's and
    2^-20, relative to exp(z - lse), and by bf16's half step."""
    M, K = h.shape
    N = ws[0].shape[0]
    w = torch.cat([t.double() for t in ws])
    w[vocab:] = 0   # padding, whatever it holds
    x = h.double()
    z = x @ w[:vocab].T
    err = (min(K / 16, 64) + K / 512 + 16) * 2 * U * (x.abs() @ w[:vocab].abs().T)
    lse = torch.logsumexp(z, 1)
    worst = err.max(1).values if M else lse
    tol_lse = worst + 2.0 ** -20 + 2 * U * lse.abs()
    t = targets.long()
    on = (t >= 0) & (t < vocab)
    at = t.clamp(0, vocab - 1)[:, None]
    loss = torch.where(on, lse - z.gather(1, at)[:, 0], 0.0)
    tol_loss = torch.where(on, 2 * worst + 2.0 ** -20 + 2 * U * loss.abs(), 0.0)
    out = [(loss, tol_loss), (lse, tol_lse)]
    if dloss is None:
        return out
    g = torch.where(on, dloss.double(), 0.0)[:, None]
    p = torch.exp(z - lse[:, None])
    hot = torch.zeros_like(p).scatter_(1, at, 1.0) * on[:, None]
    d = (p - hot) * g
    e = p * g.abs() * (err + tol_lse[:, None] + 2.0 ** -20) * 1.1
    e = e + BF16 * (d.abs() + e) + 1e-38
    dh, mag = d @ w[:vocab], d.abs() @ w[:vocab].abs()
    tol = e @ w[:vocab].abs() + (vocab / 16 + 64) * 2 * U * mag
    out.append((dh, tol + BF16 * (dh.abs() + tol) + 1e-38))
    dw = torch.zeros_like(w)
    tol = torch.zeros_like(w)
    dw[:vocab] = d.T @ x
    tol[:vocab] = e.T @ x.abs() + (M / 16 + 64) * 2 * U * (d.abs().T @ x.abs())
    tol[:vocab] += BF16 * (dw[:vocab].abs() + tol[:vocab]) + 1e-38
    return out + [(dw.view(len(ws), N, K), tol.view(len(ws), N, K))]
