"""Plain binary64 forms of the layer norm, the gradient norm and the token log
probabilities, and the bounds that binary32 arithmetic keeps against them.

u = 2^-24 is half a binary32 step.  A sum whose longest path has K additions is
within K u of the sum of its terms' magnitudes; an output is rounded once to its
type, off by at most half a step (finfo.eps / 2 relative, or half the smallest
subnormal).
"""
import math

import torch

U = 2.0 ** -24
# half of the smallest subnormal step of a type
TINY = {torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}


def half_step(v, dtype):
    return v.abs() * (torch.finfo(dtype).eps / 2) + TINY[dtype]


# ---- layer norm ---------------------------------------------------------------------------


def layernorm(x, w, b, eps):
    """y, mean, rstd of rows x (binary64)."""
    mu = x.mean(1, keepdim=True)
    r = 1 / torch.sqrt((x - mu).square().mean(1, keepdim=True) + eps)
    y = (x - mu) * r
    y = y if w is None else y * w
    y = y if b is None else y + b
    return y, mu.squeeze(1), r.squeeze(1)


def layernorm_backward(x, dy, w, mu, r):
    """dx, dw, db for given statistics."""
    xh = (x - mu[:, None]) * r[:, None]
    g = dy if w is None else dy * w
    s0, s1 = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    return r[:, None] * (g - s0 - xh * s1), (dy * xh).sum(0), dy.sum(0)


def row_paths(H):
    """Additions on the longest path of a row sum: a warp at least takes a row."""
    return H / 32 + 40


def stats_bounds(x, eps):
    """(mean, relative rstd) bounds of the two-pass statistics."""
    K, H = row_paths(x.shape[1]), x.shape[1]
    d = x - x.mean(1, keepdim=True)
    var = d.square().mean(1)
    dmu = (K + 2) * U * x.abs().mean(1)
    # each difference is off by dmu and a rounding; the squares' sum by K roundings
    dvar = (K + 6) * U * var + 2 * (dmu + U * d.abs().mean(1)) * d.abs().mean(1) + dmu.square()
    return dmu, 0.5 * dvar / (var + eps).clamp(min=1e-300) + 4 * U


def xhat_bound(x, mu, r, dmu, rr):
    xh = (x - mu[:, None]) * r[:, None]
    return xh.abs() * (rr[:, None] + 4 * U) + r[:, None] * (dmu[:, None] * (1 + 4 * U))


def layernorm_bound(x, w, b, eps, y, mu, r, dtype):
    """Bound of y."""
    e = xhat_bound(x, mu, r, *stats_bounds(x, eps))
    xh = ((x - mu[:, None]) * r[:, None]).abs()
    if w is not None:
        e, xh = e * w.abs(), xh * w.abs()
    e = e + 2 * U * (xh + y.abs())
    return e * 1.01 + half_step(y.abs() + e, dtype)


def layernorm_backward_bounds(x, dy, w, mu, r, dmu, rr, dx, dtype):
    """Bounds of dx, dw, db; dmu and rr: errors of the statistics (0 where they are inputs).
    A column sum's path: the rows of one partial sum, and the partial sums."""
    T, H = x.shape
    K, KT = row_paths(H), T / 128 + 400
    xh = (x - mu[:, None]) * r[:, None]
    ex = xhat_bound(x, mu, r, dmu, rr)
    g = dy if w is None else dy * w
    m = lambda v: v.abs().mean(1, keepdim=True)
    e0 = (K + 4) * U * m(g)
    e1 = (K + 4) * U * m(g * xh) + m(g.abs() * ex)
    s0, s1 = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    e = r[:, None] * (e0 + xh.abs() * e1 + ex * (s1.abs() + e1)
                      + 6 * U * (g.abs() + s0.abs() + (xh * s1).abs()))
    e = e + dx.abs() * (rr[:, None] + 4 * U)
    return (e * 1.01 + half_step(dx.abs() + e, dtype),
            ((dy.abs() * ex).sum(0) + (KT + 2) * U * (dy * xh).abs().sum(0)) * 1.01 + TINY[torch.float32],
            KT * U * dy.abs().sum(0) * 1.01 + TINY[torch.float32])


# ---- gradient norm ------------------------------------------------------------------------


def grad_values(g):
    """Values (binary64) of a gradient: a tensor, or E4M3 codes with block scales (each value a
    binary32 product)."""
    if isinstance(g, tuple):
        codes, scales = g
        v = codes.view(torch.float8_e4m3fn).float().view(-1, 128) * scales[:, None]
        return v.double().reshape(-1)
    return g.double().reshape(-1)


def grad_norm(grads):
    return math.sqrt(math.fsum(float(grad_values(g).square().sum()) for g in grads))


# ---- token log probabilities ----------------------------------------------------------------


def token_logprobs(x, tokens):
    """logp, entropy, lse, log probabilities of all (binary64)."""
    V = x.shape[1]
    m = x.amax(1, keepdim=True)
    empty = (m == -math.inf).squeeze(1)
    m = torch.where(m == -math.inf, 0.0, m)
    total = (x - m).exp().sum(1, keepdim=True)
    lse = m + total.log()
    # (x - m) first: m may be too large for lse to hold ln(total) beside it
    logs = torch.where(x == -math.inf, x, x - m - torch.where(total == 0, 0.0, total.log()))
    p = logs.exp()
    entropy = -torch.where(p > 0, p * logs, 0.0).sum(1)
    logp = logs.gather(1, tokens.clamp(0, V - 1)[:, None]).squeeze(1)
    logp = torch.where(tokens < 0, 0.0, torch.where(tokens >= V, math.nan, logp))
    return logp, torch.where(empty, 0.0, entropy), lse.squeeze(1), logs


def top(x, k):
    """Indices of the k largest by (value descending, index ascending)."""
    return torch.sort(x, dim=1, descending=True, stable=True).indices[:, :k]


def token_logprobs_backward(x, tokens, lse, dlogp, entropy=None, dentropy=None):
    V = x.shape[1]
    empty = (lse == -math.inf)[:, None]
    l = torch.where(x == -math.inf, x, x - torch.where(empty, 0.0, lse[:, None]))
    p = l.exp()
    d = torch.where(tokens < 0, 0.0, dlogp)[:, None]
    hot = torch.arange(V, device=x.device)[None, :] == tokens[:, None]
    grad = d * (hot.to(x.dtype) - p)
    if dentropy is not None:
        grad = grad - torch.where(p > 0, dentropy[:, None] * p * (l + entropy[:, None]), 0.0)
    grad = torch.where(empty, 0.0, grad)
    return torch.where((tokens >= V)[:, None], math.nan, grad)


def loss_gradient(logs, tokens, weights):
    """Gradient of -sum(weights * logp), from the log probabilities of all."""
    V = logs.shape[1]
    hot = torch.arange(V, device=logs.device)[None, :] == tokens[:, None]
    empty = (logs == -math.inf).all(1) | (tokens < 0)
    grad = torch.where(empty, 0.0, weights)[:, None] * (logs.exp() - hot.to(logs.dtype))
    return torch.where((tokens >= V)[:, None], math.nan, grad)


def softmax_bounds(x, logs, lse):
    """(relative bound of each probability, of the sum, of the sum of p (x - m)).  An
    exponential is off by 4 u, and by 4 u for each unit of its argument (the difference and its
    scaled product are rounded); a sum's path has V / 256 + 64 additions."""
    V = x.shape[1]
    K = V / 256 + 64
    m = x.amax(1, keepdim=True)
    d = torch.where(x == -math.inf, 0.0, x - torch.where(m == -math.inf, 0.0, m)).abs()
    p = logs.exp()
    e = (4 + 4 * d) * U
    total = K * U + (p * e).sum(1, keepdim=True)
    first = K * U * (p * d).sum(1, keepdim=True) + (p * d * (e + 2 * U)).sum(1, keepdim=True)
    return e, total, first, p, d


def token_bounds(x, logs, lse):
    """Bounds of every log probability, of the entropy and of lse."""
    e, total, first, p, d = softmax_bounds(x, logs, lse)
    ln = (lse[:, None] - x.amax(1, keepdim=True)).abs().nan_to_num(0.0, 0.0, 0.0)
    base = total + 3 * U * ln + 2.0 ** -149
    logp = base + 2 * U * (d + logs.abs().nan_to_num(0.0, 0.0, 0.0))
    mean = (p * d).sum(1, keepdim=True)
    entropy = base + first + mean * (total + 4 * U) + 2 * U * (ln + mean)
    return (logp * 1.01, (entropy * 1.01).squeeze(1),
            (base * 1.01).squeeze(1) + 2 * U * lse.abs().nan_to_num(0.0, 0.0, 0.0))


def loss_bound(x, logs, lse, weights, grad, dtype):
    e, total, _, p, _ = softmax_bounds(x, logs, lse)
    b = weights[:, None].abs() * (p * (e + total + 6 * U) + 2 * U * (grad != 0)) + 2 * U * grad.abs()
    return b * 1.01 + half_step(grad.abs() + b, dtype)


def logprobs_backward_bound(x, lse, dlogp, entropy, dentropy, grad, dtype):
    """l = x - lse is rounded (u |l|) and scaled before the exponential."""
    l = torch.where(x == -math.inf, 0.0, x - torch.where(lse == -math.inf, 0.0, lse)[:, None]).abs()
    p = torch.where(x == -math.inf, 0.0, (x - lse[:, None])).exp()
    p = torch.where((x == -math.inf) | (lse == -math.inf)[:, None], 0.0, p)
    e = (8 + 4 * l) * U
    size = dlogp[:, None].abs()
    if dentropy is not None:
        size = size + dentropy[:, None].abs() * (l + entropy[:, None].abs())
    b = p * size * (e + 6 * U) + 2 * U * grad.abs().nan_to_num(0.0, 0.0, 0.0)
    return b * 1.01 + half_step(grad.abs() + b, dtype)
