"""Plain binary64 forms of the policy and preference losses, and the bounds that binary32
arithmetic keeps against them (u = 2^-24, half a binary32 step).

expf and expm1f are within 2 steps (4 u), logf and log1pf within 2."""
import torch

from tests import plain64 as P

U = 2.0 ** -24


def policy(x, tokens, old, A, ref, w, lo, hi, coef):
    """(loss, logp, kl, c, dlogits, logs, lse) of binary64 rows x; lo and hi: the bounds of the
    ratio.  Ignored rows are 0."""
    logp, _, lse, logs = P.token_logprobs(x, tokens)
    live = tokens >= 0
    r = (logp - old).exp()
    clipped = ((A > 0) & (r > hi)) | ((A < 0) & (r < lo))
    loss = -torch.where(clipped, torch.where(A > 0, hi, lo) * A, r * A)
    c = torch.where(clipped, 0.0, r * A)
    kl = torch.zeros_like(loss)
    if ref is not None:
        d = ref - logp
        kl = torch.expm1(d) - d
        if coef:
            loss, c = loss + coef * kl, c + coef * torch.expm1(d)
    zero = lambda v: torch.where(live, v, torch.zeros_like(v))
    loss, kl, c = zero(w * loss), zero(kl), zero(w * c)
    return loss, logp, kl, c, P.loss_gradient(logs, tokens, c), logs, lse


def policy_bounds(x, tokens, old, A, ref, w, lo, hi, coef, out, dtype):
    """Bounds of loss, logp, kl and dlogits, where the ratio is not next to a bound of its own."""
    loss, logp, kl, c, grad, logs, lse = out
    V = x.shape[1]
    every, _, _ = P.token_bounds(x, logs, lse)
    elp = every.gather(1, tokens.clamp(0, V - 1)[:, None]).squeeze(1)
    r = (logp - old).exp()
    er = elp + U * (logp - old).abs() + 5 * U            # relative
    size, slope = (r * A).abs(), torch.zeros_like(r)
    eloss, ec = size * (er + 2 * U), size * (er + 2 * U)
    ekl = torch.zeros_like(r)
    if ref is not None:
        d = ref - logp
        em = torch.expm1(d).abs()
        ed = elp + U * d.abs()
        grow = d.exp()
        ekl = em * ed + grow * ed * ed + 4 * U * (em + d.abs())
        eloss = eloss + coef * (ekl + 2 * U * kl)
        ec = ec + coef * (grow * ed * 1.01 + 4 * U * em)
        size = size + coef * kl
        slope = coef * em
    eloss = w.abs() * (eloss + 3 * U * size)
    ec = w.abs() * (ec + 3 * U * ((r * A).abs() + slope))
    at = torch.arange(V, device=x.device)[None, :] == tokens[:, None]
    step = (logs.exp() - at.to(x.dtype)).abs()
    eg = P.loss_bound(x, logs, lse, c, grad, dtype) + ec[:, None] * step * (1 + torch.finfo(dtype).eps)
    tiny = 2.0 ** -148
    return eloss * 1.01 + tiny, elp, ekl * 1.01 + tiny, eg


def preference(logp, ref, offsets, w, beta, eps):
    """(loss, margin, dlogp) of binary64 values; offsets and w: lists.  dlogp is NaN at the tokens
    of no answer."""
    r = logp if ref is None else logp - ref
    P_ = len(offsets) // 2
    loss, margin, grad = [], [], torch.full_like(logp, float("nan"))
    for p in range(P_):
        a, b, c = offsets[2 * p:2 * p + 3]
        h = beta * (r[a:b].sum() - r[b:c].sum())
        soft = torch.nn.functional.softplus
        loss.append(w[p] * ((1 - eps) * soft(-h) + eps * soft(h)))
        margin.append(h)
        v = w[p] * beta * (torch.sigmoid(-h) - eps)
        grad[a:b], grad[b:c] = -v, v
    of = lambda v: torch.stack(v) if v else logp.new_zeros(0)
    return of(loss), of(margin), grad


def preference_bounds(logp, ref, offsets, w, beta, eps, margin):
    """Bounds of loss, margin and |dlogp| of each pair.  The margin's sum carries its roundings
    along: what is left is the second order, n^2 u^2 of the magnitudes, and the last rounding."""
    r = (logp if ref is None else logp.abs() + ref.abs()).abs()
    mag = torch.stack([r[offsets[2 * p]:offsets[2 * p + 2]].sum() for p in range(len(w))])
    n = torch.tensor([offsets[2 * p + 2] - offsets[2 * p] for p in range(len(w))], device=r.device)
    em = beta * mag * (n.double() * U) ** 2 + 2 * U * margin.abs() + 2.0 ** -148
    soft = torch.nn.functional.softplus
    w = torch.tensor(w, dtype=torch.float64, device=r.device).abs()
    eloss = w * (em + 12 * U * (soft(-margin) + soft(margin) * eps))
    eg = w * beta * (em + 12 * U)
    return eloss * 1.01 + 2.0 ** -148, em * 1.01, eg * 1.01 + 2.0 ** -148
