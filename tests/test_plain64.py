"""The binary64 forms that the GPU tests compare with: their gradients against
torch's derivatives of the plain forward formulas and against central
differences (CPU)."""
import torch

from tests import plain64 as P


def _differences(f, x, step=1e-6):
    out = torch.zeros_like(x)
    for i in range(x.numel()):
        e = torch.zeros_like(x).view(-1)
        e[i] = step
        out.view(-1)[i] = (f(x + e.view_as(x)) - f(x - e.view_as(x))) / (2 * step)
    return out


def test_layernorm_backward():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(3, 11, generator=g, dtype=torch.float64)
    w, b = torch.randn(11, generator=g, dtype=torch.float64), torch.randn(11, generator=g,
                                                                          dtype=torch.float64)
    dy = torch.randn(3, 11, generator=g, dtype=torch.float64)
    f = lambda x, w, b: (P.layernorm(x, w, b, 1e-5)[0] * dy).sum()
    _, mu, r = P.layernorm(x, w, b, 1e-5)
    dx, dw, db = P.layernorm_backward(x, dy, w, mu, r)
    leaves = [t.clone().requires_grad_() for t in (x, w, b)]
    for got, want in zip((dx, dw, db), torch.autograd.grad(f(*leaves), leaves)):
        assert torch.allclose(got, want, rtol=1e-10, atol=1e-12)
    assert torch.allclose(dx, _differences(lambda v: f(v, w, b), x), rtol=1e-5, atol=1e-7)
    assert torch.allclose(dw, _differences(lambda v: f(x, v, b), w), rtol=1e-5, atol=1e-7)


def test_token_logprobs_backward():
    g = torch.Generator().manual_seed(2)
    x = 2 * torch.randn(4, 9, generator=g, dtype=torch.float64)
    x[1, 3] = -torch.inf
    tokens = torch.tensor([0, 5, -1, 8])
    dl, de = torch.randn(4, generator=g, dtype=torch.float64), torch.randn(4, generator=g,
                                                                           dtype=torch.float64)

    def f(v):
        logp, ent, _, _ = P.token_logprobs(v, tokens)
        return (torch.where(tokens < 0, 0.0, dl) * logp + de * ent).sum()
    _, ent, lse, _ = P.token_logprobs(x, tokens)
    grad = P.token_logprobs_backward(x, tokens, lse, dl, ent, de)
    assert grad[1, 3] == 0
    want = _differences(f, x.masked_fill(x == -torch.inf, -80.0))
    keep = torch.isfinite(x)
    assert torch.allclose(grad[keep], want[keep], rtol=1e-5, atol=1e-7)
    _, _, _, logs = P.token_logprobs(x, tokens)
    assert torch.allclose(P.loss_gradient(logs, tokens, dl),
                          P.token_logprobs_backward(x, tokens, lse, -dl), rtol=1e-12, atol=1e-14)
    p = torch.softmax(x, 1)
    assert torch.allclose(ent, -(p * p.clamp(min=1e-300).log()).sum(1))


def test_empty_row_and_order():
    x = torch.full((2, 5), -torch.inf, dtype=torch.float64)
    x[1] = torch.tensor([1.0, 3.0, 3.0, 1.0, 3.0])
    logp, ent, lse, logs = P.token_logprobs(x, torch.tensor([2, 9]))
    assert logp[0] == -torch.inf and ent[0] == 0 and lse[0] == -torch.inf
    assert torch.isnan(logp[1])
    assert P.top(x, 5).tolist() == [[0, 1, 2, 3, 4], [1, 2, 4, 0, 3]]
    assert not P.token_logprobs_backward(x, torch.tensor([2, 0]), lse,
                                         torch.ones(2, dtype=torch.float64))[0].any()
