"""What the policy head (gradient_quantization_gb300/policy.py) asks of the library and keeps between
its calls (CPU: stand-ins that record their calls and give tensors of the right kind)."""
import weakref

import pytest
import torch

from gradient_quantization_gb300 import agoq
from gradient_quantization_gb300.policy import PolicyHead

V, H, T = 256, 128, 6


class Calls:
    """Stand-ins for the calls that the head makes."""

    def __init__(self, monkeypatch):
        self.names, self.quants, self.at = [], [], {}
        for name in ("agoq_layernorm_forward", "agoq_amax", "agoq_fp4_quant", "agoq_fp4_gemm",
                     "agoq_token_logprobs", "agoq_policy_loss", "agoq_preference_loss",
                     "agoq_token_logprobs_backward", "agoq_grad_accum_fp8", "agoq_layernorm_backward_laaq"):
            monkeypatch.setattr(agoq, name, self._recorded(name, getattr(self, name[5:])))
        monkeypatch.setattr(agoq, "GradList", lambda grads: grads)

    def _recorded(self, name, f):
        def call(*a, **kw):
            self.names.append(name)
            if name in self.at:
                self.at[name]()
            return f(*a, **kw)
        return call

    def layernorm_forward(self, x, w, b, eps, bits=0, want_stats=True):
        codes = (torch.zeros(4), torch.zeros(4)) if bits else (None, None)
        return (x.clone(), None, None, *codes)

    def amax(self, x):
        return torch.ones(1)

    def fp4_quant(self, x, fmt, amax=None, rows=True, columns=False):
        of = lambda want: torch.zeros(8, dtype=torch.uint8) if want else None
        out = of(rows), of(rows), of(columns), of(columns)
        self.quants.append((tuple(x.shape), rows, columns, out))
        return out

    def fp4_gemm(self, ac, asc, bc, bsc, M, N, K, fmt, aa, ba, dtype):
        assert all(t is not None for t in (ac, asc, bc, bsc))
        return torch.zeros(M, N, dtype=dtype)

    def token_logprobs(self, logits, tokens, want_entropy=True):
        z = torch.zeros(logits.shape[0])
        return z, None, z, None, None

    def policy_loss(self, logits, tokens, old, A, ref, w, lo, hi, coef, dlogits):
        z = torch.zeros(logits.shape[0])
        return z, z, None, dlogits

    def preference_loss(self, logp, offsets, ref, w, beta, eps):
        return logp, logp, logp

    def token_logprobs_backward(self, logits, tokens, lse, dlogp, dlogits):
        return dlogits

    def grad_accum_fp8(self, master, scales, grad):
        assert grad.shape == (V, H)

    def layernorm_backward_laaq(self, codes, scales, bits, dy, eps, w):
        return torch.zeros_like(dy), torch.zeros(H), torch.zeros(H)


@pytest.fixture
def calls(monkeypatch):
    return Calls(monkeypatch)


def _head(fmt):
    b = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    return PolicyHead(b(H), b(H), b(V, H), fmt=fmt)


X, IDS = torch.zeros(T, H, dtype=torch.bfloat16), torch.zeros(T, dtype=torch.int64)
COL = torch.zeros(T)


@pytest.mark.parametrize("fmt", [agoq.MXFP4, agoq.NVFP4])
def test_scoring_takes_rows_alone(calls, fmt):
    """Log probabilities have no backward pass: the columns of the normed input would be thrown away."""
    head = _head(fmt)
    del calls.quants[:]
    head.logprobs(X, IDS)
    assert [q[:3] for q in calls.quants] == [((T, H), True, False)]


def test_training_takes_columns_too(calls):
    head = _head(agoq.NVFP4)
    assert [q[:3] for q in calls.quants] == [((V, H), True, True)]
    for step in (lambda: head.policy(X, IDS, COL, COL), lambda: head.preference(X, IDS, IDS[:1])):
        del calls.quants[:]
        step()
        assert [q[:3] for q in calls.quants] == [((T, H), True, True), ((T, V), True, True)]


@pytest.mark.parametrize("fmt", [agoq.MXFP4, agoq.NVFP4])
def test_rows_are_not_kept_through_the_loss(calls, fmt):
    """Between the passes the head keeps the columns of the projection's operand, not its rows."""
    head = _head(fmt)
    seen = []

    def at_the_loss():
        (_, _, _, out), = calls.quants
        seen.append([weakref.ref(t) for t in out])
        calls.quants[:] = [q[:3] for q in calls.quants]
        del out
        seen[-1] = [r() is not None for r in seen[-1]]
    calls.at.update(agoq_policy_loss=at_the_loss, agoq_preference_loss=at_the_loss)
    for step in (lambda: head.policy(X, IDS, COL, COL), lambda: head.preference(X, IDS, IDS[:1])):
        del calls.quants[:]
        step()
    assert seen == [[False, False, True, True]] * 2
