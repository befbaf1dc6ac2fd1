"""The output end of a policy training step (gradient_quantization_gb300/policy.py) against
binary64 forms of the same path, in which every product's operands are quantised as the path
quantises them (tests/plain_fp4.py).

The path's values between the products are rounded to BF16 (2^-9 of a value on average over its
two roundings, 2^-8 at most), and an operand whose value lies near a border between two codes may
come out as either: a fraction of about 2 * 2^-9 / (2^-2) = 2^-6 of the codes (E2M1's values
are a quarter to a half apart, relative to themselves), each off by one step, 1/4 to 1/2 of the
value.  That is sqrt(2^-6) * 0.35 = 0.044 of an operand's norm, and a product of two such operands
is off by 0.062.  The gradient dy = dlogits W has one of them behind logits that are off by 0.044:
0.1 is taken for it and for the weight gradient, whose FP8 master adds 0.03 (E4M3's mean error);
the norm's backward pass from 4-bit codes adds 0.03 to dx."""
import pytest
import torch

from gradient_quantization_gb300 import agoq
from gradient_quantization_gb300.policy import PolicyHead
from tests import plain64 as P
from tests import plain_fp4 as F
from tests import plain_policy as Q

pytestmark = pytest.mark.gpu


def _far(got, want):
    return float((got.double() - want).norm() / want.norm())


def _held(x, fmt):
    """Values that a matrix is quantised to along its rows."""
    amax = None if fmt == agoq.MXFP4 else F.amax_of(x)
    codes, scales = F.stored(x, fmt, amax)
    v = F.values(codes, scales, x.shape[0], x.shape[1], fmt)
    return v if amax is None else v * F.tensor_scale(amax)


class Plain:
    def __init__(self, head):
        self.h = head
        self.w, self.b, self.weight = (t.double() for t in (head.norm_w, head.norm_b, head.weight))
        self.rows, self.cols = _held(self.weight, head.fmt), _held(self.weight.t(), head.fmt)

    def logits(self, x):
        x = x.double()
        y, mu, r = P.layernorm(x, self.w, self.b, self.h.eps)
        self.x, self.stats = x, (mu, r)
        self.y = y.bfloat16().double()
        return (_held(self.y, self.h.fmt) @ self.rows.t()).bfloat16().double()

    def backward(self, dlogits):
        """dx, dweight, dw, db."""
        d = dlogits.bfloat16().double()
        dweight = _held(d.t(), self.h.fmt) @ _held(self.y.t(), self.h.fmt).t()
        dy = (_held(d, self.h.fmt) @ self.cols.t()).bfloat16().double()
        return (P.layernorm_backward(self.x, dy, self.w, *self.stats)[0], dweight,
                *P.layernorm_backward(self.x, dy, self.w, *self.stats)[1:])


def _head(fmt, seed=3, H=512, V=1024, **kw):
    g = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()
    return PolicyHead(randn(H) * 0.1 + 1, randn(H) * 0.1, randn(V, H) * H ** -0.5, fmt=fmt, **kw), g


@pytest.mark.parametrize("fmt", [agoq.MXFP4, agoq.NVFP4])
@pytest.mark.parametrize("T", [1, 100, 333])
def test_policy_micro_batches(fmt, T):
    head, g = _head(fmt, kl_coef=0.1)
    V, H = head.weight.shape
    plain = Plain(head)
    total = [0.0, 0.0, 0.0]
    for k in range(2):
        x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
        ids = torch.randint(0, V, (T,), generator=g, device="cuda")
        if T > 1:
            ids[k::17] = -100
        logits = plain.logits(x)
        old = P.token_logprobs(logits, ids)[0] - 0.1 * torch.randn(T, generator=g, device="cuda").double()
        ref = old + 0.2
        A = torch.randn(T, generator=g, device="cuda")
        w = torch.full((T,), 1 / T, device="cuda")
        # (ratios of e^+-0.1: few lie near the bounds 0.8 and 1.2, where codes would decide)
        loss, kl, dx = head.policy(x, ids, old.float(), A, w, ref.float())
        want = Q.policy(logits, ids, old, A.double(), ref, w.double(), 0.8, 1.2, 0.1)
        assert abs(float(loss.sum()) - float(want[0].sum())) <= 0.05 * float(want[0].abs().sum())
        got = plain.backward(want[4])
        assert dx.shape == x.shape
        if T > 1:       # (of one token the loss's slope itself may be clipped on one side alone)
            assert _far(dx, got[0]) <= 0.13
        total = [a + b for a, b in zip(total, got[1:])]
    agoq.agoq_device_status()
    if T > 1:
        master = P.grad_values((head.master, head.master_scales)).view(V, H)
        assert _far(master, total[0]) <= 0.13
        assert _far(head.norm_dw, total[1]) <= 0.2 and _far(head.norm_db, total[2]) <= 0.13
    before = P.grad_norm([(head.master, head.master_scales), head.norm_dw, head.norm_db])
    assert abs(float(head.clip(0.5 * before)) - before) <= 1e-5 * before
    head.zero_grad()
    assert float(agoq.agoq_grad_norm(head.grads)) == 0


@pytest.mark.parametrize("fmt", [agoq.MXFP4, agoq.NVFP4])
def test_preference_micro_batch(fmt):
    head, g = _head(fmt, 5)
    V, H = head.weight.shape
    T, offsets = 300, [0, 40, 90, 90, 250, 280, 299]
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    ids = torch.randint(0, V, (T,), generator=g, device="cuda")
    ids[::13] = -100
    plain = Plain(head)
    logits = plain.logits(x)
    lp, _, lse, _ = P.token_logprobs(logits, ids)
    ref = torch.where(ids < 0, 0.0, lp + 0.05 * torch.randn(T, generator=g, device="cuda").double())
    loss, margin, dx = head.preference(x, ids, torch.tensor(offsets, device="cuda"), ref.float(), beta=0.1)
    want, h, dlogp = Q.preference(lp, ref, offsets, [1.0] * 3, 0.1, 0.0)
    assert torch.allclose(loss.double(), want, atol=0.1)
    dlogits = P.token_logprobs_backward(logits, ids, lse, dlogp.nan_to_num(0.0))
    got = plain.backward(dlogits)
    assert _far(dx, got[0]) <= 0.13 and not dx[299:].any()
    assert _far(P.grad_values((head.master, head.master_scales)).view(V, H), got[1]) <= 0.13


def test_scoring_is_the_training_pass():
    """The log probabilities of the policy itself: ratio 1, loss -A, KL 0, to the bit."""
    head, g = _head(agoq.NVFP4, 7, kl_coef=0.1)
    V, H = head.weight.shape
    x = torch.randn(70, H, generator=g, device="cuda").bfloat16()
    ids = torch.randint(0, V, (70,), generator=g, device="cuda")
    old = head.logprobs(x, ids)
    A = torch.randn(70, generator=g, device="cuda")
    loss, kl, _ = head.policy(x, ids, old, A, None, old)
    assert float((loss + A).abs().max()) <= 1e-5 and float(kl.abs().max()) <= 1e-10


def test_a_new_weight():
    head, g = _head(agoq.NVFP4, 9)
    x = torch.randn(5, head.weight.shape[1], generator=g, device="cuda").bfloat16()
    ids = torch.arange(5, device="cuda")
    before = head.logprobs(x, ids)
    head.weight.mul_(-1)
    assert torch.equal(head.logprobs(x, ids), before)      # until its operands are made again
    head.requantise()
    assert not torch.equal(head.logprobs(x, ids), before)


def test_command(capsys):
    from gradient_quantization_gb300 import policy
    policy.main(tokens=256, hidden=256, vocabulary=512)
    assert "policy loss" in capsys.readouterr().out
