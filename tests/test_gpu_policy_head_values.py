"""The policy head's losses, margins and divergences, and micro-batches of one token, against the
binary64 forms of tests/test_gpu_policy_head.py, where each value is far from its bound; and what the
head refuses.

A token's log probability is off by LOGP = 0.062 of the logits' spread (1 here) in the mean, by the
codes near a border (see there).  A sum of n of them is off by LOGP sqrt(n), and six times that is
taken."""
import math

import pytest
import torch

from gradient_quantization_gb300 import agoq
from tests import plain64 as P
from tests import plain_policy as Q
from tests.test_gpu_policy_head import Plain, _far, _head

pytestmark = pytest.mark.gpu
FORMATS = [agoq.MXFP4, agoq.NVFP4]
LOGP = 0.062
U = 2.0 ** -24


def _batch(head, g, T):
    V, H = head.weight.shape
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    ids = torch.randint(0, V, (T,), generator=g, device="cuda")
    plain = Plain(head)
    return x, ids, plain, plain.logits(x)


@pytest.mark.parametrize("fmt", FORMATS)
def test_preference_margins(fmt):
    """Margins of several units and either sign, and losses that belong to them: chosen and
    rejected tokens swapped, or a loss of ln 2, are far outside."""
    head, g = _head(fmt, 11)
    T, offsets, beta = 300, [0, 40, 90, 90, 250, 280, 299], 0.25
    x, ids, plain, logits = _batch(head, g, T)
    ids[::13] = -100
    lp = P.token_logprobs(logits, ids)[0]
    shift = torch.zeros(T, dtype=torch.float64, device="cuda")
    for p, s in enumerate((0.2, 0.1, -0.3)):             # logp - ref: s at the chosen, -s at the rejected
        a, b, c = offsets[2 * p:2 * p + 3]
        shift[a:b], shift[b:c] = s, -s
    shift[90:250] = 0.1                                  # (the pair whose chosen answer is empty)
    ref = torch.where(ids < 0, 0.0, lp - shift)
    loss, margin, _ = head.preference(x, ids, torch.tensor(offsets, device="cuda"), ref.float(), beta=beta)
    _, h, _ = Q.preference(torch.where(ids < 0, 0.0, lp), ref, offsets, [1.0] * 3, beta, 0.0)
    assert [round(float(v)) for v in h] == [4, -4, -3]
    n = torch.tensor([90.0, 160.0, 49.0], device="cuda")
    assert bool(((margin - h).abs() <= 6 * LOGP * beta * n.sqrt()).all()), (margin, h)
    soft = torch.nn.functional.softplus(-margin.double())
    assert bool(((loss - soft).abs() <= 12 * U * soft).all()), (loss, soft)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T", [100, 333])
def test_divergence_from_the_reference(fmt, T):
    """d = 2 in the plain form: kl = e^2 - 3, with a slope of e^2 - 1."""
    head, g = _head(fmt, 12, kl_coef=0.1)
    x, ids, plain, logits = _batch(head, g, T)
    ids[3::17] = -100
    lp = P.token_logprobs(logits, ids)[0]
    ref = lp + 2
    own = head.logprobs(x, ids)
    A = torch.randn(T, generator=g, device="cuda")
    loss, kl, _ = head.policy(x, ids, own, A, None, ref.float())
    live = ids >= 0
    assert not kl[~live].any() and not loss[~live].any()
    # of its own log probabilities: they are the scoring pass's within 2e-6 (a rounding of logp, 5e-7,
    # and the sum's exponentials and logarithm), once in each call, times the slope; four times that
    d = ref - own.double()
    want = torch.expm1(d) - d
    assert bool(((kl - want).abs() <= 4 * 4e-6 * d.exp())[live].all())
    assert bool(((loss - (0.1 * want - A)).abs() <= 4 * 4e-6 * (0.1 * d.exp() + A.abs()))[live].all())
    # and of the plain form's: the mean
    off = (math.exp(2) - 1) * 6 * LOGP / math.sqrt(int(live.sum())) + math.exp(2) * LOGP ** 2
    assert abs(float(kl[live].mean()) - (math.exp(2) - 3)) <= off


@pytest.mark.parametrize("fmt", FORMATS)
def test_one_token(fmt):
    """Ratio e^-1 under a positive advantage: not clipped.  The factor of the gradient is 4.4, which
    leaves the token's own gradient far from a border between codes (4 and 6, or 6 under an E4M3
    scale), and what is left of the errors is that of longer micro-batches."""
    head, g = _head(fmt, 13)
    x, ids, plain, logits = _batch(head, g, 1)
    A = torch.full((1,), 4.4 * math.e, device="cuda")
    own = head.logprobs(x, ids)
    loss, kl, dx = head.policy(x, ids, own + 1, A)
    assert kl is None and abs(float(loss) + 4.4) <= 1e-4
    lp = P.token_logprobs(logits, ids)[0]
    one = torch.ones(1, dtype=torch.float64, device="cuda")
    want = Q.policy(logits, ids, lp + 1, A.double(), None, one, 0.8, 1.2, 0.0)
    assert abs(float(want[0]) + 4.4) <= 1e-6
    wx, ww, wdw, wdb = plain.backward(want[4])
    assert dx.shape == x.shape and _far(dx, wx) <= 0.13
    V, H = head.weight.shape
    assert _far(P.grad_values((head.master, head.master_scales)).view(V, H), ww) <= 0.13
    assert _far(head.norm_dw, wdw) <= 0.2 and _far(head.norm_db, wdb) <= 0.13


def test_refusals_come_first(monkeypatch):
    """An input of another type or length is refused by the first call of a micro-batch, and no
    gradient has changed."""
    head, g = _head(agoq.NVFP4, 14)
    V, H = head.weight.shape
    ids, col = torch.zeros(4, dtype=torch.int64, device="cuda"), torch.zeros(4, device="cuda")
    offsets = torch.tensor([0, 2, 4], device="cuda")

    def late(*a, **kw):
        raise AssertionError("a later call was made")
    for name in ("agoq_amax", "agoq_fp4_quant", "agoq_fp4_gemm", "agoq_policy_loss", "agoq_token_logprobs"):
        monkeypatch.setattr(agoq, name, late)
    for norm in (torch.bfloat16, torch.float32):
        head.norm_w, head.norm_b = head.norm_w.to(norm), head.norm_b.to(norm)
        for x in (torch.zeros(4, H, device="cuda"), torch.zeros(4, H, device="cuda").half(),
                  torch.zeros(4, H + 128, device="cuda").bfloat16(), torch.zeros(4, H).bfloat16()):
            with pytest.raises((TypeError, ValueError, agoq.AgoqError)):
                head.policy(x, ids, col, col)
            with pytest.raises((TypeError, ValueError, agoq.AgoqError)):
                head.preference(x, ids, offsets)
    assert not head.master.any() and not head.norm_dw.any() and not head.norm_db.any()
