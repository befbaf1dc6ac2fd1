"""The clipped policy loss and the preference loss on the GPU against their plain binary64 forms
(tests/plain_policy.py holds formulas and bounds): types, vocabularies of one entry to ones that
fit no chip, strides and alignments, masks, both sides of both bounds, ignored and foreign tokens,
values that are not finite, empty and long answers, gradients against differences."""
import math

import pytest
import torch

from gradient_quantization_gb300 import agoq
from tests import plain_policy as Q
from tests.gpu_util import Guarded

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
TYPES = [F32, BF16, F16]


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _logits(T, V, dtype, seed, pad=0, shift=0, scale=2.5):
    g = _gen(seed)
    buf = torch.full((T * (V + pad) + shift + 16,), 50.0, dtype=dtype, device="cuda")
    x = buf[shift:shift + T * (V + pad)].view(T, V + pad)[:, :V]
    x.copy_(scale * torch.randn(T, V, generator=g, device="cuda"))
    return x


def _case(x, seed, ref=True, lo=0.8, hi=1.25, spread=0.4):
    """Tokens, old and reference log probabilities, advantages and weights for logits x; no ratio
    within 1e-3 of a bound."""
    T, V = x.shape
    g = _gen(seed)
    tokens = torch.randint(0, V, (T,), generator=g, device="cuda")
    # a token that the mask left, where there is one
    tokens = torch.where(torch.isfinite(x.gather(1, tokens[:, None]).squeeze(1)), tokens, x.argmax(1))
    logp = torch.log_softmax(x.double(), 1).gather(1, tokens[:, None]).squeeze(1)
    step = spread * torch.randn(T, generator=g, device="cuda").double()
    for edge in (math.log(lo) if lo else -1e9, math.log(hi)):
        step = torch.where((step - edge).abs() < 1e-3, edge + 2e-3, step)
    old = (logp - step).nan_to_num(-1.0).float()
    A = torch.randn(T, generator=g, device="cuda")
    r = (logp + 0.7 * torch.randn(T, generator=g, device="cuda")).nan_to_num(-1.0).float() if ref else None
    w = torch.rand(T, generator=g, device="cuda") + 0.1
    return tokens, old, A, r, w


def _close(got, want, bound, what):
    got, big = got.double(), torch.finfo(got.dtype).max
    want = torch.where(want.abs() > big, want.sign() * math.inf, want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), what
    fine = torch.isfinite(want)
    off, b = (got - want).abs()[fine], bound[fine]
    assert bool((off <= b).all()), (what, float((off / b).max()))


def _check(x, tokens, old, A, ref, w, lo=0.2, hi=0.25, coef=0.1, **kw):
    before = x.clone()
    got = agoq.agoq_policy_loss(x, tokens, old, A, ref_logp=ref, weights=w, clip_low=lo, clip_high=hi,
                                kl_coef=coef if ref is not None else 0.0, **kw)
    x64 = before.double()
    d = lambda v: None if v is None else v.double()
    w64 = torch.ones_like(old).double() if w is None else w.double()
    f = lambda v: float(torch.tensor(v, dtype=F32))
    lo, hi = float(1 - torch.tensor(lo, dtype=F32)), float(1 + torch.tensor(hi, dtype=F32))
    args = (x64, tokens, d(old), d(A), d(ref), w64, lo, hi, f(coef) if ref is not None else 0.0)
    want = Q.policy(*args)
    bloss, blogp, bkl, bgrad = Q.policy_bounds(*args, want, x.dtype)
    _close(got[0], want[0], bloss, "loss")
    _close(got[1], want[1], blogp, "logp")
    if ref is not None:
        _close(got[2], want[2], bkl, "kl")
    else:
        assert got[2] is None
    _close(got[3], want[4], bgrad, "gradient")
    return got


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,V", [(1, 1), (2, 7), (9, 100), (5, 691), (300, 1003), (33, 10000), (7, 32000),
                                 (3, 50001), (2, 131072), (2, 300001), (1, 500000)])
def test_sizes(dtype, T, V):
    x = _logits(T, V, dtype, T + V)
    for ref in (True, False):
        _check(x, *_case(x, 1, ref))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rows_that_fit_no_chip(dtype):
    x = _logits(3, 1000003, dtype, 2)
    tokens, old, A, ref, w = _case(x, 3)
    tokens[1] = -1
    _check(x, tokens, old, A, ref, w)
    _check(x, tokens, old, A, ref, w, dlogits=x)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V,pad,shift", [(333, 0, 1), (500, 3, 0), (4099, 5, 2), (32001, 0, 0), (32000, 7, 3)])
def test_strides_in_place_and_elsewhere(dtype, V, pad, shift):
    x = _logits(11, V, dtype, 4, pad, shift)
    case = _case(x, 5)
    want = _check(x, *case)
    out = torch.empty(11, V + 9, dtype=dtype, device="cuda")[:, 3:3 + V]
    got = _check(x, *case, dlogits=out)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    got = _check(x, *case, dlogits=x)
    assert got[3] is x and all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("low", ["inf", "lowest"])
def test_masks(dtype, low):
    """Most entries masked, by -inf or the lowest value; a row with one left, one with none."""
    x = _logits(12, 5003, dtype, 6)
    v = -math.inf if low == "inf" else torch.finfo(dtype).min
    x[torch.rand(12, 5003, generator=_gen(7), device="cuda") < 0.9] = v
    x[3] = v
    x[3, 77] = 1.0
    tokens, old, A, ref, w = _case(x, 8)
    if low == "lowest":
        x[5] = v
        old[5], ref[5] = math.log(1 / 5003), math.log(1 / 5000)
    _check(x, tokens, old, A, ref, w)


def test_a_row_of_nothing():
    """-inf throughout: gradient 0; ratio 0 and an infinite KL term."""
    x = torch.full((3, 400), -math.inf, dtype=BF16, device="cuda")
    x[0] = 0
    tokens = torch.tensor([3, 3, -1], device="cuda")
    old = torch.full((3,), -6.0, device="cuda")
    one = torch.ones(3, device="cuda")
    loss, logp, kl, grad = agoq.agoq_policy_loss(x, tokens, old, one)
    assert float(logp[1]) == -math.inf and float(loss[1]) == 0 and not grad[1:].any() and kl is None
    loss, _, kl, grad = agoq.agoq_policy_loss(x, tokens, old, one, ref_logp=old, kl_coef=0.1)
    assert float(kl[1]) == math.inf and float(loss[1]) == math.inf and not grad[1:].any()
    assert float(loss[2]) == 0 and float(kl[2]) == 0


def test_a_token_of_no_probability():
    x = _logits(4, 300, F32, 9)
    x[:, 5] = -math.inf
    tokens = torch.tensor([5, 5, 6, -3], device="cuda")
    old, one = torch.full((4,), -5.0, device="cuda"), torch.ones(4, device="cuda")
    loss, logp, _, grad = agoq.agoq_policy_loss(x, tokens, old, one)
    assert logp[:2].tolist() == [-math.inf] * 2 and loss[:2].tolist() == [0, 0] and not grad[:2].any()
    assert torch.isfinite(grad[2]).all() and grad[2].any() and not grad[3].any()
    loss, _, kl, grad = agoq.agoq_policy_loss(x, tokens, old, one, ref_logp=old, kl_coef=1.0)
    assert kl[:2].tolist() == [math.inf] * 2 and torch.isnan(grad[:2]).all()
    # reported, with no coefficient: it takes no part
    loss, _, kl, grad = agoq.agoq_policy_loss(x, tokens, old, one, ref_logp=old)
    assert kl[:2].tolist() == [math.inf] * 2 and loss[:2].tolist() == [0, 0] and not grad[:2].any()


@pytest.mark.parametrize("V", [50, 3000, 131072, 1000003])
def test_tokens_outside_and_not_finite(V):
    x = _logits(7, V, BF16, 10)
    x[4, V // 2], x[5, V - 1] = math.nan, math.inf
    tokens = torch.tensor([V, -7, 1 << 40, V - 1, 0, 1, -1], device="cuda")
    old, one = torch.full((7,), -3.0, device="cuda"), torch.ones(7, device="cuda")
    loss, logp, kl, grad = agoq.agoq_policy_loss(x, tokens, old, one, ref_logp=old, kl_coef=0.1)
    for v in (loss, logp, kl):
        assert torch.isnan(v[[0, 2, 4, 5]]).all() and torch.isfinite(v[[1, 3, 6]]).all()
        assert v[[1, 6]].tolist() == [0, 0]
    assert torch.isnan(grad[[0, 2, 4, 5]]).all() and not grad[[1, 6]].any()
    assert torch.isfinite(grad[3]).all()
    zero = torch.zeros(7, device="cuda")        # a weight of 0 hides no NaN
    _, _, _, grad = agoq.agoq_policy_loss(x, tokens, old, one, weights=zero)
    assert torch.isnan(grad[[0, 2, 4, 5]]).all() and not grad[[1, 3, 6]].any()


def test_statistics_that_are_not_finite():
    x = _logits(6, 1000, F32, 11)
    tokens = torch.arange(6, device="cuda")
    lp = agoq.agoq_token_logprobs(x, tokens)[0]
    old, A, ref = lp.clone(), torch.ones(6, device="cuda"), lp.clone()
    old[0], A[1], ref[2] = math.nan, math.nan, math.nan
    old[3], A[3] = -1000.0, -1.0                 # a ratio beyond binary32, not clipped
    ref[4] = 200.0                               # e^d beyond binary32
    old[5], A[5] = -1000.0, 1.0                  # the same ratio, clipped
    loss, logp, kl, grad = agoq.agoq_policy_loss(x, tokens, old, A, ref_logp=ref, kl_coef=0.1)
    assert torch.isnan(loss[:3]).all() and torch.isnan(grad[:5]).all()
    assert loss[3:5].tolist() == [math.inf, math.inf] and torch.isfinite(grad[5]).all()
    assert torch.isfinite(logp).all() and abs(float(loss[5]) + 1.2) < 1e-5


def test_bounds_of_the_ratio():
    """All of the four sides: the clipped ones have the gradient of the KL term alone."""
    x = _logits(4, 500, F32, 12)
    tokens = torch.arange(4, device="cuda")
    lp = agoq.agoq_token_logprobs(x, tokens)[0]
    step = torch.tensor([0.5, 0.5, -0.5, -0.5], device="cuda")
    A = torch.tensor([2.0, -2.0, 2.0, -2.0], device="cuda")
    loss, _, _, grad = agoq.agoq_policy_loss(x, tokens, lp - step, A, clip_low=0.2, clip_high=0.3)
    e, f = math.exp(0.5), math.exp(-0.5)
    want = torch.tensor([-2 * 1.3, 2 * e, -2 * f, 2 * 0.8], device="cuda")
    assert torch.allclose(loss, want, rtol=3e-6)
    assert not grad[0].any() and not grad[3].any() and grad[1].any() and grad[2].any()
    _check(x, tokens, lp - step, A, None, None, 0.2, 0.3)
    # clip_low 1: the ratio has no lower bound
    _, _, _, grad = agoq.agoq_policy_loss(x, tokens, lp - step, A, clip_low=1.0, clip_high=0.3)
    assert grad[3].any()


def test_gradient_against_differences():
    """Of the loss's own values in binary64: the formula's gradient is that of the formula."""
    g = torch.Generator().manual_seed(13)
    x = torch.randn(5, 30, generator=g).double()
    tokens = torch.tensor([1, 5, -1, 20, 29])
    old = torch.log_softmax(x, 1).gather(1, tokens.clamp(min=0)[:, None]).squeeze(1) - torch.tensor(
        [0.5, -0.5, 0.1, 0.05, -0.1]).double()
    A, ref, w = (torch.randn(5, generator=g).double() for _ in range(3))
    ref = old + ref
    f = lambda z: float(Q.policy(z, tokens, old, A, ref, w, 0.8, 1.25, 0.3)[0].sum())
    grad = Q.policy(x, tokens, old, A, ref, w, 0.8, 1.25, 0.3)[4]
    h = 1e-6
    for t, i in ((0, 1), (0, 3), (1, 5), (1, 6), (2, 1), (3, 20), (3, 0), (4, 29), (4, 28)):
        up, down = x.clone(), x.clone()
        up[t, i] += h
        down[t, i] -= h
        assert abs((f(up) - f(down)) / (2 * h) - float(grad[t, i])) < 1e-8
    got = agoq.agoq_policy_loss(x.float().cuda(), tokens.cuda(), old.float().cuda(), A.float().cuda(),
                                ref.float().cuda(), w.float().cuda(), 0.2, 0.25, 0.3)[3]
    assert float((got.cpu().double() - grad).abs().max()) < 1e-5


def test_small_and_large_divergences():
    """kl where its terms cancel, and where they do not."""
    x = _logits(40, 200, F32, 14)
    tokens = torch.arange(40, device="cuda")
    lp = agoq.agoq_token_logprobs(x, tokens)[0]
    d = torch.cat([torch.logspace(-5, 1.5, 20), -torch.logspace(-5, 1.5, 20)]).cuda()
    _check(x, tokens, lp, torch.ones(40, device="cuda"), lp + d, None, coef=0.5)


def test_nothing_outside_the_outputs():
    T, V = 13, 1003
    x = _logits(T, V, F16, 15)
    tokens, old, A, ref, w = _case(x, 16)
    outs = [Guarded(4 * T, F32) for _ in range(3)]
    grad = Guarded(2 * T * V, F16)
    _check(x, tokens, old, A, ref, w, loss=outs[0].view, logp=outs[1].view, kl=outs[2].view,
           dlogits=grad.view.view(T, V))
    assert all(o.intact() for o in outs + [grad])
    x3 = x.reshape(T, 1, V)
    assert agoq.agoq_policy_loss(x3, tokens, old, A)[3].shape == x3.shape


def test_as_the_token_loss():
    """Advantage 1, ratio 1: the token loss's own bits."""
    x = _logits(300, 32000, BF16, 17)
    tokens = torch.randint(0, 32000, (300,), generator=_gen(18), device="cuda")
    logp, want = agoq.agoq_token_loss(x, tokens)
    loss, lp, _, grad = agoq.agoq_policy_loss(x, tokens, logp, torch.ones(300, device="cuda"))
    assert torch.equal(lp, logp) and torch.equal(grad, want) and bool((loss == -1).all())


def test_policy_streams_and_graph():
    x = _logits(20, 5000, BF16, 19)
    case = _case(x, 20)
    call = lambda **kw: agoq.agoq_policy_loss(x, *case[:3], ref_logp=case[3], weights=case[4], kl_coef=0.1, **kw)
    want = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    x.copy_(x * 0.5)
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(got, call()))


def test_policy_refusals():
    x = _logits(4, 50, BF16, 21)
    tokens, old, A, ref, w = _case(x, 22)
    with pytest.raises(agoq.AgoqError):
        agoq.agoq_policy_loss(x, tokens, old, A, kl_coef=0.1)
    with pytest.raises(agoq.AgoqError):
        agoq.agoq_policy_loss(x, tokens, old, A, kl=torch.empty(4, device="cuda"))
    with pytest.raises(agoq.AgoqError):
        agoq.agoq_policy_loss(x, tokens, old, A, clip_low=1.5)
    with pytest.raises(TypeError):
        agoq.agoq_policy_loss(x, tokens.int(), old, A)
    with pytest.raises(ValueError):
        agoq.agoq_policy_loss(x, tokens, old[:3], A)
    with pytest.raises(TypeError):
        agoq.agoq_policy_loss(x, tokens, old.double(), A)
    with pytest.raises(agoq.AgoqError):
        agoq.agoq_policy_loss(x[:, :40], tokens, old, A, dlogits=x[:, 2:42])
    e = x[:0]
    none = torch.empty(0, device="cuda")
    assert agoq.agoq_policy_loss(e, tokens[:0], none, none)[3].shape == (0, 50)


# ---- preference -----------------------------------------------------------------------------


def _pairs(lengths, tail, seed, shift=0, ref_shift=None):
    g = _gen(seed)
    T = sum(lengths) + tail
    offsets = [0]
    for n in lengths:
        offsets.append(offsets[-1] + n)

    def placed(v, s):
        buf = torch.full((T + s + 8,), 9.0, device="cuda")
        buf[s:s + T] = v
        return buf[s:s + T]
    logp = -torch.empty(T, device="cuda").exponential_(1.0, generator=g)
    ref = placed(logp + 0.3 * torch.randn(T, generator=g, device="cuda"), shift if ref_shift is None else ref_shift)
    return placed(logp, shift), ref, offsets


def _check_pairs(logp, ref, offsets, w=None, beta=0.1, eps=0.0, **kw):
    o = torch.tensor(offsets, device="cuda")
    wt = None if w is None else torch.tensor(w, device="cuda", dtype=F32)
    got = agoq.agoq_preference_loss(logp, o, ref_logp=ref, weights=wt, beta=beta, label_smoothing=eps, **kw)
    n = len(offsets) // 2
    ws = [1.0] * n if w is None else wt.double().tolist()
    f = lambda v: float(torch.tensor(v, dtype=F32))
    args = (logp.double(), None if ref is None else ref.double(), offsets, ws, f(beta), f(eps))
    loss, margin, grad = Q.preference(*args)
    bl, bm, bg = Q.preference_bounds(*args, margin)
    _close(got[0], loss, bl, "loss")
    _close(got[1], margin, bm, "margin")
    for p in range(n):
        a, c = offsets[2 * p], offsets[2 * p + 2]
        assert bool(((got[2][a:c].double() - grad[a:c]).abs() <= bg[p]).all()), p
    return got


@pytest.mark.parametrize("lengths", [(1, 1), (0, 1), (1, 0), (0, 0), (3, 5, 0, 0, 7, 2), (1000, 900),
                                     (5000, 1), (1, 5000), (31, 33) * 50, (40000, 50001), (9, 4000, 0, 1),
                                     (300000, 200000)])
@pytest.mark.parametrize("shift", [0, 1])
def test_pairs(lengths, shift):
    logp, ref, offsets = _pairs(lengths, 5, 1, shift)
    for r, eps in ((ref, 0.0), (ref, 0.2), (None, 0.0)):
        _check_pairs(logp if r is not None else logp * 0.01, r, offsets, eps=eps)


def test_vectors_at_different_alignments():
    for a, b in ((0, 1), (1, 0), (2, 3), (3, 3)):
        logp, ref, offsets = _pairs((700, 900, 11, 12), 3, 2, a, b)
        w = [0.5, 2.0]
        out = torch.zeros(len(logp) + 7, device="cuda")[1:1 + len(logp)]
        _check_pairs(logp, ref, offsets, w, beta=0.3, dlogp=out)


def test_many_pairs_and_the_same_bits_again():
    g = torch.Generator().manual_seed(3)
    lengths = torch.randint(0, 60, (6000,), generator=g).tolist()
    logp, ref, offsets = _pairs(lengths, 0, 4)
    got = _check_pairs(logp, ref, offsets, eps=0.1)
    again = agoq.agoq_preference_loss(logp, torch.tensor(offsets, device="cuda"), ref_logp=ref,
                                      label_smoothing=0.1)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


def test_rows_of_no_answer_stay():
    logp, ref, _ = _pairs((30, 30), 10, 5)
    o = torch.tensor([4, 20, 41], device="cuda")
    out = Guarded(4 * 70, F32)
    out.view.fill_(3.0)
    _check_pairs(logp, ref, [4, 20, 41], dlogp=out.view)
    assert bool((out.view[:4] == 3).all()) and bool((out.view[41:] == 3).all()) and out.intact()
    made = agoq.agoq_preference_loss(logp, o, ref_logp=ref)[2]
    assert not made[:4].any() and not made[41:].any()


def test_margins_of_any_size():
    """Losses near 0 and far from it, and where e^h leaves binary32."""
    T = 12
    for d in (0.0, 1e-6, 5.0, 30.0, 80.0, 200.0, 5000.0):
        for sign in (1, -1):
            logp = torch.zeros(T, device="cuda")
            logp[:6], logp[6:] = sign * d / 12, -sign * d / 12
            _check_pairs(logp, None, [0, 6, 12], beta=1.0)
            _check_pairs(logp, None, [0, 6, 12], beta=1.0, eps=0.3)


def test_answers_that_are_not_finite():
    logp, ref, offsets = _pairs((5, 5) * 4, 0, 6)
    logp[1], logp[17], logp[22] = -math.inf, -math.inf, math.nan     # chosen 0, rejected 1, chosen 2
    loss, margin, dlogp = agoq.agoq_preference_loss(logp, torch.tensor(offsets, device="cuda"), ref_logp=ref)
    assert loss[:2].tolist() == [math.inf, 0.0] and margin[:2].tolist() == [-math.inf, math.inf]
    assert math.isnan(float(loss[2])) and math.isnan(float(margin[2])) and math.isfinite(float(loss[3]))
    assert torch.allclose(dlogp[:5], torch.full((5,), -0.1, device="cuda")) and not dlogp[10:20].any()
    assert torch.isnan(dlogp[20:30]).all() and torch.isfinite(dlogp[30:]).all()


def test_offsets_that_are_none():
    """Descending or outside: loss NaN, nothing written for that pair, the others as ever."""
    logp, ref, _ = _pairs((10, 10), 80, 7)
    for bad in ([0, 10, 20, 15, 30, 40, 50], [0, 10, 20, 30, 101, 60, 70], [-5, 3, 8, 20, 30, 40, 50],
                [0, 10, 20, 30, 40, 50, 1 << 50]):
        out = torch.full((100,), 2.0, device="cuda")
        o = torch.tensor(bad, device="cuda")
        loss, margin, _ = agoq.agoq_preference_loss(logp, o, ref_logp=ref, dlogp=out)
        touched = torch.zeros(100, dtype=torch.bool)
        for p in range(3):
            a, b, c = bad[2 * p:2 * p + 3]
            good = 0 <= a <= b <= c <= 100
            assert math.isnan(float(loss[p])) != good and math.isnan(float(margin[p])) != good
            if good:
                touched[a:c] = True
        assert torch.equal((out != 2).cpu(), touched)


def test_with_the_calls_around_it():
    """Log probabilities, the loss, their gradient: against binary64 autograd from the logits."""
    T, V = 60, 500
    x = _logits(T, V, F32, 23)
    g = _gen(24)
    tokens = torch.randint(0, V, (T,), generator=g, device="cuda")
    tokens[::7] = -100
    ref = torch.where(tokens < 0, 0.0, -torch.rand(T, generator=g, device="cuda") * 8)
    offsets = [0, 11, 25, 25, 47]
    logp, _, lse, _, _ = agoq.agoq_token_logprobs(x, tokens)
    loss, _, dlogp = agoq.agoq_preference_loss(logp, torch.tensor(offsets, device="cuda"), ref_logp=ref, beta=0.2)
    got = agoq.agoq_token_logprobs_backward(x, tokens, lse, dlogp)
    leaf = x.double().requires_grad_()
    lp = torch.log_softmax(leaf, 1).gather(1, tokens.clamp(min=0)[:, None]).squeeze(1)
    lp = torch.where(tokens < 0, 0.0, lp) - ref.double()
    h = torch.stack([lp[a:b].sum() - lp[b:c].sum() for a, b, c in ((0, 11, 25), (25, 25, 47))])
    want = -torch.nn.functional.logsigmoid(0.2 * h)
    want.sum().backward()
    assert torch.allclose(loss.double(), want, rtol=1e-5, atol=1e-6)
    assert float((got.double() - leaf.grad).abs().max()) < 1e-6


def test_preference_streams_and_graph():
    logp, ref, offsets = _pairs((300, 5000, 70, 80), 4, 8)
    o = torch.tensor(offsets, device="cuda")
    want = agoq.agoq_preference_loss(logp, o, ref_logp=ref)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = agoq.agoq_preference_loss(logp, o, ref_logp=ref, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = agoq.agoq_preference_loss(logp, o, ref_logp=ref)
    logp.mul_(0.9)
    o[2] += 3
    graph.replay()
    want = agoq.agoq_preference_loss(logp, o, ref_logp=ref)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_preference_refusals():
    logp = torch.zeros(10, device="cuda")
    o = torch.tensor([0, 3, 6], device="cuda")
    with pytest.raises(ValueError):
        agoq.agoq_preference_loss(logp, o[:2])
    with pytest.raises(TypeError):
        agoq.agoq_preference_loss(logp, o.int())
    with pytest.raises(TypeError):
        agoq.agoq_preference_loss(logp.half(), o)
    with pytest.raises(ValueError):
        agoq.agoq_preference_loss(logp, o, ref_logp=logp[:5])
    with pytest.raises(agoq.AgoqError):
        agoq.agoq_preference_loss(logp, o, dlogp=logp)
    with pytest.raises(agoq.AgoqError):
        agoq.agoq_preference_loss(logp, o, beta=-1.0)
    with pytest.raises(TypeError):
        agoq.agoq_preference_loss(logp.cpu(), o)
    loss, margin, dlogp = agoq.agoq_preference_loss(logp, o[:1])
    assert loss.numel() == 0 and not dlogp.any()
