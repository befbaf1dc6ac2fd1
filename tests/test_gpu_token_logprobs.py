"""Token log probabilities, their gradient and the loss on the GPU against the
plain binary64 forms (tests/plain64.py holds the formulas and the bounds): types,
vocabularies of one entry to long odd ones, strides and alignments, masks that
leave a few entries or none, ties, non-finite logits, tokens outside, in place,
streams and graphs."""
import math

import pytest
import torch

from gradient_quantization_gb300 import agoq
from tests import plain64 as P
from tests.gpu_util import Guarded

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def _logits(T, V, dtype, seed, scale=3.0, pad=0, shift=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    buf = torch.full((T * (V + pad) + shift + 16,), 50.0, dtype=dtype, device="cuda")
    x = buf[shift:shift + T * (V + pad)].view(T, V + pad)[:, :V]
    x.copy_(scale * torch.randn(T, V, generator=g, device="cuda"))
    return x


def _tokens(T, V, seed=5):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(0, V, (T,), generator=g).cuda()


def _close(got, want, bound, what):
    """Equal where the exact value is not finite, within the bound elsewhere."""
    beyond = want.abs() > torch.finfo(got.dtype).max       # rounds to an infinity
    want = torch.where(beyond, want.sign() * math.inf, want)
    got = got.double()
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), what
    off = (got - want).abs()[fine]
    b = bound[fine]
    assert bool((off <= b).all()), (what, float((off / b).max()))


def _check(x, tokens, k):
    _check_rows(x, tokens, k, slice(None), agoq.agoq_token_logprobs(x, tokens, k=k))


def _check_rows(x, tokens, k, rows, got):
    logp, ent, lse, top_logp, top_ids = (v if v is None else v[rows] for v in got)
    x, tokens = x[rows], tokens[rows]
    x64 = x.double()
    ep, ee, el, logs = P.token_logprobs(x64, tokens)
    blogp, bent, blse = P.token_bounds(x64, logs, el)
    at = tokens.clamp(0, x.shape[1] - 1)[:, None]
    _close(logp, ep, blogp.gather(1, at).squeeze(1), "logp")
    _close(ent, ee, bent, "entropy")
    _close(lse, el, blse, "lse")
    if k:
        ids = P.top(x64, k)
        assert torch.equal(top_ids, ids)
        _close(top_logp, logs.gather(1, ids), blogp.gather(1, ids), "top_logp")
    else:
        assert top_logp is None and top_ids is None


VOCABS = [(3, 1), (5, 2), (4, 7), (9, 33), (3, 257), (2, 1000), (7, 4099), (5, 32000), (3, 32003),
          (2, 50001), (1, 131072), (2, 131073), (1, 300001), (600, 130), (1, 8)]


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("T,V", VOCABS)
def test_values_and_alternatives(dtype, T, V):
    _check(_logits(T, V, dtype, 1), _tokens(T, V), min(V, (0, 1, 5, 20, 32)[(T + V) % 5]))


# Around the lengths at which a warp holds more vectors, or a CTA takes the row, from any
# start; the rows differ in kind: masked, equal, ascending, with one NaN or +inf.
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("V", [3, 31, 63, 250, 256, 505, 509, 1017, 1018, 2033, 2041, 2042, 4081,
                               4082, 4090])
@pytest.mark.parametrize("pad,shift", [(0, 0), (3, 1)])
def test_short_rows(dtype, V, pad, shift):
    x = _logits(70, V, dtype, 41, pad=pad, shift=shift)
    x[1] = -math.inf
    x[2, V // 3:] = -math.inf
    x[3, ::2] = torch.finfo(dtype).min
    x[4] = 1.5
    x[5] = torch.arange(V, device="cuda").div(64, rounding_mode="floor").to(dtype)
    x[6, V // 2] = math.nan
    x[7, V - 1] = math.inf
    tokens = _tokens(70, V)
    tokens[2], tokens[8] = 0, -100
    good = [i for i in range(70) if i not in (6, 7)]
    for k in {0, 1, min(V, 17), min(V, 32)}:
        got = agoq.agoq_token_logprobs(x, tokens, k=k)
        assert all(bool(torch.isnan(v[6:8]).all()) for v in got[:3])
        if k:
            assert torch.equal(got[4][6:8], P.top(x[6:8].double(), k))
        _check_rows(x, tokens, k, good, got)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("V", [1, 2041, 2042, 4090, 8190, 16380])
@pytest.mark.parametrize("pad,shift", [(0, 0), (5, 3)])
def test_loss_of_short_rows(dtype, V, pad, shift):
    x, tokens = _logits(300, V, dtype, 42, pad=pad, shift=shift), _tokens(300, V)
    x[1, V // 3:] = -math.inf
    tokens[1], tokens[2] = 0, -100
    w = torch.rand(300, device="cuda") + 0.1
    _check_loss(x, tokens, w, *agoq.agoq_token_loss(x, tokens, w))


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("T,V", VOCABS)
def test_loss_and_gradient(dtype, T, V):
    x, tokens = _logits(T, V, dtype, 2), _tokens(T, V)
    if T > 2:
        tokens[1] = -100
    w = torch.rand(T, device="cuda") + 0.1
    logp, grad = agoq.agoq_token_loss(x, tokens, w)
    _check_loss(x, tokens, w, logp, grad)


def _check_loss(x, tokens, w, logp, grad):
    x64 = x.double()
    ep, _, el, logs = P.token_logprobs(x64, tokens)
    blogp, _, _ = P.token_bounds(x64, logs, el)
    _close(logp, ep, blogp.gather(1, tokens.clamp(0, x.shape[1] - 1)[:, None]).squeeze(1), "logp")
    want = P.loss_gradient(logs, tokens, w.double())
    _close(grad, want, P.loss_bound(x64, logs, el, w.double(), want, x.dtype), "gradient")


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("T,V", VOCABS)
def test_gradient_of_the_statistics(dtype, T, V):
    x, tokens = _logits(T, V, dtype, 3), _tokens(T, V)
    if T > 2:
        tokens[0] = -1
    _, ent, lse, _, _ = agoq.agoq_token_logprobs(x, tokens)
    g = torch.Generator(device="cuda").manual_seed(9)
    dl, de = (torch.randn(T, generator=g, device="cuda") for _ in range(2))
    for e, d in ((None, None), (ent, de)):
        grad = agoq.agoq_token_logprobs_backward(x, tokens, lse, dl, e, d)
        _check_backward(x, tokens, lse, dl, e, d, grad)


def _check_backward(x, tokens, lse, dl, ent, de, grad):
    d = lambda t: None if t is None else t.double()
    x64 = x.double()
    want = P.token_logprobs_backward(x64, tokens, d(lse), d(dl), d(ent), d(de))
    _close(grad, want, P.logprobs_backward_bound(x64, d(lse), d(dl), d(ent), d(de), want, x.dtype),
           "gradient")


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("V,pad,shift,pad_out,shift_out", [
    (1000, 8, 0, 8, 0), (1000, 3, 0, 0, 0), (1001, 0, 1, 0, 1), (32000, 5, 3, 8, 0),
    (40001, 7, 0, 7, 8), (999, 1, 2, 4, 5)])
def test_strides_and_alignment(dtype, V, pad, shift, pad_out, shift_out):
    T = 6
    x, tokens = _logits(T, V, dtype, 4, pad=pad, shift=shift), _tokens(T, V)
    _check(x, tokens, 7)
    w = torch.rand(T, device="cuda")
    _, ent, lse, _, _ = agoq.agoq_token_logprobs(x, tokens)
    dl, de = torch.rand(T, device="cuda"), torch.rand(T, device="cuda")
    for call in ("loss", "backward"):
        out = _logits(T, V, dtype, 5, pad=pad_out, shift=shift_out)
        whole = out.as_strided((T, V + pad_out), (V + pad_out, 1), out.storage_offset())
        if call == "loss":
            logp, grad = agoq.agoq_token_loss(x, tokens, w, dlogits=out)
            _check_loss(x, tokens, w, logp, grad)
        else:
            grad = agoq.agoq_token_logprobs_backward(x, tokens, lse, dl, ent, de, dlogits=out)
            _check_backward(x, tokens, lse, dl, ent, de, grad)
        assert grad is out and bool((whole[:, V:] == 50).all())


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("V", [40, 5000, 32000, 140001])
@pytest.mark.parametrize("low", ["inf", "lowest"])
def test_masks(dtype, V, low):
    """Rows with all but few entries masked, with one left, with none, and half masked."""
    x = _logits(6, V, dtype, 6)
    value = -math.inf if low == "inf" else torch.finfo(dtype).min
    keep = torch.zeros(6, V, dtype=torch.bool, device="cuda")
    keep[0, [V - 1, 3, V // 2]] = True
    keep[1, V - 2] = True
    keep[3, ::2] = True
    keep[4, :] = True
    keep[5, -5:] = True
    x[~keep] = value
    tokens = torch.tensor([3, V - 2, 7, 1, -1, V - 1]).cuda()
    _check(x, tokens, 20)
    w = torch.ones(6, device="cuda")
    logp, grad = agoq.agoq_token_loss(x, tokens, w)
    _check_loss(x, tokens, w, logp, grad)
    if low == "inf":
        assert not grad[2].any()
    _, ent, lse, _, _ = agoq.agoq_token_logprobs(x, tokens)
    _check_backward(x, tokens, lse, w, ent, w,
                    agoq.agoq_token_logprobs_backward(x, tokens, lse, w, ent, w))


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("V", [64, 6000, 32000, 131072])
def test_ties_and_orders(dtype, V):
    """Equal logits everywhere, few distinct values, signed zeros, sorted rows, and the largest
    ones side by side."""
    x = torch.empty(8, V, device="cuda")
    x[0] = 1.25
    x[1] = torch.arange(V, device="cuda") % 3
    x[2] = torch.where(torch.arange(V, device="cuda") % 2 == 0, 0.0, -0.0)
    x[3] = torch.linspace(-8, 8, V, device="cuda")
    x[4] = torch.linspace(8, -8, V, device="cuda")
    x[5] = torch.randn(V, device="cuda")
    x[5, V // 3:V // 3 + 40] = 9.0
    x[6] = torch.randn(V, device="cuda")
    x[6, -33:] = torch.linspace(9, 11, 33, device="cuda")
    x[7] = -5.0
    x[7, V // 2:V // 2 + 30] = torch.arange(30, device="cuda") * 1.0
    _check(x.to(dtype), _tokens(8, V), 32)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V", [500, 32000, 131072])
def test_not_finite(dtype, V):
    x = _logits(5, V, dtype, 8)
    x[1, V // 2] = math.nan
    x[2, 7] = math.inf
    x[3, [5, V - 1]] = math.nan
    tokens = torch.tensor([1, 2, 7, 5, 0]).cuda()
    logp, ent, lse, top_logp, ids = agoq.agoq_token_logprobs(x, tokens, k=4)
    for v in (logp, ent):
        assert torch.isfinite(v[[0, 4]]).all() and torch.isnan(v[1:4]).all()
    assert torch.isfinite(lse[[0, 4]]).all() and not torch.isfinite(lse[1:4]).any()
    assert int(ids[1, 0]) == V // 2 and ids[3, :2].tolist() == [5, V - 1] and int(ids[2, 0]) == 7
    clean = x.clone()
    clean[1, V // 2] = clean[2, 7] = clean[3, 5] = clean[3, V - 1] = -math.inf
    rest = P.top(clean.double(), 4)
    assert torch.equal(ids[1, 1:], rest[1, :3]) and torch.equal(ids[3, 2:], rest[3, :2])
    assert torch.equal(ids[[0, 4]], rest[[0, 4]]) and torch.equal(ids[2, 1:], rest[2, :3])
    _, grad = agoq.agoq_token_loss(x, tokens, torch.ones(5, device="cuda"))
    assert torch.isfinite(grad[[0, 4]]).all() and torch.isnan(grad[1]).any()


def test_large_magnitudes():
    x = _logits(4, 3000, F32, 9, scale=1.0)
    x[0] *= 1e4
    x[1] += 3e38
    x[2] -= 3e38
    x[3] = -3.0e38
    x[3, 17] = 3.0e38
    _check(x, torch.tensor([0, 1, 2, 17]).cuda(), 3)


def test_tokens_outside():
    x = _logits(4, 100, BF16, 10)
    tokens = torch.tensor([100, -7, 1 << 40, 99]).cuda()
    _check(x, tokens, 3)
    w = torch.ones(4, device="cuda")
    logp, grad = agoq.agoq_token_loss(x, tokens, w)
    _check_loss(x, tokens, w, logp, grad)
    assert torch.isnan(grad[0]).all() and not grad[1].any()
    _, ent, lse, _, _ = agoq.agoq_token_logprobs(x, tokens)
    _check_backward(x, tokens, lse, w, None, None,
                    agoq.agoq_token_logprobs_backward(x, tokens, lse, w))


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("V,pad", [(333, 0), (32000, 0), (32001, 3), (140000, 0), (400000, 0)])
def test_in_place(dtype, V, pad):
    T = 5
    x, tokens = _logits(T, V, dtype, 11, pad=pad), _tokens(T, V)
    logp, ent, lse, _, _ = agoq.agoq_token_logprobs(x, tokens)
    w = torch.rand(T, device="cuda")
    z = x.clone() if not pad else _logits(T, V, dtype, 11, pad=pad)
    lp, want = agoq.agoq_token_loss(x, tokens, w)
    lp2, got = agoq.agoq_token_loss(z, tokens, w, dlogits=z)
    assert got is z and torch.equal(z, want) and torch.equal(lp, lp2)
    z = x.clone()
    want = agoq.agoq_token_logprobs_backward(x, tokens, lse, w, ent, w)
    assert torch.equal(agoq.agoq_token_logprobs_backward(z, tokens, lse, w, ent, w, dlogits=z),
                       want)


def test_nothing_outside_the_outputs():
    T, V, k = 11, 1003, 6
    x, tokens = _logits(T, V, F16, 12), _tokens(T, V)
    outs = [Guarded(4 * T, F32) for _ in range(3)]
    top, ids = Guarded(4 * T * k, F32), Guarded(8 * T * k, torch.int64)
    agoq.agoq_token_logprobs(x, tokens, k, logp=outs[0].view, entropy=outs[1].view,
                             lse=outs[2].view, top_logp=top.view.view(T, k),
                             top_ids=ids.view.view(T, k))
    grad, lp = Guarded(2 * T * V, F16), Guarded(4 * T, F32)
    agoq.agoq_token_loss(x, tokens, None, logp=lp.view, dlogits=grad.view.view(T, V))
    assert all(g.intact() for g in outs + [top, ids, grad, lp])
    _check_loss(x, tokens, torch.ones(T, device="cuda"), lp.view, grad.view.view(T, V))


def test_weights_and_optional_outputs():
    x, tokens = _logits(7, 500, BF16, 13), _tokens(7, 500)
    _, g1 = agoq.agoq_token_loss(x, tokens)
    _, g2 = agoq.agoq_token_loss(x, tokens, torch.ones(7, device="cuda"))
    assert torch.equal(g1, g2)
    logp, ent, lse, _, _ = agoq.agoq_token_logprobs(x, tokens, want_entropy=False)
    assert ent is None
    want = agoq.agoq_token_logprobs(x, tokens)
    assert torch.equal(logp, want[0]) and torch.equal(lse, want[2])
    x3 = x.view(7, 1, 500)
    assert agoq.agoq_token_loss(x3, tokens)[1].shape == x3.shape


def test_no_rows():
    x = torch.empty(0, 50, dtype=BF16, device="cuda")
    t = torch.empty(0, dtype=torch.int64, device="cuda")
    assert agoq.agoq_token_logprobs(x, t, k=3)[3].shape == (0, 3)
    assert agoq.agoq_token_loss(x, t)[1].shape == (0, 50)


def test_many_rows_and_the_same_bits_again():
    x, tokens = _logits(5000, 700, BF16, 14), _tokens(5000, 700)
    _check(x, tokens, 5)
    w = torch.rand(5000, device="cuda")
    logp, grad = agoq.agoq_token_loss(x, tokens, w)
    _check_loss(x, tokens, w, logp, grad)
    again = agoq.agoq_token_loss(x, tokens, w)
    assert torch.equal(logp, again[0]) and torch.equal(grad, again[1])


def test_offsets_beyond_32_bits():
    T, V, ld = 4, 3000, (1 << 30) + 8
    buf = torch.zeros(T * ld, dtype=BF16, device="cuda")
    x = buf.as_strided((T, V), (ld, 1))
    x.copy_(_logits(T, V, BF16, 15))
    tokens = _tokens(T, V)
    _check(x, tokens, 4)
    want = agoq.agoq_token_loss(x, tokens)[1]
    agoq.agoq_token_loss(x, tokens, dlogits=x)
    assert torch.equal(x, want)


def test_another_stream_and_a_graph():
    x, tokens = _logits(16, 5000, BF16, 16), _tokens(16, 5000)
    w = torch.rand(16, device="cuda")

    def step(stream=None):
        got = agoq.agoq_token_logprobs(x, tokens, k=6, stream=stream)
        return got + agoq.agoq_token_loss(x, tokens, w, stream=stream) + (
            agoq.agoq_token_logprobs_backward(x, tokens, got[2], w, got[1], w, stream=stream),)
    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = step(side)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = step()
    x.copy_(_logits(16, 5000, BF16, 17))
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(held, step()))


def test_binding_refusals():
    x, tokens = _logits(4, 50, BF16, 18), _tokens(4, 50)
    with pytest.raises(TypeError):
        agoq.agoq_token_logprobs(x, tokens.int())
    with pytest.raises(ValueError):
        agoq.agoq_token_logprobs(x, tokens[:3])
    with pytest.raises(agoq.AgoqError):
        agoq.agoq_token_logprobs(x, tokens, k=33)
    with pytest.raises(TypeError):
        agoq.agoq_token_loss(x, tokens, dlogits=torch.empty(4, 50, device="cuda"))
    with pytest.raises(ValueError):
        agoq.agoq_token_loss(x, tokens, dlogits=torch.empty(4, 51, dtype=BF16, device="cuda"))
    with pytest.raises(agoq.AgoqError):
        agoq.agoq_token_loss(x[:, :40], tokens, dlogits=x[:, 2:42])      # overlapping, not in place
