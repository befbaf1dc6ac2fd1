"""Refusals of the layer norm, gradient norm and token log probability calls: every
call below fails its host-side validation and launches nothing (CPU)."""
import ctypes

import pytest

from gradient_quantization_gb300 import agoq

OK, NULL, SHAPE, BITS, ALIGN, ALIAS, FORMAT = 0, 1, 2, 3, 4, 5, 8
F32, BF16, F16, E4M3 = 0, 1, 2, 3
A = 0x10000000          # fake addresses: never dereferenced on these paths
GAP = 1 << 24
f = ctypes.c_float


@pytest.fixture(scope="module")
def L():
    return agoq.lib()


def _at(i):
    return A + i * GAP


def _fwd(**over):
    a = dict(x=_at(0), ldx=256, w=_at(1), b=_at(2), pd=F32, T=8, H=256, dt=BF16, eps=1e-5, y=_at(3),
             ldy=256, mean=_at(4), rstd=_at(5), codes=0, scales=0, bits=0, stream=None)
    a.update(over)
    a["eps"] = f(a["eps"])
    return agoq.lib().agoq_layernorm_forward(*a.values())


@pytest.mark.parametrize("want,over", [
    (OK, dict(T=0, x=0, y=0)),
    (FORMAT, dict(dt=3)), (FORMAT, dict(dt=-1)), (FORMAT, dict(pd=F16)),
    (FORMAT, dict(dt=F32, pd=BF16)),
    (FORMAT, dict(dt=F16, pd=F32, codes=_at(6), scales=_at(7), bits=4)),
    (BITS, dict(codes=_at(6), scales=_at(7), bits=7)),
    (SHAPE, dict(T=-1)), (SHAPE, dict(H=0)), (SHAPE, dict(H=(1 << 24) + 1, ldx=1 << 25, ldy=1 << 25)),
    (SHAPE, dict(ldx=255)), (SHAPE, dict(ldy=100)), (SHAPE, dict(eps=-1.0)),
    (SHAPE, dict(eps=float("nan"))), (SHAPE, dict(T=1 << 62)),
    (SHAPE, dict(H=200, codes=_at(6), scales=_at(7), bits=4)),
    (NULL, dict(x=0)), (NULL, dict(y=0)), (NULL, dict(codes=_at(6), bits=4)),
    (NULL, dict(scales=_at(6), bits=4)),
    (ALIGN, dict(x=_at(0) + 1)), (ALIGN, dict(y=_at(3) + 1)), (ALIGN, dict(w=_at(1) + 2)),
    (ALIGN, dict(mean=_at(4) + 2)), (ALIGN, dict(codes=_at(6) + 4, scales=_at(7), bits=4)),
    (ALIAS, dict(y=_at(0) + 2)), (ALIAS, dict(y=_at(0), ldy=512)), (ALIAS, dict(mean=_at(0) + 16)),
    (ALIAS, dict(rstd=_at(4))), (ALIAS, dict(y=_at(1))), (ALIAS, dict(y=_at(0), mean=_at(0))),
    (ALIAS, dict(codes=_at(0), scales=_at(7), bits=4)),
])
def test_layernorm_forward(L, want, over):
    assert _fwd(**over) == want


def _bwd(**over):
    n = 1 << 30
    a = dict(x=_at(0), ldx=256, dy=_at(1), lddy=256, w=_at(2), pd=F32, mean=_at(3), rstd=_at(4),
             T=8, H=256, dt=BF16, dx=_at(5), lddx=256, dw=_at(6), db=_at(7), ws=_at(8), nws=n,
             stream=None)
    a.update(over)
    return agoq.lib().agoq_layernorm_backward(*a.values())


@pytest.mark.parametrize("want,over", [
    (OK, dict(T=0, dw=0, db=0)),
    (FORMAT, dict(dt=3)), (FORMAT, dict(pd=F16)),
    (SHAPE, dict(T=-1)), (SHAPE, dict(H=0)), (SHAPE, dict(lddy=8)), (SHAPE, dict(lddx=255)),
    (SHAPE, dict(nws=16)), (NULL, dict(ws=0)), (NULL, dict(mean=0)), (NULL, dict(dy=0)),
    (NULL, dict(dx=0)), (ALIGN, dict(ws=_at(8) + 8)), (ALIGN, dict(dw=_at(6) + 1)),
    (ALIAS, dict(dx=_at(0) + 256)), (ALIAS, dict(dw=_at(7))), (ALIAS, dict(ws=_at(6))),
    (ALIAS, dict(db=_at(1))), (ALIAS, dict(dx=_at(1), lddx=300)), (ALIAS, dict(dx=_at(3))),
])
def test_layernorm_backward(L, want, over):
    assert _bwd(**over) == want


def _laaq(**over):
    a = dict(codes=_at(0), scales=_at(1), bits=4, dy=_at(2), lddy=256, w=_at(3), pd=BF16, T=8,
             H=256, eps=1e-5, dx=_at(4), lddx=256, dw=_at(5), db=_at(6), ws=_at(7), nws=1 << 30,
             stream=None)
    a.update(over)
    a["eps"] = f(a["eps"])
    return agoq.lib().agoq_layernorm_backward_laaq(*a.values())


@pytest.mark.parametrize("want,over", [
    (BITS, dict(bits=0)), (BITS, dict(bits=7)), (FORMAT, dict(pd=F16)),
    (SHAPE, dict(H=192)), (SHAPE, dict(eps=-1.0)), (SHAPE, dict(nws=0)),
    (NULL, dict(scales=0)), (NULL, dict(codes=0)), (ALIGN, dict(codes=_at(0) + 8)),
    (ALIAS, dict(dx=_at(0))), (ALIAS, dict(dw=_at(1))), (OK, dict(T=0, dw=0, db=0)),
])
def test_layernorm_backward_laaq(L, want, over):
    assert _laaq(**over) == want


def test_layernorm_workspace(L):
    wb = L.agoq_layernorm_backward_workspace_bytes
    assert wb(0, 256) == 0
    assert wb(8, 256) == 8 * 2 * 256 * 4
    assert wb(100000, 4096) == 304 * 2 * 4096 * 4
    assert wb(-1, 256) == -1 and wb(8, 0) == -1 and wb(8, (1 << 24) + 1) == -1


def _tensor(data, n, dtype, out=None, scales=0):
    return agoq._GradTensor(data, scales, data if out is None else out, n, dtype, 0)


def _list(*tensors):
    return (agoq._GradTensor * max(1, len(tensors)))(*tensors)


@pytest.mark.parametrize("want,t", [
    (FORMAT, _tensor(_at(0), 5, 4)), (FORMAT, _tensor(_at(0), 5, -1)),
    (SHAPE, _tensor(_at(0), -1, F32)), (SHAPE, _tensor(_at(0), (1 << 40) + 1, F32)),
    (SHAPE, _tensor(_at(0), 100, E4M3, scales=_at(1))),
    (NULL, _tensor(0, 5, F32)), (NULL, _tensor(_at(0), 128, E4M3, out=_at(2))),
    (ALIGN, _tensor(_at(0) + 2, 5, F32)), (ALIGN, _tensor(_at(0) + 1, 5, BF16)),
    (ALIGN, _tensor(_at(0) + 8, 128, E4M3, out=_at(1), scales=_at(1))),
    (ALIGN, _tensor(_at(0), 128, E4M3, out=_at(2), scales=_at(1) + 2)),
])
def test_grad_tensor(L, want, t):
    for first in (False, True):
        l = _list(t) if first else _list(_tensor(_at(9), 3, F32), t)
        n = len(l)
        assert L.agoq_grad_list_check(l, n) == want
        assert L.agoq_grad_norm(l, n, _at(20), _at(21), 1 << 20, None) == want
        assert L.agoq_clip_grads(l, n, f(1.0), _at(20), None) == want
        assert L.agoq_clip_grad_norm(l, n, f(1.0), _at(20), _at(21), 1 << 20, None) == want


def test_grad_list_overlaps(L):
    ok = _list(_tensor(_at(0), 64, F32), _tensor(_at(0) + 256, 64, BF16, out=_at(1)),
               _tensor(_at(2), 256, E4M3, out=_at(3), scales=_at(3)), _tensor(0, 0, F16))
    assert L.agoq_grad_list_check(ok, 4) == OK
    assert L.agoq_grad_list_check(None, 0) == OK
    assert L.agoq_grad_list_check(None, 1) == NULL
    assert L.agoq_grad_list_check(ok, -1) == SHAPE
    for bad in (
            _list(_tensor(_at(0), 64, F32), _tensor(_at(0) + 252, 64, BF16)),
            _list(_tensor(_at(0), 64, F32, out=_at(1)), _tensor(_at(2), 64, F32, out=_at(1) + 128)),
            _list(_tensor(_at(0), 64, F32, out=_at(1)), _tensor(_at(1) + 4, 64, F32, out=_at(2))),
            _list(_tensor(_at(2), 256, E4M3, out=_at(3), scales=_at(4)),
                  _tensor(_at(5), 256, E4M3, out=_at(6), scales=_at(3) + 4)),
            # a long tensor that starts before several short ones
            _list(_tensor(_at(0), 1 << 20, F32, out=_at(1)), _tensor(_at(2), 4, F32, out=_at(3)),
                  _tensor(_at(1) + 4096, 4, F32, out=_at(4))),
            _list(_tensor(_at(0), 64, F32, out=_at(0) + 4), _tensor(_at(2), 4, F32))):
        assert L.agoq_grad_list_check(bad, len(bad)) == ALIAS
    assert L.agoq_clip_grads(_list(_tensor(_at(0), 64, F32, out=_at(0) + 4)), 1, f(1.0), _at(9),
                             None) == ALIAS


def test_grad_norm_arguments(L):
    l = _list(_tensor(_at(0), 64, F32))
    need = L.agoq_grad_norm_workspace_bytes(1)
    assert need == 1216 * 8 and L.agoq_grad_norm_workspace_bytes(0) == need
    assert L.agoq_grad_norm_workspace_bytes(1001) == 2 * need
    assert L.agoq_grad_norm_workspace_bytes(-1) == -1
    clip = L.agoq_clip_grad_norm
    assert L.agoq_grad_norm(l, 1, None, _at(9), need, None) == NULL
    assert L.agoq_grad_norm(l, 1, _at(8), None, need, None) == NULL
    assert L.agoq_grad_norm(l, 1, _at(8), _at(9), need - 8, None) == SHAPE
    assert L.agoq_grad_norm(l, 1, _at(8) + 2, _at(9), need, None) == ALIGN
    assert L.agoq_grad_norm(l, 1, _at(8), _at(9) + 8, need, None) == ALIGN
    assert L.agoq_grad_norm(l, 1, _at(0) + 8, _at(9), need, None) == ALIAS
    assert L.agoq_grad_norm(l, 1, _at(9), _at(9), need, None) == ALIAS
    assert L.agoq_grad_norm(l, -1, _at(8), _at(9), need, None) == SHAPE
    for bad in (-1.0, float("nan"), float("inf")):
        assert clip(l, 1, f(bad), _at(8), _at(9), need, None) == SHAPE
        assert L.agoq_clip_grads(l, 1, f(bad), _at(8), None) == SHAPE
    assert L.agoq_clip_grads(l, 1, f(1.0), None, None) == NULL
    assert L.agoq_clip_grads(l, 1, f(1.0), _at(8) + 1, None) == ALIGN
    assert L.agoq_clip_grads(l, 1, f(1.0), _at(0) + 16, None) == ALIAS


def _logprobs(**over):
    a = dict(x=_at(0), ld=100, dt=BF16, tok=_at(1), T=4, V=100, k=5, logp=_at(2), ent=_at(3),
             lse=_at(4), top=_at(5), ids=_at(6), stream=None)
    a.update(over)
    return agoq.lib().agoq_token_logprobs(*a.values())


@pytest.mark.parametrize("want,over", [
    (OK, dict(T=0)), (FORMAT, dict(dt=3)), (SHAPE, dict(T=-1)), (SHAPE, dict(V=0)),
    (SHAPE, dict(V=(1 << 30) + 1, ld=1 << 31)), (SHAPE, dict(ld=99)), (SHAPE, dict(k=33)),
    (SHAPE, dict(k=-1)), (SHAPE, dict(V=4, k=5)), (NULL, dict(x=0)), (NULL, dict(tok=0)),
    (NULL, dict(top=0)), (NULL, dict(ids=0)), (ALIGN, dict(x=_at(0) + 1)),
    (ALIGN, dict(tok=_at(1) + 4)), (ALIGN, dict(ids=_at(6) + 4)), (ALIGN, dict(lse=_at(4) + 2)),
    (ALIAS, dict(logp=_at(0))), (ALIAS, dict(ent=_at(2))), (ALIAS, dict(ids=_at(1))),
    (ALIAS, dict(top=_at(6))),
])
def test_token_logprobs(L, want, over):
    assert _logprobs(**over) == want


def _logprobs_bwd(**over):
    a = dict(x=_at(0), ld=100, dt=F32, tok=_at(1), T=4, V=100, lse=_at(2), ent=_at(3), dl=_at(4),
             de=_at(5), dx=_at(6), ldd=100, stream=None)
    a.update(over)
    return agoq.lib().agoq_token_logprobs_backward(*a.values())


@pytest.mark.parametrize("want,over", [
    (OK, dict(T=0)), (FORMAT, dict(dt=3)), (SHAPE, dict(ldd=10)), (SHAPE, dict(V=0)),
    (NULL, dict(lse=0)), (NULL, dict(dl=0)), (NULL, dict(ent=0)), (NULL, dict(dx=0)),
    (ALIGN, dict(dx=_at(6) + 2)), (ALIGN, dict(dl=_at(4) + 2)), (ALIAS, dict(dx=_at(0) + 4)),
    (ALIAS, dict(dx=_at(0), ldd=200)), (ALIAS, dict(dx=_at(2))),
])
def test_token_logprobs_backward(L, want, over):
    assert _logprobs_bwd(**over) == want


def _loss(**over):
    a = dict(x=_at(0), ld=100, dt=F16, tok=_at(1), w=_at(2), T=4, V=100, logp=_at(3), dx=_at(4),
             ldd=100, stream=None)
    a.update(over)
    return agoq.lib().agoq_token_loss(*a.values())


@pytest.mark.parametrize("want,over", [
    (OK, dict(T=0)), (FORMAT, dict(dt=5)), (SHAPE, dict(V=-1)), (SHAPE, dict(ldd=99)),
    (NULL, dict(dx=0)), (NULL, dict(tok=0)), (ALIGN, dict(w=_at(2) + 1)),
    (ALIGN, dict(dx=_at(4) + 1)), (ALIAS, dict(dx=_at(0) + 2)), (ALIAS, dict(logp=_at(2))),
    (ALIAS, dict(dx=_at(0), ldd=128)), (ALIAS, dict(logp=_at(4) + 8)),
])
def test_token_loss(L, want, over):
    assert _loss(**over) == want
