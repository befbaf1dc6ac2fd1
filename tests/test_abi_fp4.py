"""Refusals of the FP4, policy and preference calls: every call below fails its host-side
validation and launches nothing (CPU)."""
import ctypes

import pytest

from gradient_quantization_gb300 import agoq

OK, NULL, SHAPE, ALIGN, ALIAS, FORMAT = 0, 1, 2, 4, 5, 8
F32, BF16, F16, E4M3 = 0, 1, 2, 3
MX, NV = 0, 1
A = 0x10000000          # fake addresses: never dereferenced on these paths
GAP = 1 << 24
f = ctypes.c_float
NAN = float("nan")


def _at(i):
    return A + i * GAP


def test_sizes():
    L = agoq.lib()
    assert L.agoq_fp4_code_bytes(5, 33) == 5 * 32 and L.agoq_fp4_code_bytes(0, 7) == 0
    assert L.agoq_fp4_scale_bytes(1, 1, MX) == 512 and L.agoq_fp4_scale_bytes(129, 128, MX) == 1024
    assert L.agoq_fp4_scale_bytes(128, 129, MX) == 1024 and L.agoq_fp4_scale_bytes(0, 8, NV) == 0
    assert L.agoq_fp4_scale_bytes(128, 65, NV) == 1024 and L.agoq_fp4_scale_bytes(1, 64, NV) == 512
    for rows, K, fmt in ((-1, 8, 0), (1, 0, 0), (1, (1 << 24) + 1, 0), ((1 << 30) + 1, 8, 0), (1, 8, 2),
                         (1, 8, -1)):
        assert L.agoq_fp4_scale_bytes(rows, K, fmt) == -1
    assert L.agoq_fp4_code_bytes(1, 0) == -1 and L.agoq_fp4_code_bytes(-1, 8) == -1


def _amax(**over):
    a = dict(x=_at(0), ldx=64, T=4, K=64, dt=BF16, amax=_at(1), stream=None)
    a.update(over)
    return agoq.lib().agoq_amax(*a.values())


@pytest.mark.parametrize("want,over", [
    (FORMAT, dict(dt=E4M3)), (FORMAT, dict(dt=-1)), (SHAPE, dict(T=-1)), (SHAPE, dict(K=-1)),
    (SHAPE, dict(ldx=63)), (SHAPE, dict(T=(1 << 30) + 1)), (NULL, dict(x=0)), (NULL, dict(amax=0)),
    (ALIGN, dict(x=_at(0) + 1)), (ALIGN, dict(amax=_at(1) + 2)), (ALIAS, dict(amax=_at(0) + 8)),
    (ALIAS, dict(amax=_at(0) + 4 * 128 - 4)),
])
def test_amax(want, over):
    assert _amax(**over) == want


def _quant(**over):
    a = dict(x=_at(0), ldx=64, T=4, K=64, dt=BF16, fmt=NV, amax=_at(1), codes=_at(2), scales=_at(3),
             codes_t=_at(4), scales_t=_at(5), stream=None)
    a.update(over)
    return agoq.lib().agoq_fp4_quant(*a.values())


@pytest.mark.parametrize("want,over", [
    (OK, dict(T=0, x=0, amax=0)),
    (FORMAT, dict(dt=E4M3)), (FORMAT, dict(fmt=2)), (FORMAT, dict(fmt=-1)),
    (SHAPE, dict(T=-1)), (SHAPE, dict(K=0)), (SHAPE, dict(K=(1 << 24) + 1, ldx=1 << 25)),
    (SHAPE, dict(ldx=63)), (SHAPE, dict(T=(1 << 24) + 1)),
    (NULL, dict(codes=0)), (NULL, dict(scales=0)), (NULL, dict(codes_t=0)), (NULL, dict(scales_t=0)),
    (NULL, dict(codes=0, scales=0, codes_t=0, scales_t=0)), (NULL, dict(x=0)), (NULL, dict(amax=0)),
    (ALIGN, dict(x=_at(0) + 1)), (ALIGN, dict(dt=F32, x=_at(0) + 2)), (ALIGN, dict(codes=_at(2) + 8)),
    (ALIGN, dict(scales=_at(3) + 4)), (ALIGN, dict(codes_t=_at(4) + 1)),
    (ALIGN, dict(scales_t=_at(5) + 8)), (ALIGN, dict(amax=_at(1) + 1)),
    (ALIAS, dict(codes=_at(0))), (ALIAS, dict(scales=_at(2) + 64)), (ALIAS, dict(codes_t=_at(3))),
    (ALIAS, dict(scales_t=_at(4) + 512)), (ALIAS, dict(codes=_at(1))),
    (ALIAS, dict(scales_t=_at(0) + 256)),
])
def test_quant(want, over):
    assert _quant(**over) == want


def _dequant(**over):
    a = dict(codes=_at(0), scales=_at(1), amax=_at(2), T=4, K=64, fmt=NV, y=_at(3), ldy=64, dt=F32,
             stream=None)
    a.update(over)
    return agoq.lib().agoq_fp4_dequant(*a.values())


@pytest.mark.parametrize("want,over", [
    (OK, dict(T=0, codes=0, y=0)), (FORMAT, dict(dt=7)), (FORMAT, dict(fmt=9)), (SHAPE, dict(K=0)),
    (SHAPE, dict(T=-3)), (SHAPE, dict(ldy=32)), (NULL, dict(codes=0)), (NULL, dict(scales=0)),
    (NULL, dict(y=0)), (NULL, dict(amax=0)), (ALIGN, dict(codes=_at(0) + 4)),
    (ALIGN, dict(scales=_at(1) + 4)), (ALIGN, dict(y=_at(3) + 2)), (ALIGN, dict(amax=_at(2) + 3)),
    (ALIAS, dict(y=_at(0) + 64)), (ALIAS, dict(y=_at(1))), (ALIAS, dict(y=_at(2))),
])
def test_dequant(want, over):
    assert _dequant(**over) == want


def _gemm(**over):
    a = dict(ac=_at(0), as_=_at(1), aa=_at(2), bc=_at(3), bs=_at(4), ba=_at(5), M=4, N=8, K=64, fmt=NV,
             d=_at(6), ldd=8, dt=BF16, stream=None)
    a.update(over)
    return agoq.lib().agoq_fp4_gemm(*a.values())


@pytest.mark.parametrize("want,over", [
    (OK, dict(M=0, ac=0)), (OK, dict(N=0, d=0)),
    (FORMAT, dict(dt=E4M3)), (FORMAT, dict(fmt=3)),
    (SHAPE, dict(M=-1)), (SHAPE, dict(N=-1)), (SHAPE, dict(K=0)), (SHAPE, dict(ldd=7)),
    (SHAPE, dict(K=(1 << 24) + 1)), (SHAPE, dict(M=1 << 21, N=1 << 21, ldd=1 << 21)),
    (NULL, dict(ac=0)), (NULL, dict(as_=0)), (NULL, dict(bc=0)), (NULL, dict(bs=0)), (NULL, dict(d=0)),
    (NULL, dict(aa=0)), (NULL, dict(ba=0)),
    (ALIGN, dict(ac=_at(0) + 8)), (ALIGN, dict(as_=_at(1) + 8)), (ALIGN, dict(bc=_at(3) + 1)),
    (ALIGN, dict(bs=_at(4) + 2)), (ALIGN, dict(d=_at(6) + 1)), (ALIGN, dict(aa=_at(2) + 2)),
    (ALIGN, dict(ba=_at(5) + 2)),
    (ALIAS, dict(d=_at(0) + 64)), (ALIAS, dict(d=_at(1))), (ALIAS, dict(d=_at(2))),
    (ALIAS, dict(d=_at(3))), (ALIAS, dict(d=_at(4) + 256)), (ALIAS, dict(d=_at(5))),
])
def test_gemm(want, over):
    assert _gemm(**over) == want


def _policy(**over):
    a = dict(x=_at(0), ld=64, dt=BF16, tokens=_at(1), old=_at(2), ref=_at(3), adv=_at(4), w=_at(5), T=4,
             V=64, lo=0.2, hi=0.2, kl_coef=0.1, loss=_at(6), logp=_at(7), kl=_at(8), d=_at(9), ldd=64,
             stream=None)
    a.update(over)
    for k in ("lo", "hi", "kl_coef"):
        a[k] = f(a[k])
    return agoq.lib().agoq_policy_loss(*a.values())


@pytest.mark.parametrize("want,over", [
    (OK, dict(T=0, x=0)),
    (FORMAT, dict(dt=E4M3)), (SHAPE, dict(T=-1)), (SHAPE, dict(V=0)), (SHAPE, dict(ld=63)),
    (SHAPE, dict(ldd=63)), (SHAPE, dict(V=(1 << 30) + 1, ld=1 << 31, ldd=1 << 31)),
    (SHAPE, dict(lo=-0.1)), (SHAPE, dict(lo=1.5)), (SHAPE, dict(lo=NAN)), (SHAPE, dict(hi=-1.0)),
    (SHAPE, dict(hi=NAN)), (SHAPE, dict(hi=float("inf"))), (SHAPE, dict(kl_coef=-1.0)),
    (SHAPE, dict(kl_coef=NAN)),
    (NULL, dict(x=0)), (NULL, dict(tokens=0)), (NULL, dict(old=0)), (NULL, dict(adv=0)),
    (NULL, dict(d=0)), (NULL, dict(ref=0)), (NULL, dict(ref=0, kl=0)), (NULL, dict(ref=0, kl_coef=0.0)),
    (ALIGN, dict(x=_at(0) + 1)), (ALIGN, dict(tokens=_at(1) + 4)), (ALIGN, dict(old=_at(2) + 2)),
    (ALIGN, dict(ref=_at(3) + 1)), (ALIGN, dict(adv=_at(4) + 2)), (ALIGN, dict(w=_at(5) + 2)),
    (ALIGN, dict(loss=_at(6) + 2)), (ALIGN, dict(logp=_at(7) + 2)), (ALIGN, dict(kl=_at(8) + 2)),
    (ALIGN, dict(d=_at(9) + 1)),
    (ALIAS, dict(d=_at(0) + 128)), (ALIAS, dict(d=_at(0), ldd=72)), (ALIAS, dict(loss=_at(7))),
    (ALIAS, dict(kl=_at(3))), (ALIAS, dict(logp=_at(2) + 4)), (ALIAS, dict(loss=_at(0))),
    (ALIAS, dict(d=_at(5))), (ALIAS, dict(x=_at(9), loss=_at(9))),
])
def test_policy(want, over):
    assert _policy(**over) == want


def _preference(**over):
    a = dict(logp=_at(0), ref=_at(1), offsets=_at(2), w=_at(3), T=100, P=3, beta=0.1, eps=0.0,
             loss=_at(4), margin=_at(5), dlogp=_at(6), stream=None)
    a.update(over)
    for k in ("beta", "eps"):
        a[k] = f(a[k])
    return agoq.lib().agoq_preference_loss(*a.values())


@pytest.mark.parametrize("want,over", [
    (OK, dict(P=0, logp=0, offsets=0)),
    (SHAPE, dict(T=-1)), (SHAPE, dict(P=-1)), (SHAPE, dict(beta=-1.0)), (SHAPE, dict(beta=NAN)),
    (SHAPE, dict(eps=1.1)), (SHAPE, dict(eps=-0.1)), (SHAPE, dict(eps=NAN)), (SHAPE, dict(T=1 << 41)),
    (SHAPE, dict(P=(1 << 30) + 1)),
    (NULL, dict(logp=0)), (NULL, dict(offsets=0)), (NULL, dict(dlogp=0)),
    (ALIGN, dict(logp=_at(0) + 2)), (ALIGN, dict(ref=_at(1) + 2)), (ALIGN, dict(offsets=_at(2) + 4)),
    (ALIGN, dict(w=_at(3) + 2)), (ALIGN, dict(loss=_at(4) + 2)), (ALIGN, dict(margin=_at(5) + 2)),
    (ALIGN, dict(dlogp=_at(6) + 2)),
    (ALIAS, dict(dlogp=_at(0))), (ALIAS, dict(loss=_at(5))), (ALIAS, dict(margin=_at(2) + 48)),
    (ALIAS, dict(dlogp=_at(3))), (ALIAS, dict(loss=_at(6) + 396)),
])
def test_preference(want, over):
    assert _preference(**over) == want
