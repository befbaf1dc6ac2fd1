"""The global gradient norm and clipping on the GPU against binary64.

The norm's squares are summed in binary32 over at most 128 elements and in
binary64 beyond: (128 + 3) u relative on the sum, half of that on the root, and
the final rounding.  A clipped value is one binary32 product, rounded once more to
its type."""
import math

import pytest
import torch

from gradient_quantization_gb300 import agoq
from tests import plain64 as P
from tests.gpu_util import Guarded

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
NORM_REL = (131 / 2 + 2) * P.U


def _rand(n, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(n, generator=g)).to(dtype).cuda()


def _master(n, seed, scale=1e-3):
    v = _rand(n, F32, seed, scale).view(-1, 128)
    s = v.abs().amax(1) / 448
    return (v / s[:, None]).to(torch.float8_e4m3fn).view(torch.uint8).view(-1), s


def _check_norm(norm, grads):
    want = P.grad_norm(grads)
    assert abs(float(norm) - want) <= NORM_REL * want + 2.0 ** -149, (float(norm), want)


def _coef(max_norm, norm):
    c = torch.tensor(max_norm, dtype=F32) / (norm.cpu() + torch.tensor(1e-6, dtype=F32))
    return torch.clamp(c, max=1.0).cuda()


def _check_clipped(grads, outs, coef):
    """The same single binary32 product everywhere: equal bits."""
    for g, o in zip(grads, outs):
        if isinstance(g, tuple):
            assert torch.equal(o, g[1] * coef)
        else:
            assert torch.equal(o, (g.float() * coef).to(g.dtype))


LISTS = {
    "one": [(1, F32)],
    "odd": [(1, BF16), (3, F16), (0, F32), (7, F32), (127, BF16), (129, F16), (4097, F32)],
    "long": [(3_000_001, BF16), (17, F32), (1_000_003, F16), (500_000, F32)],
    "masters": [(128, "e4m3"), (128 * 300, "e4m3"), (128 * 4001, "e4m3"), (4096, F32)],
    "many": [(64 + 5 * i, (F32, BF16, F16)[i % 3]) for i in range(1100)],
    "ends": [(8192, F32), (8193, F32), (16384, BF16), (16383, F16), (32768, "e4m3"),
             (32768 + 128, "e4m3")],
}


def _grads(name):
    return [_master(n, 7 * i + 1) if t == "e4m3" else _rand(n, t, 7 * i + 1, 0.01)
            for i, (n, t) in enumerate(LISTS[name])]


def _like(grads):
    return [torch.full_like(g[1] if isinstance(g, tuple) else g, 3.0) for g in grads]


@pytest.mark.parametrize("name", sorted(LISTS))
@pytest.mark.parametrize("fraction", [0.5, 2.0])
def test_norm_and_clip(name, fraction):
    grads = _grads(name)
    outs = _like(grads)
    want = P.grad_norm(grads)
    l = agoq.GradList(grads, outs)
    norm = agoq.agoq_grad_norm(l)
    _check_norm(norm, grads)
    both = agoq.agoq_clip_grad_norm(l, want * fraction)
    assert torch.equal(both, norm)
    _check_clipped(grads, outs, _coef(want * fraction, norm))
    outs2 = _like(grads)
    agoq.agoq_clip_grads(agoq.GradList(grads, outs2), want * fraction, norm)
    assert all(torch.equal(p, q) for p, q in zip(outs, outs2))


@pytest.mark.parametrize("name", sorted(LISTS))
def test_in_place(name):
    grads = _grads(name)
    kept = [tuple(t.clone() for t in g) if isinstance(g, tuple) else g.clone() for g in grads]
    l = agoq.GradList(grads)
    norm = agoq.agoq_clip_grad_norm(l, 1e9)                       # nothing to clip
    same = lambda p, q: all(torch.equal(a, b) for a, b in zip(p, q)) if isinstance(p, tuple) \
        else torch.equal(p, q)
    assert all(same(p, q) for p, q in zip(grads, kept))
    half = 0.5 * float(norm)
    agoq.agoq_clip_grad_norm(l, half)
    _check_clipped(kept, [g[1] if isinstance(g, tuple) else g for g in grads], _coef(half, norm))
    assert all(torch.equal(g[0], k[0]) for g, k in zip(grads, kept) if isinstance(g, tuple))


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("shift_in,shift_out", [(0, 0), (1, 1), (1, 0), (0, 3), (2, 5)])
def test_alignment(dtype, shift_in, shift_out):
    n = 20_011
    buf = _rand(n + 16, dtype, 3)
    g = buf[shift_in:shift_in + n]
    size = torch.empty((), dtype=dtype).element_size()
    guard = Guarded((n + 16) * size, dtype)
    out = guard.view[shift_out:shift_out + n]
    before = guard.view.clone()
    norm = agoq.agoq_clip_grad_norm(agoq.GradList([g], [out]), 1.0)
    _check_norm(norm, [g])
    _check_clipped([g], [out], _coef(1.0, norm))
    assert guard.intact()
    b, a = before.view(torch.uint8), guard.view.view(torch.uint8)
    assert torch.equal(b[:shift_out * size], a[:shift_out * size])
    assert torch.equal(b[(shift_out + n) * size:], a[(shift_out + n) * size:])


@pytest.mark.parametrize("dtype,scale", [(F32, 1e25), (F32, 1e-30), (BF16, 1e30), (BF16, 1e-25),
                                         (F16, 1e-7), (F32, 1e-42)])
def test_range(dtype, scale):
    """Values whose squares leave the binary32 range, beside ordinary ones and zeros."""
    grads = [_rand(5000, dtype, 4, scale), torch.zeros(3000, dtype=dtype, device="cuda")]
    _check_norm(agoq.agoq_grad_norm(agoq.GradList(grads)), grads)
    grads.append(_rand(777, dtype, 5))
    _check_norm(agoq.agoq_grad_norm(agoq.GradList(grads)), grads)


def test_zero_and_nothing():
    z = torch.zeros(1000, device="cuda")
    assert float(agoq.agoq_grad_norm(agoq.GradList([z]))) == 0
    assert float(agoq.agoq_clip_grad_norm(agoq.GradList([]), 1.0)) == 0
    assert float(agoq.agoq_clip_grad_norm(agoq.GradList([z]), 0.0)) == 0
    assert not z.any()
    codes = torch.zeros(256, dtype=torch.uint8, device="cuda")
    assert float(agoq.agoq_grad_norm(agoq.GradList([(codes, torch.zeros(2, device="cuda"))]))) == 0


def test_not_finite():
    for bad in (float("inf"), float("nan")):
        for dtype in (F32, BF16, F16):
            g = _rand(40_000, dtype, 6)
            g[33_333] = bad
            norm = agoq.agoq_clip_grad_norm(agoq.GradList([g.clone()]), 1.0)
            assert math.isnan(float(norm)) if bad != bad else float(norm) == math.inf
    codes, scales = _master(1280, 8)
    codes[700] = 0x7F                                             # E4M3 NaN
    assert math.isnan(float(agoq.agoq_grad_norm(agoq.GradList([(codes, scales)]))))
    g = _rand(1000, F32, 9)
    g[5] = float("inf")
    agoq.agoq_clip_grad_norm(agoq.GradList([g]), 1.0)             # coefficient 0
    assert math.isnan(float(g[5])) and not g[:5].any()


def test_master_values_with_all_codes():
    """Every finite code, subnormals and signed zeros among them, with scales of many sizes."""
    c = [v for v in range(256) if v & 0x7F != 0x7F]
    codes = torch.tensor((c * 64)[:128 * 100], dtype=torch.uint8, device="cuda")
    scales = torch.tensor([2.0 ** (i % 60 - 40) * 1.3 for i in range(100)], device="cuda")
    _check_norm(agoq.agoq_grad_norm(agoq.GradList([(codes, scales)])), [(codes, scales)])


def test_offsets_beyond_32_bits():
    n = (1 << 32) + 12_345
    g = torch.zeros(n, dtype=BF16, device="cuda")
    g[-1], g[0], g[1 << 31] = 3.0, 4.0, 12.0
    out = torch.empty_like(g)
    norm = agoq.agoq_clip_grad_norm(agoq.GradList([g], [out]), 6.5)
    assert float(norm) == 13.0
    assert [float(out[i]) for i in (0, 1 << 31, -1, 5)] == [2.0, 6.0, 1.5, 0.0]


def test_same_bits_again_other_stream_and_graph():
    grads = _grads("long") + _grads("masters")
    outs = _like(grads)
    l = agoq.GradList(grads, outs)
    norm = agoq.agoq_clip_grad_norm(l, 1.0)
    kept = [o.clone() for o in outs]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    again = agoq.agoq_clip_grad_norm(l, 1.0, stream=side)
    side.synchronize()
    assert torch.equal(norm, again) and all(torch.equal(p, q) for p, q in zip(outs, kept))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = agoq.agoq_clip_grad_norm(l, 1.0)
    grads[0].mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    _check_norm(held, grads)
    _check_clipped(grads, outs, _coef(1.0, held))


def test_binding_refusals():
    g = _rand(100, F32, 1)
    with pytest.raises(TypeError):
        agoq.GradList([g.double()])
    with pytest.raises(TypeError):
        agoq.GradList([g.cpu()])
    with pytest.raises(ValueError):
        agoq.GradList([g], [g[:50]])
    with pytest.raises(TypeError):
        agoq.GradList([g], [g.to(BF16)])
    with pytest.raises(ValueError):
        agoq.GradList([g], [])
    with pytest.raises(agoq.AgoqError):
        agoq.GradList([g, g])                                     # one tensor twice
    with pytest.raises(agoq.AgoqError):
        agoq.agoq_clip_grad_norm(agoq.GradList([g]), -1.0)
    with pytest.raises(ValueError):
        agoq.agoq_clip_grads(agoq.GradList([g]), 1.0, g)
