"""FP4 quantisation on the GPU against the plain form (tests/plain_fp4.py), bit for bit: types,
sizes from one element on, strides and alignments, special values, both directions, and the way
back for every code under every scale."""
import math

import pytest
import torch

from gradient_quantization_gb300 import agoq
from tests import plain_fp4 as F
from tests.gpu_util import Guarded

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
TYPES = [F32, BF16, F16]
FORMATS = [agoq.MXFP4, agoq.NVFP4]


def _rows(T, K, dtype, seed, pad=0, shift=0):
    """T rows of K values, K + pad apart, `shift` elements into a buffer of other values."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    buf = torch.full((T * (K + pad) + shift + 40,), 1000.0, dtype=dtype, device="cuda")
    x = buf[shift:shift + T * (K + pad)].view(T, K + pad)[:, :K]
    v = torch.randn(T, K, generator=g, device="cuda") * torch.exp2(
        torch.randint(-6, 7, (T, K), generator=g, device="cuda").float())
    x.copy_(v)
    return x


def _check(x, fmt, amax=None, given=None):
    """Rows, columns and both of x; amax as a number, `given`: the tensor that holds it."""
    T, K = x.shape
    x64 = x.double()
    if fmt == agoq.NVFP4 and amax is None:
        given = agoq.agoq_amax(x)
        amax = F.amax_of(x64)
        assert (math.isnan(amax) and math.isnan(float(given))) or float(given) == amax
    want, want_t = F.stored(x64, fmt, amax), F.stored(x64.t(), fmt, amax)
    got = agoq.agoq_fp4_quant(x, fmt, given)
    assert got[2] is None and got[3] is None
    both = agoq.agoq_fp4_quant(x, fmt, given, columns=True)
    cols = agoq.agoq_fp4_quant(x, fmt, given, rows=False, columns=True)
    assert cols[0] is None and cols[1] is None
    for name, a, b in (("rows", got[0], want[0]), ("row scales", got[1], want[1]),
                       ("rows of both", both[0], want[0]), ("their scales", both[1], want[1]),
                       ("columns", both[2], want_t[0]), ("column scales", both[3], want_t[1]),
                       ("columns alone", cols[2], want_t[0]), ("their scales", cols[3], want_t[1])):
        assert a.shape == b.shape and torch.equal(a, b), (name, int((a != b).sum()))
    return got, both


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,K", [(1, 1), (1, 16), (2, 31), (3, 33), (1, 4096), (31, 64), (128, 128),
                                 (129, 130), (200, 511), (127, 1000), (300, 65), (4097, 20)])
def test_sizes(fmt, dtype, T, K):
    _check(_rows(T, K, dtype, T + K), fmt)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad,shift", [(8, 0), (1, 0), (0, 1), (3, 5), (16, 8), (24, 4), (5, 2)])
def test_strides_and_alignments(fmt, dtype, pad, shift):
    for T, K in ((37, 200), (130, 77)):
        _check(_rows(T, K, dtype, 3, pad, shift), fmt)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_many_rows(dtype):
    _check(_rows(20001, 48, dtype, 4), agoq.NVFP4)
    _check(_rows(3, 70000, dtype, 5, 3), agoq.MXFP4)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", TYPES)
def test_borders_between_codes(fmt, dtype):
    """Quotients at and next to every border, in blocks whose scale is known: ties and their
    neighbours in the type."""
    borders = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], dtype=dtype, device="cuda")
    up = torch.nextafter(borders, torch.full_like(borders, 100))
    down = torch.nextafter(borders, torch.zeros_like(borders))
    v = torch.cat([borders, up, down])
    v = torch.cat([v, -v])
    x = torch.zeros(len(v), 32, dtype=dtype, device="cuda")
    x[:, 0] = 6.0
    x[:, 1] = v
    x[:, 16] = 6.0
    x[:, 17] = v.flip(0)
    if fmt == agoq.MXFP4:
        _check(x, fmt)
    else:
        _check(x, fmt, 2688.0, torch.tensor([2688.0], device="cuda"))      # g = 1


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", TYPES)
def test_extremes(fmt, dtype):
    """Zeros of both signs, subnormals, the smallest and largest values, blocks far apart."""
    info = torch.finfo(dtype)
    x = torch.zeros(9, 96, dtype=dtype, device="cuda")
    x[1, ::2] = -0.0
    x[2] = info.tiny
    x[3, 1::3] = info.tiny * info.eps            # the smallest subnormal
    x[4] = -info.max
    x[4, 5:40] = info.max
    x[5, 0], x[5, 40:] = info.max, info.tiny
    x[6] = torch.linspace(-1, 1, 96, device="cuda")
    x[7] = torch.randn(96, device="cuda") * (2.0 ** -120 if dtype != F16 else 2.0 ** -14)
    x[8] = torch.randn(96, device="cuda")
    _check(x, fmt)
    for row in range(9):
        _check(x[row:row + 1], fmt)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", TYPES)
def test_not_finite(fmt, dtype):
    x = _rows(130, 150, dtype, 6)
    x[3, 7], x[40, 149], x[129, 64], x[5, 0:32] = math.nan, math.inf, -math.inf, math.nan
    given, amax = (None, None) if fmt == agoq.MXFP4 else (torch.tensor([70.0], device="cuda"), 70.0)
    got, _ = _check(x, fmt, amax, given)        # a finite amax: those blocks alone
    y = agoq.agoq_fp4_dequant(got[0], got[1], 130, 150, fmt, given, dtype=F32)
    size = 32 if fmt == agoq.MXFP4 else 16
    bad = ~torch.isfinite(x.float())
    wide = torch.zeros(130, 160, dtype=torch.bool, device="cuda")
    wide[:, :150] = bad
    want = wide.view(130, -1, size).any(2).repeat_interleave(size, 1)[:, :150]
    assert torch.equal(torch.isnan(y), want)
    if fmt == agoq.NVFP4:                       # the tensor's own: all
        got, _ = _check(x, fmt)
        assert torch.isnan(agoq.agoq_fp4_dequant(got[0], got[1], 130, 150, fmt, agoq.agoq_amax(x))).all()
        x[3, 7] = x[5, 0] = 0
        x[5, 0:32] = 0
        assert float(agoq.agoq_amax(x)) == math.inf
        _check(x, fmt)


@pytest.mark.parametrize("amax", [0.0, 1e-38, 3.0, 50.0, 1e30, 3.4e38])
def test_an_amax_from_elsewhere(amax):
    """Smaller than the tensor's (values saturate), larger, and degenerate."""
    x = _rows(40, 100, F32, 7)
    given = torch.tensor([amax], device="cuda")
    _check(x, agoq.NVFP4, float(given), given)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,K,pad,shift", [(1, 1, 0, 0), (1, 17, 0, 1), (7, 1000, 3, 0), (2000, 700, 0, 0),
                                           (900, 2001, 1, 3), (3, 400000, 0, 0)])
def test_amax(dtype, T, K, pad, shift):
    x = _rows(T, K, dtype, 8, pad, shift)
    for t, k in ((T - 1, K - 1), (0, 0), (T // 2, K // 2)):
        x[t, k] = -10000.0                      # (BF16 holds 9984)
        assert float(agoq.agoq_amax(x)) == float(torch.tensor(10000.0, dtype=dtype))
        x[t, k] = math.nan
        assert math.isnan(float(agoq.agoq_amax(x)))
        x[t, k] = -math.inf
        assert float(agoq.agoq_amax(x)) == math.inf
        x[t, k] = 1
    assert float(agoq.agoq_amax(x)) == float(x.float().abs().max())
    assert float(agoq.agoq_amax(x[:0])) == 0.0 and float(agoq.agoq_amax(x[:, :0])) == 0.0


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("fmt", FORMATS)
def test_every_code_under_every_scale(fmt, dtype):
    size, n = (32, 256) if fmt == agoq.MXFP4 else (16, 128)     # an E4M3 scale has no sign
    K = n * size
    codes = (torch.arange(K, device="cuda") % 16).to(torch.uint8).view(1, K)
    scales = F.tile(torch.arange(n, device="cuda", dtype=torch.int32).to(torch.uint8).view(1, n))
    packed = F.pack(codes)
    for amax in ((None,) if fmt == agoq.MXFP4 else (2688.0, 3.0, 1e-37, 1e38)):
        given = None if amax is None else torch.tensor([amax], device="cuda")
        y = agoq.agoq_fp4_dequant(packed, scales, 1, K, fmt, given, dtype=dtype)
        want = F.values(packed, scales, 1, K, fmt).float()
        if amax is not None:
            want = (want.double() * F.tensor_scale(float(given))).float()
        want = want.to(dtype)
        same = (y == want) | (torch.isnan(y) & torch.isnan(want))
        assert bool(same.all()) and torch.equal(torch.signbit(y) & (y == 0), torch.signbit(want) & (want == 0))


@pytest.mark.parametrize("dtype", TYPES)
def test_dequantise_into_rows(dtype):
    T, K = 150, 77
    x = _rows(T, K, F32, 9)
    amax = agoq.agoq_amax(x)
    codes, scales, _, _ = agoq.agoq_fp4_quant(x, agoq.NVFP4, amax)
    want = agoq.agoq_fp4_dequant(codes, scales, T, K, agoq.NVFP4, amax, dtype=dtype)
    for pad, shift in ((0, 1), (3, 0), (19, 0), (8, 8)):
        buf = torch.full((T * (K + pad) + shift,), 7.0, dtype=dtype, device="cuda")
        y = buf[shift:].view(T, K + pad)
        assert agoq.agoq_fp4_dequant(codes, scales, T, K, agoq.NVFP4, amax, y=y[:, :K]).dtype == dtype
        assert torch.equal(y[:, :K], want) and bool((y[:, K:] == 7).all()) and bool((buf[:shift] == 7).all())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,K", [(1, 1), (130, 77), (64, 256)])
def test_nothing_outside_the_outputs(fmt, T, K):
    x = _rows(T, K, BF16, 10, 3, 1)
    amax = agoq.agoq_amax(x) if fmt == agoq.NVFP4 else None
    want = agoq.agoq_fp4_quant(x, fmt, amax, columns=True)
    outs = [Guarded(w.numel(), torch.uint8) for w in want]
    for keys in ((0, 1), (2, 3), (0, 1, 2, 3)):
        names = ("codes", "scales", "codes_t", "scales_t")
        agoq.agoq_fp4_quant(x, fmt, amax, rows=0 in keys, columns=2 in keys,
                            **{names[k]: outs[k].view for k in keys})
        for k in keys:
            assert outs[k].intact() and torch.equal(outs[k].view, want[k].view(-1))
    y = Guarded(2 * T * K, BF16)
    agoq.agoq_fp4_dequant(want[0], want[1], T, K, fmt, amax, y=y.view.view(T, K))
    m = Guarded(4, F32)
    agoq.agoq_amax(x, amax=m.view)
    assert y.intact() and m.intact()


def test_streams_and_graphs():
    x = _rows(257, 300, BF16, 11)
    want = agoq.agoq_fp4_quant(x, agoq.NVFP4, agoq.agoq_amax(x), columns=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    amax = agoq.agoq_amax(x, stream=side)
    got = agoq.agoq_fp4_quant(x, agoq.NVFP4, amax, columns=True, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    z = x.clone()
    big = torch.zeros(3000, 700, dtype=BF16, device="cuda")
    m = torch.zeros(1, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        amax = agoq.agoq_amax(z)
        got = agoq.agoq_fp4_quant(z, agoq.NVFP4, amax, columns=True)
        agoq.agoq_amax(big, amax=m)
    for k in (2.0, 0.25):
        z.copy_(x.float() * k)
        big.fill_(-k)
        graph.replay()
        want = agoq.agoq_fp4_quant(z, agoq.NVFP4, agoq.agoq_amax(z), columns=True)
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and float(m) == k


def test_refusals():
    x = torch.zeros(4, 64, dtype=BF16, device="cuda")
    amax = torch.ones(1, device="cuda")
    with pytest.raises(agoq.AgoqError):
        agoq.agoq_fp4_quant(x, agoq.NVFP4)                               # no amax
    with pytest.raises(ValueError):
        agoq.agoq_fp4_quant(x, 2, amax)
    with pytest.raises(agoq.AgoqError):
        agoq.agoq_fp4_quant(x, agoq.MXFP4, rows=False)                   # nothing wanted
    with pytest.raises(TypeError):
        agoq.agoq_fp4_quant(x.double(), agoq.MXFP4)
    with pytest.raises(TypeError):
        agoq.agoq_fp4_quant(x.cpu(), agoq.MXFP4)
    with pytest.raises(ValueError):
        agoq.agoq_fp4_quant(x, agoq.MXFP4, codes=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        agoq.agoq_fp4_quant(x[:0], agoq.MXFP4, columns=True)
    with pytest.raises(ValueError):
        agoq.agoq_amax(x.t())
    codes, scales, _, _ = agoq.agoq_fp4_quant(x, agoq.MXFP4)
    with pytest.raises(ValueError):
        agoq.agoq_fp4_dequant(codes, scales, 5, 64, agoq.MXFP4)
    with pytest.raises(TypeError):
        agoq.agoq_fp4_dequant(codes, scales, 4, 64, agoq.MXFP4, dtype=torch.float64)
    c, s, _, _ = agoq.agoq_fp4_quant(x[:0], agoq.MXFP4)
    assert c.numel() == 0 and agoq.agoq_fp4_dequant(c, s, 0, 64, agoq.MXFP4).shape == (0, 64)
