"""The FP4 product on the GPU against binary64 products of the stored values: sizes of every
kind, types, strides, exact sums, scales far apart, NaN, streams and graphs.

Bounds.  A product of two codes and two scales is exact in binary32 (4 + 4 bits of codes, 4 + 4 of
E4M3 scales), and a binary32 sum of K of them in any order is within K 2^-24 of the sum of their
magnitudes if each addition rounds, or within K 2^-23 if it cuts off (the tensor cores' additions
are not specified): K 2^-23 is taken.  The tensor scales are two more roundings, the output one of
its type."""
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
U = 2.0 ** -24
TINY = {F32: 2.0 ** -150, BF16: 2.0 ** -134, F16: 2.0 ** -25}


class Operand:
    """A stored operand and its binary64 values."""

    def __init__(self, x, fmt):
        self.rows, self.K = x.shape
        self.amax = x.float().abs().max().view(1) if fmt == agoq.NVFP4 else None
        number = None if self.amax is None else float(self.amax)
        self.codes, self.scales = F.stored(x.double(), fmt, number)
        self.values = F.values(self.codes, self.scales, self.rows, self.K, fmt)
        if number is not None:
            self.values = self.values * F.tensor_scale(number)


def _operand(rows, K, fmt, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(rows, K, generator=g, device="cuda") * scale
    x[torch.rand(rows, K, generator=g, device="cuda") < 1e-2] *= 20
    return Operand(x, fmt)


def _gemm(a, b, fmt, **kw):
    return agoq.agoq_fp4_gemm(a.codes, a.scales, b.codes, b.scales, a.rows, b.rows, a.K, fmt,
                              a_amax=a.amax, b_amax=b.amax, **kw)


def _check(a, b, d):
    want = a.values @ b.values.t()
    bound = (a.K * 2 + 4) * U * (a.values.abs() @ b.values.abs().t())
    bound = bound + (want.abs() + bound) * (torch.finfo(d.dtype).eps / 2) + TINY[d.dtype]
    off = (d.double() - want).abs()
    assert bool((off <= bound).all()), float((off / bound).max())


SIZES = [(1, 1, 1), (1, 128, 64), (1, 300, 1000), (2, 129, 65), (17, 1000, 333), (32, 128, 4096),
         (33, 257, 777), (64, 64, 64), (64, 1000, 2000), (65, 65, 65), (65, 64, 300), (1000, 1, 500),
         (300, 31, 129), (5000, 64, 200), (128, 128, 256), (129, 127, 257), (200, 300, 512),
         (517, 1003, 1999), (100, 2500, 100), (1, 5000, 33), (3, 200, 20000), (200, 40, 9000), (300, 200, 9000),
         (513, 130, 6200)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K", SIZES)
def test_sizes(fmt, M, N, K):
    a, b = _operand(M, K, fmt, 1), _operand(N, K, fmt, 2)
    for dtype in TYPES:
        _check(a, b, _gemm(a, b, fmt, dtype=dtype))
    agoq.agoq_device_status()


# Sizes of the CTA pairs (a long K, a round or two of 256 x 256 tiles), whole and ragged.
PAIRS = [(1024, 4096, 4096), (1001, 4090, 3999), (2561, 2177, 4000), (130, 9001, 4100)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K", [(2560, 2048, 64), (2561, 2177, 300), (2304, 4097, 1000),
                                   (5000, 3000, 513)] + PAIRS)
def test_large(fmt, M, N, K):
    """Several tiles a CTA, odd edges."""
    a, b = _operand(M, K, fmt, 3), _operand(N, K, fmt, 4)
    for dtype in TYPES:
        _check(a, b, _gemm(a, b, fmt, dtype=dtype))
    agoq.agoq_device_status()


def _exact_operand(rows, K, fmt, seed):
    """Small codes under scales that are small whole numbers (NVFP4) or powers of two (MXFP4),
    so that every partial sum is a multiple of 1/4 below 2^22: exact in binary32 in any order."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    codes = torch.randint(0, 16, (rows, -(-K // 32) * 32), generator=g, device="cuda").to(torch.uint8)
    codes[:, K:] = 0
    nb = codes.shape[1] // F.BLOCK[fmt]
    if fmt == agoq.MXFP4:
        scales = torch.randint(127, 130, (rows, nb), generator=g, device="cuda").to(torch.uint8)
    else:
        pick = torch.tensor([0x38, 0x40, 0x44, 0x48], device="cuda", dtype=torch.uint8)   # 1 2 3 4
        scales = pick[torch.randint(0, 4, (rows, nb), generator=g, device="cuda")]
    op = Operand.__new__(Operand)
    op.rows, op.K, op.codes, op.scales = rows, K, F.pack(codes), F.tile(scales)
    op.amax = torch.tensor([2688.0], device="cuda") if fmt == agoq.NVFP4 else None     # g = 1
    op.values = F.values(op.codes, op.scales, rows, K, fmt)
    return op


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K", [(5, 400, 3001), (40, 300, 700), (300, 200, 1000), (2600, 2100, 500),
                                   (1, 1000, 4096), (3000, 20, 100), (300, 200, 4000),
                                   (300, 200, 6500), (1001, 4090, 3999), (1024, 4096, 4096)])
def test_exact_sums(fmt, M, N, K):
    """Bit for bit: every element of K once, with its own scale, in the right place."""
    a, b = _exact_operand(M, K, fmt, 5), _exact_operand(N, K, fmt, 6)
    want = a.values @ b.values.t()
    assert float((a.values.abs() @ b.values.abs().t()).max()) < 2 ** 22
    for dtype in TYPES:
        if dtype != F16 or float(want.abs().max()) < 65504:
            assert torch.equal(_gemm(a, b, fmt, dtype=dtype), want.float().to(dtype))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N", [(3, 300), (150, 200), (2600, 2100)])
def test_one_hot_rows_give_columns(fmt, M, N):
    """Rows of a with a single 1 select columns of b: codes and scales are paired rightly."""
    K = 600
    b = _operand(N, K, fmt, 7)
    x = torch.zeros(M, K, device="cuda")
    at = (torch.arange(M, device="cuda") * 37 + 11) % K
    x[torch.arange(M, device="cuda"), at] = 1.0
    a = Operand(x, fmt)
    if fmt == agoq.NVFP4:       # 1 / 2688 * 448 * 6 is a power of two only nearly: a's own values
        _check(a, b, _gemm(a, b, fmt, dtype=F32))
    else:
        assert torch.equal(_gemm(a, b, fmt, dtype=F32), b.values[:, at].t().float())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,N,K", [(5, 200, 200), (70, 333, 200), (333, 40, 200), (2600, 2117, 200),
                                   (1001, 4090, 3999)])
def test_rows_of_d(dtype, M, N, K):
    """Distances and alignments of d's rows; nothing between them is written."""
    a, b = _operand(M, K, agoq.NVFP4, 8), _operand(N, K, agoq.NVFP4, 9)
    want = _gemm(a, b, agoq.NVFP4, dtype=dtype)
    for pad, shift in ((0, 1), (3, 0), (-N % 8 + 8, 0), (-N % 8, 8), (5, 3)):
        buf = torch.full((M * (N + pad) + shift + 8,), 7.0, dtype=dtype, device="cuda")
        d = buf[shift:shift + M * (N + pad)].view(M, N + pad)
        _gemm(a, b, agoq.NVFP4, d=d[:, :N])
        assert torch.equal(d[:, :N], want)
        assert bool((d[:, N:] == 7).all()) and bool((buf[:shift] == 7).all()) and bool((buf[-8:] == 7).all())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K", [(2, 130, 100), (130, 100, 100), (2600, 2100, 100), (1001, 4090, 3999)])
def test_nothing_outside_d(fmt, M, N, K):
    a, b = _operand(M, K, fmt, 10), _operand(N, K, fmt, 11)
    d = Guarded(2 * M * N, BF16)
    _gemm(a, b, fmt, d=d.view.view(M, N))
    assert d.intact()
    _check(a, b, d.view.view(M, N))


@pytest.mark.parametrize("M,N,K", [(4, 300, 320), (300, 200, 320), (2600, 2100, 320), (1001, 4090, 3999)])
def test_scales_far_apart(M, N, K):
    """MXFP4 rows from 2^-40 to 2^40."""
    g = torch.Generator(device="cuda").manual_seed(12)
    spread = lambda n: torch.exp2(torch.randint(-40, 41, (n, 1), generator=g, device="cuda").float())
    a = Operand(torch.randn(M, K, generator=g, device="cuda") * spread(M), agoq.MXFP4)
    b = Operand(torch.randn(N, K, generator=g, device="cuda") * spread(N), agoq.MXFP4)
    _check(a, b, _gemm(a, b, agoq.MXFP4, dtype=F32))


def test_tensor_scales_far_apart():
    """NVFP4 tensors of 1e30 and 1e-30, and of 1e-36 twice (a product that binary32 holds as 0)."""
    for sa, sb in ((1e30, 1e-30), (1e-30, 1e30), (1e-36, 1e20), (1e-36, 1e-36)):
        a, b = _operand(70, 100, agoq.NVFP4, 13, sa), _operand(90, 100, agoq.NVFP4, 14, sb)
        d = _gemm(a, b, agoq.NVFP4, dtype=F32)
        assert torch.isfinite(d).all()
        _check(a, b, d)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K", [(5, 300, 500), (300, 200, 500), (300, 200, 6500), (2600, 2100, 500),
                                   (1001, 4090, 3999)])
def test_nan_stays_in_its_row(fmt, M, N, K):
    g = torch.Generator(device="cuda").manual_seed(15)
    x, w = torch.randn(M, K, generator=g, device="cuda"), torch.randn(N, K, generator=g, device="cuda")
    x[M // 2, 300], w[N - 1, 5] = math.nan, math.inf
    am = torch.tensor([6.0], device="cuda") if fmt == agoq.NVFP4 else None
    a, b = (agoq.agoq_fp4_quant(v, fmt, am) for v in (x, w))
    d = agoq.agoq_fp4_gemm(a[0], a[1], b[0], b[1], M, N, K, fmt, am, am)
    bad = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    bad[M // 2], bad[:, N - 1] = True, True
    assert torch.equal(torch.isnan(d), bad)


def test_zeros_and_nothing():
    for fmt in FORMATS:
        a, b = Operand(torch.zeros(70, 64, device="cuda"), fmt), _operand(80, 64, fmt, 16)
        assert not _gemm(a, b, fmt, dtype=F32).any()
        e = agoq.agoq_fp4_quant(torch.zeros(0, 64, device="cuda"), agoq.MXFP4)
        assert agoq.agoq_fp4_gemm(e[0], e[1], b.codes, b.scales, 0, 80, 64, fmt, b.amax, b.amax).shape == (0, 80)


def test_the_same_bits_again():
    for M, N, K in ((3, 500, 5000), (300, 300, 700), (2600, 2100, 300), (1001, 4090, 3999), (300, 200, 7000)):
        a, b = _operand(M, K, agoq.NVFP4, 17), _operand(N, K, agoq.NVFP4, 18)
        first = _gemm(a, b, agoq.NVFP4, dtype=F32)
        for _ in range(5):
            assert torch.equal(_gemm(a, b, agoq.NVFP4, dtype=F32), first)


def test_streams_at_the_same_time():
    """Calls of every variant in six streams at once."""
    ops = [(_operand(M, K, agoq.NVFP4, 19), _operand(N, K, agoq.NVFP4, 20))
           for M, N, K in ((2, 700, 900), (50, 700, 900), (300, 500, 900), (2600, 2100, 900), (300, 200, 4000),
                           (1001, 4090, 3999))]
    want = [_gemm(a, b, agoq.NVFP4) for a, b in ops]
    streams = [torch.cuda.Stream() for _ in ops]
    torch.cuda.synchronize()
    got = [[_gemm(a, b, agoq.NVFP4, stream=s) for (a, b), s in zip(ops, streams)] for _ in range(6)]
    torch.cuda.synchronize()
    agoq.agoq_device_status()
    assert all(torch.equal(d, w) for row in got for d, w in zip(row, want))


def test_graph():
    x = torch.randn(40, 300, device="cuda")
    b = [_operand(n, 300, agoq.NVFP4, 21) for n in (60, 700)]
    y = x.clone()
    graph = torch.cuda.CUDAGraph()

    def step():
        amax = agoq.agoq_amax(y)
        c, s, _, _ = agoq.agoq_fp4_quant(y, agoq.NVFP4, amax)
        return [agoq.agoq_fp4_gemm(c, s, o.codes, o.scales, 40, o.rows, 300, agoq.NVFP4, amax, o.amax)
                for o in b]
    step()
    with torch.cuda.graph(graph):
        got = step()
    for k in (3.0, 0.1):
        y.copy_(x * k)
        graph.replay()
        assert all(torch.equal(g, w) for g, w in zip(got, step()))


def test_a_linear_layer_and_its_gradients():
    """Y = X W^T, dX = dY W, dW = dY^T X from operands quantised along rows and columns, against
    binary64 products of the values that the operands stand for."""
    T, N, K = 300, 200, 500
    g = torch.Generator(device="cuda").manual_seed(22)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()
    x, w, dy = randn(T, K), randn(N, K), randn(T, N)
    for fmt in FORMATS:
        ops = {}
        for name, v in (("x", x), ("w", w), ("dy", dy)):
            amax = agoq.agoq_amax(v) if fmt == agoq.NVFP4 else None
            ops[name] = (*agoq.agoq_fp4_quant(v, fmt, amax, columns=True), amax)

        def part(name, turned):
            codes, scales, codes_t, scales_t, amax = ops[name]
            rows, cols = {"x": x, "w": w, "dy": dy}[name].shape
            op = Operand.__new__(Operand)
            op.codes, op.scales = (codes_t, scales_t) if turned else (codes, scales)
            op.rows, op.K = (cols, rows) if turned else (rows, cols)
            op.amax = amax
            op.values = F.values(op.codes, op.scales, op.rows, op.K, fmt)
            if amax is not None:
                op.values = op.values * F.tensor_scale(float(amax))
            return op
        for a, b, shape in ((("x", False), ("w", False), (T, N)), (("dy", False), ("w", True), (T, K)),
                            (("dy", True), ("x", True), (N, K))):
            a, b = part(*a), part(*b)
            d = _gemm(a, b, fmt, dtype=F32)
            assert d.shape == shape
            _check(a, b, d)


def test_refusals():
    a, b = _operand(8, 64, agoq.NVFP4, 23), _operand(16, 64, agoq.NVFP4, 24)
    call = lambda **kw: _gemm(a, b, agoq.NVFP4, **kw)
    with pytest.raises(TypeError):
        call(dtype=torch.float64)
    with pytest.raises(ValueError):
        call(d=torch.empty(16, 8, device="cuda"))
    with pytest.raises(ValueError):
        agoq.agoq_fp4_gemm(a.codes, a.scales, b.codes, b.scales, 8, 17, 64, agoq.NVFP4, a.amax, b.amax)
    with pytest.raises(ValueError):
        agoq.agoq_fp4_gemm(a.codes, a.scales, b.codes, b.scales, 8, 16, 96, agoq.NVFP4, a.amax, b.amax)
    with pytest.raises(agoq.AgoqError):
        agoq.agoq_fp4_gemm(a.codes, a.scales, b.codes, b.scales, 8, 16, 64, agoq.NVFP4, a.amax)
    with pytest.raises(ValueError):
        agoq.agoq_fp4_gemm(a.codes, a.scales, b.codes, b.scales, 8, 16, 64, 5, a.amax, b.amax)
    with pytest.raises(TypeError):
        agoq.agoq_fp4_gemm(a.codes.cpu(), a.scales, b.codes, b.scales, 8, 16, 64, agoq.NVFP4, a.amax, b.amax)
