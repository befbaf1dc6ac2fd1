"""agoq_fp4_gemm with several tiles to a CTA pair: the order of a tile's MMAs by halves of the
accumulator, from a K of one stage (256 elements) on to more stages than the halves hold, the next
tile's begin beside the last one's end, and tiles that D ends within."""
import pytest
import torch

from gradient_quantization_gb300 import agoq
from tests.test_gpu_fp4_gemm import FORMATS, _exact_operand, _gemm

pytestmark = pytest.mark.gpu


# 32 x 19 tiles of 256 x 256: eight to a pair
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("K", [1, 64, 256, 300, 700, 1000, 1217, 1536, 1700, 2048])
def test_exact_sums_of_every_round(fmt, K):
    """Bit for bit: partial sums are multiples of 1/4 below 2^22 (asserted), which binary32 holds in any
    order."""
    M, N = 8180, 4861 if K == 300 else 4864
    a, b = _exact_operand(M, K, fmt, 1), _exact_operand(N, K, fmt, 2)
    assert float((a.values.abs() @ b.values.abs().t()).max()) < 2 ** 22
    want = (a.values @ b.values.t()).float()
    for dtype in (torch.float32, torch.bfloat16):
        got = _gemm(a, b, fmt, dtype=dtype)
        assert torch.equal(got, want.to(dtype))
        assert torch.equal(got, _gemm(a, b, fmt, dtype=dtype))
    agoq.agoq_device_status()


@pytest.mark.parametrize("K", [200, 1000, 2000])
def test_two_streams(K):
    """Two products of many rounds at once, each as alone."""
    ops = [[_exact_operand(n, K, agoq.NVFP4, 3 + i + j) for j, n in enumerate((8192, 4864))] for i in (0, 2)]
    want = [_gemm(a, b, agoq.NVFP4) for a, b in ops]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ops]
    got = [[], []]
    for _ in range(4):
        for i, ((a, b), s) in enumerate(zip(ops, streams)):
            with torch.cuda.stream(s):
                got[i].append(_gemm(a, b, agoq.NVFP4))
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(x, w) for x in g)
    agoq.agoq_device_status()
