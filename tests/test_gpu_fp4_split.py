"""agoq_fp4_gemm where the stages of K do not divide by the CTAs that share them: 5, 6, 9 and 33
stages of 256 elements, either operand the one of few rows, and two CTAs for four stages."""
import pytest
import torch

from gradient_quantization_gb300 import agoq
from tests.test_gpu_fp4_gemm import FORMATS, TYPES, _exact_operand, _gemm

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K", [(5, 400, 1200), (400, 64, 1281), (700, 20, 1500), (40, 300, 2200),
                                   (300, 3, 2300), (3, 200, 8300), (200, 40, 8193), (2, 10000, 1000)])
def test_exact_sums(fmt, M, N, K):
    """Bit for bit: partial sums are multiples of 1/4 below 2^22 (asserted), which binary32 holds in any
    order."""
    a, b = _exact_operand(M, K, fmt, 1), _exact_operand(N, K, fmt, 2)
    assert float((a.values.abs() @ b.values.abs().t()).max()) < 2 ** 22
    want = (a.values @ b.values.t()).float()
    for dtype in TYPES:
        got = _gemm(a, b, fmt, dtype=dtype)
        assert torch.equal(got, want.to(dtype))
    agoq.agoq_device_status()
