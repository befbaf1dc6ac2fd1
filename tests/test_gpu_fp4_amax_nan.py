"""NVFP4 codes of finite blocks under an amax that is not finite (a running one that has become NaN
or infinite after the codes were made): the values and products that the formulas give, in every
variant of the product."""
import math

import pytest
import torch

from gradient_quantization_gb300 import agoq
from tests.test_gpu_fp4_gemm import TYPES, _gemm, _operand

pytestmark = pytest.mark.gpu
NV = agoq.NVFP4


def _one(v):
    return torch.tensor([v], device="cuda")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad", [0, 1])                # rows at 16-byte boundaries, and not
@pytest.mark.parametrize("T,K", [(1, 16), (130, 77), (40, 1000)])
def test_values(dtype, pad, T, K):
    op = _operand(T, K, NV, 1)
    y = torch.zeros(T, K + pad, dtype=dtype, device="cuda")[:, :K]
    agoq.agoq_fp4_dequant(op.codes, op.scales, T, K, NV, _one(math.nan), y=y)
    assert torch.isnan(y).all()
    # an infinite tensor scale: the sign of each value, and NaN for 0
    agoq.agoq_fp4_dequant(op.codes, op.scales, T, K, NV, _one(math.inf), y=y)
    zero = op.values == 0
    assert torch.isnan(y[zero]).all()
    assert torch.equal(y[~zero].float(), op.values[~zero].sign().float() * math.inf)


# 32, 64 and 128 columns with K shared, single CTAs, CTA pairs; either operand the larger
@pytest.mark.parametrize("M,N,K", [(1, 300, 1000), (300, 5, 1000), (50, 300, 500), (300, 200, 9000),
                                   (300, 200, 500), (2600, 2100, 100), (1001, 4090, 3999)])
def test_products(M, N, K):
    a, b = _operand(M, K, NV, 2), _operand(N, K, NV, 3)
    good = a.amax, b.amax
    for first, second in ((math.nan, None), (None, math.nan), (math.nan, math.nan),
                          (math.inf, math.nan), (math.nan, math.inf)):
        a.amax, b.amax = (g if v is None else _one(v) for g, v in zip(good, (first, second)))
        for dtype in TYPES:
            assert torch.isnan(_gemm(a, b, NV, dtype=dtype)).all(), (first, second, dtype)
    agoq.agoq_device_status()


@pytest.mark.parametrize("given", [math.nan, math.inf, -math.inf])
def test_codes_made_with_it(given):
    """As before: NaN scales, codes of 0."""
    x = torch.randn(130, 200, device="cuda").bfloat16()
    for rows, columns in ((True, False), (False, True), (True, True)):
        c, s, ct, st = agoq.agoq_fp4_quant(x, NV, _one(given), rows=rows, columns=columns)
        for codes, scales, T, K in ((c, s, 130, 200), (ct, st, 200, 130)):
            if codes is not None:
                assert not codes.any()
                assert torch.isnan(agoq.agoq_fp4_dequant(codes, scales, T, K, NV, _one(1.0))).all()
