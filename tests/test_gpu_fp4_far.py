"""FP4 and policy calls on tensors of more than 2^31 elements: the rows beyond are compared with
calls on those rows alone, which have small offsets."""
import pytest
import torch

from gradient_quantization_gb300 import agoq
from tests import plain_fp4 as F

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def test_long_rows():
    """130 rows of 2^24, the longest that the calls take."""
    T, K = 130, 1 << 24
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(T, K, dtype=BF16, device="cuda")
    for t in (0, 1, 127, 128, 129):
        x[t] = torch.randn(K, generator=g, device="cuda")
    x[2:127] = x[1]
    amax = agoq.agoq_amax(x)
    assert float(amax) == float(x[[0, 1, 127, 128, 129]].abs().max())
    codes, scales, _, _ = agoq.agoq_fp4_quant(x, agoq.NVFP4, amax)
    tail, tail_scales, _, _ = agoq.agoq_fp4_quant(x[128:], agoq.NVFP4, amax)
    assert torch.equal(codes[128:], tail) and torch.equal(scales[-len(tail_scales):], tail_scales)
    y = agoq.agoq_fp4_dequant(codes, scales, T, K, agoq.NVFP4, amax)
    assert torch.equal(y[128:], agoq.agoq_fp4_dequant(tail, tail_scales, 2, K, agoq.NVFP4, amax))
    want, _ = F.stored(x[129:, -4096:].double(), agoq.NVFP4, float(amax))
    assert torch.equal(codes[129:, -2048:], want)


def test_columns_of_many_rows():
    """140000 rows of 16384 along their columns: a strip of columns against the strip alone."""
    T, K = 140000, 16384
    x = torch.zeros(T, K, dtype=BF16, device="cuda")
    x[:, -256:] = torch.randn(T, 256, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda")
    _, _, codes, scales = agoq.agoq_fp4_quant(x, agoq.MXFP4, rows=False, columns=True)
    _, _, strip, strip_scales = agoq.agoq_fp4_quant(x[:, -256:], agoq.MXFP4, rows=False, columns=True)
    assert torch.equal(codes[-256:], strip) and torch.equal(scales[-len(strip_scales):], strip_scales)
    assert not codes[:-256].any()


@pytest.mark.parametrize("K", [64, 3000])
def test_a_large_product(K):
    """65600 x 33000: exact sums, the last rows against a product of those rows; by single CTAs and
    by CTA pairs."""
    M, N = 65600, 33000
    g = torch.Generator(device="cuda").manual_seed(3)
    a, b = (torch.randint(0, 16, (n, K), generator=g, device="cuda").to(torch.uint8) for n in (M, N))
    a, b = (torch.nn.functional.pad(v, (0, -K % 32)) for v in (a, b))
    sa, sb = (F.tile(torch.randint(127, 129, (n, a.shape[1] // 32), generator=g, device="cuda").to(torch.uint8)) for n in (M, N))
    d = agoq.agoq_fp4_gemm(F.pack(a), sa, F.pack(b), sb, M, N, K, agoq.MXFP4)
    agoq.agoq_device_status()
    assert d.numel() > 2 ** 31
    bv = F.values(F.pack(b), sb, N, K, agoq.MXFP4)
    av = F.values(F.pack(a), sa, M, K, agoq.MXFP4)
    for rows in (slice(0, 70), slice(M // 2, M // 2 + 70), slice(M - 70, M)):
        assert torch.equal(d[rows], (av[rows] @ bv.t()).to(BF16))


def test_policy_of_many_rows():
    T, V = 70000, 32000
    x = torch.empty(T, V, dtype=BF16, device="cuda").normal_(
        generator=torch.Generator(device="cuda").manual_seed(4))
    tokens = torch.arange(T, device="cuda") % V
    old, A = torch.full((T,), -10.0, device="cuda"), torch.ones(T, device="cuda")
    tail = x[-50:].clone()
    want = agoq.agoq_policy_loss(tail, tokens[-50:], old[-50:], A[-50:], clip_high=1e6)
    got = agoq.agoq_policy_loss(x, tokens, old, A, clip_high=1e6, dlogits=x)
    # (few rows are shared by clusters: other sums)
    assert torch.allclose(got[0][-50:], want[0], rtol=1e-5) and torch.allclose(got[1][-50:], want[1], rtol=1e-6)
    assert torch.allclose(x[-50:].float(), want[3].float(), rtol=1e-2, atol=1e-12)
