"""A token outside the vocabulary gives a row of NaN in both gradients, in a row of nothing
but -inf too."""
import math

import pytest
import torch

from gradient_quantization_gb300 import agoq

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("V,pad", [(50, 0), (50, 3), (32003, 0), (32000, 5)])
def test_a_token_beyond_in_an_empty_row(dtype, V, pad):
    x = torch.full((3, V + pad), -math.inf, dtype=dtype, device="cuda")[:, :V]
    tokens = torch.tensor([V, 2, -1]).cuda()
    logp, ent, lse, _, _ = agoq.agoq_token_logprobs(x, tokens)
    ones = torch.ones(3, device="cuda")
    for e, d in ((None, None), (ent, ones)):
        grad = agoq.agoq_token_logprobs_backward(x, tokens, lse, ones, e, d)
        assert torch.isnan(grad[0]).all() and not grad[1:].any()
    grad = agoq.agoq_token_loss(x, tokens)[1]
    assert torch.isnan(grad[0]).all() and not grad[1:].any()
