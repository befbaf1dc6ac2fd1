"""Rows of logits with a NaN or +inf, whose statistics are NaN, where the token, an
alternative or the weight is one that could hide it."""
import math

import pytest
import torch

from gradient_quantization_gb300 import agoq

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
# a warp a row, a CTA a row, a cluster a row, and (the loss) rows beyond a cluster
LENGTHS = {F32: [50, 6000, 131072, 442400], BF16: [50, 6000, 131072, 884800],
           F16: [51, 6001, 131073, 884801]}
CASES = [(d, V) for d, n in LENGTHS.items() for V in n]


def _logits(V, dtype):
    g = torch.Generator(device="cuda").manual_seed(3)
    x = (3 * torch.randn(5, V, generator=g, device="cuda")).to(dtype)
    x[1, V // 2], x[1, 5] = math.nan, -math.inf
    x[2, V - 1], x[2, 6] = math.inf, -math.inf
    x[3] = -math.inf
    x[3, 7] = math.nan
    return x, torch.tensor([1, 5, 6, 0, 4]).cuda()


@pytest.mark.parametrize("dtype,V", CASES)
def test_a_token_of_probability_zero(dtype, V):
    """Its logit is -inf, but the row's statistics are NaN, and so is its log probability."""
    x, tokens = _logits(V, dtype)
    logp = agoq.agoq_token_logprobs(x, tokens)[0]
    assert torch.isnan(logp[1:4]).all() and torch.isfinite(logp[[0, 4]]).all()
    logp = agoq.agoq_token_loss(x, tokens)[0]
    assert torch.isnan(logp[1:4]).all() and torch.isfinite(logp[[0, 4]]).all()
    tokens[1:4] = -1
    assert not agoq.agoq_token_logprobs(x, tokens)[0][1:4].any()      # ignored: 0
    assert not agoq.agoq_token_loss(x, tokens)[0][1:4].any()


@pytest.mark.parametrize("dtype,V", CASES)
def test_alternatives_of_probability_zero(dtype, V):
    x, tokens = _logits(V, dtype)
    _, _, _, top, ids = agoq.agoq_token_logprobs(x, tokens, k=4)
    assert ids[3].tolist() == [7, 0, 1, 2]                            # NaN, then -inf in order
    assert torch.isnan(top[1:4]).all() and torch.isfinite(top[[0, 4]]).all()


@pytest.mark.parametrize("dtype,V", CASES)
def test_a_weight_of_zero(dtype, V):
    """0 times the probabilities of such a row is NaN; of any other row 0."""
    x, tokens = _logits(V, dtype)
    grad = agoq.agoq_token_loss(x, tokens, torch.zeros(5, device="cuda"))[1]
    assert torch.isnan(grad[1:4]).all() and not grad[[0, 4]].any()
    tokens[1:4] = -1
    assert not agoq.agoq_token_loss(x, tokens)[1][1:4].any()          # ignored: 0
