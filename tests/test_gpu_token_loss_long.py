"""The loss of rows that no cluster holds in shared memory (more than 8 x 216 KB), against
the plain binary64 forms."""
import math

import pytest
import torch

from gradient_quantization_gb300 import agoq
from tests.test_gpu_token_logprobs import BF16, F16, F32, _check_loss, _logits, _tokens

pytestmark = pytest.mark.gpu
# 8 x 221184 bytes less a vector: the last row that a cluster takes, and the first beyond
EDGE = {F32: 442364, BF16: 884728, F16: 884728}


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("more,pad,shift", [(0, 0, 0), (1, 0, 0), (37, 5, 3), (100001, 0, 1)])
def test_loss_and_gradient(dtype, more, pad, shift):
    V = EDGE[dtype] + more
    x, tokens = _logits(6, V, dtype, 51, pad=pad, shift=shift), _tokens(6, V)
    x[1, V // 3:] = -math.inf
    x[2] = -math.inf
    x[3, ::2] = torch.finfo(dtype).min
    tokens[1], tokens[4], tokens[5] = 0, -100, V
    w = torch.rand(6, device="cuda") + 0.1
    logp, grad = agoq.agoq_token_loss(x, tokens, w)
    _check_loss(x, tokens, w, logp, grad)
    assert not grad[2].any() and not grad[4].any() and bool(torch.isnan(grad[5]).all())
    z = x.clone()                                  # another row distance, and in place
    lp, got = agoq.agoq_token_loss(z, tokens, w, dlogits=z)
    assert got is z
    _check_loss(x, tokens, w, lp, z)
    if pad == 0 and shift == 0:
        assert torch.equal(lp[:5], logp[:5]) and torch.equal(z[:5], grad[:5])
