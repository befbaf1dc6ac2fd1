"""agoq_preference_loss where the margin is infinite: each term of the loss at its limit."""
import math

import pytest
import torch

from gradient_quantization_gb300 import agoq

pytestmark = pytest.mark.gpu


# (1 - e) ln(1 + e^-h) + e ln(1 + e^h): the first term grows without bound as h falls, the second
# as it rises; one whose factor is 0 is not there.  The gradient's 1/(1 + e^h) - e is 1 - e and -e.
@pytest.mark.parametrize("eps,falls,rises", [(0.0, math.inf, 0.0), (0.5, math.inf, math.inf),
                                             (1.0, 0.0, math.inf)])
@pytest.mark.parametrize("length", [3, 400])           # a warp a pair, and a CTA
def test_infinite_margins(eps, falls, rises, length):
    logp = torch.zeros(4 * length, device="cuda")
    logp[1] = -math.inf                                # chosen answer of pair 0: h = -inf
    logp[3 * length + 1] = -math.inf                   # rejected answer of pair 1: h = inf
    offsets = torch.arange(5, device="cuda") * length
    loss, margin, dlogp = agoq.agoq_preference_loss(logp, offsets, beta=0.5, label_smoothing=eps)
    assert margin.tolist() == [-math.inf, math.inf]
    assert loss.tolist() == [falls, rises]
    for p, c in enumerate((0.5 * (1 - eps), -0.5 * eps)):      # exact in binary32
        chosen, rejected = dlogp[2 * p * length:2 * (p + 1) * length].chunk(2)
        assert bool((chosen == -c).all()) and bool((rejected == c).all())
