"""The norm of FP8 masters whose codes are zero under a scale that is not finite: a
value is the code times its block's scale, 0 times an infinity or NaN is NaN."""
import math

import pytest
import torch

from gradient_quantization_gb300 import agoq

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("zero", [0x00, 0x80])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("blocks,at", [(1, 0), (300, 0), (300, 299), (4001, 2000)])
def test_zero_codes(zero, bad, blocks, at):
    codes = torch.full((128 * blocks,), zero, dtype=torch.uint8, device="cuda")
    scales = torch.full((blocks,), 1e-3, device="cuda")
    scales[at] = bad
    assert math.isnan(float(agoq.agoq_grad_norm(agoq.GradList([(codes, scales)]))))


def test_large_finite_scales_of_zero_codes():
    codes = torch.zeros(1280, dtype=torch.uint8, device="cuda")
    scales = torch.full((10,), 3e38, device="cuda")       # whose square is beyond binary32
    assert float(agoq.agoq_grad_norm(agoq.GradList([(codes, scales)]))) == 0


def test_norm_after_clipping_by_nan():
    """A NaN gradient makes the coefficient NaN, and with it the scales of a master of zeros."""
    codes, scales = torch.zeros(256, dtype=torch.uint8, device="cuda"), torch.ones(2, device="cuda")
    agoq.agoq_clip_grads(agoq.GradList([(codes, scales)]), 1.0,
                         torch.full((1,), math.nan, device="cuda"))
    assert bool(torch.isnan(scales).all())
    assert math.isnan(float(agoq.agoq_grad_norm(agoq.GradList([(codes, scales)]))))
