"""The output end of a training step (gradient_quantization_gb300/head.py): the layer
norm, loss and clipping calls with the framework's quantizers and fused weight-gradient
product, against binary64 autograd of the same function.

What the path rounds: the norm's output, the logits and their gradient to BF16 (2^-8
each), the norm's input to 4 bits for the backward pass, the projection's operand to 4
bits, the master to E4M3 (2^-4).  4-bit codes of a normal block of 128 (absmax near 2.8
sigma, step 0.4 sigma) have an error of 0.4 / sqrt(12) = 0.12 of the signal, so the weight
gradient is within 0.12 + 0.03 (E4M3's mean error) + 0.02, and the norm's input gradient,
which sees that error through one of three terms and the BF16 roundings, within 0.03."""
import pytest
import torch

from gradient_quantization_gb300 import agoq
from gradient_quantization_gb300.head import OutputHead
from tests import plain64 as P

pytestmark = pytest.mark.gpu


def _far(got, want):
    return float((got.double() - want).norm() / want.norm())


def test_micro_batches_and_clipping():
    T, H, V = 192, 512, 1024
    g = torch.Generator(device="cuda").manual_seed(3)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()
    w, b, weight = randn(H) * 0.1 + 1, randn(H) * 0.1, randn(V, H) * H ** -0.5
    head = OutputHead(w, b, weight)
    leaves = [t.double().requires_grad_() for t in (w, b, weight)]
    for k in range(2):
        x = randn(T, H)
        ids = torch.randint(0, V, (T,), generator=g, device="cuda")
        ids[k::17] = -100
        loss, dx = head.micro_batch(x, ids, 1 / T)
        x64 = x.double().requires_grad_()
        y, _, _ = P.layernorm(x64, leaves[0], leaves[1], head.eps)
        want = -P.token_logprobs(y @ leaves[2].t(), ids)[0].sum() / T
        want.backward()
        assert abs(float(loss) - want.item()) <= 0.005 * want.item()
        assert _far(dx, x64.grad) <= 0.03
    dw, db, dweight = (t.grad for t in leaves)
    master = P.grad_values((head.master, head.master_scales)).view(V, H)
    assert _far(master, dweight) <= 0.17
    assert _far(head.norm_dw, dw) <= 0.15 and _far(head.norm_db, db) <= 0.02
    parts = [(head.master.clone(), head.master_scales.clone()), head.norm_dw.clone(),
             head.norm_db.clone()]
    before = P.grad_norm(parts)
    norm = float(head.clip(0.25 * before))
    assert abs(norm - before) <= 1e-5 * before
    after = P.grad_norm([(head.master, head.master_scales), head.norm_dw, head.norm_db])
    assert abs(after - 0.25 * before) <= 1e-5 * before
    assert torch.equal(head.master, parts[0][0])
    head.zero_grad()
    assert float(agoq.agoq_grad_norm(head.grads)) == 0
