"""The output end of a training step on the library's calls: final layer norm,
output projection, loss of the next tokens, their gradients into an FP8 master,
and the clipping of all of them ("AGoQ: Activation and Gradient Quantization for
Memory-Efficient Distributed Training of LLMs", sections 2.A and 2.B, applied to
the last layer).

Between the forward and the backward pass of a micro-batch nothing wider than the
low-bit codes of the norm's input is kept: the logits become their own gradient in
place, the weight gradient is accumulated in an FP8 master, and the norm's backward
pass works from the codes.

    head = OutputHead(norm_w, norm_b, weight)             # BF16 [H], [H], [V][H]
    for x, tokens in micro_batches:                       # BF16 [T][H], int64 [T]
        loss, dx = head.micro_batch(x, tokens, 1 / total_tokens)
    norm = head.clip(1.0)                                 # then the optimizer's step

``python -m gradient_quantization_gb300.head`` runs one on random data.
"""
import torch

from . import agoq


class OutputHead:
    """Weights (the caller's), gradients and the list that clips them.

    V and H are multiples of 128, a micro-batch's token count of 64 (the FP8
    accumulation's tiles)."""

    def __init__(self, norm_w, norm_b, weight, bits=4, eps=1e-5):
        self.norm_w, self.norm_b, self.weight = norm_w, norm_b, weight
        self.bits, self.eps = bits, eps
        V, H = weight.shape
        dev = weight.device
        self.master = torch.zeros(V * H, dtype=torch.uint8, device=dev)
        self.master_scales = torch.zeros(V * H // agoq.BLOCK, dtype=torch.float32, device=dev)
        self.norm_dw = torch.zeros(H, dtype=torch.float32, device=dev)
        self.norm_db = torch.zeros(H, dtype=torch.float32, device=dev)
        self.grads = agoq.GradList([(self.master, self.master_scales), self.norm_dw, self.norm_db])

    def micro_batch(self, x, tokens, weight_per_token):
        """Forward and backward pass of one micro-batch: returns (loss, dx), the loss
        -sum(weight_per_token * logp) over tokens >= 0, and adds this micro-batch's gradients."""
        T, H = x.shape
        V = self.weight.shape[0]
        y, _, _, codes, scales = agoq.agoq_layernorm_forward(
            x, self.norm_w, self.norm_b, self.eps, bits=self.bits, want_stats=False)
        logits = y @ self.weight.t()
        weights = torch.full((T,), weight_per_token, dtype=torch.float32, device=x.device)
        logp, dlogits = agoq.agoq_token_loss(logits, tokens, weights, dlogits=logits)
        # the projection's operand for its weight gradient, in 4 bits too
        y_codes, y_scales = agoq.agoq_quant_act(y, 4)
        agoq.agoq_wgrad_gemm_int4_accum_fp8(dlogits, y_codes, y_scales, V, H, T, self.master,
                                            self.master_scales)
        dy = dlogits @ self.weight
        dx, dw, db = agoq.agoq_layernorm_backward_laaq(codes, scales, self.bits, dy, self.eps,
                                                       self.norm_w)
        self.norm_dw += dw
        self.norm_db += db
        return -weight_per_token * logp.sum(), dx

    def clip(self, max_norm):
        """Clip the accumulated gradients in place (of the master the scales); returns their
        norm before that."""
        return agoq.agoq_clip_grad_norm(self.grads, max_norm)

    def zero_grad(self):
        for t in (self.master, self.master_scales, self.norm_dw, self.norm_db):
            t.zero_()


def main(tokens=4096, hidden=4096, vocabulary=32000, micro_batches=2):
    g = torch.Generator(device="cuda").manual_seed(0)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()
    head = OutputHead(randn(hidden) * 0.1 + 1, randn(hidden) * 0.1,
                      randn(vocabulary, hidden) * hidden ** -0.5)
    loss = 0.0
    for _ in range(micro_batches):
        ids = torch.randint(0, vocabulary, (tokens,), generator=g, device="cuda")
        part, dx = head.micro_batch(randn(tokens, hidden), ids, 1 / (tokens * micro_batches))
        loss += float(part)
    norm = float(head.clip(0.01))
    agoq.agoq_device_status()
    print("loss %.4f, gradient norm %.5f, after clipping %.5f"
          % (loss, norm, float(agoq.agoq_grad_norm(head.grads))))


if __name__ == "__main__":
    main()
