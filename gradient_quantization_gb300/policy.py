"""The output end of a policy training step on the library's calls: final layer norm, output
projection and its two gradients as micro-scaled 4-bit products, the clipped policy loss or the
preference loss in between, the weight gradient in an FP8 master ("AGoQ: Activation and Gradient
Quantization for Memory-Efficient Distributed Training of LLMs", sections 2.A and 2.B, applied to
the last layer of a policy).

Between the forward and the backward pass of a micro-batch the norm's input is kept as low-bit
codes and the projection's operand in FP4, along its columns alone; the logits become their own
gradient in place.  The gradient's operands are rounded to the nearest code, not stochastically:
elements below half a step of their block are 0.

    head = PolicyHead(norm_w, norm_b, weight)              # BF16 [H], [H], [V][H]
    old = head.logprobs(x, tokens)                         # of the sampling policy, FP32 [T]
    for x, tokens, ... in micro_batches:                   # BF16 [T][H], int64 [T]
        loss, kl, dx = head.policy(x, tokens, old, advantages, weights, ref_logp)
    norm = head.clip(1.0)                                  # then the optimizer's step
    head.requantise()                                      # of the new weight

``python -m gradient_quantization_gb300.policy`` runs one on random data.
"""
import torch

from . import agoq


class PolicyHead:
    """Weights (the caller's), the projection's FP4 operands, gradients and the list that clips
    them.  V and H are multiples of 128; a micro-batch has any number of tokens from one on."""

    def __init__(self, norm_w, norm_b, weight, fmt=agoq.NVFP4, bits=4, eps=1e-5, clip_low=0.2,
                 clip_high=0.2, kl_coef=0.0):
        self.norm_w, self.norm_b, self.weight = norm_w, norm_b, weight
        self.fmt, self.bits, self.eps = fmt, bits, eps
        self.clip_low, self.clip_high, self.kl_coef = clip_low, clip_high, kl_coef
        V, H = weight.shape
        dev = weight.device
        self.master = torch.zeros(V * H, dtype=torch.uint8, device=dev)
        self.master_scales = torch.zeros(V * H // agoq.BLOCK, dtype=torch.float32, device=dev)
        self.norm_dw = torch.zeros(H, dtype=torch.float32, device=dev)
        self.norm_db = torch.zeros(H, dtype=torch.float32, device=dev)
        self.grads = agoq.GradList([(self.master, self.master_scales), self.norm_dw, self.norm_db])
        self.requantise()

    def _operand(self, x, columns=True):
        """(codes, scales, codes_t, scales_t, amax) of a matrix."""
        amax = agoq.agoq_amax(x) if self.fmt == agoq.NVFP4 else None
        return (*agoq.agoq_fp4_quant(x, self.fmt, amax, columns=columns), amax)

    def requantise(self):
        """The projection's operands from the weight as it is now: its rows for the logits, its
        columns for the gradient of their input."""
        self.operand = self._operand(self.weight)

    def _logits(self, y, columns=True):
        """(logits, FP4 operand) of the normed input; its columns are for the weight gradient."""
        op = self._operand(y, columns)
        w = self.operand
        V, H = self.weight.shape
        return agoq.agoq_fp4_gemm(op[0], op[1], w[0], w[1], y.shape[0], V, H, self.fmt, op[4],
                                  w[4], dtype=y.dtype), op

    def logprobs(self, x, tokens):
        """Log probabilities of tokens, FP32 [T]: of the policy that samples, or a reference."""
        y = agoq.agoq_layernorm_forward(x, self.norm_w, self.norm_b, self.eps, want_stats=False)[0]
        logits, _ = self._logits(y, columns=False)
        return agoq.agoq_token_logprobs(logits, tokens, want_entropy=False)[0]

    def _forward(self, x):
        """(logits, what is kept for _backward): the columns of the projection's operand (its rows
        are done with) and the codes of the norm's input."""
        y, _, _, codes, scales = agoq.agoq_layernorm_forward(
            x, self.norm_w, self.norm_b, self.eps, bits=self.bits, want_stats=False)
        logits, op = self._logits(y)
        return logits, op[2:], codes, scales

    def _backward(self, dlogits, y_columns, codes, scales):
        """dx of the logits' gradient; adds this micro-batch's gradients."""
        T, V = dlogits.shape
        H = self.weight.shape[1]
        d, w = self._operand(dlogits), self.operand
        # dW = dlogits^T y, summed over the tokens: columns of both
        yc, ys, y_amax = y_columns
        dweight = agoq.agoq_fp4_gemm(d[2], d[3], yc, ys, V, H, T, self.fmt, d[4], y_amax,
                                     dtype=dlogits.dtype)
        agoq.agoq_grad_accum_fp8(self.master, self.master_scales, dweight)
        # dy = dlogits W, summed over the vocabulary: rows of the gradient, columns of the weight
        dy = agoq.agoq_fp4_gemm(d[0], d[1], w[2], w[3], T, H, V, self.fmt, d[4], w[4],
                                dtype=dlogits.dtype)
        dx, dw, db = agoq.agoq_layernorm_backward_laaq(codes, scales, self.bits, dy, self.eps,
                                                       self.norm_w)
        self.norm_dw += dw
        self.norm_db += db
        return dx

    def policy(self, x, tokens, old_logp, advantages, weights=None, ref_logp=None):
        """One micro-batch of sampled tokens under the clipped policy loss: returns (loss, kl, dx),
        loss and kl FP32 [T] (kl None without a reference), and adds its gradients."""
        logits, *kept = self._forward(x)
        loss, _, kl, dlogits = agoq.agoq_policy_loss(
            logits, tokens, old_logp, advantages, ref_logp, weights, self.clip_low, self.clip_high,
            self.kl_coef, dlogits=logits)
        return loss, kl, self._backward(dlogits, *kept)

    def preference(self, x, tokens, offsets, ref_logp=None, weights=None, beta=0.1,
                   label_smoothing=0.0):
        """One micro-batch of pairs of answers (offsets: agoq_preference_loss) under the preference
        loss: returns (loss, margin, dx), loss and margin FP32 [P], and adds its gradients."""
        logits, *kept = self._forward(x)
        logp, _, lse, _, _ = agoq.agoq_token_logprobs(logits, tokens, want_entropy=False)
        loss, margin, dlogp = agoq.agoq_preference_loss(logp, offsets, ref_logp, weights, beta,
                                                        label_smoothing)
        dlogits = agoq.agoq_token_logprobs_backward(logits, tokens, lse, dlogp, dlogits=logits)
        return loss, margin, self._backward(dlogits, *kept)

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
    head = PolicyHead(randn(hidden) * 0.1 + 1, randn(hidden) * 0.1,
                      randn(vocabulary, hidden) * hidden ** -0.5, kl_coef=0.05)
    weights = torch.full((tokens,), 1 / (tokens * micro_batches), device="cuda")
    total = 0.0
    for _ in range(micro_batches):
        x = randn(tokens, hidden)
        ids = torch.randint(0, vocabulary, (tokens,), generator=g, device="cuda")
        logp = head.logprobs(x, ids)
        old = logp - 0.1 * torch.randn(tokens, generator=g, device="cuda")
        advantages = torch.randn(tokens, generator=g, device="cuda")
        loss, kl, dx = head.policy(x, ids, old, advantages, weights, ref_logp=old)
        total += float(loss.sum())
    offsets = torch.arange(0, tokens + 1, tokens // 8, device="cuda")
    pair_loss, margin, dx = head.preference(x, ids, offsets, ref_logp=old)
    norm = float(head.clip(0.01))
    agoq.agoq_device_status()
    print("policy loss %.4f, preference loss %.4f, gradient norm %.5f, after clipping %.5f"
          % (total, float(pair_loss.mean()), norm, float(agoq.agoq_grad_norm(head.grads))))


if __name__ == "__main__":
    main()
