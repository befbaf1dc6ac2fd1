"""Cases of the layer norm, the gradient norm with clipping and the token log
probabilities: their inputs, their plain forms and what they have to move.

With `own` false, `run` computes a case with elementary torch operations in
binary32 (binary64 for long sums); with `own` true it makes the library's calls.
`exact` gives the same outputs from the definitions in binary64.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4, "e4m3": 1 + 4 / 128}
EPS = 1e-5              # layer norm
GRAD_STD = 1e-3         # clipping
NORM_EPS = 1e-6


def listed():
    return [
        # the norm in front of one generated token's projections: latency alone
        {"name": "ln_fwd_1x4096", "op": "ln_fwd", "T": 1, "H": 4096, "dtype": "bf16",
         "params": "same", "pad": 0},
        # a ragged batch of packed sequences, odd rows inside a wider buffer, half precision
        {"name": "ln_fwd_6151x5003_f16", "op": "ln_fwd", "T": 6151, "H": 5003, "dtype": "f16",
         "params": "f32", "pad": 13},
        # backward of one layer's norm on a training micro-batch (8192 tokens, hidden 4096)
        {"name": "ln_bwd_8192x4096", "op": "ln_bwd", "T": 8192, "H": 4096, "dtype": "bf16",
         "params": "same", "pad": 0},
        # the same norm as the quantizing framework trains it: the forward pass keeps the 4-bit
        # codes of its input only, the backward pass works from them
        {"name": "ln_step_q4_8192x4096", "op": "ln_step", "T": 8192, "H": 4096, "dtype": "bf16",
         "params": "f32", "bits": 4},
        # gradients of small adapters: many short odd tensors, latency and tensor count
        {"name": "clip_adapters_f32", "op": "clip", "layers": 16, "hidden": 65, "ffn": 173,
         "grad": "f32", "active": True},
        # BF16 gradients of two layers' worth of weights (hidden 4096, FFN 11008), clipped
        {"name": "clip_2_layers_bf16", "op": "clip", "layers": 2, "hidden": 4096, "ffn": 11008,
         "grad": "bf16", "active": True},
        # FP8 masters of eight layers after the reduce, with FP32 norm vectors beside them
        {"name": "clip_8_layers_e4m3", "op": "clip", "layers": 8, "hidden": 4096, "ffn": 11008,
         "grad": "e4m3", "active": True},
        # one decoding step of a small batch: sampled tokens' log probabilities and 8 alternatives,
        # part of the vocabulary masked out
        {"name": "logprobs_8x32000", "op": "logprobs", "T": 8, "V": 32000, "dtype": "bf16", "k": 8,
         "mask": "inf", "pad": 0},
        # scoring a batch of prompts against a large vocabulary with 20 alternatives
        {"name": "logprobs_2048x128000", "op": "logprobs", "T": 2048, "V": 128000, "dtype": "bf16",
         "k": 20, "mask": "none", "pad": 0},
        # the loss of a training micro-batch and its gradient
        {"name": "loss_8192x32000", "op": "loss", "T": 8192, "V": 32000, "dtype": "bf16",
         "mask": "none", "pad": 0},
        # the same with FP32 logits of an odd vocabulary
        {"name": "loss_1021x50001_f32", "op": "loss", "T": 1021, "V": 50001, "dtype": "f32",
         "mask": "lowest", "pad": 0},
        # policy training with an entropy bonus: gradients of both through given statistics
        {"name": "logprobs_bwd_4096x32003", "op": "logprobs_bwd", "T": 4096, "V": 32003,
         "dtype": "bf16", "mask": "none", "pad": 5},
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["ln_fwd", "ln_bwd", "ln_step", "clip", "clip", "logprobs", "logprobs",
                     "loss", "loss", "logprobs_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op in ("ln_fwd", "ln_bwd"):
        H = _log_uniform(rng, 8, 16384)
        if rng.random() < 0.6:
            H = -(-H // 64) * 64
        T = _log_uniform(rng, 1, min(32768, (1 << 24) // H))
        return {"op": op, "T": T, "H": H, "dtype": dtype,
                "params": rng.choice(["same", "f32", "none"]), "pad": rng.choice([0, 0, 8, 3])}
    if op == "ln_step":
        H = 128 * _log_uniform(rng, 1, 96)
        T = _log_uniform(rng, 1, min(32768, (1 << 25) // H))
        return {"op": op, "T": T, "H": H, "dtype": "bf16",
                "params": rng.choice(["same", "f32", "none"]), "bits": rng.choice([4, 5, 6, 8])}
    if op == "clip":
        grad = rng.choice(["f32", "bf16", "f16", "e4m3"])
        hidden = _log_uniform(rng, 32, 4096)
        ffn = hidden * 2 + rng.randrange(hidden)
        if grad == "e4m3":
            hidden, ffn = -(-hidden // 128) * 128, -(-ffn // 128) * 128
        layer = 4 * hidden * hidden + 3 * hidden * ffn
        return {"op": op, "layers": _log_uniform(rng, 1, max(1, min(64, (1 << 28) // layer))),
                "hidden": hidden, "ffn": ffn, "grad": grad, "active": rng.random() < 0.7}
    V = _log_uniform(rng, 40, 160000)
    T = _log_uniform(rng, 1, min(16384, (1 << 26) // V))
    case = {"op": op, "T": T, "V": V, "dtype": dtype,
            "mask": rng.choice(["none", "none", "inf", "lowest"]), "pad": rng.choice([0, 0, 8, 7])}
    if op == "logprobs":
        case["k"] = rng.randrange(0, 33)
    return case


# ---- inputs ---------------------------------------------------------------------------------


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _rows(values, dtype, pad):
    """[T][n] values as `dtype` rows of a buffer whose rows are n + pad elements apart."""
    T, n = values.shape
    buf = torch.zeros(T, n + pad, dtype=DTYPES[dtype], device="cuda")
    buf[:, :n] = values
    return buf[:, :n]


def _tensor_sizes(case):
    """Weight gradients of the layers (attention, gated MLP) and their norms' FP32 vectors."""
    h, f = case["hidden"], case["ffn"]
    return [h * h] * 4 + [h * f] * 3, [h, h]


def _prepare_ln(case, g):
    T, H = case["T"], case["H"]
    x = _randn(g, T, H) + 0.3 * _randn(g, T, 1)
    x[torch.rand(T, H, generator=g, device="cuda") < 1e-3] *= 20
    s = {"x": _rows(x, case["dtype"], case.get("pad", 0)), "w": None, "b": None}
    if case["params"] != "none":
        t = DTYPES[case["dtype"] if case["params"] == "same" else "f32"]
        s["w"], s["b"] = (1 + 0.1 * _randn(g, H)).to(t), (0.1 * _randn(g, H)).to(t)
    if case["op"] != "ln_fwd":
        s["dy"] = _rows(_randn(g, T, H), case["dtype"], case.get("pad", 0))
    if case["op"] == "ln_bwd":   # the statistics that the forward pass kept
        v = s["x"].double()
        s["mean"] = v.mean(1).float()
        s["rstd"] = (v.var(1, unbiased=False) + EPS).rsqrt().float()
    return s


def _prepare_clip(case, g):
    """Gradients, and buffers of the clipped ones: one flat buffer per kind, as an optimizer
    holds them (of an FP8 master the scales alone change)."""
    weights, vectors = _tensor_sizes(case)
    kind = case["grad"]
    total = case["layers"] * sum(weights)
    # an active clip halves the gradient
    s = {"grads": [], "outs": [],
         "max_norm": 0.5 * GRAD_STD * math.sqrt(total) if case["active"] else 1e6}
    flat_w = torch.empty(total // 128 if kind == "e4m3" else total, device="cuda",
                         dtype=torch.float32 if kind == "e4m3" else DTYPES[kind])
    flat_v = torch.empty(case["layers"] * sum(vectors), device="cuda")
    at = {"w": 0, "v": 0}
    for n in (weights + vectors) * case["layers"]:
        value = _randn(g, n) * GRAD_STD
        vector = n == case["hidden"]
        if not vector and kind == "e4m3":
            v = value.view(-1, 128)
            scales = v.abs().amax(1) / 448
            codes = (v / scales[:, None]).to(torch.float8_e4m3fn).view(torch.uint8).view(-1)
            s["grads"].append((codes, scales))
            s["outs"].append(flat_w[at["w"]:at["w"] + n // 128])
            at["w"] += n // 128
            continue
        s["grads"].append(value if vector else value.to(DTYPES[kind]))
        flat, key = (flat_v, "v") if vector else (flat_w, "w")
        s["outs"].append(flat[at[key]:at[key] + n])
        at[key] += n
    s["flat"] = [flat_w, flat_v]
    if own:   # the list a training program builds once, over its gradient buffers
        from gradient_quantization_gb300 import agoq
        s["list"] = agoq.GradList(s["grads"], s["outs"])
    return s


def _prepare_logits(case, g):
    T, V, dtype = case["T"], case["V"], case["dtype"]
    x = 2.5 * _randn(g, T, V)
    if case["mask"] != "none":
        low = -math.inf if case["mask"] == "inf" else torch.finfo(DTYPES[dtype]).min
        off = torch.rand(T, V, generator=g, device="cuda") < 0.6
        if case["mask"] == "inf" and T >= 8:
            off[T // 2] = True                         # a row with nothing left
        x[off] = low
    logits = _rows(x, dtype, case["pad"])
    u = torch.rand(T, V, generator=g, device="cuda").clamp_(1e-12, 1 - 1e-7)
    tokens = (logits.float() - torch.log(-torch.log(u))).argmax(1)    # sampled from the softmax
    del x, u
    s = {"logits": logits, "tokens": tokens}
    if case["op"] == "logprobs":
        s["k"] = case["k"]
        return s
    ignored = torch.rand(T, generator=g, device="cuda") < 0.05        # padding
    s["tokens"] = torch.where(ignored, -100, tokens)
    if case["op"] == "loss":
        s["weights"] = torch.full((T,), 1.0 / max(1, T), device="cuda")
        return s
    lse = torch.logsumexp(logits.double(), 1)
    p = (logits.double() - lse[:, None]).exp()
    ent = -torch.where(p > 0, p * (logits.double() - lse[:, None]), 0.0).sum(1)
    s["lse"], s["entropy"] = lse.float(), ent.float()
    s["dlogp"], s["dentropy"] = _randn(g, T), 0.01 * _randn(g, T)
    return s


def prepare(case, seed):
    g = _gen(seed)
    if case["op"].startswith("ln"):
        s = _prepare_ln(case, g)
    elif case["op"] == "clip":
        s = _prepare_clip(case, g)
    else:
        s = _prepare_logits(case, g)
    s["case"] = case
    return s


# ---- one pass -------------------------------------------------------------------------------


def _plain_ln_fwd(x, w, b):
    v = x.float()
    mean = v.mean(1, keepdim=True)
    d = v - mean
    rstd = (d.square().mean(1, keepdim=True) + EPS).rsqrt()
    y = d * rstd
    if w is not None:
        y = y * w.float() + b.float()
    return y.to(x.dtype), mean.view(-1), rstd.view(-1)


def _plain_ln_bwd(v, dy, w, mean, rstd):
    xh = (v.float() - mean[:, None]) * rstd[:, None]
    d = dy.float()
    gr = d if w is None else d * w.float()
    dx = rstd[:, None] * (gr - gr.mean(1, keepdim=True) - xh * (gr * xh).mean(1, keepdim=True))
    return dx.to(dy.dtype), (d * xh).sum(0), d.sum(0)


def _plain_codes(x, bits):
    """The values the stored codes stand for: block-wise symmetric codes of 128 elements."""
    qmax = 2 ** (bits - 1) - 1
    v = x.float().view(-1, 128)
    # by a tensor: torch divides by a number as a product with its reciprocal, which is not fl(a / b)
    scale = v.abs().amax(1, keepdim=True) / torch.tensor(float(qmax), device="cuda")
    code = torch.where(scale > 0, torch.round(v / scale), 0.0).clamp(-qmax, qmax)
    return (code * scale).to(torch.bfloat16).view(x.shape)


def _plain_ln_step(s, bits):
    y, mean, rstd = _plain_ln_fwd(s["x"], s["w"], s["b"])
    v = _plain_codes(s["x"], bits).float()
    m = v.mean(1)
    r = ((v - m[:, None]).square().mean(1) + EPS).rsqrt()
    dx, dw, db = _plain_ln_bwd(v, s["dy"], s["w"], m, r)
    return {"y": y, "mean": mean, "rstd": rstd, "dx": dx, "dw": dw, "db": db}


def _plain_square_sum(grad):
    if isinstance(grad, tuple):
        codes, scales = grad
        v = codes.view(torch.float8_e4m3fn).float().view(-1, 128) * scales[:, None]
        return v.square().sum(dtype=torch.float64)
    return grad.float().square().sum(dtype=torch.float64)


def _plain_clip(s):
    norm = torch.stack([_plain_square_sum(t) for t in s["grads"]]).sum().sqrt().float()
    coef = (s["max_norm"] / (norm + NORM_EPS)).clamp(max=1.0)
    [o.copy_((t[1] if isinstance(t, tuple) else t.float()) * coef)
     for t, o in zip(s["grads"], s["outs"])]
    return {"norm": norm.view(1), "clipped": s["flat"][0], "vectors": s["flat"][1]}


def _plain_softmax(logits):
    """Shifted logits, their exponentials and sums; a row with nothing in it has sum 0."""
    x = logits.float()
    m = x.amax(1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    d = x - m
    e = d.exp()
    return x, m, d, e, e.sum(1, keepdim=True)


def _plain_pick(x, tokens, lse):
    at = x.gather(1, tokens.clamp(min=0)[:, None])
    logp = torch.where(at == -math.inf, at, at - lse).view(-1)
    return torch.where(tokens < 0, 0.0, logp)


def _plain_logprobs(s):
    x, m, d, e, total = _plain_softmax(s["logits"])
    lse = m + total.log()
    mean = torch.where(e > 0, e * d, 0.0).sum(1, keepdim=True) / total
    entropy = torch.where(total > 0, total.log() - mean, 0.0)
    out = {"logp": _plain_pick(x, s["tokens"], lse), "entropy": entropy.view(-1),
           "lse": lse.view(-1)}
    if s["k"]:
        top, ids = torch.sort(x, dim=1, descending=True, stable=True)
        top, ids = top[:, :s["k"]], ids[:, :s["k"]]
        out["top_logp"] = torch.where(top == -math.inf, top, top - lse)
        out["top_ids"] = ids.contiguous()
    return out


def _one_hot_add(p, tokens, value):
    """p with value [T] added at each row's token; ignored rows keep p."""
    at = tokens.clamp(min=0)[:, None]
    return p.scatter_add(1, at, torch.where(tokens < 0, 0.0, value)[:, None])


def _plain_loss(s):
    x, m, d, e, total = _plain_softmax(s["logits"])
    tokens = s["tokens"]
    logp = _plain_pick(x, tokens, m + total.log())
    w = torch.where((tokens < 0) | (total.view(-1) == 0), 0.0, s["weights"])
    grad = torch.where(total > 0, e / total, 0.0) * w[:, None]
    return {"logp": logp, "dlogits": _one_hot_add(grad, tokens, -w).to(s["logits"].dtype)}


def _plain_logprobs_bwd(s):
    x, lse, tokens = s["logits"].float(), s["lse"], s["tokens"]
    l = x - torch.where(lse == -math.inf, 0.0, lse)[:, None]
    p = l.exp()
    empty = lse == -math.inf
    a = torch.where((tokens < 0) | empty, 0.0, s["dlogp"])
    c = torch.where(empty, 0.0, s["dentropy"])
    grad = -p * (a[:, None] + torch.where(p > 0, c[:, None] * (l + s["entropy"][:, None]), 0.0))
    return {"dlogits": _one_hot_add(grad, tokens, a).to(s["logits"].dtype)}


def _run_plain(s):
    op = s["case"]["op"]
    if op == "ln_fwd":
        return dict(zip(("y", "mean", "rstd"), _plain_ln_fwd(s["x"], s["w"], s["b"])))
    if op == "ln_bwd":
        return dict(zip(("dx", "dw", "db"),
                        _plain_ln_bwd(s["x"], s["dy"], s["w"], s["mean"], s["rstd"])))
    if op == "ln_step":
        return _plain_ln_step(s, s["case"]["bits"])
    return {"clip": _plain_clip, "logprobs": _plain_logprobs, "loss": _plain_loss,
            "logprobs_bwd": _plain_logprobs_bwd}[op](s)


def _run_own(s):
    from gradient_quantization_gb300 import agoq
    op = s["case"]["op"]
    if op == "ln_fwd":
        y, mean, rstd, _, _ = agoq.agoq_layernorm_forward(s["x"], s["w"], s["b"], EPS)
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "ln_bwd":
        dx, dw, db = agoq.agoq_layernorm_backward(s["x"], s["dy"], s["mean"], s["rstd"], s["w"])
        return {"dx": dx, "dw": dw, "db": db}
    if op == "ln_step":
        bits = s["case"]["bits"]
        y, mean, rstd, codes, scales = agoq.agoq_layernorm_forward(s["x"], s["w"], s["b"], EPS,
                                                                   bits=bits)
        dx, dw, db = agoq.agoq_layernorm_backward_laaq(codes, scales, bits, s["dy"], EPS, s["w"])
        return {"y": y, "mean": mean, "rstd": rstd, "dx": dx, "dw": dw, "db": db}
    if op == "clip":
        norm = agoq.agoq_clip_grad_norm(s["list"], s["max_norm"])
        return {"norm": norm, "clipped": s["flat"][0], "vectors": s["flat"][1]}
    if op == "logprobs":
        logp, entropy, lse, top_logp, top_ids = agoq.agoq_token_logprobs(
            s["logits"], s["tokens"], k=s["k"], want_entropy=True)
        out = {"logp": logp, "entropy": entropy, "lse": lse}
        if s["k"]:
            out["top_logp"], out["top_ids"] = top_logp, top_ids
        return out
    if op == "loss":
        logp, dlogits = agoq.agoq_token_loss(s["logits"], s["tokens"], s["weights"])
        return {"logp": logp, "dlogits": dlogits}
    return {"dlogits": agoq.agoq_token_logprobs_backward(
        s["logits"], s["tokens"], s["lse"], s["dlogp"], s["entropy"], s["dentropy"])}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- what a pass has to move ----------------------------------------------------------------


def work(case):
    op = case["op"]
    if op.startswith("ln"):
        T, H = case["T"], case["H"]
        n, e = T * H, SIZE[case["dtype"]]
        p = 0 if case["params"] == "none" else e if case["params"] == "same" else 4
        if op == "ln_fwd":
            return {"bytes": 2 * n * e + 2 * H * p + 8 * T, "flops": 8 * n}
        if op == "ln_bwd":
            return {"bytes": 3 * n * e + H * p + 8 * T + 8 * H, "flops": 14 * n}
        q = case["bits"] / 8 + 4 / 128
        return {"bytes": n * (2 * e + q) + 2 * H * p + 8 * T + n * (q + 2 * e) + H * p + 8 * H,
                "flops": 30 * n}
    if op == "clip":
        weights, vectors = _tensor_sizes(case)
        nw, nv = case["layers"] * sum(weights), case["layers"] * sum(vectors)
        out = 4 / 128 if case["grad"] == "e4m3" else SIZE[case["grad"]]
        return {"bytes": nw * (SIZE[case["grad"]] + out) + nv * 8, "flops": 3 * (nw + nv)}
    T, n, e = case["T"], case["T"] * case["V"], SIZE[case["dtype"]]
    if op == "logprobs":
        return {"bytes": n * e + T * (8 + 12 + 12 * case["k"]), "flops": 6 * n}
    if op == "loss":
        return {"bytes": 2 * n * e + 16 * T, "flops": 8 * n}
    return {"bytes": 2 * n * e + 24 * T, "flops": 8 * n}


# ---- the definitions in binary64 --------------------------------------------------------------


def _exact_stats(v):
    mu = v.sum(1) / v.shape[1]
    return mu, 1.0 / torch.sqrt((v - mu[:, None]).pow(2).sum(1) / v.shape[1] + EPS)


def _exact_ln_grads(v, dy, w, mu, r):
    H = v.shape[1]
    n = (v - mu.unsqueeze(1)) * r.unsqueeze(1)
    up = dy.double()
    g = up if w is None else up * w.double().unsqueeze(0)
    s0 = g.sum(1, keepdim=True)
    s1 = torch.einsum("th,th->t", g, n).unsqueeze(1)
    return {"dx": r.unsqueeze(1) * (g - (s0 + n * s1) / H), "dw": torch.einsum("th,th->h", up, n),
            "db": up.sum(0)}


def _exact_ln(s, case):
    v = s["x"].double()
    mu, r = _exact_stats(v)
    if case["op"] == "ln_bwd":   # the statistics are inputs there
        return _exact_ln_grads(v, s["dy"], s["w"], s["mean"].double(), s["rstd"].double())
    y = (v - mu[:, None]) * r[:, None]
    if s["w"] is not None:
        y = y * s["w"].double() + s["b"].double()
    out = {"y": y, "mean": mu, "rstd": r}
    if case["op"] == "ln_step":
        # the stored values are defined by binary32 roundings: the scale, the quotient, the product
        top = 2 ** (case["bits"] - 1) - 1
        blocks = s["x"].float().reshape(-1, 128)
        divisor = torch.tensor(float(top), device="cuda")   # a tensor, as in _plain_codes
        step = torch.div(blocks.abs().max(dim=1).values, divisor).unsqueeze(1)
        quotient = torch.div(blocks, torch.where(step == 0, 1.0, step))
        kept = torch.mul(torch.round(quotient), step).bfloat16().double().reshape(v.shape)
        out.update(_exact_ln_grads(kept, s["dy"], s["w"], *_exact_stats(kept)))
    return out


def _exact_clip(s):
    def value(t):
        if isinstance(t, tuple):
            return (t[0].view(torch.float8_e4m3fn).double().reshape(-1, 128)
                    * t[1].double().unsqueeze(1))
        return t.double()
    norm = math.sqrt(sum(float(torch.linalg.vector_norm(value(t))) ** 2 for t in s["grads"]))
    c = min(1.0, s["max_norm"] / (norm + NORM_EPS))
    held = [(t[1] if isinstance(t, tuple) else t).double() * c for t in s["grads"]]
    per = 9
    return {"norm": torch.tensor([norm], dtype=torch.float64, device="cuda"),
            "clipped": torch.cat([h for i, h in enumerate(held) if i % per < 7]),
            "vectors": torch.cat([h for i, h in enumerate(held) if i % per >= 7])}


def _exact_logits(s, case):
    x, tok = s["logits"].double(), s["tokens"]
    rows = torch.arange(x.shape[0], device="cuda")
    lse = torch.logsumexp(x, 1)
    gone = torch.isneginf(lse)
    l = torch.where(torch.isneginf(x), -math.inf, x - torch.where(gone, 0.0, lse)[:, None])
    p = torch.exp(l)
    named = torch.where(tok >= 0, l[rows, tok.clamp(min=0)], 0.0)
    unit = torch.zeros_like(x)
    unit[rows, tok.clamp(min=0)] = (tok >= 0).double()
    if case["op"] == "logprobs":
        out = {"logp": named, "entropy": torch.special.entr(p).sum(1), "lse": lse}
        if s["k"]:
            out["top_logp"] = torch.topk(l, s["k"], dim=1).values
            out["top_ids"] = None
        return out
    live = ((tok >= 0) & ~gone).double()
    if case["op"] == "loss":
        return {"logp": named, "dlogits": (s["weights"].double() * live)[:, None] * (p - unit)}
    h = s["entropy"].double()[:, None]
    ent = torch.where(p > 0, -p * (l + h), 0.0) * s["dentropy"].double()[:, None]
    return {"dlogits": (s["dlogp"].double() * live)[:, None] * (unit - p) + ent}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("ln"):
        return _exact_ln(s, case)
    return _exact_clip(s) if case["op"] == "clip" else _exact_logits(s, case)
