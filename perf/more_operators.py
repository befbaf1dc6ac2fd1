"""Cases of the micro-scaled 4-bit quantisation and product, the clipped policy loss and the
preference loss: their inputs, their plain forms and what they have to move.

With `own` false, `run` computes a case with elementary torch operations in binary32 (binary64
for long sums); with `own` true it makes the library's calls.  `exact` gives the same outputs
from the definitions in binary64.

The stored 4-bit format, which prepared operands have too (`_store`): codes of E2M1, two to a
byte, the even element in the low half, rows of ceil(K / 32) * 16 bytes; scales one byte a block
of 32 (mx: E8M0) or 16 (nv: E4M3, times the tensor's scale amax / 2688), in tiles of 128 rows by
4 blocks, 512 bytes each, block b of row r at byte (r % 32) * 16 + (r % 128 / 32) * 4 + b % 4.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
BLOCK = {"mx": 32, "nv": 16}
LARGEST = 6.0                    # of E2M1
TENSOR = 2688.0                  # 6 * 448: the largest value over the tensor's scale
LOWEST_SCALE = 2.0 ** -100       # of a tensor


def listed():
    return [
        # the normed input of one small decoding batch's projections: latency alone
        {"name": "fp4_16x4096_nv", "op": "fp4", "T": 16, "K": 4096, "format": "nv",
         "dtype": "bf16", "columns": False, "out": "bf16", "pad": 0},
        # the FFN activation of a training micro-batch, kept in 4 bits and read back
        {"name": "fp4_8192x11008_mx", "op": "fp4", "T": 8192, "K": 11008, "format": "mx",
         "dtype": "bf16", "columns": False, "out": "bf16", "pad": 0},
        # a gradient for both products of the backward pass, quantised along rows and columns
        {"name": "fp4_both_4096x4096_nv", "op": "fp4", "T": 4096, "K": 4096, "format": "nv",
         "dtype": "bf16", "columns": True, "out": "bf16", "pad": 0},
        # a ragged FP32 batch inside a wider buffer, both ways
        {"name": "fp4_both_1021x5003_mx_f32", "op": "fp4", "T": 1021, "K": 5003, "format": "mx",
         "dtype": "f32", "columns": True, "out": "f32", "pad": 5},
        # one generated token through the FFN's first projection: reading the weight
        {"name": "linear_1x11008x4096_nv", "op": "linear", "M": 1, "N": 11008, "K": 4096,
         "format": "nv", "dtype": "bf16", "pad": 0},
        # odd sizes throughout, half precision
        {"name": "linear_517x5003x1999_mx_f16", "op": "linear", "M": 517, "N": 5003, "K": 1999,
         "format": "mx", "dtype": "f16", "pad": 3},
        # the FFN's first projection of a training micro-batch
        {"name": "linear_8192x11008x4096_nv", "op": "linear", "M": 8192, "N": 11008, "K": 4096,
         "format": "nv", "dtype": "bf16", "pad": 0},
        # its weight gradient from operands quantised before, in FP32
        {"name": "product_11008x4096x8192_mx", "op": "product", "M": 11008, "N": 4096, "K": 8192,
         "format": "mx", "out": "f32"},
        # policy loss of a few sampled tokens, without a reference
        {"name": "policy_16x32000", "op": "policy", "T": 16, "V": 32000, "dtype": "bf16",
         "mask": "none", "ref": False, "pad": 0},
        # of a micro-batch of samples, with the KL term to a reference
        {"name": "policy_8192x32000", "op": "policy", "T": 8192, "V": 32000, "dtype": "bf16",
         "mask": "none", "ref": True, "pad": 0},
        # preference loss of a few pairs of answers
        {"name": "preference_8_pairs", "op": "preference", "pairs": 8, "longest": 1000,
         "tail": 3, "ref": True},
        # of a large batch of long answers
        {"name": "preference_512_pairs", "op": "preference", "pairs": 512, "longest": 20000,
         "tail": 77, "ref": True},
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["fp4", "fp4", "linear", "linear", "product", "policy", "policy",
                     "preference"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    pad = rng.choice([0, 0, 8, 3])
    fmt = rng.choice(["mx", "nv"])
    if op == "fp4":
        K = _log_uniform(rng, 1, 16384)
        if rng.random() < 0.6:
            K = -(-K // 32) * 32
        T = _log_uniform(rng, 1, min(16384, (1 << 26) // K))
        return {"op": op, "T": T, "K": K, "format": fmt, "dtype": dtype,
                "columns": rng.random() < 0.5, "out": rng.choice(["bf16", "f32", dtype]),
                "pad": pad}
    if op in ("linear", "product"):
        N, K = _log_uniform(rng, 8, 16384), _log_uniform(rng, 16, 16384)
        if rng.random() < 0.6:
            N, K = -(-N // 64) * 64, -(-K // 64) * 64
        M = _log_uniform(rng, 1, min(16384, max(1, (1 << 38) // (N * K))))
        case = {"op": op, "M": M, "N": N, "K": K, "format": fmt}
        case.update({"dtype": dtype, "pad": pad} if op == "linear" else {"out": dtype})
        return case
    if op == "policy":
        V = _log_uniform(rng, 40, 160000)
        T = _log_uniform(rng, 1, min(16384, (1 << 26) // V))
        return {"op": op, "T": T, "V": V, "dtype": dtype,
                "mask": rng.choice(["none", "none", "inf", "lowest"]),
                "ref": rng.random() < 0.6, "pad": pad}
    longest = _log_uniform(rng, 1, 100000)
    return {"op": op, "pairs": _log_uniform(rng, 1, max(1, min(4096, (1 << 22) // longest))),
            "longest": longest, "tail": rng.randrange(0, 200), "ref": rng.random() < 0.7}


# ---- the stored format, in elementary operations ----------------------------------------------


def _number(v):
    """A tensor: torch divides by a number as a product with its reciprocal."""
    return torch.tensor(float(v), device="cuda")


def _tensor_scale(amax):
    return torch.clamp(amax / _number(TENSOR), min=LOWEST_SCALE)


def _blocks(x, fmt):
    """FP32 rows in blocks, the last ones filled with zeros: whole runs of 32 elements."""
    T, K = x.shape
    wide = torch.zeros(T, -(-K // 32) * 32, device="cuda")
    wide[:, :K] = x
    return wide.view(T, -1, BLOCK[fmt])


def _quantise(x, fmt, amax):
    """(values of E2M1 [T][blocks][block], scale bytes [T][blocks]) of rows x."""
    b = _blocks(x, fmt)
    top = b.abs().amax(2)
    if fmt == "mx":
        e = torch.where(top > 0, torch.frexp(top)[1] - 3, -127).clamp(min=-127)
        q = b * torch.ldexp(torch.ones_like(top), -e)[:, :, None]
        scales = (e + 127).to(torch.uint8)
    else:
        g = _tensor_scale(amax)
        s = (top / (g * 6.0)).clamp(max=448.0).to(torch.float8_e4m3fn)
        sg = s.float() * g
        inverse = torch.where(sg > 0, _number(1.0) / sg, 0.0)
        q = b * inverse[:, :, None]
        scales = s.view(torch.uint8)
    a = q.abs()
    # to the nearest of 0 .5 1 1.5 2 3 4 6, ties to the even code
    v = torch.where(a < 2, torch.round(a * 2) / 2, torch.where(a < 4, torch.round(a),
                                                               torch.round(a / 2) * 2))
    return torch.copysign(v.clamp(max=LARGEST), q), scales


def _store(values, scales):
    """(codes, scales) as they are kept, of the values and scale bytes of _quantise."""
    T = values.shape[0]
    a = values.reshape(T, -1)
    m = a.abs()
    code = torch.where(m < 2, m * 2, torch.where(m < 4, m + 2, m / 2 + 4)).to(torch.uint8)
    code += torch.signbit(a).to(torch.uint8) * 8
    codes = code[:, 0::2] | (code[:, 1::2] << 4)
    nb = scales.shape[1]
    wide = torch.zeros(-(-T // 128) * 128, -(-nb // 4) * 4, dtype=torch.uint8, device="cuda")
    wide[:T, :nb] = scales
    tiles = wide.view(-1, 4, 32, wide.shape[1] // 4, 4).permute(0, 3, 2, 1, 4)
    return codes.contiguous(), tiles.contiguous().view(-1)


def _load(codes, scales, T, K, fmt):
    """FP32 [T][K] values of stored codes, without the tensor's scale (exact)."""
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0.0, -.5, -1, -1.5, -2, -3, -4, -6],
                         device="cuda")
    v = torch.stack([table[(codes & 15).int()], table[(codes >> 4).int()]], 2).view(T, -1)
    nb = v.shape[1] // BLOCK[fmt]
    up, across = -(-T // 128), -(-nb // 4)
    s = scales.view(up, across, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(up * 128, -1)[:T, :nb]
    if fmt == "mx":
        s = torch.ldexp(torch.ones(1, device="cuda"), s.int() - 127)
    else:
        s = s.contiguous().view(torch.float8_e4m3fn).float()
    return (v.view(T, nb, -1) * s[:, :, None]).view(T, -1)[:, :K]


# ---- inputs -----------------------------------------------------------------------------------


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


def _activation(g, T, K):
    """Normal values of rows of different sizes, one in a thousand twenty times as large."""
    x = _randn(g, T, K) * torch.exp(0.5 * _randn(g, T, 1))
    x[torch.rand(T, K, generator=g, device="cuda") < 1e-3] *= 20
    return x


def _operand(g, rows, K, fmt, scale):
    """A stored operand: (codes, scales, amax)."""
    x = (_activation(g, rows, K) * scale).bfloat16().float()
    amax = x.abs().amax().view(1) if fmt == "nv" else None
    return (*_store(*_quantise(x, fmt, amax)), amax)


def _prepare_policy(case, g):
    T, V, dtype = case["T"], case["V"], case["dtype"]
    x = 2.5 * _randn(g, T, V)
    if case["mask"] != "none":
        low = -math.inf if case["mask"] == "inf" else torch.finfo(DTYPES[dtype]).min
        x[torch.rand(T, V, generator=g, device="cuda") < 0.6] = low
    logits = _rows(x, dtype, case["pad"])
    u = torch.rand(T, V, generator=g, device="cuda").clamp_(1e-12, 1 - 1e-7)
    tokens = (logits.float() - torch.log(-torch.log(u))).argmax(1)    # sampled from the softmax
    del x, u
    logp = (logits.double().gather(1, tokens[:, None])
            - torch.logsumexp(logits.double(), 1, keepdim=True)).view(-1)
    step = 0.25 * _randn(g, T).double()      # of the policy since the tokens were sampled
    # The gradient jumps where the ratio meets a bound; no ratio lies within 1e-4 of one, where
    # rounding would decide.
    for edge in (math.log(0.8), math.log(1.28)):
        step = torch.where((step - edge).abs() < 1e-4, edge + 2e-4, step)
    s = {"logits": logits, "old": (logp - step).float(), "advantages": _randn(g, T),
         "weights": torch.full((T,), 1.0 / T, device="cuda"),
         "ref": (logp + 0.3 * _randn(g, T)).float() if case["ref"] else None}
    ignored = torch.rand(T, generator=g, device="cuda") < 0.05        # prompts and padding
    s["tokens"] = torch.where(ignored, -100, tokens)
    return s


def _lengths(case):
    """Lengths of the answers, in pairs: some of one token, a few empty."""
    rng = random.Random(case["pairs"] * 1000003 + case["longest"])
    return [0 if rng.random() < 0.02 else _log_uniform(rng, 1, case["longest"])
            for _ in range(2 * case["pairs"])]


def _prepare_preference(case, g):
    lengths = _lengths(case)
    T = sum(lengths) + case["tail"]
    offsets = torch.tensor([0] + lengths, device="cuda").cumsum(0)
    logp = -torch.empty(T, device="cuda").exponential_(1.0, generator=g)
    ref = logp + 0.2 * _randn(g, T) if case["ref"] else None
    if not case["ref"]:
        logp = logp * 0.02
    # a buffer that the program keeps: rows behind the last answer stay as they are
    return {"logp": logp, "ref": ref, "offsets": offsets, "dlogp": torch.zeros(T, device="cuda")}


POLICY = {"clip_low": 0.2, "clip_high": 0.28, "kl_coef": 0.05}
PREFERENCE = {"beta": 0.1, "label_smoothing": 0.1}


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "fp4":
        s = {"x": _rows(_activation(g, case["T"], case["K"]), case["dtype"], case["pad"])}
    elif op == "linear":
        s = {"x": _rows(_activation(g, case["M"], case["K"]), case["dtype"], case["pad"]),
             "b": _operand(g, case["N"], case["K"], case["format"], case["K"] ** -0.5)}
    elif op == "product":
        s = {"a": _operand(g, case["M"], case["K"], case["format"], 1e-2),
             "b": _operand(g, case["N"], case["K"], case["format"], 1.0)}
    elif op == "policy":
        s = _prepare_policy(case, g)
    else:
        s = _prepare_preference(case, g)
    s["case"] = case
    return s


# ---- one pass ---------------------------------------------------------------------------------


def _plain_fp4(s, case):
    fmt, dtype = case["format"], DTYPES[case["out"]]
    x = s["x"].float()
    amax = x.abs().amax() if fmt == "nv" else None
    g = _tensor_scale(amax) if fmt == "nv" else 1.0
    out = {}
    for name, v in (("y", x), ("yt", x.t())) if case["columns"] else (("y", x),):
        stored = _store(*_quantise(v, fmt, amax))
        out[name] = (_load(*stored, *v.shape, fmt) * g).to(dtype)
    return out


def _plain_product(a, b, M, N, K, fmt, dtype):
    d = _load(a[0], a[1], M, K, fmt) @ _load(b[0], b[1], N, K, fmt).t()
    if fmt == "nv":
        d = d * _tensor_scale(a[2]) * _tensor_scale(b[2])
    return d.to(dtype)


def _plain_linear(s, case):
    fmt = case["format"]
    x = s["x"].float()
    amax = x.abs().amax() if fmt == "nv" else None
    a = (*_store(*_quantise(x, fmt, amax)), amax)
    return {"y": _plain_product(a, s["b"], case["M"], case["N"], case["K"], fmt, s["x"].dtype)}


def _plain_policy(s):
    x, tokens = s["logits"].float(), s["tokens"]
    live = tokens >= 0
    m = x.amax(1, keepdim=True)
    e = (x - m).exp()
    total = e.sum(1, keepdim=True)
    at = tokens.clamp(min=0)[:, None]
    # the ratio is compared with its bounds, and the KL term cancels: binary64
    logp = ((x.gather(1, at) - m).double() - total.double().log()).view(-1)
    A, w = s["advantages"].double(), s["weights"].double()
    ratio = (logp - s["old"].double()).exp()
    lo, hi = 1 - POLICY["clip_low"], 1 + POLICY["clip_high"]
    clipped = ((A > 0) & (ratio > hi)) | ((A < 0) & (ratio < lo))
    loss = -torch.minimum(ratio * A, ratio.clamp(lo, hi) * A)
    c = torch.where(clipped, 0.0, ratio * A)
    out = {"logp": torch.where(live, logp, 0.0).float()}
    if s["ref"] is not None:
        d = s["ref"].double() - logp
        kl = torch.expm1(d) - d
        loss = loss + POLICY["kl_coef"] * kl
        c = c + POLICY["kl_coef"] * torch.expm1(d)
        out["kl"] = torch.where(live, kl, 0.0).float()
    out["loss"] = torch.where(live, w * loss, 0.0).float()
    c = torch.where(live, w * c, 0.0).float()
    grad = e / total * c[:, None]
    out["dlogits"] = grad.scatter_add(1, at, -c[:, None]).to(s["logits"].dtype)
    return out


def _plain_preference(s):
    ref = s["ref"]
    r = s["logp"].double() if ref is None else s["logp"].double() - ref.double()
    total = torch.cat([torch.zeros(1, device="cuda", dtype=torch.float64), r.cumsum(0)])
    o = s["offsets"]
    sums = (total[o[1:]] - total[o[:-1]]).view(-1, 2)
    beta, eps = PREFERENCE["beta"], PREFERENCE["label_smoothing"]
    h = beta * (sums[:, 0] - sums[:, 1])
    softplus = lambda v: v.clamp(min=0) + torch.log1p(torch.exp(-v.abs()))
    loss = (1 - eps) * softplus(-h) + eps * softplus(h)
    c = -beta * ((1 - eps) / (1 + h.exp()) - eps / (1 + (-h).exp()))
    each = torch.stack([c, -c], 1).view(-1)
    n = int(s["case"]["tail"])
    rows = torch.repeat_interleave(each, o[1:] - o[:-1], output_size=r.numel() - n)
    s["dlogp"][:r.numel() - n] = rows.float()
    return {"loss": loss.float(), "margin": h.float(), "dlogp": s["dlogp"]}


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "fp4":
        return _plain_fp4(s, case)
    if op == "linear":
        return _plain_linear(s, case)
    if op == "product":
        return {"d": _plain_product(s["a"], s["b"], case["M"], case["N"], case["K"],
                                    case["format"], DTYPES[case["out"]])}
    return _plain_policy(s) if op == "policy" else _plain_preference(s)


def _run_own(s):
    from gradient_quantization_gb300 import agoq
    case = s["case"]
    op = case["op"]
    if op == "policy":
        terms = POLICY if s["ref"] is not None else dict(POLICY, kl_coef=0.0)
        loss, logp, kl, dlogits = agoq.agoq_policy_loss(
            s["logits"], s["tokens"], s["old"], s["advantages"], ref_logp=s["ref"],
            weights=s["weights"], **terms)
        out = {"logp": logp, "loss": loss, "dlogits": dlogits}
        if s["ref"] is not None:
            out["kl"] = kl
        return out
    if op == "preference":
        loss, margin, dlogp = agoq.agoq_preference_loss(s["logp"], s["offsets"],
                                                        ref_logp=s["ref"], dlogp=s["dlogp"],
                                                        **PREFERENCE)
        return {"loss": loss, "margin": margin, "dlogp": dlogp}
    fmt = agoq.NVFP4 if case["format"] == "nv" else agoq.MXFP4
    if op == "product":
        a, b = s["a"], s["b"]
        return {"d": agoq.agoq_fp4_gemm(a[0], a[1], b[0], b[1], case["M"], case["N"], case["K"],
                                        fmt, a_amax=a[2], b_amax=b[2],
                                        dtype=DTYPES[case["out"]])}
    x = s["x"]
    amax = agoq.agoq_amax(x) if fmt == agoq.NVFP4 else None
    columns = case.get("columns", False)
    codes, scales, codes_t, scales_t = agoq.agoq_fp4_quant(x, fmt, amax, columns=columns)
    if op == "linear":
        b = s["b"]
        return {"y": agoq.agoq_fp4_gemm(codes, scales, b[0], b[1], case["M"], case["N"],
                                        case["K"], fmt, a_amax=amax, b_amax=b[2], dtype=x.dtype)}
    T, K, dtype = case["T"], case["K"], DTYPES[case["out"]]
    out = {"y": agoq.agoq_fp4_dequant(codes, scales, T, K, fmt, amax, dtype=dtype)}
    if columns:
        out["yt"] = agoq.agoq_fp4_dequant(codes_t, scales_t, K, T, fmt, amax, dtype=dtype)
    return out


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- what a pass has to move ------------------------------------------------------------------


def work(case):
    op = case["op"]
    if op == "fp4":
        n = case["T"] * case["K"]
        ways = 2 if case["columns"] else 1
        return {"bytes": n * (SIZE[case["dtype"]] + ways * SIZE[case["out"]]),
                "flops": 4 * n * ways}
    if op in ("linear", "product"):
        M, N, K = case["M"], case["N"], case["K"]
        e = 0.5 + 1 / BLOCK[case["format"]]
        if op == "linear":
            size = SIZE[case["dtype"]]
            return {"bytes": M * K * size + N * K * e + M * N * size, "flops": 2 * M * N * K}
        return {"bytes": (M + N) * K * e + M * N * SIZE[case["out"]], "flops": 2 * M * N * K}
    if op == "policy":
        n = case["T"] * case["V"]
        return {"bytes": 2 * n * SIZE[case["dtype"]] + case["T"] * (32 if case["ref"] else 24),
                "flops": 8 * n}
    n = sum(_lengths(case))
    return {"bytes": n * (12 if case["ref"] else 8) + 24 * case["pairs"], "flops": 3 * n}


# ---- the definitions in binary64 --------------------------------------------------------------


def _exact_values(x, fmt, amax):
    """Binary64 values that rows x [T][K] are stored as.  The stored values are defined by
    binary32 roundings (of the scale and of the scaled element), which are made here from
    binary64 results."""
    T, K = x.shape
    size = BLOCK[fmt]
    pad = torch.nn.functional.pad(x.float().double(), (0, -K % size)).reshape(T, -1, size)
    most = pad.abs().max(dim=2).values
    if fmt == "mx":
        field = (most.float().view(torch.int32) >> 23).double() - 127
        step = torch.pow(2.0, torch.clamp(field - 2, min=-127.0))
        inverse = 1.0 / step
    else:
        g = max(float(torch.tensor(float(amax) / TENSOR, dtype=torch.float64).float()),
                LOWEST_SCALE)
        six = float(torch.tensor(6 * g, dtype=torch.float64).float())
        want = torch.clamp((most / six).float().double(), max=448.0)
        power = torch.floor(torch.log2(torch.clamp(want, min=2.0 ** -6)))
        grid = torch.pow(2.0, power - 3)
        kept = torch.round(want / grid) * grid
        step = kept * g                             # the value: not rounded
        inner = step.float().double()
        inverse = torch.where(inner > 0, 1.0 / torch.where(inner > 0, inner, 1.0), 0.0)
        inverse = inverse.float().double()
    scaled = (pad * inverse[:, :, None]).float().double()
    # the sum of a step at every border passed; a border itself goes to the even code
    size_of = scaled.abs()
    level = torch.zeros_like(size_of)
    for border, rise, up in ((.25, .5, False), (.75, .5, True), (1.25, .5, False),
                             (1.75, .5, True), (2.5, 1., False), (3.5, 1., True), (5., 2., False)):
        level += rise * (size_of >= border if up else size_of > border)
    signed = torch.where(scaled < 0, -level, level)
    return (signed * step[:, :, None]).reshape(T, -1)[:, :K]


def _exact_stored(operand, rows, K, fmt):
    """Binary64 values of a stored operand, read element by element from its definition."""
    codes, scales, amax = operand
    k = torch.arange(K, device="cuda")
    r = torch.arange(rows, device="cuda")[:, None]
    nibble = (codes[:, k // 2].int() >> (4 * (k % 2))) & 15
    exponent, half = (nibble >> 1) & 3, nibble & 1
    v = torch.where(exponent == 0, 0.5 * half.double(),
                    torch.pow(2.0, (exponent - 1).double()) * (1 + 0.5 * half.double()))
    v = torch.where(nibble >= 8, -v, v)
    size = BLOCK[fmt]
    b = k // size
    across = -(-(-(-K // 32) * 32 // size) // 4)
    at = ((r // 128) * across + b // 4) * 512 + (r % 32) * 16 + (r % 128 // 32) * 4 + b % 4
    byte = scales[at].int()
    if fmt == "mx":
        return v * torch.pow(2.0, (byte - 127).double())
    e, f = byte >> 3, (byte & 7).double()
    s = torch.where(e == 0, f * 2.0 ** -9, torch.pow(2.0, (e - 7).double()) * (1 + f / 8))
    g = max(float(torch.tensor(float(amax) / TENSOR, dtype=torch.float64).float()), LOWEST_SCALE)
    return v * s * g


def _exact_policy(s):
    x, tok = s["logits"].double(), s["tokens"]
    rows = torch.arange(x.shape[0], device="cuda")
    at = tok.clamp(min=0)
    logs = torch.log_softmax(x, 1)
    lp = logs[rows, at]
    gone = tok < 0                  # such a row's token may be one of probability 0
    A, r = s["advantages"].double(), torch.exp(lp - s["old"].double())
    bounded = r.clamp(1 - POLICY["clip_low"], 1 + POLICY["clip_high"])
    gain = torch.minimum(A * r, A * bounded)
    slope = torch.where(A * r <= A * bounded, A * r, 0.0)
    out = {}
    if s["ref"] is not None:
        d = s["ref"].double() - lp
        kl = torch.exp(d) - 1 - d
        gain = gain - POLICY["kl_coef"] * kl
        slope = slope + POLICY["kl_coef"] * (torch.exp(d) - 1)
        out["kl"] = kl.masked_fill(gone, 0.0)
    weight = s["weights"].double()
    grad = torch.exp(logs)
    grad[rows, at] -= 1
    out.update(logp=lp.masked_fill(gone, 0.0), loss=(-weight * gain).masked_fill(gone, 0.0),
               dlogits=(weight * slope).masked_fill(gone, 0.0)[:, None] * grad)
    return out


def _exact_preference(s):
    diff = s["logp"].double() - (0.0 if s["ref"] is None else s["ref"].double())
    ends = s["offsets"].tolist()
    beta, eps = PREFERENCE["beta"], PREFERENCE["label_smoothing"]
    loss, margin, grad = [], [], torch.zeros_like(diff)
    sums = [float(diff[a:b].sum()) for a, b in zip(ends, ends[1:])]
    for p in range(len(sums) // 2):
        h = beta * (sums[2 * p] - sums[2 * p + 1])
        # ln(1 + e^-h) without overflow
        low = math.log1p(math.exp(-h)) if h > 0 else -h + math.log1p(math.exp(h))
        loss.append(low + eps * h)
        margin.append(h)
        sig = 1 / (1 + math.exp(-h)) if h > 0 else math.exp(h) / (1 + math.exp(h))
        slope = beta * (sig - 1 + eps)
        grad[ends[2 * p]:ends[2 * p + 1]] = slope
        grad[ends[2 * p + 1]:ends[2 * p + 2]] = -slope
    of = lambda v: torch.tensor(v, dtype=torch.float64, device="cuda")
    return {"loss": of(loss), "margin": of(margin), "dlogp": grad}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "policy":
        return _exact_policy(s)
    if op == "preference":
        return _exact_preference(s)
    fmt = case["format"]
    if op == "product":
        a = _exact_stored(s["a"], case["M"], case["K"], fmt)
        return {"d": a @ _exact_stored(s["b"], case["N"], case["K"], fmt).t()}
    amax = s["x"].double().abs().max() if fmt == "nv" else None
    values = _exact_values(s["x"], fmt, amax)
    if op == "linear":
        return {"y": values @ _exact_stored(s["b"], case["N"], case["K"], fmt).t()}
    out = {"y": values}
    if case["columns"]:
        out["yt"] = _exact_values(s["x"].t(), fmt, amax)
    return out
