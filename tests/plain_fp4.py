"""Plain binary64 forms of the micro-scaled 4-bit format: quantisation, storage, values.

The format's own roundings to binary32 (quotients and products of binary32 numbers) are made
by rounding the binary64 result, which is the same: a product of two has 48 bits, and a
quotient rounded to 53 bits and then to 24 is the quotient rounded to 24."""
import torch

MX, NV = 0, 1
BLOCK = {MX: 32, NV: 16}
GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def f32(v):
    return v.float().double()


def exponent(v):
    """floor(log2 v) of positive binary64 values (log2 itself may round across a whole number)."""
    return torch.frexp(v)[1].double() - 1


def pow2(e):
    """2^e of whole numbers e, -1022 .. 1023, by its bits (the GPU's pow may be off by a step,
    which would decide ties)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def e2m1(q):
    """Codes 0 .. 15 of binary64 values: nearest, ties to the even code, beyond 6 to 6."""
    grid = GRID.to(q.device)
    a = q.abs().clamp(max=6.0)
    lo = torch.bucketize(a, grid, right=True) - 1
    hi = (lo + 1).clamp(max=7)
    below, above = a - grid[lo], grid[hi] - a
    up = (above < below) | ((above == below) & (lo % 2 == 1))
    return (torch.where(up, hi, lo) + 8 * torch.signbit(q)).to(torch.uint8)


def e4m3(v):
    """(byte, value) of non-negative binary64 values: nearest even, beyond 448 to 448."""
    v = v.clamp(max=448.0)
    e = exponent(v.clamp(min=2.0 ** -6))
    n = torch.round(v * pow2(3 - e))           # 0 .. 16 steps of 2^(e-3)
    value = n * pow2(e - 3)
    byte = torch.where(n == 16, (e + 8) * 8, torch.where(n < 8, n, (e + 7) * 8 + n - 8))
    return byte.to(torch.uint8), value


def tensor_scale(amax):
    """g of a largest magnitude (a number)."""
    g = f32(torch.tensor(amax, dtype=torch.float64) / 2688)
    return float(g.clamp(min=2.0 ** -100))


def amax_of(x):
    return float("nan") if torch.isnan(x).any() else float(x.abs().max()) if x.numel() else 0.0


def quantise(x, fmt, amax=None):
    """(codes [T][K'], scale bytes [T][blocks], step of each block) of x [T][K]; K' is K up to a
    multiple of 32."""
    T, K = x.shape
    b = torch.zeros(T, -(-K // 32) * 32, dtype=torch.float64, device=x.device)
    b[:, :K] = x.double()
    b = b.view(T, -1, BLOCK[fmt])
    fine = torch.isfinite(b).all(2)
    b = torch.where(fine[:, :, None], b, torch.zeros_like(b))
    top = b.abs().amax(2)
    if fmt == MX:
        e = (exponent(top.clamp(min=2.0 ** -149)) - 2).clamp(min=-127.0)
        byte, step, inverse = (e + 127).to(torch.uint8), pow2(e), pow2(-e)
        nan = 255
    else:
        g = tensor_scale(amax) if amax == amax and abs(amax) != float("inf") else 1.0
        fine = fine & (amax == amax and abs(amax) != float("inf"))
        byte, s = e4m3(f32(top / f32(torch.tensor(6 * g, dtype=torch.float64))))
        inner = f32(s * g)
        inverse = torch.where(byte > 0, f32(1.0 / torch.where(byte > 0, inner, 1.0)), 0.0)
        step = s * g
        nan = 127
    codes = e2m1(f32(b * inverse[:, :, None]))
    codes = torch.where(fine[:, :, None], codes, torch.zeros_like(codes)).view(T, -1)
    byte = torch.where(fine, byte, torch.full_like(byte, nan))
    byte[:, -(-K // BLOCK[fmt]):] = 0               # no block begins there
    return codes, byte, step


def pack(codes):
    return codes[:, 0::2] | (codes[:, 1::2] << 4)


def tile(scales, fill=0):
    """Scale bytes [rows][blocks] in their tiles."""
    R, nb = scales.shape
    across = -(-nb // 4)
    out = torch.full((-(-R // 128) * across * 512,), fill, dtype=torch.uint8, device=scales.device)
    r = torch.arange(R, device=scales.device)[:, None]
    b = torch.arange(nb, device=scales.device)[None, :]
    out[place(r, b, across)] = scales
    return out


def place(r, b, across):
    return (r // 128 * across + b // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + b % 4


def stored(x, fmt, amax=None):
    """(codes, scales) as the library writes them."""
    codes, scales, _ = quantise(x, fmt, amax)
    return pack(codes), tile(scales)


def scale_values(byte, fmt):
    if fmt == MX:
        v = pow2(byte.double() - 127)
        return torch.where(byte == 255, torch.full_like(v, float("nan")), v)
    e, m = (byte >> 3).double(), (byte & 7).double()
    v = torch.where(e == 0, m * 2.0 ** -9, pow2(e - 7) * (1 + m / 8))
    return torch.where(byte == 127, torch.full_like(v, float("nan")), v)


def code_values(codes):
    v = GRID.to(codes.device)[(codes & 7).long()]
    return torch.where(codes >= 8, -v, v)


def values(codes, scales, rows, K, fmt):
    """Binary64 [rows][K] of stored codes and scales: code times block scale."""
    c = torch.stack([codes & 15, codes >> 4], 2).view(rows, -1)[:, :K]
    k = torch.arange(K, device=codes.device)[None, :]
    r = torch.arange(rows, device=codes.device)[:, None]
    nb = -(-K // 32) * 32 // BLOCK[fmt]
    s = scale_values(scales[place(r, k // BLOCK[fmt], -(-nb // 4))], fmt)
    return code_values(c) * s
