"""Pins of tests/plain_fp4.py, by hand and by brute force (CPU)."""
from fractions import Fraction

import pytest
import torch

from tests import plain_fp4 as F


def test_codes_are_the_nearest_values():
    """Against exact rational distances; at equal ones the even code."""
    grid = [Fraction(v) for v in (0, "1/2", 1, "3/2", 2, 3, 4, 6)]
    q = [Fraction(n, 64) for n in range(0, 64 * 8)]
    got = F.e2m1(torch.tensor([float(v) for v in q], dtype=torch.float64)).tolist()
    for v, c in zip(q, got):
        best = min(abs(v - g) for g in grid)
        near = [i for i, g in enumerate(grid) if abs(v - g) == best]
        assert c == (near[0] if len(near) == 1 else [i for i in near if i % 2 == 0][0]), v
    neg = F.e2m1(torch.tensor([-float(v) for v in q[1:]], dtype=torch.float64)).tolist()
    assert neg == [c + 8 for c in got[1:]]


def test_e4m3_is_torchs():
    v = torch.cat([torch.linspace(0, 448, 20001), torch.logspace(-12, 8.8, 20001, base=2.0)]).double()
    byte, value = F.e4m3(v)
    want = v.float().to(torch.float8_e4m3fn)
    assert torch.equal(byte, want.view(torch.uint8)) and torch.equal(value, want.double())


@pytest.mark.parametrize("top,byte", [(0.0, 0), (6.0, 127), (7.9, 127), (8.0, 128), (4.0, 127),
                                      (3.9999998, 126), (2.0 ** -126, 0), (2.0 ** -124, 1),
                                      (2.0 ** -149, 0), (3.4028234663852886e38, 252)])
def test_mx_scale(top, byte):
    x = torch.zeros(1, 32, dtype=torch.float64)
    x[0, 5] = -top
    codes, scales, step = F.quantise(x, F.MX)
    assert int(scales[0, 0]) == byte and float(step[0, 0]) == 2.0 ** (byte - 127)


def test_nv_block():
    """amax 2688: the tensor scale is 1, a block with 6 has scale 1, one with 2688 has 448."""
    x = torch.zeros(1, 64, dtype=torch.float64)
    x[0, :4] = torch.tensor([6.0, -2.4, 0.24, -0.26])
    x[0, 16] = 2688.0
    x[0, 32] = 6 * 2.0 ** -11                       # half the smallest scale: a tie, to 0
    codes, scales, step = F.quantise(x, F.NV, 2688.0)
    assert scales[0].tolist() == [0x38, 0x7E, 0, 0]
    assert codes[0, :4].tolist() == [7, 12, 0, 9] and int(codes[0, 16]) == 7
    assert not codes[0, 32:].any()


def test_places_are_distinct():
    r = torch.arange(300)[:, None]
    b = torch.arange(11)[None, :]
    at = F.place(r, b, 3).reshape(-1)
    assert at.unique().numel() == 3300 and int(at.max()) < 3 * 3 * 512


def test_values_of_what_is_stored():
    g = torch.Generator().manual_seed(0)
    x = torch.randn(130, 100, generator=g).double()
    for fmt, amax in ((F.MX, None), (F.NV, float(x.float().abs().max()))):
        codes, scales = F.stored(x, fmt, amax)
        v = F.values(codes, scales, 130, 100, fmt) * (F.tensor_scale(amax) if amax else 1.0)
        c, _, step = F.quantise(x, fmt, amax)
        err = (v - x).abs()
        half = step.repeat_interleave(F.BLOCK[fmt], 1)[:, :100]
        # half of E2M1's widest step (2), and what lies beyond 6 (MXFP4: below 8)
        assert bool((err <= (2.0 if fmt == F.MX else 1.25) * half).all())
