"""A row of the layer norm does not depend on the rows beside it, nor on what earlier
kernels left in shared memory: equal bits alone, in a batch with rows whose mean is
far off 0 (whose variance takes a second pass), and after other calls."""
import pytest
import torch

from gradient_quantization_gb300 import agoq

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
EPS = 1e-5


def _rows(T, H, dtype, seed, far=0.0):
    """Rows of mean 0.3 and deviation 1.5; every third has `far` added."""
    g = torch.Generator().manual_seed(seed)
    x = 0.3 + 1.5 * torch.randn(T, H, generator=g)
    x[1::3] += far
    return x.to(dtype).cuda()


# groups of 8 and 16 lanes, of a warp, of several warps, the whole CTA; parts of a
# cluster; rows of any alignment, whole and in parts
LENGTHS = [64, 128, 256, 512, 1024, 4096, 8320, 777, 5003, 17001]


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("H", LENGTHS)
def test_forward_row_alone(dtype, H):
    x = _rows(13, H, dtype, 1, 40.0)
    w = _rows(1, H, F32, 2)[0]
    got = agoq.agoq_layernorm_forward(x, w, None, EPS)[:3]
    for t in range(13):
        alone = agoq.agoq_layernorm_forward(x[t:t + 1], w, None, EPS)[:3]
        for p, q, what in zip(got, alone, ("y", "mean", "rstd")):
            assert torch.equal(p[t:t + 1], q), (t, what)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("H", [128, 512, 4096, 8320])
def test_forward_row_alone_with_codes(bits, H):
    x = _rows(7, H, BF16, 3, 40.0)
    got = agoq.agoq_layernorm_forward(x, None, None, EPS, bits=bits)[:3]
    for t in range(7):
        alone = agoq.agoq_layernorm_forward(x[t:t + 1], None, None, EPS, bits=bits)[:3]
        assert all(torch.equal(p[t:t + 1], q) for p, q in zip(got, alone)), t


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("T,H", [(1, 4096), (3, 4096), (1, 1024), (5, 64), (1, 128), (3, 8320)])
def test_forward_after_other_calls(dtype, T, H):
    """Ring slots of rows that do not exist hold what the last call left there."""
    xs = [_rows(T, H, dtype, 10 + i) for i in range(8)]
    wanted = None
    for offset in (0.0, 300.0, -7.0):
        kept = []
        for x in xs:
            left = (offset + torch.randn(4096, H, device="cuda")).to(dtype)
            agoq.agoq_layernorm_forward(left, None, None, EPS)
            kept.append(agoq.agoq_layernorm_forward(x, None, None, EPS)[:3])
        if wanted is None:
            wanted = kept
        for i, (p, q) in enumerate(zip(kept, wanted)):
            assert all(torch.equal(a, b) for a, b in zip(p, q)), (offset, i)


@pytest.mark.parametrize("bits", [4, 5, 6, 8])
@pytest.mark.parametrize("H", [128, 256, 640, 4096, 8320])
def test_backward_row_alone_from_codes(bits, H):
    """dx of a row, and its terms of dw and db where all other rows' dy is 0 (sums with zeros
    are exact)."""
    T = 7
    x = _rows(T, H, BF16, 4, 40.0)
    dy, w = _rows(T, H, BF16, 5), _rows(1, H, BF16, 6)[0]
    _, _, _, codes, scales = agoq.agoq_layernorm_forward(x, w, None, EPS, bits=bits)
    codes, scales = codes.view(T, -1), scales.view(T, -1)
    dx = agoq.agoq_layernorm_backward_laaq(codes, scales, bits, dy, EPS, w)[0]
    for t in range(T):
        only = torch.zeros_like(dy)
        only[t] = dy[t]
        _, dw, db = agoq.agoq_layernorm_backward_laaq(codes, scales, bits, only, EPS, w)
        ax, aw, ab = agoq.agoq_layernorm_backward_laaq(codes[t], scales[t], bits, dy[t:t + 1], EPS, w)
        assert torch.equal(dx[t:t + 1], ax) and torch.equal(dw, aw) and torch.equal(db, ab), t
