"""Layer norm on the GPU against the plain binary64 form (tests/plain64.py holds
the formulas and the bounds): types, lengths from one element to long rows, odd
sizes, strides and alignments, in place, codes, both backward forms, streams and
graphs."""
import pytest
import torch

from gradient_quantization_gb300 import agoq
from tests import plain64 as P
from tests.gpu_util import Guarded

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
EPS = 1e-5


def _rand(shape, dtype, seed, scale=1.0, offset=0.0):
    g = torch.Generator().manual_seed(seed)
    return (offset + scale * torch.randn(shape, generator=g)).to(dtype).cuda()


def _strided(t, pad, shift=0):
    """The rows of t inside a buffer with `pad` more elements a row, `shift` elements in."""
    T, H = t.shape
    buf = torch.full((T * (H + pad) + shift + 64,), 7.0, dtype=t.dtype, device="cuda")
    v = buf[shift:shift + T * (H + pad)].view(T, H + pad)[:, :H]
    v.copy_(t)
    return v


def _params(kind, dtype, H):
    if kind == "none":
        return None, None
    t = F32 if kind == "f32" else dtype
    return _rand((H,), t, 91, 0.3, 1.0), _rand((H,), t, 92, 0.3)


def _d(t):
    return None if t is None else t.double()


def _check_forward(x, w, b, y, mean, rstd, eps=EPS):
    x64 = x.double()
    ey, em, er = P.layernorm(x64, _d(w), _d(b), eps)
    dmu, rr = P.stats_bounds(x64, eps)
    assert bool(((mean.double() - em).abs() <= dmu * 1.01 + 1e-45).all())
    assert bool(((rstd.double() - er).abs() <= (rr * 1.01) * er).all())
    off = (y.double() - ey).abs()
    bound = P.layernorm_bound(x64, _d(w), _d(b), eps, ey, em, er, x.dtype)
    assert bool((off <= bound).all()), float((off / bound).max())


SHAPES = [(1, 1), (5, 2), (3, 7), (17, 33), (4, 128), (9, 640), (6, 1000), (3, 4096), (2, 5003),
          (5, 8192), (2, 12288), (1, 16389), (2, 40000), (700, 96), (3, 65536)]


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("T,H", SHAPES)
def test_forward_and_backward(dtype, T, H):
    kind = ("none", "same", "f32")[(T + H) % 3]
    x = _rand((T, H), dtype, 1, 1.5, 0.5)
    dy = _rand((T, H), dtype, 2)
    w, b = _params(kind, dtype, H)
    y, mean, rstd, codes, _ = agoq.agoq_layernorm_forward(x, w, b, EPS)
    assert codes is None
    _check_forward(x, w, b, y, mean, rstd)
    _check_backward(x, dy, w, mean, rstd, *agoq.agoq_layernorm_backward(x, dy, mean, rstd, w))


def _check_backward(x, dy, w, mean, rstd, dx, dw, db, dmu=None, rr=None):
    x64, dy64, w64 = x.double(), dy.double(), _d(w)
    mu, r = mean.double(), rstd.double()
    zero = torch.zeros_like(mu)
    dmu, rr = zero if dmu is None else dmu, zero if rr is None else rr
    ex, ew, eb = P.layernorm_backward(x64, dy64, w64, mu, r)
    bx, bw, bb = P.layernorm_backward_bounds(x64, dy64, w64, mu, r, dmu, rr, ex, dx.dtype)
    for got, want, bound, what in ((dx, ex, bx, "dx"), (dw, ew, bw, "dw"), (db, eb, bb, "db")):
        if got is not None:
            off = (got.double() - want).abs()
            assert bool((off <= bound).all()), (what, float((off / bound).max()))


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("H,pad,shift", [(256, 8, 0), (256, 3, 0), (500, 12, 1), (1024, 0, 1),
                                         (4096, 16, 8), (130, 6, 0)])
def test_strides_and_alignment(dtype, H, pad, shift):
    x = _strided(_rand((13, H), dtype, 3), pad, shift)
    dy = _strided(_rand((13, H), dtype, 4), pad + 8, 0)
    w, b = _params("f32", dtype, H + 1)
    w, b = w[1:], b[1:]                                  # 4-byte aligned only
    y = _strided(torch.zeros(13, H, dtype=dtype, device="cuda"), pad, 8)
    y2, mean, rstd, _, _ = agoq.agoq_layernorm_forward(x, w, b, EPS, y=y)
    assert y2 is y
    _check_forward(x, w, b, y, mean, rstd)
    assert pad == 0 or bool((y.as_strided((13, pad), (H + pad, 1), y.storage_offset() + H)
                             == 7).all())                # nothing between the rows
    dx = _strided(torch.zeros(13, H, dtype=dtype, device="cuda"), pad, shift)
    _check_backward(x, dy, w, mean, rstd,
                    *agoq.agoq_layernorm_backward(x, dy, mean, rstd, w, dx=dx))


# Rows that one CTA does not hold: of whole vectors and of any alignment, from the first
# such length to the last, and beyond; few rows, and more than the GPU takes at a time.
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("T,H,pad", [(3, 8200, 0), (301, 12296, 8), (2, 32768, 0), (2, 32776, 0),
                                     (5, 4999, 0), (3, 8065, 3), (307, 11137, 2), (3, 16257, 0),
                                     (2, 27651, 1), (2, 39937, 0), (1300, 9001, 0)])
def test_long_rows(dtype, T, H, pad):
    x, dy = _rand((T, H), dtype, 31, 1.5, 0.5), _rand((T, H), dtype, 32)
    x[T - 1] += 50                                       # a row whose mean is far off 0
    if pad:
        x, dy = _strided(x, pad), _strided(dy, pad, 1)
    w, b = _params(("none", "same", "f32")[H % 3], dtype, H)
    y, mean, rstd, _, _ = agoq.agoq_layernorm_forward(x, w, b, EPS)
    _check_forward(x, w, b, y, mean, rstd)
    got = agoq.agoq_layernorm_backward(x, dy, mean, rstd, w)
    _check_backward(x, dy, w, mean, rstd, *got)
    again = agoq.agoq_layernorm_backward(x, dy, mean, rstd, w)
    assert all(torch.equal(p, q) for p, q in zip(got, again))        # sums in a fixed order
    if pad == 0:
        agoq.agoq_layernorm_backward(x, dy, mean, rstd, w, dx=dy)
        assert torch.equal(dy, got[0])
        agoq.agoq_layernorm_forward(x, w, b, EPS, y=x)
        assert torch.equal(x, y)


@pytest.mark.parametrize("bits", [4, 5, 6, 8])
@pytest.mark.parametrize("T,H", [(3, 8320), (330, 12288), (2, 32768), (1, 32896)])
def test_codes_of_long_rows(bits, T, H):
    x = _rand((T, H), BF16, 33, 2.0, 0.2)
    x[T - 1] += 30                                       # a row whose mean is far off 0
    w, b = _params("same", BF16, H)
    y, mean, rstd, codes, scales = agoq.agoq_layernorm_forward(x, w, b, EPS, bits=bits)
    _check_forward(x, w, b, y, mean, rstd)
    qc, qs = agoq.agoq_quant_act(x, bits)
    assert torch.equal(codes, qc) and torch.equal(scales, qs)
    kept = agoq.agoq_dequant_act(codes, scales, T * H, bits).view(T, H)
    dy = _rand((T, H), BF16, 34)
    got = agoq.agoq_layernorm_backward_laaq(codes, scales, bits, dy, EPS, w)
    k64 = kept.double()
    _, mu, r = P.layernorm(k64, None, None, EPS)
    _check_backward(kept, dy, w, mu, r, *got, *P.stats_bounds(k64, EPS))


def test_nothing_outside_the_outputs():
    T, H = 37, 1000
    x, dy = _rand((T, H), F16, 5), _rand((T, H), F16, 6)
    w, b = _params("same", F16, H)
    y, dx = Guarded(T * H * 2, F16), Guarded(T * H * 2, F16)
    mean, rstd = Guarded(T * 4, F32), Guarded(T * 4, F32)
    dw, db = Guarded(H * 4, F32), Guarded(H * 4, F32)
    ws = Guarded(agoq.agoq_layernorm_backward_workspace_bytes(T, H), torch.uint8)
    agoq.agoq_layernorm_forward(x, w, b, EPS, y=y.view.view(T, H), mean=mean.view, rstd=rstd.view)
    agoq.agoq_layernorm_backward(x, dy, mean.view, rstd.view, w, dx=dx.view.view(T, H),
                                 dw=dw.view, db=db.view, workspace=ws.view)
    assert all(g.intact() for g in (y, dx, mean, rstd, dw, db, ws))
    _check_backward(x, dy, w, mean.view, rstd.view, dx.view.view(T, H), dw.view, db.view)


@pytest.mark.parametrize("offset,scale", [(1000.0, 1e-2), (0.0, 0.0), (-3e4, 1.0), (0.0, 1e-18)])
def test_hard_rows(offset, scale):
    """A large common offset, constant rows, tiny values (the variance is not a difference of
    two large sums)."""
    x = _rand((6, 768), F32, 7, scale, offset)
    y, mean, rstd, _, _ = agoq.agoq_layernorm_forward(x, None, None, EPS)
    _check_forward(x, None, None, y, mean, rstd)


def test_a_bad_row_stays_alone():
    x = _rand((5, 512), BF16, 8)
    x[2, 100], x[3, 7] = float("nan"), float("inf")
    y, mean, rstd, _, _ = agoq.agoq_layernorm_forward(x, None, None, EPS)
    assert bool(torch.isnan(y[2:4]).all()) and bool(torch.isfinite(y[[0, 1, 4]]).all())


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("H", [1024, 777])
def test_in_place(dtype, H):
    x, dy = _rand((9, H), dtype, 10), _rand((9, H), dtype, 11)
    w, b = _params("f32", dtype, H)
    y, mean, rstd, _, _ = agoq.agoq_layernorm_forward(x, w, b, EPS)
    z = x.clone()
    agoq.agoq_layernorm_forward(z, w, b, EPS, y=z)
    assert torch.equal(z, y)
    dx, dw, db = agoq.agoq_layernorm_backward(x, dy, mean, rstd, w)
    for on in ("x", "dy"):
        xc, dc = x.clone(), dy.clone()
        got = agoq.agoq_layernorm_backward(xc, dc, mean, rstd, w, dx=xc if on == "x" else dc)
        assert all(torch.equal(p, q) for p, q in zip(got, (dx, dw, db))), on


@pytest.mark.parametrize("bits", [4, 5, 6, 8])
@pytest.mark.parametrize("T,H,pad", [(1, 128, 0), (7, 384, 0), (33, 1024, 0), (5, 4096, 0),
                                     (3, 8192, 8), (4, 640, 3), (2, 20480, 0), (600, 256, 0)])
def test_codes_and_backward_from_them(bits, T, H, pad):
    x = _rand((T, H), BF16, 12, 2.0, 0.2)
    x[0, :128] = 0                                       # an all-zero block
    if pad:
        x = _strided(x, pad)
    w, b = _params(("same", "f32", "none")[(T + bits) % 3], BF16, H)
    y, mean, rstd, codes, scales = agoq.agoq_layernorm_forward(x, w, b, EPS, bits=bits)
    _check_forward(x, w, b, y, mean, rstd)
    qc, qs = agoq.agoq_quant_act(x.contiguous(), bits)
    assert torch.equal(codes, qc) and torch.equal(scales, qs)
    kept = agoq.agoq_dequant_act(codes, scales, T * H, bits).view(T, H)
    dy = _rand((T, H), BF16, 13)
    if pad:
        dy = _strided(dy, pad)
    dx, dw, db = agoq.agoq_layernorm_backward_laaq(codes, scales, bits, dy, EPS, w)
    k64 = kept.double()
    _, mu, r = P.layernorm(k64, None, None, EPS)
    dmu, rr = P.stats_bounds(k64, EPS)
    _check_backward(kept, dy, w, mu, r, dx, dw, db, dmu, rr)


def test_gradient_sums_on_their_own():
    T, H = 50, 640
    x, dy = _rand((T, H), BF16, 14), _rand((T, H), BF16, 15)
    _, mean, rstd, codes, scales = agoq.agoq_layernorm_forward(x, None, None, EPS, bits=4)
    dx, dw, db = agoq.agoq_layernorm_backward(x, dy, mean, rstd)
    qx, qw, qb = agoq.agoq_layernorm_backward_laaq(codes, scales, 4, dy, EPS)
    for want_dw, want_db in ((True, False), (False, True), (False, False)):
        for got, want in ((agoq.agoq_layernorm_backward(x, dy, mean, rstd, want_dw=want_dw,
                                                        want_db=want_db), (dx, dw, db)),
                          (agoq.agoq_layernorm_backward_laaq(codes, scales, 4, dy, EPS,
                                                             want_dw=want_dw, want_db=want_db),
                           (qx, qw, qb))):
            assert torch.equal(got[0], want[0])
            assert got[1] is None if not want_dw else torch.equal(got[1], want[1])
            assert got[2] is None if not want_db else torch.equal(got[2], want[2])


def test_no_rows():
    x = torch.empty(0, 256, dtype=BF16, device="cuda")
    y, mean, rstd, _, _ = agoq.agoq_layernorm_forward(x)
    assert y.shape == (0, 256) and mean.numel() == 0
    dw, db = (torch.full((256,), 5.0, device="cuda") for _ in range(2))
    agoq.agoq_layernorm_backward(x, x, mean, rstd, dw=dw, db=db)
    assert not dw.any() and not db.any()


def test_many_rows_in_order():
    """More rows than CTAs; twice the same bits."""
    T, H = 20000, 128
    x, dy = _rand((T, H), BF16, 16), _rand((T, H), BF16, 17)
    w, b = _params("same", BF16, H)
    y, mean, rstd, _, _ = agoq.agoq_layernorm_forward(x, w, b, EPS)
    _check_forward(x, w, b, y, mean, rstd)
    first = agoq.agoq_layernorm_backward(x, dy, mean, rstd, w)
    _check_backward(x, dy, w, mean, rstd, *first)
    again = agoq.agoq_layernorm_backward(x, dy, mean, rstd, w)
    assert all(torch.equal(p, q) for p, q in zip(first, again))


def test_offsets_beyond_32_bits():
    """Rows whose byte offsets pass 2^32: a long row distance, the first and last rows checked."""
    T, H, ld = 5, 512, (1 << 29) + 64
    buf = torch.zeros(T * ld, dtype=BF16, device="cuda")
    x = buf.as_strided((T, H), (ld, 1))
    x.copy_(_rand((T, H), BF16, 18))
    y, mean, rstd, _, _ = agoq.agoq_layernorm_forward(x, None, None, EPS)
    _check_forward(x, None, None, y, mean, rstd)
    agoq.agoq_layernorm_forward(x, None, None, EPS, y=x)
    assert torch.equal(x, y)


def test_another_stream_and_a_graph():
    T, H = 64, 1024
    x, dy = _rand((T, H), BF16, 19), _rand((T, H), BF16, 20)
    w, b = _params("same", BF16, H)

    def step(stream=None):
        y, m, r, c, s = agoq.agoq_layernorm_forward(x, w, b, EPS, bits=4, stream=stream)
        return (y, m, r) + agoq.agoq_layernorm_backward(x, dy, m, r, w, stream=stream) + \
            agoq.agoq_layernorm_backward_laaq(c, s, 4, dy, EPS, w, stream=stream)
    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = step(side)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = step()
    x.copy_(_rand((T, H), BF16, 21))
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(held, step()))


def test_binding_refusals():
    x = _rand((4, 64), BF16, 22)
    with pytest.raises(TypeError):
        agoq.agoq_layernorm_forward(x.double())
    with pytest.raises(TypeError):
        agoq.agoq_layernorm_forward(x.cpu())
    with pytest.raises(ValueError):
        agoq.agoq_layernorm_forward(x.t())
    with pytest.raises(ValueError):
        agoq.agoq_layernorm_forward(x, w=torch.ones(63, device="cuda"))
    with pytest.raises(TypeError):
        agoq.agoq_layernorm_forward(x, w=torch.ones(64, dtype=F16, device="cuda"))
    with pytest.raises(agoq.AgoqError):
        agoq.agoq_layernorm_forward(x, bits=4)          # rows of 64: no whole block
    with pytest.raises(ValueError):
        agoq.agoq_layernorm_forward(x.expand(4, 4, 64)[0].as_strided((4, 64), (1, 1)))
