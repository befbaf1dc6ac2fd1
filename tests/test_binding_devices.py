"""The layer norm, gradient norm and token calls refuse operands that are not on the current
device, before anything is launched (CPU: tensors that claim a device, and a library that
only counts its calls)."""
import torch
import pytest

from gradient_quantization_gb300 import agoq

F32, BF16, I64, U8 = torch.float32, torch.bfloat16, torch.int64, torch.uint8


class Claims(torch.Tensor):
    """A CPU tensor that says it is on cuda:`index`."""
    index = 0
    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", self.index))

    def get_device(self):
        return self.index


def _on(index, shape, dtype):
    t = torch.zeros(shape, dtype=dtype).as_subclass(Claims)
    t.index = index
    return t


class Library:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*a):
            self.calls.append(name)
            return 1 << 16 if name.endswith("bytes") else 0
        return call


@pytest.fixture
def library(monkeypatch):
    L = Library()
    monkeypatch.setattr(agoq, "lib", lambda: L)
    monkeypatch.setattr(agoq, "_current_device", lambda: 0, raising=False)
    monkeypatch.setattr(agoq, "_raw_stream", lambda i: 0)
    real = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **k: real(*a, **dict(k, device="cpu")))
    return L


T, H, V = 4, 256, 50
X, ROW, COL, TOK, OUT = ((T, H), BF16), ((H,), F32), ((T,), F32), ((T,), I64), ((T, V), BF16)
CODES, SCALES = ((T * H // 2,), U8), ((T * H // 128,), F32)
CALLS = {
    "forward": (dict(x=X, w=ROW, b=ROW, y=X, mean=COL, rstd=COL, codes=CODES, scales=SCALES),
                lambda a: agoq.agoq_layernorm_forward(bits=4, **a)),
    "backward": (dict(x=X, dy=X, mean=COL, rstd=COL, w=ROW, dx=X, dw=ROW, db=ROW,
                      workspace=((1 << 16,), U8)), lambda a: agoq.agoq_layernorm_backward(**a)),
    "backward_laaq": (dict(codes=CODES, scales=SCALES, dy=X, w=ROW, dx=X, dw=ROW, db=ROW,
                           workspace=((1 << 16,), U8)),
                      lambda a: agoq.agoq_layernorm_backward_laaq(bits=4, **a)),
    "logprobs": (dict(logits=OUT, tokens=TOK, logp=COL, entropy=COL, lse=COL, top_logp=((T, 3), F32),
                      top_ids=((T, 3), I64)), lambda a: agoq.agoq_token_logprobs(k=3, **a)),
    "logprobs_backward": (dict(logits=OUT, tokens=TOK, lse=COL, dlogp=COL, entropy=COL, dentropy=COL,
                               dlogits=OUT), lambda a: agoq.agoq_token_logprobs_backward(**a)),
    "loss": (dict(logits=OUT, tokens=TOK, weights=COL, logp=COL, dlogits=OUT),
             lambda a: agoq.agoq_token_loss(**a)),
    "grad_norm": (dict(g=ROW, codes=CODES, scales=((T * H // 2 // 128,), F32), norm=((1,), F32)),
                  lambda a: agoq.agoq_grad_norm(agoq.GradList([a["g"], (a["codes"], a["scales"])]),
                                                a["norm"])),
    "clip": (dict(g=ROW, out=ROW, norm=((1,), F32)),
             lambda a: agoq.agoq_clip_grads(agoq.GradList([a["g"]], [a["out"]]), 1.0, a["norm"])),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_an_operand_on_another_device(library, name):
    kinds, call = CALLS[name]
    call({k: _on(0, *v) for k, v in kinds.items()})
    launches = [c for c in library.calls if not c.endswith(("bytes", "check"))]
    assert len(launches) == 1
    for bad in kinds:
        del library.calls[:]
        with pytest.raises(ValueError, match="cuda:1"):
            call({k: _on(int(k == bad), *v) for k, v in kinds.items()})
        assert launches[0] not in library.calls, bad


@pytest.mark.parametrize("name", sorted(CALLS))
def test_all_on_a_device_that_is_not_current(library, name, monkeypatch):
    kinds, call = CALLS[name]
    with pytest.raises(ValueError, match="cuda:1.*current device is cuda:0"):
        call({k: _on(1, *v) for k, v in kinds.items()})
    monkeypatch.setattr(agoq, "_current_device", lambda: 1, raising=False)
    call({k: _on(1, *v) for k, v in kinds.items()})


def test_a_list_of_another_device(library, monkeypatch):
    grads = agoq.GradList([_on(0, (64,), F32)])
    monkeypatch.setattr(agoq, "_current_device", lambda: 1, raising=False)
    for call in (lambda: agoq.agoq_grad_norm(grads, _on(1, (1,), F32)),
                 lambda: agoq.agoq_clip_grad_norm(grads, 1.0, _on(1, (1,), F32)),
                 lambda: agoq.agoq_clip_grads(grads, 1.0, _on(1, (1,), F32))):
        with pytest.raises(ValueError, match="current device is cuda:1"):
            call()


def test_host_tensors(library):
    with pytest.raises(TypeError, match="CUDA"):
        agoq.agoq_layernorm_forward(torch.zeros(2, 8))
    with pytest.raises(TypeError, match="CUDA"):
        agoq.agoq_token_loss(_on(0, (2, 8), F32), torch.zeros(2, dtype=I64), logp=_on(0, (2,), F32),
                             dlogits=_on(0, (2, 8), F32))
    with pytest.raises(TypeError, match="CUDA"):
        agoq.GradList([torch.zeros(3)])


@pytest.mark.parametrize("bad", [None, 3.0, (None, None), ("x", "y"), (None,), ()])
def test_what_is_no_gradient(library, bad):
    """A parameter without a gradient, say."""
    for grads in ([bad], [_on(0, (64,), F32), bad]):
        with pytest.raises(TypeError, match="gradient"):
            agoq.GradList(grads)
