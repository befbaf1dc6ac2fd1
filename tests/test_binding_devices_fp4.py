"""The FP4, policy and preference calls refuse operands that are not on the current device, before
anything is launched (CPU: tensors that claim a device, and a library that only counts its
calls)."""
import pytest
import torch

from gradient_quantization_gb300 import agoq
from tests.test_binding_devices import Library, _on

F32, BF16, I64, U8 = torch.float32, torch.bfloat16, torch.int64, torch.uint8


@pytest.fixture
def library(monkeypatch):
    L = Library()
    monkeypatch.setattr(agoq, "lib", lambda: L)
    monkeypatch.setattr(agoq, "_current_device", lambda: 0, raising=False)
    monkeypatch.setattr(agoq, "_raw_stream", lambda i: 0)
    return L


T, V = 4, 50
X, COL, TOK, ONE = ((T, V), BF16), ((T,), F32), ((T,), I64), ((1,), F32)
CODES, SCALES, CODES_T, BYTES = ((T * 32,), U8), ((512,), U8), ((V * 16,), U8), ((1600,), U8)
CALLS = {
    "amax": (dict(x=X, amax=ONE), lambda a: agoq.agoq_amax(**a)),
    "quant": (dict(x=X, amax=ONE, codes=CODES, scales=SCALES, codes_t=CODES_T, scales_t=SCALES),
              lambda a: agoq.agoq_fp4_quant(fmt=agoq.NVFP4, columns=True, **a)),
    "dequant": (dict(codes=CODES, scales=SCALES, amax=ONE, y=X),
                lambda a: agoq.agoq_fp4_dequant(T=T, K=V, fmt=agoq.NVFP4, **a)),
    "gemm": (dict(a_codes=CODES, a_scales=SCALES, b_codes=BYTES, b_scales=SCALES, a_amax=ONE, b_amax=ONE,
                  d=X), lambda a: agoq.agoq_fp4_gemm(M=T, N=V, K=64, fmt=agoq.NVFP4, **a)),
    "policy": (dict(logits=X, tokens=TOK, old_logp=COL, advantages=COL, ref_logp=COL, weights=COL,
                    loss=COL, logp=COL, kl=COL, dlogits=X), lambda a: agoq.agoq_policy_loss(**a)),
    "preference": (dict(logp=COL, offsets=((3,), I64), ref_logp=COL, weights=ONE, loss=ONE, margin=ONE,
                        dlogp=COL), lambda a: agoq.agoq_preference_loss(**a)),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_an_operand_on_another_device(library, name):
    kinds, call = CALLS[name]
    call({k: _on(0, *v) for k, v in kinds.items()})
    launches = [c for c in library.calls if not c.endswith("bytes")]
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


@pytest.mark.parametrize("name", sorted(CALLS))
def test_host_tensors(library, name):
    kinds, call = CALLS[name]
    for bad in kinds:
        with pytest.raises(TypeError, match="CUDA"):
            call({k: torch.zeros(*v[:1], dtype=v[1]) if k == bad else _on(0, *v) for k, v in kinds.items()})


def test_sizes_are_the_librarys():
    """The binding's own sizes against the library's."""
    for rows in (0, 1, 127, 128, 129, 1000, 1 << 30):
        for K in (1, 16, 17, 32, 33, 64, 65, 127, 128, 129, 5003, 1 << 24):
            for fmt in (agoq.MXFP4, agoq.NVFP4):
                row, codes, scales = agoq._fp4_sizes(rows, K, fmt)
                assert codes == agoq.agoq_fp4_code_bytes(rows, K) == rows * row
                assert scales == agoq.agoq_fp4_scale_bytes(rows, K, fmt)
    for bad in ((-1, 8, 0), (1, 0, 0), (1, (1 << 24) + 1, 0), ((1 << 30) + 1, 8, 0), (1, 8, 2), (1, 8, None)):
        with pytest.raises(ValueError):
            agoq._fp4_sizes(*bad)
