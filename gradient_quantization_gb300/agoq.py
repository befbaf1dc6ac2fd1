"""Python binding of libagoq.so: argument marshalling only.

Every function has the name of the C entry point it calls (include/agoq.h) and
takes torch CUDA tensors; all arithmetic runs in the library's CUDA kernels.
Outputs that are not supplied are allocated with torch (device memory is the
caller's, as in the C ABI).  Calls are asynchronous on ``stream`` (default:
torch's current stream).  A non-zero status raises ``AgoqError``.

The library is built in-tree by ``python -m gradient_quantization_gb300.build``
(``__graft_entry__.build()`` does it too); importing a function without the
built library raises immediately -- there is no fallback implementation.
"""
import ctypes
import os
import re

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libagoq.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "agoq.h")
BLOCK = 128

STATUS = {0: "AGOQ_OK", 1: "AGOQ_ERR_NULL", 2: "AGOQ_ERR_SHAPE", 3: "AGOQ_ERR_BITS",
          4: "AGOQ_ERR_ALIGN", 5: "AGOQ_ERR_ALIAS", 6: "AGOQ_ERR_CUDA", 7: "AGOQ_ERR_TIMEOUT",
          8: "AGOQ_ERR_FORMAT"}


class AgoqError(RuntimeError):
    def __init__(self, status, what):
        self.status = status
        super().__init__("%s failed: %s" % (what, _lib_handle().agoq_status_string(status).decode()))


_L = None


def _lib_handle():
    global _L
    if _L is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libagoq.so is not built (%s); run "
                               "`python -m gradient_quantization_gb300.build`" % LIB_PATH)
        L = ctypes.CDLL(LIB_PATH)
        vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
        L.agoq_status_string.argtypes = [i32]
        L.agoq_status_string.restype = ctypes.c_char_p
        L.agoq_version.argtypes = []
        L.agoq_version.restype = i32
        L.agoq_quant_act.argtypes = [vp, i64, i32, vp, vp, vp]
        L.agoq_dequant_act.argtypes = [vp, vp, i64, i32, vp, vp]
        L.agoq_grad_accum_fp8.argtypes = [vp, vp, vp, i64, vp]
        L.agoq_silu_backward.argtypes = [vp, vp, vp, i64, i32, vp, vp, vp]
        L.agoq_rmsnorm_backward.argtypes = [vp, vp, vp, vp, i64, i64, i32, ctypes.c_float, vp,
                                            vp, vp, vp]
        L.agoq_rmsnorm_backward_ws.argtypes = [vp, vp, vp, vp, i64, i64, i32, ctypes.c_float, vp,
                                               vp, vp, vp, i64, vp]
        L.agoq_rmsnorm_backward_noalloc.argtypes = [vp, vp, vp, vp, i64, i64, i32, ctypes.c_float,
                                                    vp, vp, vp, vp]
        L.agoq_rmsnorm_backward_workspace_bytes.argtypes = [i64]
        L.agoq_rmsnorm_backward_workspace_bytes.restype = i64
        L.agoq_grad_accum_fp8_mid.argtypes = [vp, vp, vp, i64, i32, vp]
        L.agoq_reduce_fp8_shards.argtypes = [vp, vp, i32, i64, vp, vp, vp, vp]
        L.agoq_wgrad_gemm_int4.argtypes = [vp, vp, vp, i32, i32, i32, vp, vp]
        L.agoq_wgrad_gemm_int4_f32out.argtypes = [vp, vp, vp, i32, i32, i32, vp, vp]
        L.agoq_wgrad_gemm_int4_accum_fp8.argtypes = [vp, vp, vp, i32, i32, i32, vp, vp, vp]
        L.agoq_device_status.argtypes = [vp]
        L.agoq_test_wait_timeout.argtypes = [i64, vp]
        L.agoq_dbca_pp_bits.argtypes = [i32, i32, i32, vp]
        f32 = ctypes.c_float
        L.agoq_layernorm_forward.argtypes = [vp, i64, vp, vp, i32, i64, i64, i32, f32, vp, i64,
                                             vp, vp, vp, vp, i32, vp]
        L.agoq_layernorm_backward_workspace_bytes.argtypes = [i64, i64]
        L.agoq_layernorm_backward_workspace_bytes.restype = i64
        L.agoq_layernorm_backward.argtypes = [vp, i64, vp, i64, vp, i32, vp, vp, i64, i64, i32,
                                              vp, i64, vp, vp, vp, i64, vp]
        L.agoq_layernorm_backward_laaq.argtypes = [vp, vp, i32, vp, i64, vp, i32, i64, i64, f32,
                                                   vp, i64, vp, vp, vp, i64, vp]
        L.agoq_grad_list_check.argtypes = [vp, i32]
        L.agoq_grad_norm_workspace_bytes.argtypes = [i32]
        L.agoq_grad_norm_workspace_bytes.restype = i64
        L.agoq_grad_norm.argtypes = [vp, i32, vp, vp, i64, vp]
        L.agoq_clip_grads.argtypes = [vp, i32, f32, vp, vp]
        L.agoq_clip_grad_norm.argtypes = [vp, i32, f32, vp, vp, i64, vp]
        L.agoq_token_logprobs.argtypes = [vp, i64, i32, vp, i64, i64, i32, vp, vp, vp, vp, vp, vp]
        L.agoq_token_logprobs_backward.argtypes = [vp, i64, i32, vp, i64, i64, vp, vp, vp, vp,
                                                   vp, i64, vp]
        L.agoq_token_loss.argtypes = [vp, i64, i32, vp, vp, i64, i64, vp, vp, i64, vp]
        L.agoq_fwd_gemm_quant.argtypes = [vp, vp, i32, i32, i32, i32, vp, vp, vp, vp]
        for name in ("agoq_quant_act", "agoq_dequant_act", "agoq_grad_accum_fp8",
                     "agoq_reduce_fp8_shards", "agoq_wgrad_gemm_int4",
                     "agoq_wgrad_gemm_int4_f32out", "agoq_device_status",
                     "agoq_wgrad_gemm_int4_accum_fp8", "agoq_grad_accum_fp8_mid",
                     "agoq_silu_backward", "agoq_rmsnorm_backward", "agoq_rmsnorm_backward_ws",
                     "agoq_rmsnorm_backward_noalloc",
                     "agoq_dbca_pp_bits",
                     "agoq_fwd_gemm_quant", "agoq_test_wait_timeout",
                     "agoq_layernorm_forward", "agoq_layernorm_backward",
                     "agoq_layernorm_backward_laaq", "agoq_grad_list_check", "agoq_grad_norm",
                     "agoq_clip_grads", "agoq_clip_grad_norm", "agoq_token_logprobs",
                     "agoq_token_logprobs_backward", "agoq_token_loss"):
            getattr(L, name).restype = i32
        _L = L
    return _L


def lib():
    """The loaded ctypes library (raises if it is not built)."""
    return _lib_handle()


def declared_entry_points():
    """Names of the functions include/agoq.h declares."""
    with open(HEADER) as f:
        text = f.read()
    return sorted(set(re.findall(r"^\s*(?:agoq_status|const char \*|int)\s*\*?\s*(agoq_\w+)\s*\(",
                                 text, flags=re.M)))


def _stream(stream):
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _need(t, dtype, what):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % what)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (what, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % what)


def _check(rc, what):
    if rc != 0:
        raise AgoqError(rc, what)


def record_bytes(bits):
    """Bytes of one packed record of 128 codes of `bits` bits."""
    return 16 * bits


def agoq_quant_act(x, bits, codes=None, scales=None, stream=None):
    """LAAQ quantize BF16 `x` (any shape, numel % 128 == 0) -> (codes uint8, scales float32)."""
    _need(x, torch.bfloat16, "x")
    n = x.numel()
    if codes is None:
        codes = torch.empty(n // BLOCK * record_bytes(max(bits, 0)), dtype=torch.uint8,
                            device=x.device)
    if scales is None:
        scales = torch.empty(n // BLOCK, dtype=torch.float32, device=x.device)
    _need(codes, torch.uint8, "codes")
    _need(scales, torch.float32, "scales")
    if bits in (4, 5, 6, 8) and (codes.numel() < n // BLOCK * record_bytes(bits)
                                 or scales.numel() < n // BLOCK):
        raise ValueError("codes/scales too small for %d elements at %d bits" % (n, bits))
    _check(lib().agoq_quant_act(_ptr(x), n, bits, _ptr(codes), _ptr(scales), _stream(stream)),
           "agoq_quant_act")
    return codes, scales


def agoq_dequant_act(codes, scales, n, bits, y=None, stream=None):
    """LAAQ dequantize -> BF16 tensor of n elements (or into `y`)."""
    _need(codes, torch.uint8, "codes")
    _need(scales, torch.float32, "scales")
    if bits in (4, 5, 6, 8) and (codes.numel() < n // BLOCK * record_bytes(bits)
                                 or scales.numel() < n // BLOCK):
        raise ValueError("codes/scales too small for %d elements at %d bits" % (n, bits))
    if y is None:
        y = torch.empty(n, dtype=torch.bfloat16, device=codes.device)
    _need(y, torch.bfloat16, "y")
    if y.numel() < n:
        raise ValueError("y too small")
    _check(lib().agoq_dequant_act(_ptr(codes), _ptr(scales), n, bits, _ptr(y), _stream(stream)),
           "agoq_dequant_act")
    return y


def agoq_grad_accum_fp8(master, master_scales, grad, stream=None):
    """In-place QuanGrad accumulation of BF16 `grad` into the FP8 master (uint8 codes)."""
    _need(master, torch.uint8, "master")
    _need(master_scales, torch.float32, "master_scales")
    _need(grad, torch.bfloat16, "grad")
    n = grad.numel()
    if master.numel() != n or master_scales.numel() != n // BLOCK:
        raise ValueError("master/scales do not match the gradient size")
    _check(lib().agoq_grad_accum_fp8(_ptr(master), _ptr(master_scales), _ptr(grad), n,
                                     _stream(stream)), "agoq_grad_accum_fp8")
    return master, master_scales


def agoq_silu_backward(codes, scales, dy, n, bits, dx=None, y=None, want_y=False, stream=None):
    """SiLU backward recomputed from LAAQ codes: returns (dx, y) as BF16 tensors
    (y is None unless `y` is given or want_y is set)."""
    _need(codes, torch.uint8, "codes")
    _need(scales, torch.float32, "scales")
    _need(dy, torch.bfloat16, "dy")
    if dx is None:
        dx = torch.empty(n, dtype=torch.bfloat16, device=dy.device)
    if y is None and want_y:
        y = torch.empty(n, dtype=torch.bfloat16, device=dy.device)
    _need(dx, torch.bfloat16, "dx")
    if y is not None:
        _need(y, torch.bfloat16, "y")
    _check(lib().agoq_silu_backward(_ptr(codes), _ptr(scales), _ptr(dy), n, bits, _ptr(dx),
                                    _ptr(y), _stream(stream)), "agoq_silu_backward")
    return dx, y


def agoq_rmsnorm_backward(codes, scales, dy, w, T, H, bits, eps, dx=None, rstd=None, dw=None,
                          want_dw=True, stream=None):
    """RMSNorm backward recomputed from LAAQ codes of x [T][H]: returns (dx BF16 [T][H],
    rstd FP32 [T], dw FP32 [H] or None)."""
    _need(codes, torch.uint8, "codes")
    _need(scales, torch.float32, "scales")
    _need(dy, torch.bfloat16, "dy")
    _need(w, torch.bfloat16, "w")
    dev = dy.device
    if dx is None:
        dx = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
    if rstd is None:
        rstd = torch.empty(T, dtype=torch.float32, device=dev)
    if dw is None and want_dw:
        dw = torch.empty(H, dtype=torch.float32, device=dev)
    _check(lib().agoq_rmsnorm_backward(_ptr(codes), _ptr(scales), _ptr(dy), _ptr(w), T, H, bits,
                                       float(eps), _ptr(dx), _ptr(rstd), _ptr(dw),
                                       _stream(stream)), "agoq_rmsnorm_backward")
    return dx, rstd, dw


def agoq_rmsnorm_backward_workspace_bytes(H):
    """Bytes of scratch agoq_rmsnorm_backward_ws needs for rows of H elements."""
    return int(lib().agoq_rmsnorm_backward_workspace_bytes(int(H)))


def agoq_rmsnorm_backward_ws(codes, scales, dy, w, T, H, bits, eps, workspace, dx=None, rstd=None,
                             dw=None, stream=None):
    """The RMSNorm backward in one read of the input (H <= 4096), dw included; `workspace`
    is a CUDA tensor of at least agoq_rmsnorm_backward_workspace_bytes(H) bytes.
    Returns (dx, rstd, dw)."""
    _need(codes, torch.uint8, "codes")
    _need(scales, torch.float32, "scales")
    _need(dy, torch.bfloat16, "dy")
    _need(w, torch.bfloat16, "w")
    dev = dy.device
    if dx is None:
        dx = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
    if rstd is None:
        rstd = torch.empty(T, dtype=torch.float32, device=dev)
    if dw is None:
        dw = torch.empty(H, dtype=torch.float32, device=dev)
    nbytes = workspace.numel() * workspace.element_size()
    _check(lib().agoq_rmsnorm_backward_ws(_ptr(codes), _ptr(scales), _ptr(dy), _ptr(w), T, H, bits,
                                          float(eps), _ptr(dx), _ptr(rstd), _ptr(dw),
                                          _ptr(workspace), nbytes, _stream(stream)),
           "agoq_rmsnorm_backward_ws")
    return dx, rstd, dw


def agoq_rmsnorm_backward_noalloc(codes, scales, dy, w, T, H, bits, eps, dx, rstd, dw,
                                  stream=None):
    """agoq_rmsnorm_backward_ws with the library's own static scratch (H <= 4096), for
    callers that cannot allocate device memory at the call: every output is
    caller-provided and the call allocates nothing."""
    _need(codes, torch.uint8, "codes")
    _need(scales, torch.float32, "scales")
    _need(dy, torch.bfloat16, "dy")
    _need(w, torch.bfloat16, "w")
    _check(lib().agoq_rmsnorm_backward_noalloc(_ptr(codes), _ptr(scales), _ptr(dy), _ptr(w), T, H,
                                               bits, float(eps), _ptr(dx), _ptr(rstd), _ptr(dw),
                                               _stream(stream)), "agoq_rmsnorm_backward_noalloc")
    return dx, rstd, dw


def agoq_dbca_pp_bits(stages, microbatches, base_bits=4):
    """DBCA-PP widths per pipeline stage (host-side): a list of `stages` ints."""
    out = (ctypes.c_int * max(int(stages), 1))()
    _check(lib().agoq_dbca_pp_bits(int(stages), int(microbatches), int(base_bits), out),
           "agoq_dbca_pp_bits")
    return list(out)[:stages]


def agoq_fwd_gemm_quant(x, w, T, N, K, bits, y=None, codes=None, scales=None, stream=None):
    """Forward GEMM Y = bf16(X W^T) (X [T][K], W [N][K], BF16) with the LAAQ
    quantization of Y fused: returns (Y [T][N], codes, scales)."""
    _need(x, torch.bfloat16, "x")
    _need(w, torch.bfloat16, "w")
    dev = x.device
    if y is None:
        y = torch.empty((T, N), dtype=torch.bfloat16, device=dev)
    if codes is None:
        codes = torch.empty(T * N // BLOCK * record_bytes(bits), dtype=torch.uint8, device=dev)
    if scales is None:
        scales = torch.empty(T * N // BLOCK, dtype=torch.float32, device=dev)
    _check(lib().agoq_fwd_gemm_quant(_ptr(x), _ptr(w), T, N, K, bits, _ptr(y), _ptr(codes),
                                     _ptr(scales), _stream(stream)), "agoq_fwd_gemm_quant")
    return y, codes, scales


MID_FP32, MID_BF16, MID_FP16 = 0, 1, 2


def agoq_grad_accum_fp8_mid(master, master_scales, grad, mid_format, stream=None):
    """In-place QuanGrad accumulation with the intermediate held in binary32
    (MID_FP32), BF16 (MID_BF16) or FP16 (MID_FP16)."""
    _need(master, torch.uint8, "master")
    _need(master_scales, torch.float32, "master_scales")
    _need(grad, torch.bfloat16, "grad")
    n = grad.numel()
    if master.numel() != n or master_scales.numel() != n // BLOCK:
        raise ValueError("master/scales do not match the gradient size")
    _check(lib().agoq_grad_accum_fp8_mid(_ptr(master), _ptr(master_scales), _ptr(grad), n,
                                         int(mid_format), _stream(stream)),
           "agoq_grad_accum_fp8_mid")
    return master, master_scales


def agoq_reduce_fp8_shards(shards, shard_scales, W, n, out=None, out_scales=None,
                           naive_overflow_count=None, stream=None):
    """Local reduce of W shard-major FP8 shards -> (codes, scales).  Pass a one-element
    int64 CUDA tensor as `naive_overflow_count` to receive the naive-sum overflow count."""
    _need(shards, torch.uint8, "shards")
    _need(shard_scales, torch.float32, "shard_scales")
    if shards.numel() != W * n or shard_scales.numel() != W * (n // BLOCK):
        raise ValueError("shards/shard_scales do not match W and n")
    if out is None:
        out = torch.empty(n, dtype=torch.uint8, device=shards.device)
    if out_scales is None:
        out_scales = torch.empty(n // BLOCK, dtype=torch.float32, device=shards.device)
    _need(out, torch.uint8, "out")
    _need(out_scales, torch.float32, "out_scales")
    if naive_overflow_count is not None:
        _need(naive_overflow_count, torch.int64, "naive_overflow_count")
    _check(lib().agoq_reduce_fp8_shards(_ptr(shards), _ptr(shard_scales), W, n, _ptr(out),
                                        _ptr(out_scales), _ptr(naive_overflow_count),
                                        _stream(stream)), "agoq_reduce_fp8_shards")
    return out, out_scales


def agoq_wgrad_gemm_int4(dY, x_codes, x_scales, M, N, K, dW=None, stream=None):
    """dW[M][N] (BF16) = dY^T Xhat for dY BF16 [K][M] and LAAQ INT4 X (codes [K][N/2])."""
    _need(dY, torch.bfloat16, "dY")
    _need(x_codes, torch.uint8, "x_codes")
    _need(x_scales, torch.float32, "x_scales")
    if dW is None:
        dW = torch.empty((M, N), dtype=torch.bfloat16, device=dY.device)
    _need(dW, torch.bfloat16, "dW")
    _check(lib().agoq_wgrad_gemm_int4(_ptr(dY), _ptr(x_codes), _ptr(x_scales), M, N, K, _ptr(dW),
                                      _stream(stream)), "agoq_wgrad_gemm_int4")
    return dW


def agoq_wgrad_gemm_int4_f32out(dY, x_codes, x_scales, M, N, K, dW=None, stream=None):
    """The same GEMM with the FP32 accumulator as output."""
    _need(dY, torch.bfloat16, "dY")
    _need(x_codes, torch.uint8, "x_codes")
    _need(x_scales, torch.float32, "x_scales")
    if dW is None:
        dW = torch.empty((M, N), dtype=torch.float32, device=dY.device)
    _need(dW, torch.float32, "dW")
    _check(lib().agoq_wgrad_gemm_int4_f32out(_ptr(dY), _ptr(x_codes), _ptr(x_scales), M, N, K,
                                             _ptr(dW), _stream(stream)),
           "agoq_wgrad_gemm_int4_f32out")
    return dW


def agoq_wgrad_gemm_int4_accum_fp8(dY, x_codes, x_scales, M, N, K, master, master_scales,
                                   stream=None):
    """The GEMM with the QuanGrad accumulation as its epilogue: the product is
    added to the FP8 master [M][N] (uint8 E4M3 codes, float32 scales [M][N/128])
    in place.  Returns (master, master_scales)."""
    _need(dY, torch.bfloat16, "dY")
    _need(x_codes, torch.uint8, "x_codes")
    _need(x_scales, torch.float32, "x_scales")
    _need(master, torch.uint8, "master")
    _need(master_scales, torch.float32, "master_scales")
    _check(lib().agoq_wgrad_gemm_int4_accum_fp8(_ptr(dY), _ptr(x_codes), _ptr(x_scales), M, N, K,
                                                _ptr(master), _ptr(master_scales),
                                                _stream(stream)),
           "agoq_wgrad_gemm_int4_accum_fp8")
    return master, master_scales


DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
F32, BF16, F16, E4M3 = 0, 1, 2, 3


_empty = torch.empty
_raw_stream = torch._C._cuda_getCurrentRawStream      # torch.cuda.current_stream() costs 2 us
_current_device = torch._C._cuda_getDevice


def _refuse(t, what, at):
    """Raise for an operand that is not on the device `at` of the others."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % what)
    raise ValueError("%s is on cuda:%d, the other operands are on cuda:%d"
                     % (what, t.get_device(), at))


def _launch(stream, device):
    """(handle, other) of a call's stream: other is None for torch's current stream, else the
    stream to allocate on (see _new).  The operands' device must be the current one: a handle
    may mean another device's stream there (0 is every device's default stream), whose kernels
    would meet foreign addresses."""
    at = device.index
    if at != _current_device():
        raise ValueError("the operands are on cuda:%d, but the current device is cuda:%d (make the "
                         "call within torch.cuda.device)" % (at, _current_device()))
    current = _raw_stream(at)
    if stream is None:
        return current, None
    handle = stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)
    if handle == current:
        return handle, None
    return handle, torch.cuda.ExternalStream(handle, device=device)


def _new(other, shape, dtype, device):
    """A tensor allocated for a call's stream: it belongs to that stream, so memory that
    torch's current stream still uses is not written by another one.  (Inputs are the caller's
    to order and keep alive.)"""
    if other is None:
        return _empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(other):
        return _empty(shape, dtype=dtype, device=device)


def _rows(t, what, n=None, T=None, dtype=None, at=None):
    """(address, rows, row length, row distance) of a CUDA tensor (on device `at`, where given)
    of FP32, BF16 or FP16 whose last dimension is contiguous: two-dimensional, or contiguous
    throughout."""
    if not isinstance(t, torch.Tensor) or (not t.is_cuda if at is None else t.get_device() != at):
        _refuse(t, what, at)
    if t.dtype not in DTYPES or (dtype is not None and t.dtype != dtype):
        raise TypeError("%s must be %s, got %s" % (what, dtype or "float32, bfloat16 or float16",
                                                   t.dtype))
    if t.dim() == 2:
        rows, length = t.shape
        ld, step = t.stride()
        if length > 1 and step != 1:
            raise ValueError("the last dimension of %s must be contiguous" % what)
        if rows <= 1 or ld < length:
            if rows > 1:
                raise ValueError("rows of %s overlap" % what)
            ld = length
    else:
        if t.dim() == 0 or not t.is_contiguous():
            raise ValueError("%s must be contiguous, or two-dimensional" % what)
        length = ld = t.shape[-1]
        rows = t.numel() // length if length else 0
    if (n is not None and length != n) or (T is not None and rows != T):
        raise ValueError("%s must hold %s rows of %s" % (what, T, n))
    return t.data_ptr(), rows, length, ld


def _vector(t, n, what, dtypes, at):
    """Address of a contiguous tensor of n elements on device `at` (None: 0)."""
    if t is None:
        return 0
    if not isinstance(t, torch.Tensor) or t.get_device() != at:
        _refuse(t, what, at)
    if t.dtype not in dtypes:
        raise TypeError("%s must be %s, got %s" % (what, " or ".join(map(str, dtypes)), t.dtype))
    if t.numel() != n or not t.is_contiguous():
        raise ValueError("%s must be contiguous and hold %d values" % (what, n))
    return t.data_ptr()


_F32 = (torch.float32,)


def _out(t, n, other, shape, dtype, device, what):
    """(tensor, address) of an output: the caller's `t` of n values, or a new one."""
    if t is None:
        t = _new(other, shape, dtype, device)
        return t, t.data_ptr()
    return t, _vector(t, n, what, (dtype,), device.index)


def _params(x_dtype, H, at, w, b=None):
    """(w, b, param_dtype): weight and bias of one type, FP32 or the activation's."""
    kinds = (torch.float32, x_dtype)
    wp, bp = _vector(w, H, "w", kinds, at), _vector(b, H, "b", kinds, at)
    if w is not None and b is not None and w.dtype != b.dtype:
        raise TypeError("w and b must have one type")
    ref = w if w is not None else b
    return wp, bp, DTYPES[ref.dtype] if ref is not None else F32


def agoq_layernorm_forward(x, w=None, b=None, eps=1e-5, bits=0, y=None, mean=None, rstd=None,
                           codes=None, scales=None, want_stats=True, stream=None):
    """Layer norm over the last dimension of `x` (FP32, BF16 or FP16; two-dimensional with any
    row distance, or contiguous).  `bits` 4, 5, 6 or 8 also writes the LAAQ codes of x (BF16,
    rows a multiple of 128).  Returns (y, mean, rstd, codes, scales); codes and scales are None
    for bits = 0, mean and rstd None unless given or wanted."""
    xp, T, H, ldx = _rows(x, "x")
    dev = x.device
    handle, other = _launch(stream, dev)
    wp, bp, pd = _params(x.dtype, H, dev.index, w, b)
    if y is None:
        y = _new(other, x.shape, x.dtype, dev)
        yp, ldy = y.data_ptr(), H
    else:
        yp, _, _, ldy = _rows(y, "y", H, T, x.dtype, dev.index)
    mp = rp = cp = sp = 0
    if mean is not None or want_stats:
        mean, mp = _out(mean, T, other, T, torch.float32, dev, "mean")
    if rstd is not None or want_stats:
        rstd, rp = _out(rstd, T, other, T, torch.float32, dev, "rstd")
    if bits:
        n = T * H // BLOCK
        m = n * record_bytes(bits)
        codes, cp = _out(codes, m, other, m, torch.uint8, dev, "codes")
        scales, sp = _out(scales, n, other, n, torch.float32, dev, "scales")
    else:
        codes = scales = None
    rc = lib().agoq_layernorm_forward(xp, ldx, wp, bp, pd, T, H, DTYPES[x.dtype], eps, yp, ldy,
                                      mp, rp, cp, sp, bits, handle)
    if rc:
        raise AgoqError(rc, "agoq_layernorm_forward")
    return y, mean, rstd, codes, scales


def agoq_layernorm_backward_workspace_bytes(T, H):
    """Bytes of scratch the layer norm's backward calls need for dw or db."""
    return int(lib().agoq_layernorm_backward_workspace_bytes(int(T), int(H)))


def _norm_sums(other, T, H, dev, dw, db, want_dw, want_db, workspace):
    """(dw, db, workspace) and the addresses and size that the backward calls take."""
    wp = bp = 0
    if dw is not None or want_dw:
        dw, wp = _out(dw, H, other, H, torch.float32, dev, "dw")
    if db is not None or want_db:
        db, bp = _out(db, H, other, H, torch.float32, dev, "db")
    if workspace is None:
        if not wp and not bp:
            return dw, db, None, 0, 0, 0, 0
        n = lib().agoq_layernorm_backward_workspace_bytes(T, H)
        workspace = _new(other, max(n, 0), torch.uint8, dev)
        return dw, db, workspace, wp, bp, workspace.data_ptr(), n
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    if workspace.get_device() != dev.index:
        _refuse(workspace, "workspace", dev.index)
    return (dw, db, workspace, wp, bp, workspace.data_ptr(),
            workspace.numel() * workspace.element_size())


def agoq_layernorm_backward(x, dy, mean, rstd, w=None, dx=None, dw=None, db=None, want_dw=True,
                            want_db=True, workspace=None, stream=None):
    """Layer norm backward from the input and its statistics: returns (dx, dw, db), dw and db
    FP32 (None unless given or wanted).  dx may be dy or x."""
    xp, T, H, ldx = _rows(x, "x")
    dev = x.device
    at = dev.index
    handle, other = _launch(stream, dev)
    dyp, _, _, lddy = _rows(dy, "dy", H, T, x.dtype, at)
    wp, _, pd = _params(x.dtype, H, at, w)
    if dx is None:
        dx = _new(other, dy.shape, dy.dtype, dev)
        dxp, lddx = dx.data_ptr(), H
    else:
        dxp, _, _, lddx = _rows(dx, "dx", H, T, x.dtype, at)
    dw, db, workspace, dwp, dbp, ws, nws = _norm_sums(other, T, H, dev, dw, db, want_dw, want_db,
                                                      workspace)
    rc = lib().agoq_layernorm_backward(
        xp, ldx, dyp, lddy, wp, pd, _vector(mean, T, "mean", _F32, at),
        _vector(rstd, T, "rstd", _F32, at), T, H, DTYPES[x.dtype], dxp, lddx, dwp, dbp, ws, nws,
        handle)
    if rc:
        raise AgoqError(rc, "agoq_layernorm_backward")
    return dx, dw, db


def agoq_layernorm_backward_laaq(codes, scales, bits, dy, eps=1e-5, w=None, dx=None, dw=None,
                                 db=None, want_dw=True, want_db=True, workspace=None, stream=None):
    """Layer norm backward from the LAAQ codes of the input (statistics recomputed from the
    dequantized values): returns (dx, dw, db) as agoq_layernorm_backward."""
    dyp, T, H, lddy = _rows(dy, "dy", dtype=torch.bfloat16)
    dev = dy.device
    at = dev.index
    handle, other = _launch(stream, dev)
    wp, _, pd = _params(dy.dtype, H, at, w)
    if dx is None:
        dx = _new(other, dy.shape, dy.dtype, dev)
        dxp, lddx = dx.data_ptr(), H
    else:
        dxp, _, _, lddx = _rows(dx, "dx", H, T, dy.dtype, at)
    dw, db, workspace, dwp, dbp, ws, nws = _norm_sums(other, T, H, dev, dw, db, want_dw, want_db,
                                                      workspace)
    blocks = T * H // BLOCK
    rc = lib().agoq_layernorm_backward_laaq(
        _vector(codes, blocks * record_bytes(bits), "codes", (torch.uint8,), at),
        _vector(scales, blocks, "scales", _F32, at), bits, dyp, lddy, wp, pd, T, H, eps, dxp, lddx,
        dwp, dbp, ws, nws, handle)
    if rc:
        raise AgoqError(rc, "agoq_layernorm_backward_laaq")
    return dx, dw, db


class _GradTensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("out", ctypes.c_void_p),
                ("n", ctypes.c_int64), ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class GradList:
    """The gradients that agoq_grad_norm and the clipping calls take, built once and kept.

    grads: CUDA tensors (FP32, BF16 or FP16) and (codes, scales) pairs (FP8 masters: uint8
    E4M3 codes and FP32 block scales).  outs: for each the tensor that receives the clipped
    gradient (for a pair: the clipped scales), or None to clip in place.  All are contiguous.
    The list keeps references to them and a workspace on their device; calls on one list must
    not overlap in time on the GPU."""

    def __init__(self, grads, outs=None):
        grads = list(grads)
        outs = [None] * len(grads) if outs is None else list(outs)
        if len(outs) != len(grads):
            raise ValueError("outs must match grads")
        self.entries = (_GradTensor * max(1, len(grads)))()
        self.count = len(grads)
        pairs = [g if isinstance(g, tuple) else (g, None) for g in grads]
        for p in pairs:
            if len(p) != 2 or not isinstance(p[0], torch.Tensor) or not p[0].is_cuda:
                raise TypeError("a gradient must be a CUDA tensor or a pair of codes and scales")
        at = pairs[0][0].get_device() if pairs else _current_device()
        for e, (codes, scales), o in zip(self.entries, pairs, outs):
            n = codes.numel()
            if scales is None:
                e.data = _vector(codes, n, "gradient", tuple(DTYPES), at)
                e.out = e.data if o is None else _vector(o, n, "out", (codes.dtype,), at)
                e.dtype = DTYPES[codes.dtype]
            else:
                e.data = _vector(codes, n, "codes", (torch.uint8,), at)
                e.scales = _vector(scales, n // BLOCK, "scales", _F32, at)
                e.out = e.scales if o is None else _vector(o, n // BLOCK, "out", _F32, at)
                e.dtype = E4M3
            e.n = n
        self.device = torch.device("cuda", at)
        self.tensors = (grads, outs)
        _check(lib().agoq_grad_list_check(self.entries, self.count), "agoq_grad_list_check")
        self.workspace = torch.empty(
            int(lib().agoq_grad_norm_workspace_bytes(self.count)), dtype=torch.uint8,
            device=self.device)

    def _scratch(self):
        return self.workspace.data_ptr(), self.workspace.numel()


def agoq_grad_norm(grads, norm=None, stream=None):
    """Global L2 norm of a GradList -> FP32 CUDA tensor of one element."""
    handle, other = _launch(stream, grads.device)
    if norm is None:
        norm = _new(other, 1, torch.float32, grads.device)
    _check(lib().agoq_grad_norm(grads.entries, grads.count,
                                _vector(norm, 1, "norm", _F32, grads.device.index),
                                *grads._scratch(), handle), "agoq_grad_norm")
    return norm


def agoq_clip_grads(grads, max_norm, norm, stream=None):
    """Clip a GradList by the norm in the one-element FP32 CUDA tensor `norm`: every gradient
    times min(1, max_norm / (norm + 1e-6)); of FP8 masters the scales alone change."""
    handle, other = _launch(stream, grads.device)
    _check(lib().agoq_clip_grads(grads.entries, grads.count, max_norm,
                                 _vector(norm, 1, "norm", _F32, grads.device.index), handle),
           "agoq_clip_grads")


def agoq_clip_grad_norm(grads, max_norm, norm=None, stream=None):
    """agoq_grad_norm and agoq_clip_grads in one call; returns the norm before clipping."""
    handle, other = _launch(stream, grads.device)
    if norm is None:
        norm = _new(other, 1, torch.float32, grads.device)
    _check(lib().agoq_clip_grad_norm(grads.entries, grads.count, max_norm,
                                     _vector(norm, 1, "norm", _F32, grads.device.index),
                                     *grads._scratch(), handle), "agoq_clip_grad_norm")
    return norm


_I64 = (torch.int64,)


def agoq_token_logprobs(logits, tokens, k=0, want_entropy=True, logp=None, entropy=None, lse=None,
                        top_logp=None, top_ids=None, stream=None):
    """Log probabilities of `tokens` (int64, one a row; negative: ignored) under `logits`
    (FP32, BF16 or FP16 rows), and the k most likely alternatives of each row.  Returns (logp,
    entropy, lse, top_logp, top_ids): FP32 [T] each, FP32 and int64 [T][k] (None for k = 0);
    entropy is None unless given or wanted."""
    xp, T, V, ld = _rows(logits, "logits")
    dev = logits.device
    at = dev.index
    handle, other = _launch(stream, dev)
    f32 = torch.float32
    logp, pp = _out(logp, T, other, T, f32, dev, "logp")
    lse, lp = _out(lse, T, other, T, f32, dev, "lse")
    ep = tp = ip = 0
    if entropy is not None or want_entropy:
        entropy, ep = _out(entropy, T, other, T, f32, dev, "entropy")
    if k > 0:
        top_logp, tp = _out(top_logp, T * k, other, (T, k), f32, dev, "top_logp")
        top_ids, ip = _out(top_ids, T * k, other, (T, k), torch.int64, dev, "top_ids")
    rc = lib().agoq_token_logprobs(xp, ld, DTYPES[logits.dtype],
                                   _vector(tokens, T, "tokens", _I64, at), T, V, k, pp, ep, lp, tp,
                                   ip, handle)
    if rc:
        raise AgoqError(rc, "agoq_token_logprobs")
    return logp, entropy, lse, top_logp, top_ids


def agoq_token_logprobs_backward(logits, tokens, lse, dlogp, entropy=None, dentropy=None,
                                 dlogits=None, stream=None):
    """Gradient of agoq_token_logprobs' logp (and entropy, with `dentropy`) -> dlogits of the
    logits' type; `dlogits` may be the logits themselves."""
    xp, T, V, ld = _rows(logits, "logits")
    dev = logits.device
    at = dev.index
    handle, other = _launch(stream, dev)
    if dlogits is None:
        dlogits = _new(other, logits.shape, logits.dtype, dev)
        dp, ldd = dlogits.data_ptr(), V
    else:
        dp, _, _, ldd = _rows(dlogits, "dlogits", V, T, logits.dtype, at)
    rc = lib().agoq_token_logprobs_backward(
        xp, ld, DTYPES[logits.dtype], _vector(tokens, T, "tokens", _I64, at), T, V,
        _vector(lse, T, "lse", _F32, at), _vector(entropy, T, "entropy", _F32, at),
        _vector(dlogp, T, "dlogp", _F32, at), _vector(dentropy, T, "dentropy", _F32, at), dp, ldd,
        handle)
    if rc:
        raise AgoqError(rc, "agoq_token_logprobs_backward")
    return dlogits


def agoq_token_loss(logits, tokens, weights=None, logp=None, dlogits=None, stream=None):
    """Log probabilities of `tokens` and the gradient of the loss -sum(weights * logp) ->
    (logp FP32 [T], dlogits of the logits' type); `dlogits` may be the logits themselves."""
    xp, T, V, ld = _rows(logits, "logits")
    dev = logits.device
    at = dev.index
    handle, other = _launch(stream, dev)
    logp, pp = _out(logp, T, other, T, torch.float32, dev, "logp")
    if dlogits is None:
        dlogits = _new(other, logits.shape, logits.dtype, dev)
        dp, ldd = dlogits.data_ptr(), V
    else:
        dp, _, _, ldd = _rows(dlogits, "dlogits", V, T, logits.dtype, at)
    rc = lib().agoq_token_loss(xp, ld, DTYPES[logits.dtype], _vector(tokens, T, "tokens", _I64, at),
                               _vector(weights, T, "weights", _F32, at), T, V, pp, dp, ldd, handle)
    if rc:
        raise AgoqError(rc, "agoq_token_loss")
    return logp, dlogits


def agoq_test_wait_timeout(limit_cycles, stream=None):
    """Launch the failure-path probe whose one pipeline wait gives up after
    `limit_cycles` SM cycles (test-only; see include/agoq.h)."""
    _check(lib().agoq_test_wait_timeout(int(limit_cycles), _stream(stream)),
           "agoq_test_wait_timeout")


def agoq_device_status(stream=None):
    """Synchronise and check the device status words (raises AgoqError if a pipeline wait timed out)."""
    _check(lib().agoq_device_status(_stream(stream)), "agoq_device_status")
