// agoq_api.cu -- the extern "C" entry points declared in include/agoq.h.
//
// Each entry point validates its arguments on the host (null pointers, sizes,
// widths, alignment, overlap of outputs with inputs) before launching
// anything, then launches on the caller's stream and maps a launch failure to
// AGOQ_ERR_CUDA.  No entry point allocates or synchronises (except
// agoq_device_status, whose purpose is to synchronise).
#include "../../include/agoq.h"
#include "agoq_launch.h"

#include <algorithm>
#include <cstdint>
#include <new>

namespace agoq {

int sm_count() {
    static int cache[kMaxDevices];
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= kMaxDevices) dev = 0;
    if (cache[dev] == 0) {
        int sms = 0;
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        cache[dev] = sms > 0 ? sms : 1;
    }
    return cache[dev];
}

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Half-open byte ranges [a, a+na) and [b, b+nb) overlap.
bool overlap(const void *a, uint64_t na, const void *b, uint64_t nb) {
    if (na == 0 || nb == 0) return false;
    const uintptr_t pa = reinterpret_cast<uintptr_t>(a), pb = reinterpret_cast<uintptr_t>(b);
    return pa < pb + nb && pb < pa + na;
}

bool bits_ok(int bits) { return bits == 4 || bits == 5 || bits == 6 || bits == 8; }

agoq_status from_cuda(cudaError_t e) { return e == cudaSuccess ? AGOQ_OK : AGOQ_ERR_CUDA; }

cudaStream_t as_stream(void *s) { return static_cast<cudaStream_t>(s); }

// A byte range of an argument; empty for a NULL pointer.
struct Range {
    const void *p;
    uint64_t n;
};

// Half-open byte range of T rows of `len` elements of `size` bytes, `ld` apart.
Range rows(const void *p, int64_t T, int64_t len, int64_t ld, int size) {
    return {p, p && T > 0 ? ((uint64_t)(T - 1) * ld + len) * size : 0};
}
Range vec(const void *p, int64_t n, int size) { return {p, p ? (uint64_t)n * size : 0}; }

// A range of a gradient list's tensor, ordered by address.
struct Span {
    uintptr_t from, to;
    int tensor;
    bool out;
    bool operator<(const Span &o) const { return from < o.from; }
};

// Some output overlaps an input or another output.
template <int O, int I>
bool any_overlap(const Range (&out)[O], const Range (&in)[I]) {
    for (int o = 0; o < O; ++o) {
        for (int i = 0; i < I; ++i)
            if (overlap(out[o].p, out[o].n, in[i].p, in[i].n)) return true;
        for (int i = 0; i < o; ++i)
            if (overlap(out[o].p, out[o].n, out[i].p, out[i].n)) return true;
    }
    return false;
}

bool float_dtype(int d) { return d == AGOQ_F32 || d == AGOQ_BF16 || d == AGOQ_F16; }
int elem_size(int d) { return d == AGOQ_F32 ? 4 : d == AGOQ_E4M3 ? 1 : 2; }

// Sizes of rows that the typed calls take: T rows of n elements, `ld` apart,
// whose byte offsets stay within 62 bits.
bool rows_ok(int64_t T, int64_t n, int64_t ld) {
    return ld >= n && ld <= (1ll << 40) && T <= (1ll << 60) / (ld > 0 ? ld : 1);
}

constexpr int64_t kMaxHidden = 1ll << 24, kMaxVocab = 1ll << 30;
constexpr int kMaxTop = 32;

}  // namespace
}  // namespace agoq

extern "C" {

const char *agoq_status_string(agoq_status s) {
    switch (s) {
        case AGOQ_OK: return "AGOQ_OK";
        case AGOQ_ERR_NULL: return "AGOQ_ERR_NULL: a required pointer is NULL";
        case AGOQ_ERR_SHAPE: return "AGOQ_ERR_SHAPE: size not supported (n % 128, GEMM tiles)";
        case AGOQ_ERR_BITS: return "AGOQ_ERR_BITS: bits must be 4, 5, 6 or 8";
        case AGOQ_ERR_ALIGN: return "AGOQ_ERR_ALIGN: pointer not aligned as required";
        case AGOQ_ERR_ALIAS: return "AGOQ_ERR_ALIAS: an output overlaps an input";
        case AGOQ_ERR_CUDA: return "AGOQ_ERR_CUDA: CUDA runtime error";
        case AGOQ_ERR_TIMEOUT: return "AGOQ_ERR_TIMEOUT: a pipeline wait gave up";
        case AGOQ_ERR_FORMAT: return "AGOQ_ERR_FORMAT: unsupported intermediate format or element type";
    }
    return "AGOQ_ERR_UNKNOWN";
}

int agoq_version(void) { return 100; }

agoq_status agoq_quant_act(const void *x_bf16, int64_t n, int bits, void *codes, float *scales,
                           void *stream) {
    using namespace agoq;
    if (!bits_ok(bits)) return AGOQ_ERR_BITS;
    if (n < 0 || n % kBlockElems) return AGOQ_ERR_SHAPE;
    if (n == 0) return AGOQ_OK;
    if (!x_bf16 || !codes || !scales) return AGOQ_ERR_NULL;
    if (!aligned(x_bf16, 16) || !aligned(codes, 16) || !aligned(scales, 4)) return AGOQ_ERR_ALIGN;
    const uint64_t nb = (uint64_t)n / kBlockElems;
    const uint64_t xb = 2ull * n, cb = nb * 16 * bits, sb = nb * 4;
    if (overlap(codes, cb, x_bf16, xb) || overlap(scales, sb, x_bf16, xb) ||
        overlap(codes, cb, scales, sb))
        return AGOQ_ERR_ALIAS;
    return from_cuda(launch_laaq_quant(x_bf16, n, bits, codes, scales, as_stream(stream)));
}

agoq_status agoq_dequant_act(const void *codes, const float *scales, int64_t n, int bits,
                             void *y_bf16, void *stream) {
    using namespace agoq;
    if (!bits_ok(bits)) return AGOQ_ERR_BITS;
    if (n < 0 || n % kBlockElems) return AGOQ_ERR_SHAPE;
    if (n == 0) return AGOQ_OK;
    if (!codes || !scales || !y_bf16) return AGOQ_ERR_NULL;
    if (!aligned(codes, 16) || !aligned(scales, 4) || !aligned(y_bf16, 16)) return AGOQ_ERR_ALIGN;
    const uint64_t nb = (uint64_t)n / kBlockElems;
    const uint64_t yb = 2ull * n, cb = nb * 16 * bits, sb = nb * 4;
    if (overlap(y_bf16, yb, codes, cb) || overlap(y_bf16, yb, scales, sb)) return AGOQ_ERR_ALIAS;
    return from_cuda(launch_laaq_dequant(codes, scales, n, bits, y_bf16, as_stream(stream)));
}

agoq_status agoq_silu_backward(const void *codes, const float *scales, const void *dy_bf16,
                               int64_t n, int bits, void *dx_bf16, void *y_bf16, void *stream) {
    using namespace agoq;
    if (!bits_ok(bits)) return AGOQ_ERR_BITS;
    if (n < 0 || n % kBlockElems) return AGOQ_ERR_SHAPE;
    if (n == 0) return AGOQ_OK;
    if (!codes || !scales || !dy_bf16 || !dx_bf16) return AGOQ_ERR_NULL;
    if (!aligned(codes, 16) || !aligned(scales, 4) || !aligned(dy_bf16, 16) ||
        !aligned(dx_bf16, 16) || (y_bf16 && !aligned(y_bf16, 16)))
        return AGOQ_ERR_ALIGN;
    const uint64_t nb = (uint64_t)n / kBlockElems;
    const uint64_t cb = nb * 16 * bits, sb = nb * 4, vb = 2ull * n, yb = y_bf16 ? vb : 0;
    if (overlap(dx_bf16, vb, codes, cb) || overlap(dx_bf16, vb, scales, sb) ||
        overlap(dx_bf16, vb, dy_bf16, vb) || overlap(y_bf16, yb, codes, cb) ||
        overlap(y_bf16, yb, scales, sb) || overlap(y_bf16, yb, dy_bf16, vb) ||
        overlap(y_bf16, yb, dx_bf16, vb))
        return AGOQ_ERR_ALIAS;
    return from_cuda(
        launch_silu_backward(codes, scales, dy_bf16, n, bits, dx_bf16, y_bf16, as_stream(stream)));
}

agoq_status agoq_rmsnorm_backward(const void *codes, const float *scales, const void *dy_bf16,
                                  const void *w_bf16, int64_t T, int64_t H, int bits, float eps,
                                  void *dx_bf16, float *rstd, float *dw, void *stream) {
    using namespace agoq;
    if (!bits_ok(bits)) return AGOQ_ERR_BITS;
    if (T < 0 || H <= 0 || H % 256 || H > 8192 || !(eps >= 0.0f) || eps > 3.0e38f)
        return AGOQ_ERR_SHAPE;
    if (T == 0 && !dw) return AGOQ_OK;
    if (!codes || !scales || !dy_bf16 || !w_bf16 || !dx_bf16 || !rstd) return AGOQ_ERR_NULL;
    if (!aligned(codes, 16) || !aligned(scales, 4) || !aligned(dy_bf16, 16) ||
        !aligned(w_bf16, 16) || !aligned(dx_bf16, 16) || !aligned(rstd, 4) ||
        (dw && !aligned(dw, 4)))
        return AGOQ_ERR_ALIGN;
    const uint64_t n = (uint64_t)T * H, nb = n / kBlockElems;
    const uint64_t cb = nb * 16 * bits, sb = nb * 4, vb = 2 * n, wb = 2ull * H;
    const uint64_t rb = 4ull * T, db = dw ? 4ull * H : 0;
    const void *in[4] = {codes, scales, dy_bf16, w_bf16};
    const uint64_t inb[4] = {cb, sb, vb, wb};
    for (int i = 0; i < 4; ++i)
        if (overlap(dx_bf16, vb, in[i], inb[i]) || overlap(rstd, rb, in[i], inb[i]) ||
            overlap(dw, db, in[i], inb[i]))
            return AGOQ_ERR_ALIAS;
    if (overlap(dx_bf16, vb, rstd, rb) || overlap(dx_bf16, vb, dw, db) || overlap(rstd, rb, dw, db))
        return AGOQ_ERR_ALIAS;
    if (T == 0) return from_cuda(cudaMemsetAsync(dw, 0, 4ull * H, as_stream(stream)));
    return from_cuda(launch_rmsnorm_backward(codes, scales, dy_bf16, w_bf16, T, H, bits, eps,
                                             dx_bf16, rstd, dw, as_stream(stream)));
}

int64_t agoq_rmsnorm_backward_workspace_bytes(int64_t H) {
    using namespace agoq;
    if (H <= 0 || H % 256 || H > 8192) return -1;
    return H <= rmsnorm_fused_max_h() ? (int64_t)rmsnorm_fused_partials() * H * 4 : 0;
}

agoq_status agoq_rmsnorm_backward_ws(const void *codes, const float *scales, const void *dy_bf16,
                                     const void *w_bf16, int64_t T, int64_t H, int bits, float eps,
                                     void *dx_bf16, float *rstd, float *dw, void *workspace,
                                     int64_t workspace_bytes, void *stream) {
    using namespace agoq;
    if (!bits_ok(bits)) return AGOQ_ERR_BITS;
    if (T < 0 || H <= 0 || H % 256 || H > 8192 || !(eps >= 0.0f) || eps > 3.0e38f)
        return AGOQ_ERR_SHAPE;
    const int64_t need = agoq_rmsnorm_backward_workspace_bytes(H);
    if (workspace_bytes < need) return AGOQ_ERR_SHAPE;
    if (!dw || (need > 0 && !workspace)) return AGOQ_ERR_NULL;
    if (need == 0 || T == 0)
        return agoq_rmsnorm_backward(codes, scales, dy_bf16, w_bf16, T, H, bits, eps, dx_bf16,
                                     rstd, dw, stream);
    if (!codes || !scales || !dy_bf16 || !w_bf16 || !dx_bf16 || !rstd) return AGOQ_ERR_NULL;
    if (!aligned(codes, 16) || !aligned(scales, 4) || !aligned(dy_bf16, 16) ||
        !aligned(w_bf16, 16) || !aligned(dx_bf16, 16) || !aligned(rstd, 4) || !aligned(dw, 4) ||
        !aligned(workspace, 16))
        return AGOQ_ERR_ALIGN;
    const uint64_t n = (uint64_t)T * H, nb = n / kBlockElems;
    const uint64_t cb = nb * 16 * bits, sb = nb * 4, vb = 2 * n, wb = 2ull * H;
    const uint64_t rb = 4ull * T, db = 4ull * H, kb = (uint64_t)need;
    const void *in[4] = {codes, scales, dy_bf16, w_bf16};
    const uint64_t inb[4] = {cb, sb, vb, wb};
    for (int i = 0; i < 4; ++i)
        if (overlap(dx_bf16, vb, in[i], inb[i]) || overlap(rstd, rb, in[i], inb[i]) ||
            overlap(dw, db, in[i], inb[i]) || overlap(workspace, kb, in[i], inb[i]))
            return AGOQ_ERR_ALIAS;
    if (overlap(dx_bf16, vb, rstd, rb) || overlap(dx_bf16, vb, dw, db) || overlap(rstd, rb, dw, db) ||
        overlap(workspace, kb, dx_bf16, vb) || overlap(workspace, kb, rstd, rb) ||
        overlap(workspace, kb, dw, db))
        return AGOQ_ERR_ALIAS;
    return from_cuda(launch_rmsnorm_backward_fused(codes, scales, dy_bf16, w_bf16, T, H, bits, eps,
                                                   dx_bf16, rstd, dw,
                                                   static_cast<float *>(workspace),
                                                   as_stream(stream)));
}

agoq_status agoq_rmsnorm_backward_noalloc(const void *codes, const float *scales,
                                          const void *dy_bf16, const void *w_bf16, int64_t T,
                                          int64_t H, int bits, float eps, void *dx_bf16,
                                          float *rstd, float *dw, void *stream) {
    using namespace agoq;
    if (!bits_ok(bits)) return AGOQ_ERR_BITS;
    if (T < 0 || H <= 0 || H % 256 || H > rmsnorm_fused_max_h() || !(eps >= 0.0f) ||
        eps > 3.0e38f)
        return AGOQ_ERR_SHAPE;
    if (!dw) return AGOQ_ERR_NULL;
    if (T == 0) {
        if (!aligned(dw, 4)) return AGOQ_ERR_ALIGN;
        return from_cuda(cudaMemsetAsync(dw, 0, 4ull * H, as_stream(stream)));
    }
    if (!codes || !scales || !dy_bf16 || !w_bf16 || !dx_bf16 || !rstd) return AGOQ_ERR_NULL;
    if (!aligned(codes, 16) || !aligned(scales, 4) || !aligned(dy_bf16, 16) ||
        !aligned(w_bf16, 16) || !aligned(dx_bf16, 16) || !aligned(rstd, 4) || !aligned(dw, 4))
        return AGOQ_ERR_ALIGN;
    const uint64_t n = (uint64_t)T * H, nb = n / kBlockElems;
    const uint64_t cb = nb * 16 * bits, sb = nb * 4, vb = 2 * n, wb = 2ull * H;
    const uint64_t rb = 4ull * T, db = 4ull * H;
    const void *in[4] = {codes, scales, dy_bf16, w_bf16};
    const uint64_t inb[4] = {cb, sb, vb, wb};
    for (int i = 0; i < 4; ++i)
        if (overlap(dx_bf16, vb, in[i], inb[i]) || overlap(rstd, rb, in[i], inb[i]) ||
            overlap(dw, db, in[i], inb[i]))
            return AGOQ_ERR_ALIAS;
    if (overlap(dx_bf16, vb, rstd, rb) || overlap(dx_bf16, vb, dw, db) || overlap(rstd, rb, dw, db))
        return AGOQ_ERR_ALIAS;
    return from_cuda(launch_rmsnorm_backward_noalloc(codes, scales, dy_bf16, w_bf16, T, H, bits,
                                                     eps, dx_bf16, rstd, dw, as_stream(stream)));
}

agoq_status agoq_grad_accum_fp8(void *master_e4m3, float *master_scales, const void *grad_bf16,
                                int64_t n, void *stream) {
    return agoq_grad_accum_fp8_mid(master_e4m3, master_scales, grad_bf16, n, AGOQ_MID_FP32, stream);
}

agoq_status agoq_grad_accum_fp8_mid(void *master_e4m3, float *master_scales,
                                    const void *grad_bf16, int64_t n, int mid_format,
                                    void *stream) {
    using namespace agoq;
    if (mid_format != AGOQ_MID_FP32 && mid_format != AGOQ_MID_BF16 && mid_format != AGOQ_MID_FP16)
        return AGOQ_ERR_FORMAT;
    if (n < 0 || n % kBlockElems) return AGOQ_ERR_SHAPE;
    if (n == 0) return AGOQ_OK;
    if (!master_e4m3 || !master_scales || !grad_bf16) return AGOQ_ERR_NULL;
    if (!aligned(master_e4m3, 16) || !aligned(master_scales, 4) || !aligned(grad_bf16, 16))
        return AGOQ_ERR_ALIGN;
    const uint64_t nb = (uint64_t)n / kBlockElems;
    const uint64_t mb = (uint64_t)n, sb = nb * 4, gb = 2ull * n;
    if (overlap(master_e4m3, mb, grad_bf16, gb) || overlap(master_scales, sb, grad_bf16, gb) ||
        overlap(master_e4m3, mb, master_scales, sb))
        return AGOQ_ERR_ALIAS;
    return from_cuda(
        launch_grad_accum(master_e4m3, master_scales, grad_bf16, n, mid_format, as_stream(stream)));
}

agoq_status agoq_reduce_fp8_shards(const void *shards_e4m3, const float *shard_scales, int W,
                                   int64_t n, void *out_e4m3, float *out_scales,
                                   unsigned long long *naive_overflow_count, void *stream) {
    using namespace agoq;
    if (W < 1 || n < 0 || n % kBlockElems) return AGOQ_ERR_SHAPE;
    if (n == 0) {
        if (naive_overflow_count)
            return from_cuda(cudaMemsetAsync(naive_overflow_count, 0, sizeof(unsigned long long),
                                             as_stream(stream)));
        return AGOQ_OK;
    }
    if (!shards_e4m3 || !shard_scales || !out_e4m3 || !out_scales) return AGOQ_ERR_NULL;
    if (!aligned(shards_e4m3, 16) || !aligned(shard_scales, 4) || !aligned(out_e4m3, 16) ||
        !aligned(out_scales, 4) || (naive_overflow_count && !aligned(naive_overflow_count, 8)))
        return AGOQ_ERR_ALIGN;
    const uint64_t nb = (uint64_t)n / kBlockElems;
    const uint64_t shb = (uint64_t)W * n, ssb = (uint64_t)W * nb * 4, ob = (uint64_t)n, osb = nb * 4;
    const uint64_t cntb = naive_overflow_count ? 8 : 0;
    if (overlap(out_e4m3, ob, shards_e4m3, shb) || overlap(out_e4m3, ob, shard_scales, ssb) ||
        overlap(out_scales, osb, shards_e4m3, shb) || overlap(out_scales, osb, shard_scales, ssb) ||
        overlap(out_e4m3, ob, out_scales, osb) ||
        overlap(naive_overflow_count, cntb, shards_e4m3, shb) ||
        overlap(naive_overflow_count, cntb, shard_scales, ssb) ||
        overlap(naive_overflow_count, cntb, out_e4m3, ob) ||
        overlap(naive_overflow_count, cntb, out_scales, osb))
        return AGOQ_ERR_ALIAS;
    return from_cuda(launch_reduce_shards(shards_e4m3, shard_scales, W, n, out_e4m3, out_scales,
                                          naive_overflow_count, as_stream(stream)));
}

static agoq_status wgrad_common(const void *dY, const void *xc, const float *xs, int M, int N,
                                int K, void *dW, bool f32_out, void *stream) {
    using namespace agoq;
    if (M <= 0 || N <= 0 || K <= 0 || M % 128 || N % 128 || K % 64) return AGOQ_ERR_SHAPE;
    if (!dY || !xc || !xs || !dW) return AGOQ_ERR_NULL;
    if (!aligned(dY, 16) || !aligned(xc, 16) || !aligned(xs, 4) || !aligned(dW, 16))
        return AGOQ_ERR_ALIGN;
    const uint64_t dyb = 2ull * K * M, xcb = (uint64_t)K * N / 2, xsb = (uint64_t)K * (N / 128) * 4;
    const uint64_t dwb = (uint64_t)M * N * (f32_out ? 4 : 2);
    if (overlap(dW, dwb, dY, dyb) || overlap(dW, dwb, xc, xcb) || overlap(dW, dwb, xs, xsb))
        return AGOQ_ERR_ALIAS;
    return from_cuda(launch_wgrad_gemm(dY, xc, xs, M, N, K, dW, f32_out, as_stream(stream)));
}

agoq_status agoq_wgrad_gemm_int4(const void *dY_bf16, const void *x_codes, const float *x_scales,
                                 int M, int N, int K, void *dW_bf16, void *stream) {
    return wgrad_common(dY_bf16, x_codes, x_scales, M, N, K, dW_bf16, false, stream);
}

agoq_status agoq_wgrad_gemm_int4_f32out(const void *dY_bf16, const void *x_codes,
                                        const float *x_scales, int M, int N, int K, float *dW_f32,
                                        void *stream) {
    return wgrad_common(dY_bf16, x_codes, x_scales, M, N, K, dW_f32, true, stream);
}

agoq_status agoq_wgrad_gemm_int4_accum_fp8(const void *dY_bf16, const void *x_codes,
                                           const float *x_scales, int M, int N, int K,
                                           void *master_e4m3, float *master_scales,
                                           void *stream) {
    using namespace agoq;
    if (M <= 0 || N <= 0 || K <= 0 || M % 128 || N % 128 || K % 64) return AGOQ_ERR_SHAPE;
    if (!dY_bf16 || !x_codes || !x_scales || !master_e4m3 || !master_scales) return AGOQ_ERR_NULL;
    if (!aligned(dY_bf16, 16) || !aligned(x_codes, 16) || !aligned(x_scales, 4) ||
        !aligned(master_e4m3, 16) || !aligned(master_scales, 4))
        return AGOQ_ERR_ALIGN;
    const uint64_t dyb = 2ull * K * M, xcb = (uint64_t)K * N / 2, xsb = (uint64_t)K * (N / 128) * 4;
    const uint64_t mb = (uint64_t)M * N, msb = (uint64_t)M * (N / 128) * 4;
    if (overlap(master_e4m3, mb, dY_bf16, dyb) || overlap(master_e4m3, mb, x_codes, xcb) ||
        overlap(master_e4m3, mb, x_scales, xsb) || overlap(master_scales, msb, dY_bf16, dyb) ||
        overlap(master_scales, msb, x_codes, xcb) || overlap(master_scales, msb, x_scales, xsb) ||
        overlap(master_e4m3, mb, master_scales, msb))
        return AGOQ_ERR_ALIAS;
    return from_cuda(launch_wgrad_accum_fp8(dY_bf16, x_codes, x_scales, M, N, K, master_e4m3,
                                            master_scales, as_stream(stream)));
}

agoq_status agoq_dbca_pp_bits(int stages, int microbatches, int base_bits, int *bits) {
    if (stages < 1 || microbatches < 1) return AGOQ_ERR_SHAPE;
    if (base_bits != 4 && base_bits != 5 && base_bits != 6 && base_bits != 8) return AGOQ_ERR_BITS;
    if (!bits) return AGOQ_ERR_NULL;
    static const int kWidths[4] = {4, 5, 6, 8};
    const long long first = stages < microbatches ? stages : microbatches;   // stage 0's batches
    const long long cap = first * base_bits;
    for (int s = 0; s < stages; ++s) {
        const long long live = (stages - s) < microbatches ? (stages - s) : microbatches;
        int b = base_bits;
        for (int i = 0; i < 4; ++i)
            if (kWidths[i] >= base_bits && live * kWidths[i] <= cap) b = kWidths[i];
        bits[s] = b;
    }
    return AGOQ_OK;
}

agoq_status agoq_fwd_gemm_quant(const void *x_bf16, const void *w_bf16, int T, int N, int K,
                                int bits, void *y_bf16, void *codes, float *scales, void *stream) {
    using namespace agoq;
    if (!bits_ok(bits)) return AGOQ_ERR_BITS;
    if (T <= 0 || N <= 0 || K <= 0 || T % 128 || N % 256 || K % 64) return AGOQ_ERR_SHAPE;
    if (!x_bf16 || !w_bf16 || !y_bf16 || !codes || !scales) return AGOQ_ERR_NULL;
    if (!aligned(x_bf16, 16) || !aligned(w_bf16, 16) || !aligned(y_bf16, 16) ||
        !aligned(codes, 16) || !aligned(scales, 4))
        return AGOQ_ERR_ALIGN;
    const uint64_t n = (uint64_t)T * N, nb = n / kBlockElems;
    const uint64_t xb = 2ull * T * K, wb = 2ull * N * K, yb = 2 * n, cb = nb * 16 * bits,
                   sb = nb * 4;
    const void *in[2] = {x_bf16, w_bf16};
    const uint64_t inb[2] = {xb, wb};
    for (int i = 0; i < 2; ++i)
        if (overlap(y_bf16, yb, in[i], inb[i]) || overlap(codes, cb, in[i], inb[i]) ||
            overlap(scales, sb, in[i], inb[i]))
            return AGOQ_ERR_ALIAS;
    if (overlap(y_bf16, yb, codes, cb) || overlap(y_bf16, yb, scales, sb) ||
        overlap(codes, cb, scales, sb))
        return AGOQ_ERR_ALIAS;
    return from_cuda(launch_fwd_gemm_quant(x_bf16, w_bf16, T, N, K, bits, y_bf16, codes, scales,
                                           as_stream(stream)));
}

agoq_status agoq_layernorm_forward(const void *x, int64_t ldx, const void *w, const void *b,
                                   int param_dtype, int64_t T, int64_t H, int dtype, float eps,
                                   void *y, int64_t ldy, float *mean, float *rstd, void *codes,
                                   float *scales, int bits, void *stream) {
    using namespace agoq;
    if (!float_dtype(dtype) || (param_dtype != AGOQ_F32 && param_dtype != dtype))
        return AGOQ_ERR_FORMAT;
    const bool quant = codes || scales;
    if (quant && dtype != AGOQ_BF16) return AGOQ_ERR_FORMAT;
    if (quant && !bits_ok(bits)) return AGOQ_ERR_BITS;
    if (T < 0 || H < 1 || H > kMaxHidden || !rows_ok(T, H, ldx) || !rows_ok(T, H, ldy) ||
        !(eps >= 0.0f) || eps > 3.0e38f || (quant && H % kBlockElems))
        return AGOQ_ERR_SHAPE;
    if (T == 0) return AGOQ_OK;
    if (!x || !y || (quant && (!codes || !scales))) return AGOQ_ERR_NULL;
    const int es = elem_size(dtype), ps = elem_size(param_dtype);
    if (!aligned(x, es) || !aligned(y, es) || !aligned(w, ps) || !aligned(b, ps) ||
        !aligned(mean, 4) || !aligned(rstd, 4) || !aligned(codes, 16) || !aligned(scales, 4))
        return AGOQ_ERR_ALIGN;
    const uint64_t nb = quant ? (uint64_t)T * H / kBlockElems : 0;
    const Range xr = rows(x, T, H, ldx, es), yr = rows(y, T, H, ldy, es);
    const bool in_place = x == y && ldx == ldy;
    const Range out[5] = {in_place ? Range{y, 0} : yr, vec(mean, T, 4), vec(rstd, T, 4),
                          {codes, nb * 16 * bits}, {scales, nb * 4}};
    const Range in[3] = {xr, vec(w, H, ps), vec(b, H, ps)};
    if (any_overlap(out, in) || (in_place && (overlap(y, yr.n, w, in[1].n) ||
                                              overlap(y, yr.n, b, in[2].n))))
        return AGOQ_ERR_ALIAS;
    const LnForward a{x, ldx, w, b, param_dtype == AGOQ_F32, T, H, dtype, eps, y, ldy,
                      mean, rstd, codes, scales, bits};
    return from_cuda(launch_ln_forward(a, as_stream(stream)));
}

int64_t agoq_layernorm_backward_workspace_bytes(int64_t T, int64_t H) {
    using namespace agoq;
    if (T < 0 || H < 1 || H > kMaxHidden || !rows_ok(T, H, H)) return -1;
    return ln_workspace_floats(T, H) * 4;
}

static agoq_status layernorm_backward_common(agoq::LnBackward a, int param_dtype,
                                             int64_t workspace_bytes, void *stream) {
    using namespace agoq;
    if (!float_dtype(a.dtype) || (param_dtype != AGOQ_F32 && param_dtype != a.dtype))
        return AGOQ_ERR_FORMAT;
    if (a.T < 0 || a.H < 1 || a.H > kMaxHidden || !rows_ok(a.T, a.H, a.ldx) ||
        !rows_ok(a.T, a.H, a.lddy) || !rows_ok(a.T, a.H, a.lddx) ||
        (a.bits && (a.H % kBlockElems || !(a.eps >= 0.0f) || a.eps > 3.0e38f)))
        return AGOQ_ERR_SHAPE;
    const bool sums = a.dw || a.db;
    if (a.T == 0 && !sums) return AGOQ_OK;
    if (a.T > 0) {
        if (!a.x || !a.dy || !a.dx) return AGOQ_ERR_NULL;
        if (a.bits ? !a.scales : (!a.mean || !a.rstd)) return AGOQ_ERR_NULL;
        if (sums && !a.workspace) return AGOQ_ERR_NULL;
        if (sums && workspace_bytes < ln_workspace_floats(a.T, a.H) * 4) return AGOQ_ERR_SHAPE;
    }
    const int es = elem_size(a.dtype), ps = elem_size(param_dtype);
    if (!aligned(a.x, a.bits ? 16 : es) || !aligned(a.scales, 4) || !aligned(a.dy, es) ||
        !aligned(a.w, ps) || !aligned(a.mean, 4) || !aligned(a.rstd, 4) || !aligned(a.dx, es) ||
        !aligned(a.dw, 4) || !aligned(a.db, 4) || (sums && !aligned(a.workspace, 16)))
        return AGOQ_ERR_ALIGN;
    const uint64_t nb = (uint64_t)a.T * a.H / kBlockElems;
    const Range xr = a.bits ? Range{a.x, nb * 16 * a.bits} : rows(a.x, a.T, a.H, a.ldx, es);
    const Range dyr = rows(a.dy, a.T, a.H, a.lddy, es), dxr = rows(a.dx, a.T, a.H, a.lddx, es);
    const bool on_dy = a.dx == a.dy && a.lddx == a.lddy;
    const bool on_x = !a.bits && a.dx == a.x && a.lddx == a.ldx;
    const Range out[4] = {vec(a.dw, a.H, 4), vec(a.db, a.H, 4),
                          {a.workspace, sums && a.T > 0
                                            ? (uint64_t)ln_workspace_floats(a.T, a.H) * 4 : 0},
                          dxr};
    const Range in[6] = {on_x ? Range{a.x, 0} : xr, on_dy ? Range{a.dy, 0} : dyr,
                         vec(a.w, a.H, ps), vec(a.mean, a.T, 4), vec(a.rstd, a.T, 4),
                         {a.scales, a.scales ? nb * 4 : 0}};
    if (any_overlap(out, in)) return AGOQ_ERR_ALIAS;
    // x and dy with dx on one of them: the other must be clear of it
    if (a.T > 0 && on_x && on_dy) return AGOQ_ERR_ALIAS;
    if (a.T == 0) {
        cudaError_t e = cudaSuccess;
        if (a.dw) e = cudaMemsetAsync(a.dw, 0, 4ull * a.H, as_stream(stream));
        if (e == cudaSuccess && a.db) e = cudaMemsetAsync(a.db, 0, 4ull * a.H, as_stream(stream));
        return from_cuda(e);
    }
    return from_cuda(launch_ln_backward(a, as_stream(stream)));
}

agoq_status agoq_layernorm_backward(const void *x, int64_t ldx, const void *dy, int64_t lddy,
                                    const void *w, int param_dtype, const float *mean,
                                    const float *rstd, int64_t T, int64_t H, int dtype, void *dx,
                                    int64_t lddx, float *dw, float *db, void *workspace,
                                    int64_t workspace_bytes, void *stream) {
    agoq::LnBackward a{};
    a.x = x, a.ldx = ldx, a.dy = dy, a.lddy = lddy, a.w = w;
    a.param_f32 = param_dtype == AGOQ_F32;
    a.mean = mean, a.rstd = rstd, a.T = T, a.H = H, a.dtype = dtype, a.dx = dx, a.lddx = lddx;
    a.dw = dw, a.db = db, a.workspace = static_cast<float *>(workspace);
    return layernorm_backward_common(a, param_dtype, workspace_bytes, stream);
}

agoq_status agoq_layernorm_backward_laaq(const void *codes, const float *scales, int bits,
                                         const void *dy_bf16, int64_t lddy, const void *w,
                                         int param_dtype, int64_t T, int64_t H, float eps,
                                         void *dx_bf16, int64_t lddx, float *dw, float *db,
                                         void *workspace, int64_t workspace_bytes, void *stream) {
    if (!agoq::bits_ok(bits)) return AGOQ_ERR_BITS;
    agoq::LnBackward a{};
    a.x = codes, a.ldx = H, a.scales = scales, a.bits = bits, a.dy = dy_bf16, a.lddy = lddy, a.w = w;
    a.param_f32 = param_dtype == AGOQ_F32;
    a.T = T, a.H = H, a.dtype = AGOQ_BF16, a.eps = eps, a.dx = dx_bf16, a.lddx = lddx;
    a.dw = dw, a.db = db, a.workspace = static_cast<float *>(workspace);
    return layernorm_backward_common(a, param_dtype, workspace_bytes, stream);
}

// One tensor of a gradient list; `clip`: its output too.
static agoq_status grad_tensor_check(const agoq_grad_tensor &t, bool clip) {
    using namespace agoq;
    const bool fp8 = t.dtype == AGOQ_E4M3;
    if (!fp8 && !float_dtype(t.dtype)) return AGOQ_ERR_FORMAT;
    if (t.n < 0 || t.n > (1ll << 40) || (fp8 && t.n % kBlockElems)) return AGOQ_ERR_SHAPE;
    if (t.n == 0) return AGOQ_OK;
    if (!t.data || (fp8 && !t.scales) || (clip && !t.out)) return AGOQ_ERR_NULL;
    const int es = fp8 ? 4 : elem_size(t.dtype);
    if (!aligned(t.data, fp8 ? 16 : es) || (fp8 && !aligned(t.scales, 4)) ||
        (clip && !aligned(t.out, es)))
        return AGOQ_ERR_ALIGN;
    if (!clip) return AGOQ_OK;
    const Range out = fp8 ? vec(t.out, t.n / kBlockElems, 4) : vec(t.out, t.n, es);
    if (fp8 && overlap(out.p, out.n, t.data, t.n)) return AGOQ_ERR_ALIAS;
    const void *from = fp8 ? t.scales : t.data;
    return t.out != from && overlap(out.p, out.n, from, out.n) ? AGOQ_ERR_ALIAS : AGOQ_OK;
}

static agoq_status grad_list_ok(const agoq_grad_tensor *tensors, int count, bool clip) {
    if (count < 0) return AGOQ_ERR_SHAPE;
    if (count > 0 && !tensors) return AGOQ_ERR_NULL;
    int64_t total = 0;
    for (int i = 0; i < count; ++i) {
        const agoq_status s = grad_tensor_check(tensors[i], clip);
        if (s != AGOQ_OK) return s;
        total += tensors[i].n;
        if (total > (1ll << 43)) return AGOQ_ERR_SHAPE;
    }
    return AGOQ_OK;
}

agoq_status agoq_grad_list_check(const agoq_grad_tensor *tensors, int count) {
    using namespace agoq;
    const agoq_status s = grad_list_ok(tensors, count, true);
    if (s != AGOQ_OK) return s;
    // Every range that is read or written, by address: a written one must not
    // meet another tensor's range.
    Span *spans = new (std::nothrow) Span[count > 0 ? 3 * (size_t)count : 1];
    if (!spans) return AGOQ_ERR_CUDA;
    size_t m = 0;
    for (int i = 0; i < count; ++i) {
        const agoq_grad_tensor &t = tensors[i];
        if (t.n == 0) continue;
        const bool fp8 = t.dtype == AGOQ_E4M3;
        const uintptr_t d = reinterpret_cast<uintptr_t>(t.data),
                        o = reinterpret_cast<uintptr_t>(t.out),
                        c = reinterpret_cast<uintptr_t>(t.scales);
        const uint64_t db = (uint64_t)t.n * (fp8 ? 1 : elem_size(t.dtype));
        const uint64_t ob = fp8 ? (uint64_t)t.n / kBlockElems * 4 : db;
        spans[m++] = {d, d + db, i, false};
        if (fp8) spans[m++] = {c, c + ob, i, false};
        spans[m++] = {o, o + ob, i, true};
    }
    std::sort(spans, spans + m);
    bool bad = false;
    for (size_t i = 0; i < m && !bad; ++i)
        for (size_t j = i + 1; j < m && spans[j].from < spans[i].to && !bad; ++j)
            bad = (spans[i].out || spans[j].out) && spans[i].tensor != spans[j].tensor;
    delete[] spans;
    return bad ? AGOQ_ERR_ALIAS : AGOQ_OK;
}

int64_t agoq_grad_norm_workspace_bytes(int count) {
    return count < 0 ? -1 : agoq::grad_norm_workspace_bytes(count);
}

static agoq_status grad_norm_ok(const agoq_grad_tensor *tensors, int count, bool clip,
                                const float *norm, const void *workspace,
                                int64_t workspace_bytes) {
    using namespace agoq;
    const agoq_status s = grad_list_ok(tensors, count, clip);
    if (s != AGOQ_OK) return s;
    if (!norm || !workspace) return AGOQ_ERR_NULL;
    if (workspace_bytes < agoq::grad_norm_workspace_bytes(count)) return AGOQ_ERR_SHAPE;
    if (!aligned(norm, 4) || !aligned(workspace, 16)) return AGOQ_ERR_ALIGN;
    const uint64_t wb = (uint64_t)agoq::grad_norm_workspace_bytes(count);
    if (overlap(norm, 4, workspace, wb)) return AGOQ_ERR_ALIAS;
    const uintptr_t pn = reinterpret_cast<uintptr_t>(norm), pw = reinterpret_cast<uintptr_t>(workspace);
    for (int i = 0; i < count; ++i) {
        const agoq_grad_tensor &t = tensors[i];
        const bool fp8 = t.dtype == AGOQ_E4M3;
        const uint64_t db = (uint64_t)t.n * elem_size(t.dtype), sb = (uint64_t)t.n / kBlockElems * 4;
        const Range in[3] = {{t.data, db}, {t.scales, fp8 ? sb : 0}, {t.out, clip ? (fp8 ? sb : db) : 0}};
        for (int k = 0; k < 3; ++k) {
            const uintptr_t p = reinterpret_cast<uintptr_t>(in[k].p), e = p + in[k].n;
            if (in[k].n && ((p < pn + 4 && pn < e) || (p < pw + wb && pw < e))) return AGOQ_ERR_ALIAS;
        }
    }
    return AGOQ_OK;
}

agoq_status agoq_grad_norm(const agoq_grad_tensor *tensors, int count, float *norm,
                           void *workspace, int64_t workspace_bytes, void *stream) {
    using namespace agoq;
    const agoq_status s = grad_norm_ok(tensors, count, false, norm, workspace, workspace_bytes);
    if (s != AGOQ_OK) return s;
    return from_cuda(launch_grad_norm(tensors, count, norm, static_cast<double *>(workspace),
                                      as_stream(stream)));
}

agoq_status agoq_clip_grads(const agoq_grad_tensor *tensors, int count, float max_norm,
                            const float *norm, void *stream) {
    using namespace agoq;
    const agoq_status s = grad_list_ok(tensors, count, true);
    if (s != AGOQ_OK) return s;
    if (!(max_norm >= 0.0f) || max_norm > 3.0e38f) return AGOQ_ERR_SHAPE;
    if (!norm) return AGOQ_ERR_NULL;
    if (!aligned(norm, 4)) return AGOQ_ERR_ALIGN;
    for (int i = 0; i < count; ++i) {
        const agoq_grad_tensor &t = tensors[i];
        const bool fp8 = t.dtype == AGOQ_E4M3;
        if (overlap(norm, 4, t.out, fp8 ? (uint64_t)t.n / kBlockElems * 4
                                        : (uint64_t)t.n * elem_size(t.dtype)))
            return AGOQ_ERR_ALIAS;
    }
    return from_cuda(launch_clip_grads(tensors, count, max_norm, norm, as_stream(stream)));
}

agoq_status agoq_clip_grad_norm(const agoq_grad_tensor *tensors, int count, float max_norm,
                                float *norm, void *workspace, int64_t workspace_bytes,
                                void *stream) {
    using namespace agoq;
    const agoq_status s = grad_norm_ok(tensors, count, true, norm, workspace, workspace_bytes);
    if (s != AGOQ_OK) return s;
    if (!(max_norm >= 0.0f) || max_norm > 3.0e38f) return AGOQ_ERR_SHAPE;
    return from_cuda(launch_clip_grad_norm(tensors, count, max_norm, norm,
                                           static_cast<double *>(workspace), as_stream(stream)));
}

agoq_status agoq_token_logprobs(const void *logits, int64_t ld, int dtype, const int64_t *tokens,
                                int64_t T, int64_t V, int k, float *logp, float *entropy,
                                float *lse, float *top_logp, int64_t *top_ids, void *stream) {
    using namespace agoq;
    if (!float_dtype(dtype)) return AGOQ_ERR_FORMAT;
    if (T < 0 || V < 1 || V > kMaxVocab || !rows_ok(T, V, ld) || k < 0 || k > kMaxTop || k > V)
        return AGOQ_ERR_SHAPE;
    if (T == 0) return AGOQ_OK;
    if (!logits || !tokens || (k > 0 && (!top_logp || !top_ids))) return AGOQ_ERR_NULL;
    const int es = elem_size(dtype);
    if (k == 0) top_logp = nullptr, top_ids = nullptr;
    if (!aligned(logits, es) || !aligned(tokens, 8) || !aligned(logp, 4) || !aligned(entropy, 4) ||
        !aligned(lse, 4) || !aligned(top_logp, 4) || !aligned(top_ids, 8))
        return AGOQ_ERR_ALIGN;
    const Range out[5] = {vec(logp, T, 4), vec(entropy, T, 4), vec(lse, T, 4),
                          vec(top_logp, T * k, 4), vec(top_ids, T * k, 8)};
    const Range in[2] = {rows(logits, T, V, ld, es), vec(tokens, T, 8)};
    if (any_overlap(out, in)) return AGOQ_ERR_ALIAS;
    TokenLogprobs a{};
    a.logits = logits, a.ld = ld, a.dtype = dtype, a.tokens = tokens, a.T = T, a.V = V, a.k = k;
    a.logp = logp, a.entropy = entropy, a.lse = lse, a.top_logp = top_logp, a.top_ids = top_ids;
    return from_cuda(launch_token_logprobs(a, as_stream(stream)));
}

agoq_status agoq_token_logprobs_backward(const void *logits, int64_t ld, int dtype,
                                         const int64_t *tokens, int64_t T, int64_t V,
                                         const float *lse, const float *entropy,
                                         const float *dlogp, const float *dentropy, void *dlogits,
                                         int64_t ldd, void *stream) {
    using namespace agoq;
    if (!float_dtype(dtype)) return AGOQ_ERR_FORMAT;
    if (T < 0 || V < 1 || V > kMaxVocab || !rows_ok(T, V, ld) || !rows_ok(T, V, ldd))
        return AGOQ_ERR_SHAPE;
    if (T == 0) return AGOQ_OK;
    if (!logits || !tokens || !lse || !dlogp || !dlogits || (dentropy && !entropy))
        return AGOQ_ERR_NULL;
    const int es = elem_size(dtype);
    if (!aligned(logits, es) || !aligned(tokens, 8) || !aligned(lse, 4) || !aligned(entropy, 4) ||
        !aligned(dlogp, 4) || !aligned(dentropy, 4) || !aligned(dlogits, es))
        return AGOQ_ERR_ALIGN;
    const Range out[1] = {rows(dlogits, T, V, ldd, es)};
    const bool in_place = logits == dlogits && ld == ldd;
    const Range lr = rows(logits, in_place ? 0 : T, V, ld, es);
    const Range in[6] = {lr,
                         vec(tokens, T, 8), vec(lse, T, 4), vec(entropy, T, 4), vec(dlogp, T, 4),
                         vec(dentropy, T, 4)};
    if (any_overlap(out, in)) return AGOQ_ERR_ALIAS;
    const TokenLogprobsBackward a{logits, ld, dtype, tokens, T, V, lse, entropy, dlogp, dentropy,
                                  dlogits, ldd};
    return from_cuda(launch_token_logprobs_backward(a, as_stream(stream)));
}

agoq_status agoq_token_loss(const void *logits, int64_t ld, int dtype, const int64_t *tokens,
                            const float *weights, int64_t T, int64_t V, float *logp, void *dlogits,
                            int64_t ldd, void *stream) {
    using namespace agoq;
    if (!float_dtype(dtype)) return AGOQ_ERR_FORMAT;
    if (T < 0 || V < 1 || V > kMaxVocab || !rows_ok(T, V, ld) || !rows_ok(T, V, ldd))
        return AGOQ_ERR_SHAPE;
    if (T == 0) return AGOQ_OK;
    if (!logits || !tokens || !dlogits) return AGOQ_ERR_NULL;
    const int es = elem_size(dtype);
    if (!aligned(logits, es) || !aligned(tokens, 8) || !aligned(weights, 4) || !aligned(logp, 4) ||
        !aligned(dlogits, es))
        return AGOQ_ERR_ALIGN;
    const Range out[2] = {rows(dlogits, T, V, ldd, es), vec(logp, T, 4)};
    const bool in_place = logits == dlogits && ld == ldd;
    const Range lr = rows(logits, in_place ? 0 : T, V, ld, es);
    const Range in[3] = {lr,
                         vec(tokens, T, 8), vec(weights, T, 4)};
    if (any_overlap(out, in)) return AGOQ_ERR_ALIAS;
    TokenLogprobs a{};
    a.logits = logits, a.ld = ld, a.dtype = dtype, a.tokens = tokens, a.T = T, a.V = V;
    a.logp = logp, a.weights = weights, a.dlogits = dlogits, a.ldd = ldd;
    return from_cuda(launch_token_logprobs(a, as_stream(stream)));
}

agoq_status agoq_test_wait_timeout(int64_t limit_cycles, void *stream) {
    if (limit_cycles <= 0 || limit_cycles > 4000000000ll) return AGOQ_ERR_SHAPE;
    return agoq::from_cuda(agoq::launch_wait_timeout_probe(limit_cycles, agoq::as_stream(stream)));
}

agoq_status agoq_device_status(void *stream) {
    unsigned status = 0, fwd = 0, red = 0, rms = 0;
    if (agoq::read_and_clear_device_status(agoq::as_stream(stream), &status) != cudaSuccess ||
        agoq::read_and_clear_fwd_status(&fwd) != cudaSuccess ||
        agoq::read_and_clear_reduce_status(&red) != cudaSuccess ||
        agoq::read_and_clear_rmsnorm_status(&rms) != cudaSuccess)
        return AGOQ_ERR_CUDA;
    return (status || fwd || red || rms) ? AGOQ_ERR_TIMEOUT : AGOQ_OK;
}

}  // extern "C"
