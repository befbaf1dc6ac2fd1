// layernorm.cu -- layer norm: the forward pass, which can keep the LAAQ codes
// of its input in the same pass, and the backward pass, from the input itself
// or from those codes ("AGoQ: Activation and Gradient Quantization for
// Memory-Efficient Distributed Training of LLMs", section 2.A "Herberekening
// versus Caching": only the quantized input is kept; the backward pass
// dequantizes it and recomputes the row statistics).
//
// Per row of H elements, in binary32:
//   mu = sum x / H,  var = sum (x - mu)^2 / H,  r = 1 / sqrt(var + eps),
//   xh = (x - mu) r,  y = xh w + b;
//   g = dy w,  dx = r (g - sum(g)/H - xh sum(g xh)/H),
//   dw = sum_t dy xh,  db = sum_t dy.
#include "agoq_launch.h"
#include "typed_io.cuh"

namespace agoq {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;

// Weight or bias element i (FP32, or the type of the activation), `none` where
// there is no such vector.
template <int DT>
__device__ __forceinline__ float param(const void *p, bool f32, int64_t i, float none) {
    if (!p) return none;
    return f32 ? load_elem<kF32>(p, i) : load_elem<DT>(p, i);
}

// LAAQ codes of a block of 128 BF16 values held by a half warp, lane c (0..15)
// having elements 8c..8c+7; the same codes and scale as agoq_quant_act.  All
// lanes of the warp call it; `valid` gates the stores.
template <int BITS>
__device__ __forceinline__ void quantize_block16(const uint4 &v, int c, uint32_t *rec, float *scale,
                                                 bool valid) {
    constexpr int kQmax = (1 << (BITS - 1)) - 1;
    constexpr int kBias = BITS < 8 ? 1 << (BITS - 1) : 0;
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    const float s = bf16_div_qmax<kQmax>(halfwarp_max(bf16_absmax<4>(w)));
    float f[8];
    Elem<kBF16>::unpack(v, f);
    uint32_t cb[8], lo, hi;
    integer_codes_n<kQmax, 8, kBias>(f, s, cb);
    if constexpr (BITS < 8) pack_biased8<BITS>(cb, lo, hi);
    else pack_fields8<BITS>(cb, lo, hi);
    store_chunk<BITS>(rec, c, lo, hi, valid);
    if (valid && c == 0) *scale = s;
}

// ---- forward ------------------------------------------------------------------

// One CTA a row, one element a thread and step; any length, stride and
// alignment.
template <int DT>
__global__ void __launch_bounds__(kThreads) ln_forward_kernel(
    const void *x, int64_t ldx, const void *__restrict__ w, const void *__restrict__ b, bool pf32,
    int64_t T, int64_t H, float eps, void *y, int64_t ldy, float *__restrict__ mean, float *__restrict__ rstd) {
    pdl_wait_and_release();
    __shared__ float red[2][kWarps];
    for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
        const char *xr = elem_at<DT>(x, t * ldx);
        char *yr = elem_at<DT>(y, t * ldy);
        float s = 0.0f;
        for (int64_t i = threadIdx.x; i < H; i += kThreads) s = __fadd_rn(s, load_now<DT>(xr, i));
        const float mu = __fdiv_rn(cta_sum<kWarps>(s, red[0]), (float)H);
        float q = 0.0f;
        for (int64_t i = threadIdx.x; i < H; i += kThreads) {
            const float d = __fsub_rn(load_now<DT>(xr, i), mu);
            q = __fmaf_rn(d, d, q);
        }
        const float var = __fdiv_rn(cta_sum<kWarps>(q, red[1]), (float)H);
        const float r = __frcp_rn(__fsqrt_rn(__fadd_rn(var, eps)));
        for (int64_t i = threadIdx.x; i < H; i += kThreads) {
            const float xh = __fmul_rn(__fsub_rn(load_now<DT>(xr, i), mu), r);
            store_elem<DT>(yr, i, __fmaf_rn(xh, param<DT>(w, pf32, i, 1.0f),
                                            param<DT>(b, pf32, i, 0.0f)));
        }
        if (threadIdx.x == 0) {
            if (mean) mean[t] = mu;
            if (rstd) rstd[t] = r;
        }
    }
}

// The codes of x, a half warp a block.
template <int BITS>
__global__ void __launch_bounds__(kThreads) ln_codes_kernel(const void *__restrict__ x, int64_t ldx,
                                                            int64_t T, int64_t H,
                                                            uint32_t *__restrict__ codes,
                                                            float *__restrict__ scales) {
    pdl_wait_and_release();
    const int64_t per_row = H / kBlock, blocks = T * per_row;
    const int c = threadIdx.x & 15;
    const int64_t stride = (int64_t)gridDim.x * (kThreads / 16);
    // every lane of a warp takes the same number of steps
    for (int64_t b0 = (int64_t)blockIdx.x * (kThreads / 16) + (threadIdx.x >> 5) * 2; b0 < blocks;
         b0 += stride) {
        const int64_t blk = b0 + ((threadIdx.x >> 4) & 1);
        const bool valid = blk < blocks;
        uint32_t v[4] = {0, 0, 0, 0};
        if (valid) {
            const uint16_t *p = static_cast<const uint16_t *>(x) + (blk / per_row) * ldx +
                                (blk % per_row) * kBlock + 8 * c;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] = (uint32_t)__ldg(p + 2 * i) | ((uint32_t)__ldg(p + 2 * i + 1) << 16);
        }
        quantize_block16<BITS>(make_uint4(v[0], v[1], v[2], v[3]), c, codes + blk * 4 * BITS,
                               scales + blk, valid);
    }
}

// ---- backward -----------------------------------------------------------------

// Where the backward pass finds its input: a tensor of type DT (BITS 0), or
// codes of BITS bits.
template <int DT, int BITS>
struct Input {
    const void *x;          // tensor, or codes
    const float *scales;
    int64_t ld;             // row distance in elements
    __device__ __forceinline__ float get(int64_t t, int64_t i) const {
        if constexpr (BITS == 0) {
            return load_now<DT>(x, t * ld + i);   // dx may be in its place
        } else {
            const int64_t blk = (t * ld + i) / kBlock;
            const int bit = (int)(i % kBlock) * BITS;
            const uint32_t *rec = static_cast<const uint32_t *>(x) + blk * 4 * BITS;
            const int word = bit >> 5;
            const uint32_t lo = __ldg(rec + word);
            const uint32_t hi = word + 1 < 4 * BITS ? __ldg(rec + word + 1) : 0u;
            const float c = field_value<BITS>(lo, hi, bit & 31);
            return Elem<kBF16>::up(Elem<kBF16>::down(__fmul_rn(c, __ldg(scales + blk))));
        }
    }
};

// One CTA a row and step, one element a thread and step.  From codes the
// statistics are recomputed; else they are arguments.  Thread i adds the row's
// terms of the columns i, i + 256, ... to row blockIdx.x of the partial sums
// ([grid][2][H]), if `partials` is given.
template <int DT, int BITS>
__global__ void __launch_bounds__(kThreads) ln_backward_kernel(
    Input<DT, BITS> in, const void *dy, int64_t lddy, const void *__restrict__ w, bool pf32,
    const float *__restrict__ mean, const float *__restrict__ rstd, int64_t T, int64_t H,
    float eps, void *dx, int64_t lddx, float *__restrict__ partials) {
    pdl_wait_and_release();
    __shared__ float red[4][kWarps];
    float *sums = partials ? partials + (int64_t)blockIdx.x * 2 * H : nullptr;
    for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
        float mu, r;
        if constexpr (BITS == 0) {
            mu = __ldg(mean + t);
            r = __ldg(rstd + t);
        } else {
            float s = 0.0f, q = 0.0f;
            for (int64_t i = threadIdx.x; i < H; i += kThreads) s = __fadd_rn(s, in.get(t, i));
            mu = __fdiv_rn(cta_sum<kWarps>(s, red[0]), (float)H);
            for (int64_t i = threadIdx.x; i < H; i += kThreads) {
                const float d = __fsub_rn(in.get(t, i), mu);
                q = __fmaf_rn(d, d, q);
            }
            const float var = __fdiv_rn(cta_sum<kWarps>(q, red[1]), (float)H);
            r = __frcp_rn(__fsqrt_rn(__fadd_rn(var, eps)));
        }
        float s0 = 0.0f, s1 = 0.0f;
        for (int64_t i = threadIdx.x; i < H; i += kThreads) {
            const float xh = __fmul_rn(__fsub_rn(in.get(t, i), mu), r);
            const float d = load_now<DT>(dy, t * lddy + i);
            const float g = __fmul_rn(d, param<DT>(w, pf32, i, 1.0f));
            s0 = __fadd_rn(s0, g);
            s1 = __fmaf_rn(g, xh, s1);
            if (sums) {
                const bool first = t < gridDim.x;
                sums[i] = __fmaf_rn(d, xh, first ? 0.0f : sums[i]);
                sums[H + i] = __fadd_rn(d, first ? 0.0f : sums[H + i]);
            }
        }
        s0 = __fdiv_rn(cta_sum<kWarps>(s0, red[2]), (float)H);
        s1 = __fdiv_rn(cta_sum<kWarps>(s1, red[3]), (float)H);
        for (int64_t i = threadIdx.x; i < H; i += kThreads) {
            const float xh = __fmul_rn(__fsub_rn(in.get(t, i), mu), r);
            const float g =
                __fmul_rn(load_now<DT>(dy, t * lddy + i), param<DT>(w, pf32, i, 1.0f));
            store_elem<DT>(dx, t * lddx + i,
                           __fmul_rn(r, __fmaf_rn(-xh, s1, __fsub_rn(g, s0))));
        }
        __syncthreads();   // red is rewritten for the next row
    }
}

// dw and db: the P partial rows in order.
__global__ void __launch_bounds__(kThreads) ln_backward_join_kernel(
    const float *__restrict__ partials, int64_t H, int P, float *__restrict__ dw,
    float *__restrict__ db) {
    pdl_wait_and_release();
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < 2 * H;
         i += (int64_t)gridDim.x * kThreads) {
        float *out = i < H ? dw : db;
        if (!out) continue;
        float s = 0.0f;
        for (int p = 0; p < P; ++p) s = __fadd_rn(s, __ldg(partials + (int64_t)p * 2 * H + i));
        out[i < H ? i : i - H] = s;
    }
}

int grid_for(int64_t units, int per_sm) {
    const int64_t most = (int64_t)sm_count() * per_sm;
    return (int)(units < most ? (units > 0 ? units : 1) : most);
}

template <int DT, int BITS>
cudaError_t backward(const Input<DT, BITS> &in, const LnBackward &a, cudaStream_t st) {
    const bool sums = a.dw || a.db;
    const int P = sums ? ln_partials(a.T) : grid_for(a.T, 8);
    const cudaError_t e = launch_pdl(ln_backward_kernel<DT, BITS>, P, kThreads, 0, st, in, a.dy,
                                     a.lddy, a.w, a.param_f32, a.mean, a.rstd, a.T, a.H, a.eps,
                                     a.dx, a.lddx, sums ? a.workspace : nullptr);
    if (e != cudaSuccess || !sums) return e;
    return launch_pdl(ln_backward_join_kernel, grid_for((2 * a.H + kThreads - 1) / kThreads, 8),
                      kThreads, 0, st, a.workspace, a.H, P, a.dw, a.db);
}

template <int DT>
cudaError_t forward(const LnForward &a, cudaStream_t st) {
    return launch_pdl(ln_forward_kernel<DT>, grid_for(a.T, 8), kThreads, 0, st, a.x, a.ldx, a.w, a.b,
                      a.param_f32, a.T, a.H, a.eps, a.y, a.ldy, a.mean, a.rstd);
}

template <int BITS>
cudaError_t codes(const LnForward &a, cudaStream_t st) {
    const int64_t blocks = a.T * (a.H / kBlock);
    return launch_pdl(ln_codes_kernel<BITS>, grid_for((blocks + 15) / 16, 8), kThreads, 0, st, a.x,
                      a.ldx, a.T, a.H, static_cast<uint32_t *>(a.codes), a.scales);
}

}  // namespace

// Rows of partial sums of dw and db: at most kLnPartials.
int ln_partials(int64_t T) { return (int)(T < kLnPartials ? T : kLnPartials); }

cudaError_t launch_ln_forward(const LnForward &a, cudaStream_t st) {
    cudaError_t e = a.dtype == kF32    ? forward<kF32>(a, st)
                    : a.dtype == kBF16 ? forward<kBF16>(a, st)
                                       : forward<kF16>(a, st);
    if (e != cudaSuccess || !a.codes) return e;
    switch (a.bits) {
        case 4: return codes<4>(a, st);
        case 5: return codes<5>(a, st);
        case 6: return codes<6>(a, st);
        default: return codes<8>(a, st);
    }
}

cudaError_t launch_ln_backward(const LnBackward &a, cudaStream_t st) {
    if (a.bits) {
        const Input<kBF16, 4> i4{a.x, a.scales, a.H};
        switch (a.bits) {
            case 4: return backward(i4, a, st);
            case 5: return backward(Input<kBF16, 5>{a.x, a.scales, a.H}, a, st);
            case 6: return backward(Input<kBF16, 6>{a.x, a.scales, a.H}, a, st);
            default: return backward(Input<kBF16, 8>{a.x, a.scales, a.H}, a, st);
        }
    }
    switch (a.dtype) {
        case kF32: return backward(Input<kF32, 0>{a.x, nullptr, a.ldx}, a, st);
        case kBF16: return backward(Input<kBF16, 0>{a.x, nullptr, a.ldx}, a, st);
        default: return backward(Input<kF16, 0>{a.x, nullptr, a.ldx}, a, st);
    }
}

}  // namespace agoq
