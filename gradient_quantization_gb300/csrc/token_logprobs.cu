// token_logprobs.cu -- log probabilities of given tokens under a row of logits,
// with the row's entropy and its most likely alternatives; their gradient; and
// the loss of given tokens with its gradient in one call.
//
// Per row x of V logits, in binary32:
//   m = max x,  S = sum e^(x - m),  lse = m + ln S,  logp = x[token] - lse,
//   entropy = ln S - sum (x - m) e^(x - m) / S,
//   the k largest logits by (value descending, index ascending);
//   loss: d x_i = w (p_i - [i = token]),  p_i = e^(x_i - m) / S;
//   gradient of the statistics:
//     d x_i = dlogp ([i = token] - p_i) - dentropy p_i (ln p_i + entropy).
// A logit of -inf has probability 0.  A row of nothing but -inf has lse = -inf,
// logp = -inf, entropy 0 and gradient 0.
#include "agoq_launch.h"
#include "typed_io.cuh"

namespace agoq {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;

// A logit's place in the order of alternatives: larger values first, NaN before
// all, equal values (-0 and +0 among them) by ascending index.
__device__ __forceinline__ uint64_t order_key(float x, uint32_t i) {
    const uint32_t b = __float_as_uint(__fadd_rn(x, 0.0f));
    const uint32_t k = x != x ? 0xFFFFFFFFu : (b & 0x80000000u) ? ~b : b | 0x80000000u;
    return (static_cast<uint64_t>(k) << 32) | (0xFFFFFFFFu - i);
}

__device__ __forceinline__ float cta_max(float v, float *red) {
    v = warp_max(v);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = red[0];
#pragma unroll
    for (int i = 1; i < kWarps; ++i) s = fmaxf(s, red[i]);
    return s;
}

// x - m, not below -1000 (where its exponential is 0 too): for x = -inf the
// product with the exponential must be 0.  NaN stays NaN.
__device__ __forceinline__ float below_max(float x, float m) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(__fsub_rn(x, m)), "f"(-1000.0f));
    return d;
}

template <int DT>
__global__ void __launch_bounds__(kThreads) token_logprobs_kernel(const TokenLogprobs a) {
    pdl_wait_and_release();
    __shared__ float red[3][kWarps];
    __shared__ unsigned long long best;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        const char *row = elem_at<DT>(a.logits, t * a.ld);
        const int64_t token = a.tokens[t];
        const float at = token >= 0 && token < a.V ? load_now<DT>(row, token) : 0.0f;
        float m = -INFINITY;
        for (int64_t i = threadIdx.x; i < a.V; i += kThreads) m = fmaxf(m, load_now<DT>(row, i));
        m = cta_max(m, red[0]);
        if (m == -INFINITY) m = 0.0f;
        float s = 0.0f, u = 0.0f;
        for (int64_t i = threadIdx.x; i < a.V; i += kThreads) {
            const float x = load_now<DT>(row, i);
            const float d = below_max(x, m), e = expf(d);
            s = __fadd_rn(s, e);
            u = __fmaf_rn(d, e, u);
        }
        s = cta_sum<kWarps>(s, red[1]);
        u = cta_sum<kWarps>(u, red[2]);
        const float ls = logf(s);
        const bool ignored = token < 0, beyond = token >= a.V, empty = s == 0.0f;
        if (threadIdx.x == 0) {
            float lp = at == -INFINITY ? at : __fsub_rn(__fsub_rn(at, m), ls);
            if (ignored) lp = 0.0f;
            if (beyond) lp = NAN;
            if (a.logp) a.logp[t] = lp;
            if (a.entropy) a.entropy[t] = empty ? 0.0f : __fsub_rn(ls, __fdiv_rn(u, s));
            if (a.lse) a.lse[t] = __fadd_rn(m, ls);
        }
        uint64_t last = ~0ull;
        for (int j = 0; j < a.k; ++j) {
            uint64_t b = 0;
            for (int64_t i = threadIdx.x; i < a.V; i += kThreads) {
                const uint64_t k = order_key(load_now<DT>(row, i), (uint32_t)i);
                if (k < last && k > b) b = k;
            }
            if (threadIdx.x == 0) best = 0;
            __syncthreads();
            atomicMax(&best, b);
            __syncthreads();
            last = best;
            __syncthreads();
            if (threadIdx.x == 0) {
                const uint32_t i = 0xFFFFFFFFu - (uint32_t)last;
                const float x = load_now<DT>(row, i);
                a.top_ids[t * a.k + j] = i;
                a.top_logp[t * a.k + j] =
                    x == -INFINITY ? x : __fsub_rn(__fsub_rn(x, m), ls);
            }
        }
        if (a.dlogits) {
            float w = a.weights ? a.weights[t] : 1.0f;
            if (ignored || empty) w = 0.0f;
            if (beyond) w = NAN;
            char *out = elem_at<DT>(a.dlogits, t * a.ldd);
            for (int64_t i = threadIdx.x; i < a.V; i += kThreads) {
                const float x = load_now<DT>(row, i);
                float g = 0.0f;
                if (w != 0.0f) {
                    g = __fdiv_rn(expf(__fsub_rn(x, m)), s);
                    g = __fmul_rn(w, i == token ? __fsub_rn(g, 1.0f) : g);
                }
                store_elem<DT>(out, i, g);
            }
        }
        __syncthreads();
    }
}

template <int DT>
__global__ void __launch_bounds__(kThreads)
token_logprobs_backward_kernel(const TokenLogprobsBackward a) {
    pdl_wait_and_release();
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        const char *row = elem_at<DT>(a.logits, t * a.ld);
        char *out = elem_at<DT>(a.dlogits, t * a.ldd);
        const int64_t token = a.tokens[t];
        const float lse = a.lse[t];
        const bool empty = lse == -INFINITY;
        float dl = a.dlogp[t], de = a.dentropy ? a.dentropy[t] : 0.0f;
        const float h = a.dentropy ? a.entropy[t] : 0.0f;
        if (token < 0 || empty) dl = 0.0f;
        if (token >= a.V) dl = NAN;
        if (empty) de = 0.0f;
        for (int64_t i = threadIdx.x; i < a.V; i += kThreads) {
            const float x = load_now<DT>(row, i);
            float g = 0.0f;
            if (!empty) {
                const float l = below_max(x, lse), p = expf(l);
                g = -__fmul_rn(p, __fmaf_rn(de, __fadd_rn(l, h), dl));
                if (i == token) g = __fadd_rn(g, dl);
            }
            store_elem<DT>(out, i, g);
        }
    }
}

int grid_for(int64_t rows) {
    const int64_t most = (int64_t)sm_count() * 8;
    return (int)(rows < most ? rows : most);
}

}  // namespace

cudaError_t launch_token_logprobs(const TokenLogprobs &a, cudaStream_t st) {
    auto k = a.dtype == kF32    ? token_logprobs_kernel<kF32>
             : a.dtype == kBF16 ? token_logprobs_kernel<kBF16>
                                : token_logprobs_kernel<kF16>;
    return launch_pdl(k, grid_for(a.T), kThreads, 0, st, a);
}

cudaError_t launch_token_logprobs_backward(const TokenLogprobsBackward &a, cudaStream_t st) {
    auto k = a.dtype == kF32    ? token_logprobs_backward_kernel<kF32>
             : a.dtype == kBF16 ? token_logprobs_backward_kernel<kBF16>
                                : token_logprobs_backward_kernel<kF16>;
    return launch_pdl(k, grid_for(a.T), kThreads, 0, st, a);
}

}  // namespace agoq
