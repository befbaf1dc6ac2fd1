// preference.cu -- the preference loss of pairs of answers from the log probabilities of their
// tokens, with its gradient in those.
//
// Pair p has the chosen answer's tokens [o_2p, o_2p+1) and the rejected one's [o_2p+1, o_2p+2).
// With S the sums of logp - ref_logp over an answer's tokens:
//   h = beta (S_chosen - S_rejected)
//   loss = w ((1 - e) ln(1 + e^-h) + e ln(1 + e^h))          e: label smoothing
//   dlogp = -c at the chosen tokens, c at the rejected ones,  c = w beta (1/(1 + e^h) - e)
// since d loss / dh = -w ((1 - e) s(-h) - e s(h)) and s(h) + s(-h) = 1.
#include <cooperative_groups.h>

#include "agoq_launch.h"
#include "typed_io.cuh"

namespace agoq {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256, kWarps = kThreads / 32, kMaxCluster = 8;

// A sum of binary32 differences held in two binary32 numbers: the roundings of every
// difference and addition are added up too (binary64 additions would take longer than the
// loads).
struct Sum {
    float s = 0.0f, c = 0.0f;
    __device__ __forceinline__ void add(float a, float b) {      // a - b
        const float d = __fsub_rn(a, b);
        const float bb = __fsub_rn(a, d);
        c = __fadd_rn(c, __fadd_rn(__fsub_rn(a, __fadd_rn(d, bb)), __fsub_rn(bb, b)));
        const float t = __fadd_rn(s, d);
        const float z = __fsub_rn(t, s);
        c = __fadd_rn(c, __fadd_rn(__fsub_rn(s, __fsub_rn(t, z)), __fsub_rn(d, z)));
        s = t;
    }
    // (c of a sum that is not finite is NaN.)
    __device__ __forceinline__ double value() const {
        return fabsf(s) <= 3.402823466e38f ? (double)s + (double)c : (double)s;
    }
};

// The [from, to) part of a range that a CTA of a cluster of C takes, cut at multiples of 4.
__device__ __forceinline__ void cut(int64_t a, int64_t b, int C, int rank, int64_t &from,
                                    int64_t &to) {
    const int64_t per = ((b - a + C - 1) / C + 3) / 4 * 4;
    from = a + per * rank < b ? a + per * rank : b;
    to = from + per < b ? from + per : b;
}

// f(i) for single elements and g(i) for four from i on, where the address of p + i is a
// multiple of 16 bytes.
template <typename F, typename G>
__device__ __forceinline__ void each(const float *p, int64_t from, int64_t to, F f, G g) {
    const int64_t skip = (16 - (reinterpret_cast<uintptr_t>(p + from) & 15u)) / 4 % 4;
    const int64_t head = from + skip < to ? from + skip : to, n = (to - head) / 4;
    for (int64_t i = from + threadIdx.x; i < head; i += kThreads) f(i);
#pragma unroll 4
    for (int64_t j = threadIdx.x; j < n; j += kThreads) g(head + 4 * j);
    for (int64_t i = head + 4 * n + threadIdx.x; i < to; i += kThreads) f(i);
}

__device__ __forceinline__ float4 load4(const float *p) {
    return __ldg(reinterpret_cast<const float4 *>(p));
}
// Four values at any alignment.
__device__ __forceinline__ float4 load4_any(const float *p) {
    return make_float4(__ldg(p), __ldg(p + 1), __ldg(p + 2), __ldg(p + 3));
}

__global__ void __launch_bounds__(kThreads) preference_kernel(const PreferenceLoss a) {
    __shared__ double part[kWarps], mine;
    cg::cluster_group cluster = cg::this_cluster();
    const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait_and_release();
    for (int64_t p = blockIdx.x / C; p < a.P; p += gridDim.x / C) {
        const int64_t o0 = __ldg(a.offsets + 2 * p), o1 = __ldg(a.offsets + 2 * p + 1),
                      o2 = __ldg(a.offsets + 2 * p + 2);
        const bool valid = o0 >= 0 && o0 <= o1 && o1 <= o2 && o2 <= a.T;
        int64_t from[2] = {0, 0}, to[2] = {0, 0};
        if (valid) {
            cut(o0, o1, C, rank, from[0], to[0]);
            cut(o1, o2, C, rank, from[1], to[1]);
        }
        const bool together =
            ((reinterpret_cast<uintptr_t>(a.logp) ^ reinterpret_cast<uintptr_t>(a.ref_logp)) & 15u) == 0;
        double h = 0.0;
#pragma unroll
        for (int side = 0; side < 2; ++side) {
            Sum s;
            each(a.logp, from[side], to[side],
                 [&](int64_t i) { s.add(__ldg(a.logp + i), a.ref_logp ? __ldg(a.ref_logp + i) : 0.0f); },
                 [&](int64_t i) {
                     const float4 l = load4(a.logp + i);
                     const float4 r = !a.ref_logp ? make_float4(0, 0, 0, 0)
                                      : together  ? load4(a.ref_logp + i)
                                                  : load4_any(a.ref_logp + i);
                     s.add(l.x, r.x);
                     s.add(l.y, r.y);
                     s.add(l.z, r.z);
                     s.add(l.w, r.w);
                 });
            h += side ? -s.value() : s.value();
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) h += __shfl_xor_sync(0xFFFFFFFFu, h, o);
        if (lane == 0) part[warp] = h;
        __syncthreads();
        double total = 0.0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) total += part[w];
        if (C > 1) {
            if (threadIdx.x == 0) mine = total;
            cluster.sync();
            total = 0.0;
            for (int r = 0; r < C; ++r) total += *cluster.map_shared_rank(&mine, r);
            cluster.sync();                    // all have read before the next pair
        } else {
            __syncthreads();
        }
        const float hf = valid ? (float)((double)a.beta * total) : NAN;
        const float w = a.weights ? __ldg(a.weights + p) : 1.0f;
        const float small = expf(-fabsf(hf)), tail = log1pf(small);
        if (rank == 0 && threadIdx.x == 0) {
            const float down = __fadd_rn(fmaxf(-hf, 0.0f), tail), up = __fadd_rn(fmaxf(hf, 0.0f), tail);
            float loss = __fmul_rn(1.0f - a.smoothing, down);
            if (a.smoothing > 0.0f) loss = __fmaf_rn(a.smoothing, up, loss);   // up may be infinite
            if (a.loss) a.loss[p] = hf != hf ? NAN : __fmul_rn(w, loss);
            if (a.margin) a.margin[p] = hf;
        }
        // 1 / (1 + e^h)
        const float s = __fdiv_rn(hf >= 0.0f ? small : 1.0f, __fadd_rn(1.0f, small));
        const float c = hf != hf ? NAN : __fmul_rn(__fmul_rn(w, a.beta), __fsub_rn(s, a.smoothing));
#pragma unroll
        for (int side = 0; side < 2; ++side) {
            const float v = side ? c : -c;
            each(a.dlogp, from[side], to[side], [&](int64_t i) { a.dlogp[i] = v; },
                 [&](int64_t i) {
                     *reinterpret_cast<float4 *>(a.dlogp + i) = make_float4(v, v, v, v);
                 });
        }
    }
}

}  // namespace

cudaError_t launch_preference_loss(const PreferenceLoss &a, cudaStream_t st) {
    // a CTA for 2048 tokens of an average pair
    const int64_t mean = a.T / a.P;
    int c = 1;
    while (c < kMaxCluster && mean > c * 2048ll) c *= 2;
    const int64_t most = (1 << 24) / c;
    return launch_pdl_clusters(preference_kernel, (int)(a.P < most ? a.P : most) * c, kThreads, c,
                               0, st, a);
}

}  // namespace agoq
