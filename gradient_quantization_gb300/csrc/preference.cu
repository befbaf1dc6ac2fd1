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

constexpr int kThreads = 128, kWarps = kThreads / 32, kMaxCluster = 8;

// A sum of binary32 differences held in two binary32 numbers: the roundings of every
// difference and addition are added up too.  (No binary64: of its additions an SM makes a few a
// clock, and 30 of them a thread, to join the threads' sums, took 86 us for 4000 short pairs.)
struct Sum {
    float s = 0.0f, c = 0.0f;
    __device__ __forceinline__ void plus(float d) {
        const float t = __fadd_rn(s, d);
        const float z = __fsub_rn(t, s);
        c = __fadd_rn(c, __fadd_rn(__fsub_rn(s, __fsub_rn(t, z)), __fsub_rn(d, z)));
        s = t;
    }
    __device__ __forceinline__ void add(float a, float b) {      // a - b
        const float d = __fsub_rn(a, b);
        const float bb = __fsub_rn(a, d);
        c = __fadd_rn(c, __fadd_rn(__fsub_rn(a, __fadd_rn(d, bb)), __fsub_rn(bb, b)));
        plus(d);
    }
    __device__ __forceinline__ void join(const Sum &o) {
        plus(o.s);
        c = __fadd_rn(c, o.c);
    }
    // (c of a sum that is not finite is NaN.)
    __device__ __forceinline__ float times(float k) const {
        const float p = __fmul_rn(k, s);
        if (!(fabsf(p) <= 3.402823466e38f)) return p;
        return __fadd_rn(p, __fmaf_rn(k, c, __fmaf_rn(k, s, -p)));
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
// multiple of 16 bytes, by THREADS threads.
template <int THREADS, typename F, typename G>
__device__ __forceinline__ void each(const float *p, int64_t from, int64_t to, F f, G g) {
    const int me = threadIdx.x % THREADS;
    const int64_t skip = (16 - (reinterpret_cast<uintptr_t>(p + from) & 15u)) / 4 % 4;
    const int64_t head = from + skip < to ? from + skip : to, n = (to - head) / 4;
    for (int64_t i = from + me; i < head; i += THREADS) f(i);
#pragma unroll 4
    for (int64_t j = me; j < n; j += THREADS) g(head + 4 * j);
    for (int64_t i = head + 4 * n + me; i < to; i += THREADS) f(i);
}

__device__ __forceinline__ float4 load4(const float *p) {
    return __ldg(reinterpret_cast<const float4 *>(p));
}
// Four values at any alignment.
__device__ __forceinline__ float4 load4_any(const float *p) {
    return make_float4(__ldg(p), __ldg(p + 1), __ldg(p + 2), __ldg(p + 3));
}

// A pair by THREADS threads: a warp, or the CTAs of a cluster.  Bound by the latency of loads one
// after another (offsets, tokens) and the join: 8 pairs of 423 tokens 4.4 us; 512 pairs of 3400,
// 1.7 million tokens, 13.6 us (1.5 TB/s: the longest pairs end last).  128 threads a CTA: with 256
// 15.3 us and with 64 19.7 us.
template <int THREADS>
__global__ void __launch_bounds__(kThreads) preference_kernel(const PreferenceLoss a) {
    constexpr bool kOne = THREADS == 32;
    __shared__ Sum part[kWarps], mine;
    cg::cluster_group cluster = cg::this_cluster();
    const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait_and_release();
    const int64_t p0 = kOne ? (int64_t)blockIdx.x * kWarps + warp : blockIdx.x / C;
    const int64_t step = kOne ? (int64_t)gridDim.x * kWarps : gridDim.x / C;
    for (int64_t p = p0; p < a.P; p += step) {
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
        Sum total;
#pragma unroll
        for (int side = 0; side < 2; ++side) {
            const float *l = a.logp, *r = a.ref_logp;
            Sum s[4];                          // four chains: each addition waits for the last
            each<THREADS>(l, from[side], to[side], [&](int64_t i) { s[0].add(__ldg(l + i), r ? __ldg(r + i) : 0.0f); },
                 [&](int64_t i) {
                     const float4 x = load4(l + i);
                     const float4 y = !r ? make_float4(0, 0, 0, 0) : together ? load4(r + i) : load4_any(r + i);
                     s[0].add(x.x, y.x);
                     s[1].add(x.y, y.y);
                     s[2].add(x.z, y.z);
                     s[3].add(x.w, y.w);
                 });
            s[0].join(s[1]);
            s[2].join(s[3]);
            s[0].join(s[2]);
            if (side) s[0].s = -s[0].s, s[0].c = -s[0].c;
            total.join(s[0]);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            Sum other;
            other.s = __shfl_xor_sync(0xFFFFFFFFu, total.s, o);
            other.c = __shfl_xor_sync(0xFFFFFFFFu, total.c, o);
            total.join(other);
        }
        if constexpr (!kOne) {
            if (lane == 0) part[warp] = total;
            __syncthreads();
            total = part[0];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) total.join(part[w]);
        }
        if (kOne) {
        } else if (C > 1) {
            if (threadIdx.x == 0) mine = total;
            cluster.sync();
            total = *cluster.map_shared_rank(&mine, 0);
            for (int r = 1; r < C; ++r) total.join(*cluster.map_shared_rank(&mine, r));
            cluster.sync();                    // all have read before the next pair
        } else {
            __syncthreads();
        }
        const float hf = valid ? total.times(a.beta) : NAN;
        const float w = a.weights ? __ldg(a.weights + p) : 1.0f;
        const float small = expf(-fabsf(hf)), tail = log1pf(small);
        if (rank == 0 && threadIdx.x % THREADS == 0) {
            const float down = __fadd_rn(fmaxf(-hf, 0.0f), tail), up = __fadd_rn(fmaxf(hf, 0.0f), tail);
            // (down or up may be infinite: a factor of 0 takes no part)
            float loss = a.smoothing < 1.0f ? __fmul_rn(1.0f - a.smoothing, down) : 0.0f;
            if (a.smoothing > 0.0f) loss = __fmaf_rn(a.smoothing, up, loss);
            if (a.loss) a.loss[p] = hf != hf ? NAN : __fmul_rn(w, loss);
            if (a.margin) a.margin[p] = hf;
        }
        // 1 / (1 + e^h)
        const float s = __fdiv_rn(hf >= 0.0f ? small : 1.0f, __fadd_rn(1.0f, small));
        const float c = hf != hf ? NAN : __fmul_rn(__fmul_rn(w, a.beta), __fsub_rn(s, a.smoothing));
#pragma unroll
        for (int side = 0; side < 2; ++side) {
            const float v = side ? c : -c;
            each<THREADS>(a.dlogp, from[side], to[side], [&](int64_t i) { a.dlogp[i] = v; },
                 [&](int64_t i) {
                     *reinterpret_cast<float4 *>(a.dlogp + i) = make_float4(v, v, v, v);
                 });
        }
    }
}

}  // namespace

cudaError_t launch_preference_loss(const PreferenceLoss &a, cudaStream_t st) {
    // A warp for a pair of up to 256 tokens on average (4000 pairs of 73: 8.0 us, 17.8 us with a CTA
    // each; 8 pairs of 423: 5.7 us, 4.4 us); else a CTA for 2048 of them (512 pairs of 3400: 13.6 us
    // with two CTAs a pair, 20 us with one, 27 us with eight).
    const int64_t mean = a.T / a.P;
    if (mean <= 256) {
        const int64_t ctas = (a.P + kWarps - 1) / kWarps, most = 1 << 24;
        return launch_pdl_clusters(preference_kernel<32>, (int)(ctas < most ? ctas : most), kThreads,
                                   1, 0, st, a);
    }
    int c = 1;
    while (c < kMaxCluster && mean > c * 2048ll) c *= 2;
    const int64_t most = (1 << 24) / c;
    return launch_pdl_clusters(preference_kernel<kThreads>, (int)(a.P < most ? a.P : most) * c,
                               kThreads, c, 0, st, a);
}

}  // namespace agoq
