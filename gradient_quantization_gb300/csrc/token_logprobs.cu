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
#include <cooperative_groups.h>

#include "agoq_launch.h"
#include "typed_io.cuh"

namespace agoq {
namespace {

namespace cg = cooperative_groups;

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

// Rows too long for a cluster's shared memory: a CTA a row, every pass reading
// the logits again, the alternatives one by one.
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

// ---- rows held on chip ----------------------------------------------------------
//
// A cluster of C CTAs takes a row; each CTA copies its slice of the row into
// shared memory once and makes every pass over it there: the maximum, the sums
// and the candidates for the alternatives, and the gradient.  The slices are cut
// at the 16-byte boundaries of memory, so a row may start anywhere; the up to two
// vectors that the row fills only in part are padded with -inf.  CTAs work with
// their slice's maximum; the C maxima and sums meet once, through distributed
// shared memory.
//
// Alternatives: a slice's vectors fall into 64 groups by the thread that holds
// them.  The k-th largest of the groups' maxima is a bound that at least k
// elements reach and, when large logits are not all in few groups, few others: about
// 1.2 k for k = 20.  The elements above it and those equal to it are collected in
// two lists and ranked by counting.  Too many equal ones (masks, constant rows):
// the first of them are found in order.  Too many above it, or NaN: the k largest
// are found one by one.
constexpr int kRowThreads = 512, kRowWarps = kRowThreads / 32;
constexpr int kGroups = 64, kGroupLanes = kRowThreads / kGroups;
constexpr int kTopMax = 32;
constexpr int kList = 256;                    // entries of a candidate list
constexpr int kMaxCluster = 8;
constexpr int kSliceBytes = 70 * 1024;        // three CTAs an SM
constexpr int kMaxSliceBytes = 212 * 1024;    // one CTA an SM
static_assert(kTopMax <= kGroups && kMaxCluster * kTopMax <= kList, "lists hold what they must");

struct RowShared {
    float red[2][kRowWarps];
    float groups[kGroups];
    float bound;                  // the k-th largest of the groups' maxima
    int above, equal;             // entries of the lists (may exceed kList)
    float max, sum, first;        // of the slice: m, sum e^(x-m), sum (x-m) e^(x-m)
    float token;                  // the token's logit, in the CTA that holds it
    float all[3];                 // of the row: m, sum, first
    unsigned long long best;
    unsigned long long top[kTopMax];
    unsigned long long list[2][kList];
};

__device__ __forceinline__ float exp2_approx(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float exp_approx(float x) { return exp2_approx(__fmul_rn(x, kLog2e)); }

__device__ __forceinline__ void copy16(uint32_t to, const void *from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
template <int N>
__device__ __forceinline__ void copies_left() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ float key_value(uint64_t key) {
    const uint32_t k = (uint32_t)(key >> 32);
    return __uint_as_float((k & 0x80000000u) ? k & 0x7FFFFFFFu : ~k);
}
__device__ __forceinline__ uint32_t key_index(uint64_t key) { return 0xFFFFFFFFu - (uint32_t)key; }

// A row's slice in this CTA, as vectors of kVec elements: vector j of the slice is
// at byte 16 j of shared memory and holds the row's elements at(j) ...
template <int DT>
struct Slice {
    using E = Elem<DT>;
    const uint4 *data;
    int n;                        // vectors
    int64_t start;                // element of the first vector's first lane (may be negative)
    int64_t V;
    __device__ __forceinline__ int64_t at(int j) const { return start + (int64_t)j * E::kVec; }
    __device__ __forceinline__ bool whole(int j) const { return at(j) >= 0 && at(j) + E::kVec <= V; }
};

// The k largest keys of the slice that `keep` accepts, one by one.
template <int DT>
__device__ __noinline__ void top_one_by_one(const Slice<DT> s, int k, RowShared &sh) {
    uint64_t last = ~0ull;
    for (int j = 0; j < k; ++j) {
        uint64_t b = 0;
        for (int v = threadIdx.x; v < s.n; v += kRowThreads) {
            float f[Elem<DT>::kVec];
            Elem<DT>::unpack(s.data[v], f);
#pragma unroll
            for (int i = 0; i < Elem<DT>::kVec; ++i) {
                const int64_t e = s.at(v) + i;
                if (e < 0 || e >= s.V) continue;
                const uint64_t key = order_key(f[i], (uint32_t)e);
                if (key < last && key > b) b = key;
            }
        }
        if (threadIdx.x == 0) sh.best = 0;
        __syncthreads();
        atomicMax(&sh.best, (unsigned long long)b);
        __syncthreads();
        last = sh.best;
        if (threadIdx.x == 0) sh.top[j] = last;
        __syncthreads();
        if (last == 0) break;     // fewer than k elements: the rest of top stays 0
    }
}

// The first `want` elements equal to the bound, in order, by one warp.
template <int DT>
__device__ __noinline__ void first_equal(const Slice<DT> s, int want, RowShared &sh) {
    const int lane = threadIdx.x & 31;
    int found = 0;
    for (int v0 = 0; v0 < s.n && found < want; v0 += 32) {
        const int v = v0 + lane;
        uint32_t hits = 0;
        float f[Elem<DT>::kVec];
        if (v < s.n) {
            Elem<DT>::unpack(s.data[v], f);
#pragma unroll
            for (int i = 0; i < Elem<DT>::kVec; ++i) {
                const int64_t e = s.at(v) + i;
                if (e >= 0 && e < s.V && f[i] == sh.bound) hits |= 1u << i;
            }
        }
        int before = __popc(hits);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xFFFFFFFFu, before, o);
            if (lane >= o) before += up;
        }
        const int total = __shfl_sync(0xFFFFFFFFu, before, 31);
        int at = found + before - __popc(hits);
#pragma unroll
        for (int i = 0; i < Elem<DT>::kVec; ++i) {
            if ((hits >> i) & 1u) {
                if (at < want) sh.list[1][at] = order_key(sh.bound, (uint32_t)(s.at(v) + i));
                ++at;
            }
        }
        found += total;
    }
}

// Place the k largest of n + m keys (two lists) into top, by counting.
__device__ __forceinline__ void rank_keys(const unsigned long long *a, int n,
                                          const unsigned long long *b, int m, int k,
                                          unsigned long long *top) {
    for (int i = threadIdx.x; i < n + m; i += kRowThreads) {
        const uint64_t key = i < n ? a[i] : b[i - n];
        int rank = 0;
        for (int j = 0; j < n; ++j) rank += a[j] > key;
        for (int j = 0; j < m; ++j) rank += b[j] > key;
        if (rank < k) top[rank] = key;
    }
}

// Gradient of the loss for eight (four) logits: w e^(x - m) / S.
template <int DT>
__device__ __forceinline__ void loss_grad(const uint4 &v, float m, float scale, float *g) {
    constexpr int N = Elem<DT>::kVec;
    float f[N];
    Elem<DT>::unpack(v, f);
    const uint64_t m2 = f32x2(m, m), l2 = f32x2(kLog2e, kLog2e), s2 = f32x2(scale, scale);
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        const uint64_t t = mul_f32x2(sub_f32x2(f32x2(f[i], f[i + 1]), m2), l2);
        const uint64_t p = mul_f32x2(f32x2(exp2_approx(lo_f32(t)), exp2_approx(hi_f32(t))), s2);
        g[i] = lo_f32(p);
        g[i + 1] = hi_f32(p);
    }
}

// LOSS: logp and the gradient; else logp, entropy, lse and the alternatives.
template <int DT, bool LOSS>
__global__ void __launch_bounds__(kRowThreads) token_rows_kernel(const TokenLogprobs a) {
    using E = Elem<DT>;
    constexpr int N = E::kVec;
    extern __shared__ __align__(16) uint4 slice[];
    __shared__ RowShared sh;
    cg::cluster_group cluster = cg::this_cluster();
    const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t base = static_cast<uint32_t>(__cvta_generic_to_shared(slice));
    pdl_wait_and_release();
    for (int64_t t = blockIdx.x / C; t < a.T; t += gridDim.x / C) {
        const char *row = elem_at<DT>(a.logits, t * a.ld);
        const int skip = (int)(reinterpret_cast<uintptr_t>(row) & 15u) / E::kSize;
        const int64_t vectors = (a.V + skip + N - 1) / N, per = (vectors + C - 1) / C;
        const int64_t v0 = rank * per, left = vectors - v0;
        const int64_t token = a.tokens[t];
        Slice<DT> s;
        s.data = slice;
        s.n = (int)(left < 0 ? 0 : left < per ? left : per);
        s.start = v0 * N - skip;
        s.V = a.V;
        const int steps = (int)((per + kRowThreads - 1) / kRowThreads);
        // in four groups of copies, so that the maximum starts with the first
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            for (int i = steps * q / 4; i < steps * (q + 1) / 4; ++i) {
                const int j = i * kRowThreads + threadIdx.x;
                if (j >= s.n) break;
                if (s.whole(j)) {
                    copy16(base + 16u * j, elem_at<DT>(row, s.at(j)));
                } else {
                    typename E::Word *to = reinterpret_cast<typename E::Word *>(slice + j);
                    const typename E::Word *from =
                        reinterpret_cast<const typename E::Word *>(row);
                    slice[j] = make_uint4(kNegInfWord<DT>, kNegInfWord<DT>, kNegInfWord<DT>,
                                          kNegInfWord<DT>);
#pragma unroll
                    for (int k = 0; k < N; ++k)
                        if (s.at(j) + k >= 0 && s.at(j) + k < a.V) to[k] = from[s.at(j) + k];
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
        uint32_t top = kNegInfWord<DT>;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if (q == 0) copies_left<3>();
            if (q == 1) copies_left<2>();
            if (q == 2) copies_left<1>();
            if (q == 3) copies_left<0>();
            for (int i = steps * q / 4; i < steps * (q + 1) / 4; ++i) {
                const int j = i * kRowThreads + threadIdx.x;
                if (j >= s.n) break;
                const uint4 v = slice[j];
                top = max_word<DT>(top, max_word<DT>(max_word<DT>(v.x, v.y),
                                                     max_word<DT>(v.z, v.w)));
            }
        }
        float m = word_max<DT>(top);
#pragma unroll
        for (int o = 1; o < kGroupLanes; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        if (threadIdx.x % kGroupLanes == 0) sh.groups[threadIdx.x / kGroupLanes] = m;
        m = warp_max(m);
        if (lane == 0) sh.red[0][warp] = m;
        __syncthreads();
        m = sh.red[0][0];
#pragma unroll
        for (int i = 1; i < kRowWarps; ++i) m = fmaxf(m, sh.red[0][i]);
        const float slice_max = m;
        if (m == -INFINITY) m = 0.0f;
        const int want = (int)(a.k < a.V ? a.k : a.V);
        bool collect = false;
        float bound = 0.0f;
        if constexpr (!LOSS) {
            collect = want > 0;
            if (collect) {
                if (threadIdx.x < kGroups) {
                    const float g = sh.groups[threadIdx.x];
                    int larger = 0;
                    for (int i = 0; i < kGroups; ++i) {
                        const float o = sh.groups[i];
                        larger += o > g || (o == g && i < (int)threadIdx.x);
                    }
                    if (larger == want - 1) sh.bound = g;
                }
                if (threadIdx.x < kTopMax) sh.top[threadIdx.x] = 0;
                if (threadIdx.x == 0) sh.above = sh.equal = 0;
                __syncthreads();
                bound = sh.bound;
            }
        }
        // the token's logit
        if (threadIdx.x == 0 && token >= 0 && token < a.V) {
            const int64_t e = token - s.start;
            if (e >= 0 && e < (int64_t)s.n * N)
                sh.token = E::up(reinterpret_cast<const typename E::Word *>(slice)[e]);
        }
        uint64_t sum2 = 0, first2 = 0;
        const uint64_t m2 = f32x2(m, m), l2 = f32x2(kLog2e, kLog2e);
        for (int j = threadIdx.x; j < s.n; j += kRowThreads) {
            const uint4 v = slice[j];
            float f[N];
            E::unpack(v, f);
#pragma unroll
            for (int i = 0; i < N; i += 2) {
                uint64_t d = sub_f32x2(f32x2(f[i], f[i + 1]), m2);
                if constexpr (!LOSS) {
                    // not below -1000, so that (x - m) e^(x - m) is 0 for x = -inf
                    float lo = lo_f32(d), hi = hi_f32(d);
                    asm("max.NaN.f32 %0, %0, %1;" : "+f"(lo) : "f"(-1000.0f));
                    asm("max.NaN.f32 %0, %0, %1;" : "+f"(hi) : "f"(-1000.0f));
                    d = f32x2(lo, hi);
                }
                const uint64_t x = mul_f32x2(d, l2);
                const uint64_t e = f32x2(exp2_approx(lo_f32(x)), exp2_approx(hi_f32(x)));
                sum2 = add_f32x2(sum2, e);
                if constexpr (!LOSS) first2 = fma_f32x2(d, e, first2);
            }
            if (collect) {
                const float most = word_max<DT>(max_word<DT>(max_word<DT>(v.x, v.y),
                                                             max_word<DT>(v.z, v.w)));
                if (most >= bound) {
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        const int64_t e = s.at(j) + i;
                        if (!(f[i] >= bound) || e < 0 || e >= a.V) continue;
                        const int which = f[i] > bound ? 0 : 1;
                        const int at = atomicAdd(which ? &sh.equal : &sh.above, 1);
                        if (at < kList) sh.list[which][at] = order_key(f[i], (uint32_t)e);
                    }
                }
            }
        }
        float sum = warp_sum(__fadd_rn(lo_f32(sum2), hi_f32(sum2)));
        float first = LOSS ? 0.0f : warp_sum(__fadd_rn(lo_f32(first2), hi_f32(first2)));
        __syncthreads();   // red has been read
        if (lane == 0) {
            sh.red[0][warp] = sum;
            sh.red[1][warp] = first;
        }
        __syncthreads();
        sum = first = 0.0f;
#pragma unroll
        for (int i = 0; i < kRowWarps; ++i) {
            sum = __fadd_rn(sum, sh.red[0][i]);
            first = __fadd_rn(first, sh.red[1][i]);
        }
        if (threadIdx.x == 0) {
            sh.max = slice_max;
            sh.sum = sum;
            sh.first = first;
        }
        if constexpr (!LOSS) {
            if (collect) {
                const int above = sh.above, equal = sh.equal;
                if (above > kList || sum != sum) {
                    top_one_by_one<DT>(s, want, sh);
                } else {
                    int ties = above >= want ? 0 : equal;
                    if (ties > kList) {
                        ties = want - above;
                        if (warp == 0) first_equal<DT>(s, ties, sh);
                        __syncthreads();
                    }
                    rank_keys(sh.list[0], above, sh.list[1], ties, want, sh.top);
                }
            }
        }
        if (C > 1) cluster.sync();
        else __syncthreads();
        // the row's maximum and sums
        if (warp == 0) {
            float mc = -INFINITY, sc = 0.0f, fc = 0.0f;
            if (lane < C) {
                const RowShared *o = cluster.map_shared_rank(&sh, lane);
                mc = o->max;
                sc = o->sum;
                fc = o->first;
            }
            const float mr = warp_max(mc), ref = mr == -INFINITY ? 0.0f : mr;
            const float d = __fsub_rn(mc, ref), f = lane < C ? exp_approx(d) : 0.0f;
            // a slice that counts for nothing may have d = -inf
            const bool none = f == 0.0f && sc == sc;
            const float rs = warp_sum(none ? 0.0f : __fmul_rn(f, sc));
            const float rf = warp_sum(none ? 0.0f : __fmul_rn(f, __fmaf_rn(d, sc, fc)));
            if (lane == 0) {
                sh.all[0] = ref;
                sh.all[1] = rs;
                sh.all[2] = rf;
            }
        }
        __syncthreads();
        const float rm = sh.all[0], rs = sh.all[1], rf = sh.all[2];
        const float ls = logf(rs);
        const bool ignored = token < 0, beyond = token >= a.V, empty = rs == 0.0f;
        if (rank == 0) {
            if (threadIdx.x == 0) {
                float lp = 0.0f;
                if (beyond) lp = NAN;
                else if (!ignored) {
                    const float x = cluster.map_shared_rank(&sh, (int)((token + skip) / N / per))->token;
                    lp = x == -INFINITY ? x : __fsub_rn(__fsub_rn(x, rm), ls);
                }
                if (a.logp) a.logp[t] = lp;
                if (!LOSS && a.entropy)
                    a.entropy[t] = empty ? 0.0f : __fsub_rn(ls, __fdiv_rn(rf, rs));
                if (!LOSS && a.lse) a.lse[t] = __fadd_rn(rm, ls);
            }
            if constexpr (!LOSS) {
                if (collect && C > 1) {
                    // the slices' alternatives: those that reach every slice's k-th
                    const int i = threadIdx.x;
                    uint64_t key = 0, least = 0;
                    if (i < C * want) key = cluster.map_shared_rank(&sh, i / want)->top[i % want];
                    for (int c = 0; c < C; ++c) {
                        const uint64_t o = cluster.map_shared_rank(&sh, c)->top[want - 1];
                        least = o > least ? o : least;
                    }
                    if (threadIdx.x == 0) sh.above = 0;
                    __syncthreads();
                    if (key != 0 && key >= least) sh.list[0][atomicAdd(&sh.above, 1)] = key;
                    __syncthreads();
                    rank_keys(sh.list[0], sh.above, nullptr, 0, want, sh.top);
                    __syncthreads();
                }
                if (threadIdx.x < want) {
                    const uint64_t key = sh.top[threadIdx.x];
                    const float x = key_value(key);
                    a.top_ids[t * want + threadIdx.x] = key_index(key);
                    a.top_logp[t * want + threadIdx.x] =
                        x == -INFINITY ? x : __fsub_rn(__fsub_rn(x, rm), ls);
                }
            }
        }
        if constexpr (LOSS) {
            float w = a.weights ? a.weights[t] : 1.0f;
            if (ignored || empty) w = 0.0f;
            if (beyond) w = NAN;
            const float scale = __fdiv_rn(w, rs);
            // Vectors of the output row: its 16-byte boundaries may lie elsewhere.
            char *out = elem_at<DT>(a.dlogits, t * a.ldd);
            const int oskip = (int)(reinterpret_cast<uintptr_t>(out) & 15u) / E::kSize;
            const int64_t e0 = s.start < 0 ? 0 : s.start;
            const int64_t stop = s.start + (int64_t)s.n * N, e1 = stop < a.V ? stop : a.V;
            const int64_t o0 = (e0 + oskip) / N;
            const int no = e1 > e0 ? (int)((e1 + oskip + N - 1) / N - o0) : 0;
            const typename E::Word *words = reinterpret_cast<const typename E::Word *>(slice);
            for (int j = threadIdx.x; j < no; j += kRowThreads) {
                const int64_t e = (o0 + j) * N - oskip;
                if (e >= e0 && e + N <= e1) {
                    const int at = (int)(e - s.start), sh_bytes = at % N * E::kSize;
                    uint4 v = slice[at / N];
                    if (sh_bytes) v = bytes_from(v, slice[at / N + 1], sh_bytes);
                    float g[N];
                    loss_grad<DT>(v, rm, scale, g);
                    if (w == 0.0f) {
#pragma unroll
                        for (int i = 0; i < N; ++i) g[i] = 0.0f;
                    }
                    if (token >= e && token < e + N) {
#pragma unroll
                        for (int i = 0; i < N; ++i)
                            if (token == e + i) g[i] = __fsub_rn(g[i], w);
                    }
                    *reinterpret_cast<uint4 *>(elem_at<DT>(out, e)) = E::pack(g);
                } else {
                    for (int i = 0; i < N; ++i) {
                        if (e + i < e0 || e + i >= e1) continue;
                        const float x = E::up(words[e + i - s.start]);
                        float g = 0.0f;
                        if (w != 0.0f) g = __fmul_rn(exp_approx(__fsub_rn(x, rm)), scale);
                        if (token == e + i) g = __fsub_rn(g, w);
                        store_elem<DT>(out, e + i, g);
                    }
                }
            }
        }
        if (C > 1) cluster.sync();     // the others have read this CTA's shared memory
        else __syncthreads();
    }
}

// The CTAs of a row's cluster: slices of at most kSliceBytes where eight CTAs
// allow it (three CTAs an SM, whose copies and passes overlap), and more CTAs a
// row while the rows alone do not fill two CTAs an SM, down to 4 KB.  0: the row
// does not fit on chip.
int row_cluster(int64_t T, int64_t V, int size) {
    const int64_t bytes = V * size + 16;
    int c = 1;
    while (c < kMaxCluster && bytes > c * (int64_t)kSliceBytes) c *= 2;
    if (bytes > c * (int64_t)kMaxSliceBytes) return 0;
    while (c < kMaxCluster && T * c < 2 * sm_count() && bytes > c * 8192ll) c *= 2;
    return c;
}

template <int DT, bool LOSS>
cudaError_t launch_rows(const TokenLogprobs &a, int c, cudaStream_t st) {
    static bool ready[kMaxDevices];
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= kMaxDevices) dev = 0;
    auto kernel = token_rows_kernel<DT, LOSS>;
    if (!ready[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(
            kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSliceBytes + 32);
        if (e != cudaSuccess) return e;
        ready[dev] = true;
    }
    // a row that starts inside a vector has one vector more
    const int64_t vectors = (a.V + 2 * Elem<DT>::kVec - 2) / Elem<DT>::kVec;
    const size_t smem = (size_t)((vectors + c - 1) / c) * 16;
    const int64_t rows = a.T < (1 << 24) ? a.T : 1 << 24;
    return launch_pdl_clusters(kernel, (int)(rows * c), kRowThreads, c, smem, st, a);
}

template <bool LOSS>
cudaError_t rows_of_type(const TokenLogprobs &a, int c, cudaStream_t st) {
    return a.dtype == kF32    ? launch_rows<kF32, LOSS>(a, c, st)
           : a.dtype == kBF16 ? launch_rows<kBF16, LOSS>(a, c, st)
                              : launch_rows<kF16, LOSS>(a, c, st);
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
    const int c = row_cluster(a.T, a.V, a.dtype == kF32 ? 4 : 2);
    if (c) return a.dlogits ? rows_of_type<true>(a, c, st) : rows_of_type<false>(a, c, st);
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
