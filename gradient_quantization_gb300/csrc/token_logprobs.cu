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

// x - m, not below -1000 (where its exponential is 0 too): for x = -inf its product
// with the exponential must be 0.  NaN stays NaN.
__device__ __forceinline__ float below_max(float x, float m) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(__fsub_rn(x, m)), "f"(-1000.0f));
    return d;
}

// Log probability of a logit x, from the row's reference, its sum and the sum's logarithm.
// (x = -inf in a row of nothing else would be a difference of infinities; in a row whose
// statistics are NaN it is NaN like every other.)
__device__ __forceinline__ float log_prob(float x, float ref, float sum, float ln) {
    return x == -INFINITY && sum == sum ? x : __fsub_rn(__fsub_rn(x, ref), ln);
}

// The loss of rows too long for a cluster's shared memory: a CTA a row, every pass
// reading the logits again.
template <int DT>
__global__ void __launch_bounds__(kThreads) token_loss_long_kernel(const TokenLogprobs a) {
    pdl_wait_and_release();
    __shared__ float red[2][kWarps];
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        const char *row = elem_at<DT>(a.logits, t * a.ld);
        const int64_t token = a.tokens[t];
        const float at = token >= 0 && token < a.V ? load_now<DT>(row, token) : 0.0f;
        float m = -INFINITY;
        for (int64_t i = threadIdx.x; i < a.V; i += kThreads) m = fmaxf(m, load_now<DT>(row, i));
        m = cta_max(m, red[0]);
        if (m == -INFINITY) m = 0.0f;
        float s = 0.0f;
        for (int64_t i = threadIdx.x; i < a.V; i += kThreads)
            s = __fadd_rn(s, expf(__fsub_rn(load_now<DT>(row, i), m)));
        s = cta_sum<kWarps>(s, red[1]);
        const bool ignored = token < 0, beyond = token >= a.V, empty = s == 0.0f;
        if (threadIdx.x == 0 && a.logp) {
            const float lp = log_prob(at, m, s, logf(s));
            a.logp[t] = ignored ? 0.0f : beyond ? NAN : lp;
        }
        float w = a.weights ? a.weights[t] : 1.0f;
        if (beyond || s != s) w = NAN;                // 0 times a row of NaN is NaN too
        if (ignored || (empty && !beyond)) w = 0.0f;
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
        __syncthreads();
    }
}

// ---- one pass over a row --------------------------------------------------------
//
// A thread adds e^(x - ref) and (x - ref) e^(x - ref) with a reference of its own:
// a vector whose largest element exceeds it by more than 8 raises it (rare after
// the first vectors), so there is no pass for the maximum, and the exponentials of
// the largest elements stay below e^8.  References and sums of the threads, warps and
// CTAs of a row are joined at its end.

// (0 where the result would be below 2^-126.)
__device__ __forceinline__ float exp2_approx(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float exp_approx(float x) { return exp2_approx(__fmul_rn(x, kLog2e)); }

constexpr float kLowest = -3.402823466e38f;   // reference of a thread that has seen nothing

// x moved from reference `from` to `to` >= from: the factor of the sums.  A factor
// of 0 keeps NaN sums and makes all others 0.
struct Sums {
    float ref, sum, first;
    __device__ __forceinline__ void move(float to) {
        const float d = __fsub_rn(ref, to), f = exp_approx(d);
        first = __fmul_rn(f, f == 0.0f ? first : __fmaf_rn(d, sum, first));
        sum = __fmul_rn(f, sum);
        ref = to;
    }
};

// The sums of a warp's lanes (every lane gets them).
__device__ __forceinline__ Sums warp_join(Sums s) {
    s.move(warp_max(s.ref));
    s.sum = warp_sum(s.sum);
    s.first = warp_sum(s.first);
    return s;
}

template <int DT>
__device__ __forceinline__ uint32_t vec_max(const uint4 &v) {
    return max_word<DT>(max_word<DT>(v.x, v.y), max_word<DT>(v.z, v.w));
}

// ENTROPY: with the sums of (x - ref) e^(x - ref).
template <int DT, bool ENTROPY>
struct Online {
    float ref = kLowest, limit = kLowest;      // limit = ref + 8
    uint64_t sum2 = 0, first2 = 0;
    // The sums of (x - ref) e^(x - ref) must not see x = -inf.  Where the exponential
    // is 0 anyway, 16-bit types raise x to `low` two at a time: -1000 below a
    // positive reference, the lowest finite value below one in (kLowRef, 0], which is
    // still more than 500 above it.  Below kLowRef values are so far apart that
    // every product is 0 (or, of FP16, less than 1e-12), and none is added.
    uint32_t low = kNegInfWord<DT>;
    static constexpr float kLowRef = DT == kF16 ? -65000.0f : -1e38f;

    __device__ __forceinline__ void raise(float to) {
        Sums s = sums();
        s.move(to);
        ref = to;
        limit = __fadd_rn(to, 8.0f);
        sum2 = f32x2(s.sum, 0.0f);
        first2 = f32x2(s.first, 0.0f);
        if constexpr (ENTROPY && DT == kBF16)
            low = to > 0.0f ? 0xC47AC47Au : to > kLowRef ? 0xFF7FFF7Fu : kNegInfWord<DT>;
        if constexpr (ENTROPY && DT == kF16)
            low = to > 0.0f ? 0xE3D0E3D0u : to > kLowRef ? 0xFBFFFBFFu : kNegInfWord<DT>;
    }

    // Add a vector whose largest element is at most `most`.
    __device__ __forceinline__ void add(const uint4 &v, float most) {
        if (most > limit) raise(most);
        add(v);
    }
    // Add a vector whose elements do not exceed the limit.
    __device__ __forceinline__ void add(uint4 v) {
        constexpr int N = Elem<DT>::kVec;
        if constexpr (ENTROPY && DT != kF32) {
            v.x = raised(v.x);
            v.y = raised(v.y);
            v.z = raised(v.z);
            v.w = raised(v.w);
        }
        const bool products = ENTROPY && (DT == kF32 || ref > kLowRef);
        const uint64_t l2 = f32x2(kLog2e, kLog2e);
        uint64_t d[N / 2];
        differences<DT>(v, ref, d);
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            if constexpr (ENTROPY && DT == kF32) {
                float lo = lo_f32(d[i]), hi = hi_f32(d[i]);
                asm("max.NaN.f32 %0, %0, %1;" : "+f"(lo) : "f"(-1000.0f));
                asm("max.NaN.f32 %0, %0, %1;" : "+f"(hi) : "f"(-1000.0f));
                d[i] = f32x2(lo, hi);
            }
            const uint64_t x = mul_f32x2(d[i], l2);
            const uint64_t e = f32x2(exp2_approx(lo_f32(x)), exp2_approx(hi_f32(x)));
            sum2 = add_f32x2(sum2, e);
            if (products) first2 = fma_f32x2(d[i], e, first2);
        }
    }

    __device__ __forceinline__ uint32_t raised(uint32_t w) const {
        uint32_t r;
        if constexpr (DT == kBF16) asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(w), "r"(low));
        else asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(w), "r"(low));
        return r;
    }

    __device__ __forceinline__ Sums sums() const {
        return {ref, __fadd_rn(lo_f32(sum2), hi_f32(sum2)),
                __fadd_rn(lo_f32(first2), hi_f32(first2))};
    }
};

// The vector of a row of V elements from element e on, -inf where there is none.
template <int DT>
__device__ __noinline__ uint4 partial(const typename Elem<DT>::Word *row, int V, int e) {
    typename Elem<DT>::Word w[Elem<DT>::kVec];
#pragma unroll
    for (int i = 0; i < Elem<DT>::kVec; ++i) {
        w[i] = Elem<DT>::down(-INFINITY);
        if (e + i >= 0 && e + i < V) w[i] = row[e + i];
    }
    uint4 v;
    __builtin_memcpy(&v, w, 16);
    return v;
}

// A CTA's slice of a row, cut at the 16-byte boundaries of memory: n vectors, of
// which the row's first and last may be filled in part only; those in [from, to) are
// whole.  (Elements are counted in 32 bits: a row has at most 2^30.)
template <int DT>
struct Slice {
    using E = Elem<DT>;
    const typename E::Word *row;
    const uint4 *vec;             // vector 0, 16-byte aligned (maybe before the row's start)
    int V, start;                 // start: element of vector 0's first lane (may be negative)
    int n, from, to;
    __device__ __forceinline__ Slice(const char *row_, int V_, int C, int rank)
        : row(reinterpret_cast<const typename E::Word *>(row_)), V(V_) {
        const int skip = (int)(reinterpret_cast<uintptr_t>(row_) & 15u) / E::kSize;
        const int vectors = (V + skip + E::kVec - 1) / E::kVec;
        const int per = C > 1 ? (vectors + C - 1) / C : vectors, left = vectors - rank * per;
        n = left < 0 ? 0 : left < per ? left : per;
        start = rank * per * E::kVec - skip;
        vec = reinterpret_cast<const uint4 *>(row_ + (int64_t)start * E::kSize);
        from = start < 0 && n > 0 ? 1 : 0;
        to = n > from && at(n) > V ? n - 1 : n;
    }
    __device__ __forceinline__ int at(int j) const { return start + j * E::kVec; }
    __device__ __forceinline__ int first() const { return start < 0 ? 0 : start; }
    __device__ __forceinline__ int end() const { return at(n) < V ? at(n) : V; }
    __device__ __forceinline__ bool has(int64_t e) const { return e >= first() && e < end(); }
    // Vector j with -inf where the row has no element.
    __device__ __forceinline__ uint4 part(int j) const { return partial<DT>(row, V, at(j)); }
    __device__ __forceinline__ uint4 load(int j) const {
        uint4 v;
        asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                     : "l"(vec + j));
        return v;
    }
    __device__ __forceinline__ uint4 any(int j) const {
        return j >= from && j < to ? load(j) : part(j);
    }
};

// ---- statistics and alternatives ------------------------------------------------
//
// A CTA (for few rows: a cluster, each CTA a slice) streams its rows once, through a
// ring of shared memory whose copies run ahead of the sums and across rows; a
// thread reads only what it copied, so the ring needs no barrier.
//
// Alternatives: a row's vectors fall into 64 groups by the threads that hold them.
// The k-th largest of the groups' maxima is a bound that at least k elements reach
// and, unless the large logits sit in few groups, few others (about 1.2 k for k = 20).
// The bounds of the first batch, of the first 4, 16, ... let the pass collect
// candidate vectors as it goes; the bound of the whole row selects their elements,
// and counting ranks what is left.  Where that fails (more candidates than the list
// holds, as in ascending rows; fewer than k finite logits; NaN) the slice is read
// again: elements above the bound and equal to it in two lists, of the equal ones the
// first in order; and where even the former are too many, the k largest one by one, a
// reading each (2048 x 128000 BF16, k = 20: all rows ascending, or finite in every eighth
// vector only, or with a NaN 6 to 7 ms; all equal 0.48 ms).
//
// 2048 x 128000 BF16 with 20 alternatives: 108 us (4.9 TB/s), without them 91 us.  Bound by
// instruction issue (71%: the exponential, its two sums and the maximum of each element)
// and by the last round, since 2048 rows on 912 CTAs are 2.25 rounds.  128 threads and six
// CTAs an SM, so that one CTA's end of a row hides behind another's stream (8208 x 32000
// 155 us, with 256 threads and three 190 us, before the bound was found by bits; now 144).
constexpr int kStatThreads = 128, kStatWarps = kStatThreads / 32;
constexpr int kBatch = 4;                     // vectors a thread and stage
constexpr int kStages = 3;                    // of shared memory, each thread's own
constexpr int kStep = kBatch * kStatThreads;
constexpr int kGroups = 64, kGroupLanes = kStatThreads / kGroups;
constexpr int kTopMax = 32;
constexpr int kWarpList = 128;                // candidate vectors of a warp
constexpr int kList = kWarpList * kStatWarps, kShortList = 256;
constexpr int kMaxCluster = 8;
static_assert(kTopMax <= kGroups && kGroups == 64 && kMaxCluster * kTopMax <= kShortList && 3 * kShortList <= 2 * kList,
              "lists hold what they must");

struct StatShared {
    uint32_t groups[kGroups];     // ordered() of the largest element of each; 16-byte aligned
    Sums warps[kStatWarps];
    Sums slice;                   // of the CTA's slice
    float bound;
    float token;                  // the token's logit, in the CTA that holds it
    int found[kStatWarps];        // candidate vectors (may exceed kWarpList)
    int count;                    // entries of a list
    int above, equal;             // entries of the shorter lists
    unsigned long long best;
    unsigned long long top[kTopMax];
    // Candidate vectors, by warp, and their first elements' indices; later lists of keys.
    union {
        uint4 vec[kStatWarps][kWarpList];
        unsigned long long list[2 * kList];
    };
    int element[kStatWarps][kWarpList];
    unsigned long long few[kShortList];
    uint4 ring[kStages][kBatch][kStatThreads];
};

__device__ __forceinline__ uint32_t key_index(uint64_t key) { return 0xFFFFFFFFu - (uint32_t)key; }

// A float's place in the order of its values, and back.
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t b = __float_as_uint(x);
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float from_ordered(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? k & 0x7FFFFFFFu : ~k);
}

// sh.bound: the want-th largest maximum of the groups, whose threads hold `most`.  Of the
// 16-bit types, whose values as binary32 differ in the upper 16 (BF16) or 19 bits only, one
// warp finds it bit by bit, each time counting the maxima that reach the bits so far; of
// FP32 a thread a group counts the larger ones.  (2048 x 128000 BF16 108 us, counting 113
// us; 8208 x 32000 144 us, 155 us; 2048 x 64000 FP32 106 us, counting 101 us.)
template <int DT>
__device__ __forceinline__ void find_bound(float most, int want, StatShared &sh) {
#pragma unroll
    for (int o = 1; o < kGroupLanes; o <<= 1)
        most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
    if (threadIdx.x % kGroupLanes == 0) sh.groups[threadIdx.x / kGroupLanes] = ordered(most);
    __syncthreads();
    if constexpr (DT == kF32) {
        if (threadIdx.x < kGroups) {
            const uint32_t g = sh.groups[threadIdx.x];
            int larger = 0;
#pragma unroll
            for (int i = 0; i < kGroups; i += 4) {
                const uint4 o = *reinterpret_cast<const uint4 *>(sh.groups + i);
                const int me = threadIdx.x;
                larger += (o.x > g || (o.x == g && i < me)) + (o.y > g || (o.y == g && i + 1 < me)) +
                          (o.z > g || (o.z == g && i + 2 < me)) + (o.w > g || (o.w == g && i + 3 < me));
            }
            if (larger == want - 1) sh.bound = from_ordered(g);
        }
    } else if (threadIdx.x < 32) {
        constexpr int kLow = DT == kBF16 ? 16 : 13;
        const uint32_t a = sh.groups[threadIdx.x], b = sh.groups[threadIdx.x + 32];
        uint32_t key = 0;
#pragma unroll
        for (int bit = 31; bit >= kLow; --bit) {
            const uint32_t next = key | 1u << bit;
            const int reach = __popc(__ballot_sync(0xFFFFFFFFu, a >= next)) +
                              __popc(__ballot_sync(0xFFFFFFFFu, b >= next));
            if (reach >= want) key = next;
        }
        if (!(key & 0x80000000u)) key |= (1u << kLow) - 1u;
        if (threadIdx.x == 0) sh.bound = from_ordered(key);
    }
    __syncthreads();
}

// Place the k largest of n keys into top, by counting.
__device__ __forceinline__ void rank_keys(const unsigned long long *keys, int n, int k,
                                          unsigned long long *top) {
    for (int i = threadIdx.x; i < n; i += kStatThreads) {
        const uint64_t key = keys[i];
        int rank = 0;
#pragma unroll 4
        for (int j = 0; j < n; ++j) rank += keys[j] > key;
        if (rank < k) top[rank] = key;
    }
}

// The k largest keys of the slice, one by one.
template <int DT>
__device__ __noinline__ void top_one_by_one(const Slice<DT> s, int k, StatShared &sh) {
    uint64_t last = ~0ull;
    for (int j = 0; j < k; ++j) {
        uint64_t b = 0;
        for (int v = threadIdx.x; v < s.n; v += kStatThreads) {
            float f[Elem<DT>::kVec];
            Elem<DT>::unpack(s.any(v), f);
#pragma unroll
            for (int i = 0; i < Elem<DT>::kVec; ++i) {
                if (!s.has(s.at(v) + i)) continue;
                const uint64_t key = order_key(f[i], (uint32_t)(s.at(v) + i));
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

// The first `want` elements equal to the bound, in order, by one warp, into `to`.
template <int DT>
__device__ __noinline__ void first_equal(const Slice<DT> s, int want, float bound,
                                         unsigned long long *to) {
    const int lane = threadIdx.x & 31;
    int found = 0;
    for (int v0 = 0; v0 < s.n && found < want; v0 += 32) {
        const int v = v0 + lane;
        uint32_t hits = 0;
        if (v < s.n) {
            float f[Elem<DT>::kVec];
            Elem<DT>::unpack(s.any(v), f);
#pragma unroll
            for (int i = 0; i < Elem<DT>::kVec; ++i)
                if (s.has(s.at(v) + i) && f[i] == bound) hits |= 1u << i;
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
                if (at < want) to[at] = order_key(bound, (uint32_t)(s.at(v) + i));
                ++at;
            }
        }
        found += total;
    }
}

// The alternatives from a second reading, with the bound of the whole slice.
template <int DT>
__device__ __noinline__ void read_again(const Slice<DT> s, int want, bool nan, StatShared &sh) {
    const float bound = sh.bound;
    unsigned long long *above = sh.list, *equal = sh.list + kShortList;
    __syncthreads();
    if (threadIdx.x == 0) sh.above = sh.equal = 0;
    if (nan) {
        top_one_by_one<DT>(s, want, sh);
        return;
    }
    __syncthreads();
    for (int v = threadIdx.x; v < s.n; v += kStatThreads) {
        float f[Elem<DT>::kVec];
        Elem<DT>::unpack(s.any(v), f);
#pragma unroll
        for (int i = 0; i < Elem<DT>::kVec; ++i) {
            if (!(f[i] >= bound) || !s.has(s.at(v) + i)) continue;
            const bool more = f[i] > bound;
            // equal ones are counted no further than it matters
            if (!more && *(volatile int *)&sh.equal > kShortList) continue;
            const int at = atomicAdd(more ? &sh.above : &sh.equal, 1);
            if (at < kShortList) (more ? above : equal)[at] = order_key(f[i], (uint32_t)(s.at(v) + i));
        }
    }
    __syncthreads();
    const int na = sh.above;
    int ne = sh.equal;
    if (na > kShortList) {
        top_one_by_one<DT>(s, want, sh);
        return;
    }
    if (na >= want) ne = 0;
    if (ne > kShortList) {
        ne = want - na;
        if (threadIdx.x < 32) first_equal<DT>(s, ne, bound, equal);
        __syncthreads();
    }
    // one list: all equal ones rank behind
    for (int i = threadIdx.x; i < ne; i += kStatThreads) sh.list[2 * kShortList + i] = equal[i];
    __syncthreads();
    for (int i = threadIdx.x; i < ne; i += kStatThreads) above[na + i] = sh.list[2 * kShortList + i];
    __syncthreads();
    rank_keys(above, na + ne, want, sh.top);
}

// The copies of a CTA's rows into the ring, ahead of the sums and across rows.
template <int DT>
struct Fetch {
    const TokenLogprobs &a;
    StatShared &sh;
    int C, rank, stage = 0;
    int64_t t;
    const uint4 *vec;             // of the row being fetched: its next vector for this thread
    int left;                     // vectors of the slice from that one on
    __device__ __forceinline__ Fetch(const TokenLogprobs &a_, StatShared &sh_, int64_t t_, int C_,
                                     int rank_)
        : a(a_), sh(sh_), C(C_), rank(rank_), t(t_) {
        row();
    }
    // Start row t, or the next one that has whole vectors.
    __device__ __forceinline__ void row() {
        left = 0;
        vec = nullptr;
        for (; t < a.T; t += gridDim.x / C) {
            const Slice<DT> s(elem_at<DT>(a.logits, t * a.ld), (int)a.V, C, rank);
            if (s.to <= s.from) continue;
            vec = s.vec + s.from + threadIdx.x;
            left = s.to - s.from;
            return;
        }
    }
    __device__ __forceinline__ void next() {
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            if ((int)threadIdx.x + i * kStatThreads < left)
                copy16(&sh.ring[stage][i][threadIdx.x], vec + i * kStatThreads);
        copies_commit();
        stage = stage + 1 == kStages ? 0 : stage + 1;
        vec += kStep;
        left -= kStep;
        if (left <= 0 && t < a.T) {
            t += gridDim.x / C;
            row();
        }
    }
};

template <int DT>
__global__ void __launch_bounds__(kStatThreads, 6) token_stats_kernel(const TokenLogprobs a) {
    constexpr int N = Elem<DT>::kVec;
    extern __shared__ __align__(16) uint8_t shared_bytes[];
    StatShared &sh = *reinterpret_cast<StatShared *>(shared_bytes);
    cg::cluster_group cluster = cg::this_cluster();
    const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int want = a.k;
    pdl_wait_and_release();
    Fetch<DT> fetch(a, sh, blockIdx.x / C, C, rank);
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch.next();
    int stage = 0;
    for (int64_t t = blockIdx.x / C; t < a.T; t += gridDim.x / C) {
        const Slice<DT> s(elem_at<DT>(a.logits, t * a.ld), (int)a.V, C, rank);
        const int64_t token = a.tokens[t];
        if (threadIdx.x == 0) {
            sh.above = 0;
            if (s.has(token)) sh.token = Elem<DT>::up(s.row[token]);
        }
        if (threadIdx.x < kTopMax) sh.top[threadIdx.x] = 0;
        Online<DT, true> sums;
        uint32_t most = kNegInfWord<DT>;
        float bound = kLowest;                        // -inf is no candidate
        // The vectors of the lanes that call with `yes` join the warp's list, in the order
        // of the lanes; all lanes call.
        int found = 0;
        auto candidates = [&](bool yes, const uint4 &v, int j) {
            const unsigned who = __ballot_sync(0xFFFFFFFFu, yes);
            const int at = found + __popc(who & ((1u << lane) - 1u));
            if (yes && at < kWarpList) {
                sh.vec[warp][at] = v;
                sh.element[warp][at] = s.at(j);
            }
            found += __popc(who);
        };
        for (int j0 = s.from, b = 0; j0 < s.to; j0 += kStep, ++b) {
            const int j = j0 + threadIdx.x;
            copies_left<kStages - 2>();
            uint4 cur[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) cur[i] = sh.ring[stage][i][threadIdx.x];
            if (j0 + kStep > s.to) {
#pragma unroll
                for (int i = 0; i < kBatch; ++i)
                    if (j + i * kStatThreads >= s.to)
                        cur[i] = make_uint4(kNegInfWord<DT>, kNegInfWord<DT>, kNegInfWord<DT>,
                                            kNegInfWord<DT>);
            }
            stage = stage + 1 == kStages ? 0 : stage + 1;
            fetch.next();
            // one check a batch against the sums' reference and the candidates' bound
            uint32_t w[kBatch], all = kNegInfWord<DT>;
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                w[i] = vec_max<DT>(cur[i]);
                all = max_word<DT>(all, w[i]);
            }
            const float vm = word_max<DT>(all);
            // a bound from the first batch, from the first 4, 16, 64, ...
            if (want && (b == 0 || ((b & (b - 1)) == 0 && (b & 0x55555554)))) {
                find_bound<DT>(b == 0 ? vm : word_max<DT>(most), want, sh);
                bound = fmaxf(sh.bound, kLowest);
            }
            most = max_word<DT>(most, all);
            if (vm > sums.limit) sums.raise(vm);
            if (want && __any_sync(0xFFFFFFFFu, vm >= bound)) {
#pragma unroll
                for (int i = 0; i < kBatch; ++i)
                    candidates(word_max<DT>(w[i]) >= bound, cur[i], j + i * kStatThreads);
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) sums.add(cur[i]);
        }
        // the vectors filled in part
        const int edge = threadIdx.x == 0 && s.from > 0 ? 0
                         : threadIdx.x == 32 && s.to < s.n ? s.to : -1;
        uint4 v = make_uint4(0, 0, 0, 0);
        float vm = -INFINITY;
        if (edge >= 0) {
            v = s.part(edge);
            const uint32_t wv = vec_max<DT>(v);
            most = max_word<DT>(most, wv);
            vm = word_max<DT>(wv);
            sums.add(v, vm);
        }
        if (want) {
            candidates(vm >= bound, v, edge);
            if (lane == 0) sh.found[warp] = found;
        }
        const Sums mine = warp_join(sums.sums());
        if (lane == 0) sh.warps[warp] = mine;
        if (want) find_bound<DT>(word_max<DT>(most), want, sh);
        else __syncthreads();
        Sums all = warp_join(lane < kStatWarps ? sh.warps[lane] : Sums{kLowest, 0.0f, 0.0f});
        if (want) {
            const float full = sh.bound;
            const bool nan = all.sum != all.sum;
            bool over = false;
#pragma unroll
            for (int i = 0; i < kStatWarps; ++i) over |= sh.found[i] > kWarpList;
            if (over || nan) {
                read_again<DT>(s, want, nan, sh);
            } else {
                // their elements that reach it, usually few
                const float least = fmaxf(full, kLowest);
                for (int i = lane; i < found; i += 32) {
                    const uint4 v = sh.vec[warp][i];
                    if (!(word_max<DT>(vec_max<DT>(v)) >= least)) continue;
                    float f[N];
                    Elem<DT>::unpack(v, f);
#pragma unroll
                    for (int k = 0; k < N; ++k) {
                        if (!(f[k] >= least)) continue;
                        const int at = atomicAdd(&sh.above, 1);
                        if (at < kShortList) sh.few[at] = order_key(f[k], sh.element[warp][i] + k);
                    }
                }
                __syncthreads();
                int few = sh.above;
                if (full == -INFINITY && few < want) {
                    // all finite ones, and the first of the others
                    if (warp == 0) first_equal<DT>(s, want - few, full, sh.few + few);
                    few = min(want, s.end() - s.first());
                    __syncthreads();
                }
                if (few > kShortList) read_again<DT>(s, want, false, sh);
                else rank_keys(sh.few, few, want, sh.top);
            }
        }
        if (C > 1) {
            if (threadIdx.x == 0) sh.slice = all;
            cluster.sync();
            if (rank == 0)
                all = warp_join(lane < C ? cluster.map_shared_rank(&sh, lane)->slice
                                         : Sums{kLowest, 0.0f, 0.0f});
        } else {
            __syncthreads();
        }
        if (rank == 0) {
            const float ls = logf(all.sum);
            if (threadIdx.x == 0) {
                float lp = 0.0f;
                if (token >= a.V) {
                    lp = NAN;
                } else if (token >= 0) {
                    // (rank 0's slice is the longest, and starts at -skip)
                    const int owner = C > 1 ? ((int)token - s.start) / N / s.n : 0;
                    const float x = cluster.map_shared_rank(&sh, owner)->token;
                    lp = log_prob(x, all.ref, all.sum, ls);
                }
                if (a.logp) a.logp[t] = lp;
                if (a.entropy)
                    a.entropy[t] = all.sum == 0.0f ? 0.0f : __fsub_rn(ls, __fdiv_rn(all.first, all.sum));
                if (a.lse) a.lse[t] = __fadd_rn(all.ref, ls);
            }
            if (want && C > 1) {
                // the slices' alternatives: those that reach every slice's last one
                uint64_t least = 0;
                if (lane < C) least = cluster.map_shared_rank(&sh, lane)->top[want - 1];
#pragma unroll
                for (int o = 1; o < kMaxCluster; o <<= 1) {
                    const uint64_t other = __shfl_xor_sync(0xFFFFFFFFu, least, o);
                    least = other > least ? other : least;
                }
                least = __shfl_sync(0xFFFFFFFFu, least, 0);
                if (threadIdx.x == 0) sh.count = 0;
                __syncthreads();
                for (int i = threadIdx.x; i < C * want; i += kStatThreads) {
                    const uint64_t key = cluster.map_shared_rank(&sh, i / want)->top[i % want];
                    if (key != 0 && key >= least) sh.list[atomicAdd(&sh.count, 1)] = key;
                }
                __syncthreads();
                rank_keys(sh.list, sh.count, want, sh.top);
                __syncthreads();
            }
            if (threadIdx.x < want) {
                const uint64_t key = sh.top[threadIdx.x];
                const float x = from_ordered((uint32_t)(key >> 32));
                a.top_ids[t * want + threadIdx.x] = key_index(key);
                a.top_logp[t * want + threadIdx.x] = log_prob(x, all.ref, all.sum, ls);
            }
        }
        if (C > 1) cluster.sync();     // the leader has read this CTA's shared memory
        else __syncthreads();
    }
}

// Short rows: a warp a row, its vectors (at most NV a lane) in registers.  The bound of the
// alternatives is the k-th largest of the lanes' maxima; what reaches it is ranked by
// counting, and where that fails (NaN, a full list) the k largest are taken one by one.
// Without a barrier and with 20 or more rows in flight an SM: 16384 x 100 BF16, k = 8,
// 19 us (162 us with a CTA a row), 7195 x 2018 25 us (57 us), 7195 x 3500, k = 20, 48 us
// (62 us).  Far from HBM (25 us: 17%): one row a warp with nothing loaded ahead, and for k
// near 32 the bound is the lowest of the lanes' maxima, which many keys reach (9870 x 691
// FP16, k = 32: 82 us).
constexpr int kShortWarps = 4, kShortKeys = 512;
template <int DT, int NV>
__global__ void __launch_bounds__(kShortWarps * 32) token_stats_short_kernel(const TokenLogprobs a) {
    using E = Elem<DT>;
    constexpr int N = E::kVec;
    __shared__ unsigned long long lists[kShortWarps][kShortKeys], tops[kShortWarps][kTopMax];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, want = a.k;
    unsigned long long *list = lists[warp], *top = tops[warp];
    pdl_wait_and_release();
    for (int64_t t = (int64_t)blockIdx.x * kShortWarps + warp; t < a.T;
         t += (int64_t)gridDim.x * kShortWarps) {
        const Slice<DT> s(elem_at<DT>(a.logits, t * a.ld), (int)a.V, 1, 0);
        const int64_t token = a.tokens[t];
        const float at_token = s.has(token) ? E::up(s.row[token]) : 0.0f;
        uint4 v[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = lane + 32 * i;
            v[i] = make_uint4(kNegInfWord<DT>, kNegInfWord<DT>, kNegInfWord<DT>, kNegInfWord<DT>);
            if (j >= s.from && j < s.to) v[i] = s.load(j);
        }
        // the vectors filled in part (at most the first and the last)
        if (s.from > 0 && lane == 0) v[0] = s.part(0);
        if (s.to < s.n && lane == (s.to & 31)) {
            const uint4 last = s.part(s.to);
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (lane + 32 * i == s.to) v[i] = last;
        }
        Online<DT, true> sums;
        float most = -INFINITY;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const float vm = word_max<DT>(vec_max<DT>(v[i]));
            most = fmaxf(most, vm);
            sums.add(v[i], vm);
        }
        const Sums all = warp_join(sums.sums());
        if (want) {
            int larger = 0;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const float o = __shfl_sync(0xFFFFFFFFu, most, i);
                larger += o > most || (o == most && i < lane);
            }
            const unsigned who = __ballot_sync(0xFFFFFFFFu, larger == want - 1);
            const float bound = __shfl_sync(0xFFFFFFFFu, most, who ? __ffs(who) - 1 : 0);
            const float least = fmaxf(bound, kLowest);        // -inf is no candidate
            int few = 0;
            bool fails = all.sum != all.sum;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (fails) break;
                float f[N];
                E::unpack(v[i], f);
                uint32_t hits = 0;
#pragma unroll
                for (int k = 0; k < N; ++k) hits |= (f[k] >= least ? 1u : 0u) << k;
                if (!__any_sync(0xFFFFFFFFu, hits)) continue;
                int before = __popc(hits);
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int up = __shfl_up_sync(0xFFFFFFFFu, before, o);
                    if (lane >= o) before += up;
                }
                const int total = __shfl_sync(0xFFFFFFFFu, before, 31);
                int at = few + before - __popc(hits);
                few += total;
                fails = few > kShortKeys;
                if (fails) break;
#pragma unroll
                for (int k = 0; k < N; ++k)
                    if ((hits >> k) & 1u)
                        list[at++] = order_key(f[k], (uint32_t)(s.at(lane + 32 * i) + k));
            }
            if (fails) {
                uint64_t last = ~0ull;
                for (int q = 0; q < want; ++q) {
                    uint64_t best = 0;
#pragma unroll 1
                    for (int j = lane; j < s.n; j += 32) {
                        float f[N];
                        E::unpack(s.any(j), f);
#pragma unroll
                        for (int k = 0; k < N; ++k) {
                            if (!s.has(s.at(j) + k)) continue;
                            const uint64_t key = order_key(f[k], (uint32_t)(s.at(j) + k));
                            if (key < last && key > best) best = key;
                        }
                    }
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) {
                        const uint64_t other = __shfl_xor_sync(0xFFFFFFFFu, best, o);
                        best = other > best ? other : best;
                    }
                    last = best;
                    if (lane == 0) top[q] = best;
                }
            } else {
                if (bound == -INFINITY && few < want) {
                    // all finite ones, and the first of the others
                    first_equal<DT>(s, want - few, bound, list + few);
                    few = want;
                }
                __syncwarp();
                for (int i = lane; i < few; i += 32) {
                    const uint64_t key = list[i];
                    int rank = 0;
#pragma unroll 4
                    for (int j = 0; j < few; ++j) rank += list[j] > key;
                    if (rank < want) top[rank] = key;
                }
            }
            __syncwarp();
        }
        const float ls = logf(all.sum);
        if (lane == 0) {
            float lp = 0.0f;
            if (token >= a.V) lp = NAN;
            else if (token >= 0)
                lp = log_prob(at_token, all.ref, all.sum, ls);
            if (a.logp) a.logp[t] = lp;
            if (a.entropy)
                a.entropy[t] = all.sum == 0.0f ? 0.0f : __fsub_rn(ls, __fdiv_rn(all.first, all.sum));
            if (a.lse) a.lse[t] = __fadd_rn(all.ref, ls);
        }
        if (lane < want) {
            const uint64_t key = top[lane];
            const float x = from_ordered((uint32_t)(key >> 32));
            a.top_ids[t * want + lane] = key_index(key);
            a.top_logp[t * want + lane] = log_prob(x, all.ref, all.sum, ls);
        }
        __syncwarp();                             // the lists are written again
    }
}

// ---- the loss and its gradient --------------------------------------------------
//
// A cluster of C CTAs takes a row; each CTA copies its slice into shared memory,
// adds its exponentials as it arrives, and writes its gradient from there: the
// logits are read once.  Join of the CTAs' sums through distributed shared memory.
// Bound by HBM: 8192 x 32000 BF16 151 us (6.9 TB/s, what a copy reaches), 1021 x 50001
// FP32 74 us (5.5 TB/s: four slices a row at any alignment).
constexpr int kRowThreads = 256, kRowWarps = kRowThreads / 32;
constexpr int kSliceBytes = 72 * 1024;        // three CTAs an SM
constexpr int64_t kOneSliceBytes = 108 * 1024;   // two, where that saves the cluster
constexpr int kMaxSliceBytes = 216 * 1024;    // one CTA an SM

__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

struct RowShared {
    Sums warps[kRowWarps];
    Sums slice, row;
    float token;                  // the token's logit, in the CTA that holds it
};

// Gradient of a vector of logits: scale e^(x - ref).
template <int DT>
__device__ __forceinline__ void loss_grad(const uint4 &v, float ref, float scale, float *g) {
    constexpr int N = Elem<DT>::kVec;
    uint64_t d[N / 2];
    differences<DT>(v, ref, d);
    const uint64_t l2 = f32x2(kLog2e, kLog2e), s2 = f32x2(scale, scale);
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        const uint64_t t = mul_f32x2(d[i], l2);
        const uint64_t p = mul_f32x2(f32x2(exp2_approx(lo_f32(t)), exp2_approx(hi_f32(t))), s2);
        g[2 * i] = lo_f32(p);
        g[2 * i + 1] = hi_f32(p);
    }
}

template <int DT, int THREADS>
__global__ void __launch_bounds__(THREADS, 768 / THREADS) token_loss_kernel(const TokenLogprobs a) {
    using E = Elem<DT>;
    using Word = typename E::Word;
    constexpr int N = E::kVec;
    extern __shared__ __align__(16) uint4 data[];
    __shared__ RowShared sh;
    cg::cluster_group cluster = cg::this_cluster();
    const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    constexpr int kWarpsHere = THREADS / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Word *words = reinterpret_cast<const Word *>(data);
    pdl_wait_and_release();
    for (int64_t t = blockIdx.x / C; t < a.T; t += gridDim.x / C) {
        const Slice<DT> s(elem_at<DT>(a.logits, t * a.ld), (int)a.V, C, rank);
        const int64_t token = a.tokens[t];
        const int steps = (s.to - s.from + THREADS - 1) / THREADS;
        auto part_of = [&](int q) {       // vectors of the q-th of four groups of copies
            return min(s.to, s.from + steps * q / 4 * THREADS);
        };
        // four groups, so that the sums start with the first
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int stop = part_of(q + 1);
#pragma unroll 2
            for (int j = part_of(q) + threadIdx.x; j < stop; j += THREADS)
                copy16(data + j, s.vec + j);
            copies_commit();
        }
        // the vectors filled in part, while the copies run
        Online<DT, false> sums;
        const int edge = threadIdx.x == 0 && s.from > 0 ? 0
                         : threadIdx.x == THREADS - 1 && s.to < s.n ? s.to : -1;
        if (edge >= 0) {
            const uint4 v = s.part(edge);
            data[edge] = v;
            sums.add(v, word_max<DT>(vec_max<DT>(v)));
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if (q == 0) copies_left<3>();
            if (q == 1) copies_left<2>();
            if (q == 2) copies_left<1>();
            if (q == 3) copies_left<0>();
            const int stop = part_of(q + 1);
#pragma unroll 2
            for (int j = part_of(q) + threadIdx.x; j < stop; j += THREADS) {
                const uint4 v = data[j];
                sums.add(v, word_max<DT>(vec_max<DT>(v)));
            }
        }
        const Sums mine = warp_join(sums.sums());
        if (lane == 0) sh.warps[warp] = mine;
        __syncthreads();
        Sums all = warp_join(lane < kWarpsHere ? sh.warps[lane] : Sums{kLowest, 0.0f, 0.0f});
        if (threadIdx.x == 0 && s.has(token)) sh.token = E::up(words[token - s.start]);
        if (C > 1) {
            if (threadIdx.x == 0) sh.slice = all;
            cluster.sync();
            if (warp == 0) {
                all = warp_join(lane < C ? cluster.map_shared_rank(&sh, lane)->slice
                                         : Sums{kLowest, 0.0f, 0.0f});
                if (lane == 0) sh.row = all;
            }
            __syncthreads();
            all = sh.row;
            cluster_arrive();              // the others' shared memory has been read
        }
        const bool ignored = token < 0, beyond = token >= a.V, empty = all.sum == 0.0f;
        // the CTA that holds the token (the first one for a token outside)
        if (threadIdx.x == 0 && a.logp && (ignored || beyond ? rank == 0 : s.has(token))) {
            const float x = sh.token;
            const float lp = log_prob(x, all.ref, all.sum, logf(all.sum));
            a.logp[t] = ignored ? 0.0f : beyond ? NAN : lp;
        }
        float w = a.weights ? a.weights[t] : 1.0f;
        if (beyond || all.sum != all.sum) w = NAN;    // 0 times a row of NaN is NaN too
        if (ignored || (empty && !beyond)) w = 0.0f;
        const float scale = __fdiv_rn(w, all.sum);
        char *out = elem_at<DT>(a.dlogits, t * a.ldd);
        const int mine_token = s.has(token) ? (int)token : -1;
        // The vectors of the output row (its 16-byte boundaries may lie elsewhere) that
        // hold elements of the slice only, and the elements before and after them.
        const int oskip = (int)(reinterpret_cast<uintptr_t>(out) & 15u) / E::kSize;
        const int e0 = s.first(), e1 = s.end();
        const int o0 = (e0 + oskip + N - 1) / N, o1 = e1 > e0 ? (e1 + oskip) / N : o0;
        uint4 *ovec = reinterpret_cast<uint4 *>(out - oskip * E::kSize);
        const int token_vec = mine_token >= 0 ? (mine_token + oskip) / N : -1;
        const int shift = (e0 + oskip + N - 1) / N * N - oskip - s.start;   // of o0 in the slice
        const uint4 *from = data + shift / N;
        const int off = shift % N * E::kSize;
        auto one = [&](const uint4 &v, int o) {
            float g[N];
            loss_grad<DT>(v, all.ref, scale, g);
            if (o == token_vec) {
#pragma unroll
                for (int i = 0; i < N; ++i)
                    if (o * N - oskip + i == mine_token) g[i] = __fsub_rn(g[i], w);
            }
            ovec[o] = E::pack(g);
        };
        if (w == 0.0f) {
            for (int o = o0 + threadIdx.x; o < o1; o += THREADS) ovec[o] = make_uint4(0, 0, 0, 0);
        } else if (off == 0) {
#pragma unroll 2
            for (int o = o0 + threadIdx.x; o < o1; o += THREADS) one(from[o - o0], o);
        } else {
            for (int o = o0 + threadIdx.x; o < o1; o += THREADS)
                one(bytes_from(from[o - o0], from[o - o0 + 1], off), o);
        }
        // elements of output vectors shared with other slices or rows
        const int head = min(e1, o0 * N - oskip), tail = max(head, o1 * N - oskip);
        const int i = threadIdx.x;
        if (i < head - e0 + e1 - tail) {
            const int e = i < head - e0 ? e0 + i : tail + i - (head - e0);
            float g = 0.0f;
            if (w != 0.0f) g = __fmul_rn(exp_approx(__fsub_rn(E::up(words[e - s.start]), all.ref)), scale);
            if (e == mine_token) g = __fsub_rn(g, w);
            store_elem<DT>(out, e, g);
        }
        if (C > 1) cluster_wait();
        __syncthreads();
    }
}

// The CTAs of a row's cluster in the loss: one for rows of up to kOneSliceBytes (4096
// rows of 100 KB: 126 us, 138 us as two slices), else slices of at most kSliceBytes
// where eight CTAs allow it (three CTAs an SM, whose copies and passes overlap: 1021
// rows of 200 KB took 91 us as four slices, 98 us as two), and more CTAs a row while
// the rows alone do not fill two CTAs an SM, down to 4 KB.  0: the row does not fit on
// chip.
int loss_cluster(int64_t T, int64_t V, int size) {
    const int64_t bytes = V * size + 16;
    int c = 1;
    while (c < kMaxCluster && bytes > (c == 1 ? kOneSliceBytes : c * (int64_t)kSliceBytes)) c *= 2;
    if (bytes > c * (int64_t)kMaxSliceBytes) return 0;
    while (c < kMaxCluster && T * c < 2 * sm_count() && bytes > c * 8192ll) c *= 2;
    return c;
}

// The CTAs of a row's cluster in the statistics: one, and more while the rows do not
// fill two CTAs an SM, down to 4 KB.
int stats_cluster(int64_t T, int64_t V, int size) {
    int c = 1;
    while (c < kMaxCluster && T * c < 2 * sm_count() && V * size > c * 8192ll) c *= 2;
    return c;
}

int row_grid(int64_t T, int c) { return (int)(T < (1 << 24) ? T : 1 << 24) * c; }

template <int DT, int THREADS>
cudaError_t launch_loss_threads(const TokenLogprobs &a, int c, int64_t slice, cudaStream_t st) {
    static bool ready[kMaxDevices];
    auto kernel = token_loss_kernel<DT, THREADS>;
    const cudaError_t e =
        allow_shared(kernel, THREADS == kRowThreads ? kMaxSliceBytes + 32 : 16 * THREADS * 16, ready);
    if (e != cudaSuccess) return e;
    return launch_pdl_clusters(kernel, row_grid(a.T, c), THREADS, c, (size_t)slice * 16, st, a);
}

// A CTA of as few threads as leave each at least eight vectors of its slice: 9870 rows of
// 691 FP16 values take 28 us with a warp a row, 49 us with eight; 4000 rows of 10000 BF16
// values 27 us with four warps, 45 us with eight.
template <int DT>
cudaError_t launch_loss(const TokenLogprobs &a, int c, cudaStream_t st) {
    // a row that starts inside a vector has one vector more
    const int64_t vectors = (a.V + 2 * Elem<DT>::kVec - 2) / Elem<DT>::kVec;
    const int64_t slice = (vectors + c - 1) / c;
    return slice >= 8 * kRowThreads ? launch_loss_threads<DT, kRowThreads>(a, c, slice, st)
           : slice >= 8 * 128       ? launch_loss_threads<DT, 128>(a, c, slice, st)
           : slice >= 8 * 64        ? launch_loss_threads<DT, 64>(a, c, slice, st)
                                    : launch_loss_threads<DT, 32>(a, c, slice, st);
}

template <int DT>
cudaError_t launch_stats(const TokenLogprobs &a, cudaStream_t st) {
    constexpr int N = Elem<DT>::kVec;
    const int64_t vectors = (a.V + 2 * N - 2) / N;
    if (vectors <= 32 * 16) {
        auto kernel = vectors <= 32 * 2   ? token_stats_short_kernel<DT, 2>
                      : vectors <= 32 * 4 ? token_stats_short_kernel<DT, 4>
                      : vectors <= 32 * 8 ? token_stats_short_kernel<DT, 8>
                                          : token_stats_short_kernel<DT, 16>;
        const int64_t ctas = (a.T + kShortWarps - 1) / kShortWarps, most = 1 << 30;
        return launch_pdl(kernel, (int)(ctas < most ? ctas : most), kShortWarps * 32, 0, st, a);
    }
    static bool ready[kMaxDevices];
    auto kernel = token_stats_kernel<DT>;
    const cudaError_t e = allow_shared(kernel, sizeof(StatShared), ready);
    if (e != cudaSuccess) return e;
    const int c = stats_cluster(a.T, a.V, Elem<DT>::kSize);
    const int64_t most = 6 * sm_count() / c;
    const int rows = (int)(a.T < most ? a.T : most);
    return launch_pdl_clusters(kernel, rows * c, kStatThreads, c, sizeof(StatShared), st, a);
}

// ---- the gradient of the statistics ----------------------------------------------
//
// One reading and one writing, nothing kept: a CTA takes a tile of a row, four vectors
// a thread at the 16-byte boundaries of the output, its copies or loads issued before
// the row's five scalars are used.  SHIFTED: some rows' logits lie across the output's
// boundaries; the tile then passes through shared memory, where an output vector is cut
// from two of the input's.  4096 x 32000 BF16 76 us (6.9 TB/s, HBM); 4096 x 32003 to rows
// at other alignments 84 us (6.2 TB/s, issue 82%; cut from registers 101 us).
constexpr int kTilePart = 4;
constexpr int kTile = kTilePart * kThreads;             // vectors

template <int DT, bool SHIFTED>
__global__ void __launch_bounds__(kThreads)
token_logprobs_backward_kernel(const TokenLogprobsBackward a, int tiles) {
    using E = Elem<DT>;
    using Word = typename E::Word;
    constexpr int N = E::kVec;
    __shared__ uint4 input[SHIFTED ? kTile + 1 : 1];
    pdl_wait_and_release();
    const int V = (int)a.V;
    for (int64_t unit = blockIdx.x; unit < a.T * tiles; unit += gridDim.x) {
        const int64_t t = unit / tiles;
        const int tile = (int)(unit - t * tiles) * kTile;
        const Word *row = reinterpret_cast<const Word *>(elem_at<DT>(a.logits, t * a.ld));
        Word *out = reinterpret_cast<Word *>(elem_at<DT>(a.dlogits, t * a.ldd));
        const int skip = (int)(reinterpret_cast<uintptr_t>(row) & 15u) / E::kSize;
        const int oskip = (int)(reinterpret_cast<uintptr_t>(out) & 15u) / E::kSize;
        const int shift = SHIFTED ? (skip - oskip + N) & (N - 1) : 0;     // elements
        // the input vector that holds the first element of an output vector
        const uint4 *vec = reinterpret_cast<const uint4 *>(row - skip) - (SHIFTED && skip < oskip);
        uint4 *ovec = reinterpret_cast<uint4 *>(out - oskip);
        const int vectors = (V + oskip + N - 1) / N;
        uint4 v[SHIFTED ? 1 : kTilePart];
        if constexpr (SHIFTED) {
            for (int i = threadIdx.x; i <= kTile; i += kThreads) {
                const int e = (tile + i) * N - oskip - shift;
                if (e >= 0 && e + N <= V) copy16(input + i, vec + tile + i);
            }
            copies_commit();
        } else {
#pragma unroll
            for (int i = 0; i < kTilePart; ++i) {
                const int o = tile + i * kThreads + threadIdx.x, e = o * N - oskip;
                if (e >= 0 && e + N <= V) v[i] = vec[o];
            }
        }
        const int64_t token = a.tokens[t];
        float lse = a.lse[t], dl = a.dlogp[t], de = 0.0f, h = 0.0f;
        if (a.dentropy) {
            de = a.dentropy[t];
            h = a.entropy[t];
        }
        if (token < 0) dl = 0.0f;
        if (token >= a.V) lse = NAN;              // a row of NaN, empty or not
        const bool empty = lse == -INFINITY;
        // g = p (c0 + c1 l), l = x - lse
        const float c0 = -__fmaf_rn(de, h, dl), c1 = -de;
        const int at = token >= 0 && token < a.V ? (int)token : -1;
        if constexpr (SHIFTED) {
            copies_left<0>();
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < kTilePart; ++i) {
            const int k0 = i * kThreads + threadIdx.x, o = tile + k0, e = o * N - oskip;
            if (o >= vectors) break;
            // (a shifted vector needs two whole input vectors)
            if (SHIFTED && shift ? e >= N && e + 2 * N <= V : e >= 0 && e + N <= V) {
                if (empty) {
                    ovec[o] = make_uint4(0, 0, 0, 0);
                    continue;
                }
                uint4 x;
                if constexpr (SHIFTED) x = bytes_from(input[k0], input[k0 + 1], shift * E::kSize);
                else x = v[i];
                uint64_t l[N / 2];
                differences<DT>(x, lse, l);
                float g[N];
#pragma unroll
                for (int k = 0; k < N / 2; ++k) {
                    float lo = lo_f32(l[k]), hi = hi_f32(l[k]);
                    asm("max.NaN.f32 %0, %0, %1;" : "+f"(lo) : "f"(-1000.0f));
                    asm("max.NaN.f32 %0, %0, %1;" : "+f"(hi) : "f"(-1000.0f));
                    l[k] = f32x2(lo, hi);
                    const uint64_t y = mul_f32x2(l[k], f32x2(kLog2e, kLog2e));
                    const uint64_t p = f32x2(exp2_approx(lo_f32(y)), exp2_approx(hi_f32(y)));
                    const uint64_t q = mul_f32x2(p, fma_f32x2(l[k], f32x2(c1, c1), f32x2(c0, c0)));
                    g[2 * k] = lo_f32(q);
                    g[2 * k + 1] = hi_f32(q);
                }
                if ((unsigned)(at - e) < (unsigned)N) {
#pragma unroll
                    for (int k = 0; k < N; ++k)
                        if (e + k == at) g[k] = __fadd_rn(g[k], dl);
                }
                ovec[o] = E::pack(g);
            } else {
                for (int k = 0; k < N; ++k) {
                    if (e + k < 0 || e + k >= V) continue;
                    float g = 0.0f;
                    if (!empty) {
                        const float l = below_max(E::up(row[e + k]), lse);
                        g = __fmul_rn(exp_approx(l), __fmaf_rn(l, c1, c0));
                        if (e + k == at) g = __fadd_rn(g, dl);
                    }
                    out[e + k] = E::down(g);
                }
            }
        }
        if constexpr (SHIFTED) __syncthreads();       // input is copied again
    }
}

int grid_for(int64_t rows) {
    const int64_t most = (int64_t)sm_count() * 8;
    return (int)(rows < most ? rows : most);
}

}  // namespace

cudaError_t launch_token_logprobs(const TokenLogprobs &a, cudaStream_t st) {
    if (!a.dlogits) {
        return a.dtype == kF32    ? launch_stats<kF32>(a, st)
               : a.dtype == kBF16 ? launch_stats<kBF16>(a, st)
                                  : launch_stats<kF16>(a, st);
    }
    const int c = loss_cluster(a.T, a.V, a.dtype == kF32 ? 4 : 2);
    if (c) {
        return a.dtype == kF32    ? launch_loss<kF32>(a, c, st)
               : a.dtype == kBF16 ? launch_loss<kBF16>(a, c, st)
                                  : launch_loss<kF16>(a, c, st);
    }
    auto k = a.dtype == kF32    ? token_loss_long_kernel<kF32>
             : a.dtype == kBF16 ? token_loss_long_kernel<kBF16>
                                : token_loss_long_kernel<kF16>;
    return launch_pdl(k, grid_for(a.T), kThreads, 0, st, a);
}

namespace {

template <int DT>
cudaError_t launch_backward(const TokenLogprobsBackward &a, cudaStream_t st) {
    constexpr int kSize = Elem<DT>::kSize, N = Elem<DT>::kVec;
    // rows of both tensors that all start at the same place between 16-byte boundaries
    const bool level = ((reinterpret_cast<uintptr_t>(a.logits) ^ reinterpret_cast<uintptr_t>(a.dlogits)) & 15u) == 0 &&
                       (a.T == 1 || (a.ld - a.ldd) * kSize % 16 == 0);
    const int64_t tiles = (a.V + N - 1 + (int64_t)kTile * N - 1) / ((int64_t)kTile * N);
    const int64_t units = a.T * tiles, most = 1 << 30;
    return launch_pdl(level ? token_logprobs_backward_kernel<DT, false>
                            : token_logprobs_backward_kernel<DT, true>,
                      (int)(units < most ? units : most), kThreads, 0, st, a, (int)tiles);
}

}  // namespace

cudaError_t launch_token_logprobs_backward(const TokenLogprobsBackward &a, cudaStream_t st) {
    return a.dtype == kF32    ? launch_backward<kF32>(a, st)
           : a.dtype == kBF16 ? launch_backward<kBF16>(a, st)
                              : launch_backward<kF16>(a, st);
}

}  // namespace agoq
