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

// fl(s / n) for n >= 1 with inv = fl(1 / n): the product, corrected by its remainder
// (P. Markstein, IBM J. Res. Dev. 34(1), 1990); a quotient that overflows or is not
// finite stays as the product gives it.
__device__ __forceinline__ float divided(float s, float n, float inv) {
    const float q = __fmul_rn(s, inv);
    const float c = __fmaf_rn(__fmaf_rn(-q, n, s), inv, q);
    return fabsf(q) < 3e38f && fabsf(s) > 1e-30f ? c : q;
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

// Threads that share a row: the CTA, or for short rows one of several groups of
// whole warps in it, each with rows of its own and a barrier of its own.
struct Group {
    int size, id, tid;            // threads; which of the CTA's groups; thread in the group
    __device__ __forceinline__ explicit Group(int size_)
        : size(size_), id(threadIdx.x / size_), tid(threadIdx.x % size_) {}
    __device__ __forceinline__ void sync() const {
        asm volatile("bar.sync %0, %1;" ::"r"(id + 1), "r"(size) : "memory");
    }
};

// The sums of the group's values (each thread gets them), in a fixed order; `red`
// holds 32 floats a value and is free again after the group's next barrier.
template <int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float *red, const Group &g) {
    const int lane = threadIdx.x & 31, warp = g.tid >> 5, warps = g.size >> 5;
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
    if (warps == 1) return;
    if (lane == 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) red[32 * i + warp] = v[i];
    }
    g.sync();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = warp_sum(lane < warps ? red[32 * i + lane] : 0.0f);
}
constexpr int kMaxGroups = 8;                 // of a CTA

__device__ __forceinline__ void copy16(void *to, const void *from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                     static_cast<uint32_t>(__cvta_generic_to_shared(to))),
                 "l"(from)
                 : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_left() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Parameters of the elements that a thread of a group holds: vectors tid, tid + size,
// ..., NV of them.
template <int DT, int NV>
__device__ __forceinline__ void load_params(const void *p, bool f32, int vectors, float none,
                                            const Group &g, float *f) {
    constexpr int V = Elem<DT>::kVec;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int j = g.tid + i * g.size;
#pragma unroll
        for (int k = 0; k < V; ++k)
            f[i * V + k] = j < vectors ? param<DT>(p, f32, (int64_t)j * V + k, none) : 0.0f;
    }
}

// Rows that start at 16-byte boundaries and hold whole vectors: a group of threads a
// row and step, NV vectors a thread, the row in registers from its one reading to
// its writing.  Copies into a ring of shared memory run kRing - 1 rows ahead; a thread
// reads only what it copied, so the ring needs no barrier.  BITS: the codes of x too,
// a half warp holding a block of 128.
template <int NV>
constexpr int kRing = NV == 4 ? 3 : 4;       // stages (1024 threads: 192 KB)

template <int DT, int BITS, int NV>
__global__ void __launch_bounds__(NV == 4 ? 1024 : 512)
ln_forward_rows_kernel(const LnForward a, int size) {
    using E = Elem<DT>;
    constexpr int V = E::kVec, F = NV * V;
    constexpr int kStages = kRing<NV>;
    constexpr bool kKeep = F <= 16;      // w and b stay in registers
    extern __shared__ __align__(16) uint4 ring[];
    __shared__ float red[kMaxGroups][2][32];
    const Group g(size);
    const int threads = blockDim.x, vectors = (int)(a.H / V);
    const int64_t step = (int64_t)gridDim.x * (threads / size);
    const int64_t first = (int64_t)blockIdx.x * (threads / size) + g.id;
    const float inv = __frcp_rn((float)a.H);
    pdl_wait_and_release();
    auto fetch = [&](int64_t t, int stage) {
        if (t < a.T) {
            const uint4 *row = reinterpret_cast<const uint4 *>(elem_at<DT>(a.x, t * a.ldx));
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (g.tid + i * size < vectors)
                    copy16(ring + (stage * NV + i) * threads + threadIdx.x, row + g.tid + i * size);
        }
        copies_commit();
    };
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) fetch(first + s * step, s);
    float w[kKeep ? F : 1], b[kKeep ? F : 1];
    if constexpr (kKeep) {
        load_params<DT, NV>(a.w, a.param_f32, vectors, 1.0f, g, w);
        load_params<DT, NV>(a.b, a.param_f32, vectors, 0.0f, g, b);
    }
    int stage = 0;
    for (int64_t t = first; t < a.T; t += step) {
        copies_left<kStages - 2>();
        uint4 v[NV];
        float f[F];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            v[i] = make_uint4(0, 0, 0, 0);
            if (g.tid + i * size < vectors) v[i] = ring[(stage * NV + i) * threads + threadIdx.x];
            E::unpack(v[i], f + i * V);
        }
        fetch(t + (kStages - 1) * step, (stage + kStages - 1) % kStages);
        stage = (stage + 1) % kStages;
        float s[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < F; ++i) s[0] = __fadd_rn(s[0], f[i]);
        row_sums(s, red[g.id][0], g);
        const float mu = divided(s[0], (float)a.H, inv);
        float q[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (g.tid + i * size >= vectors) continue;
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const float d = __fsub_rn(f[i * V + k], mu);
                q[0] = __fmaf_rn(d, d, q[0]);
            }
        }
        row_sums(q, red[g.id][1], g);
        const float var = divided(q[0], (float)a.H, inv);
        const float r = __frcp_rn(__fsqrt_rn(__fadd_rn(var, a.eps)));
        uint4 *out = reinterpret_cast<uint4 *>(elem_at<DT>(a.y, t * a.ldy));
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = g.tid + i * size;
            if (j < vectors) {
                float y[V];
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    const float xh = __fmul_rn(__fsub_rn(f[i * V + k], mu), r);
                    const int64_t e = (int64_t)j * V + k;
                    y[k] = kKeep ? __fmaf_rn(xh, w[kKeep ? i * V + k : 0], b[kKeep ? i * V + k : 0])
                                 : __fmaf_rn(xh, param<DT>(a.w, a.param_f32, e, 1.0f),
                                             param<DT>(a.b, a.param_f32, e, 0.0f));
                }
                out[j] = E::pack(y);
            }
            if constexpr (BITS != 0) {
                const int64_t blk = t * (a.H / kBlock) + j / 16;
                quantize_block16<BITS>(v[i], threadIdx.x & 15,
                                       static_cast<uint32_t *>(a.codes) + blk * 4 * BITS,
                                       a.scales + blk, j < vectors);
            }
        }
        if (g.tid == 0) {
            if (a.mean) a.mean[t] = mu;
            if (a.rstd) a.rstd[t] = r;
        }
    }
}

// Rows of any alignment: the same, an element a thread and step, NE elements a
// thread; the next row's elements are loaded before this one's sums.
template <int DT, int NE>
__global__ void __launch_bounds__(1024) ln_forward_elems_kernel(const LnForward a) {
    using E = Elem<DT>;
    using Word = typename E::Word;
    __shared__ float red[2][32];
    const Group g(blockDim.x);
    const int threads = blockDim.x, tid = threadIdx.x, H = (int)a.H;
    const float inv = __frcp_rn((float)a.H);
    pdl_wait_and_release();
    Word next[NE];
    auto fetch = [&](int64_t t) {
        const Word *row = reinterpret_cast<const Word *>(elem_at<DT>(a.x, t * a.ldx));
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            next[i] = Word(0);
            if (tid + i * threads < H) next[i] = row[tid + i * threads];
        }
    };
    if (blockIdx.x < a.T) fetch(blockIdx.x);
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        float f[NE];
#pragma unroll
        for (int i = 0; i < NE; ++i) f[i] = E::up(next[i]);
        if (t + gridDim.x < a.T) fetch(t + gridDim.x);
        float s[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < NE; ++i) s[0] = __fadd_rn(s[0], f[i]);
        row_sums(s, red[0], g);
        const float mu = divided(s[0], (float)a.H, inv);
        float q[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            const float d = __fsub_rn(f[i], mu);
            if (tid + i * threads < H) q[0] = __fmaf_rn(d, d, q[0]);
        }
        row_sums(q, red[1], g);
        const float var = divided(q[0], (float)a.H, inv);
        const float r = __frcp_rn(__fsqrt_rn(__fadd_rn(var, a.eps)));
        char *out = elem_at<DT>(a.y, t * a.ldy);
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            const int e = tid + i * threads;
            if (e >= H) break;
            const float xh = __fmul_rn(__fsub_rn(f[i], mu), r);
            store_elem<DT>(out, e, __fmaf_rn(xh, param<DT>(a.w, a.param_f32, e, 1.0f),
                                             param<DT>(a.b, a.param_f32, e, 0.0f)));
        }
        if (tid == 0) {
            if (a.mean) a.mean[t] = mu;
            if (a.rstd) a.rstd[t] = r;
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

// Rows that start at 16-byte boundaries and hold whole vectors: as the forward pass,
// x and dy read once, dx written once.  A thread adds its columns' terms of dw and db
// in registers over all rows of its group; the groups of a CTA join theirs in order,
// and the CTA writes one row of the partial sums ([grid][2][H]).
template <int DT, int BITS, int NV>
__global__ void __launch_bounds__(512) ln_backward_rows_kernel(const LnBackward a, int size) {
    using E = Elem<DT>;
    constexpr int V = E::kVec, F = NV * V;
    constexpr int kStages = kRing<NV>, kWords = 4 * BITS;
    constexpr int kParts = BITS ? 1 : 2;             // dy, and x
    extern __shared__ __align__(16) uint4 ring[];
    __shared__ float red[kMaxGroups][2][64];
    const Group g(size);
    const int threads = blockDim.x, vectors = (int)(a.H / V), groups = threads / size;
    const int64_t step = (int64_t)gridDim.x * groups;
    const int64_t first = (int64_t)blockIdx.x * groups + g.id;
    const float inv = __frcp_rn((float)a.H);
    const bool sums = a.dw || a.db;
    pdl_wait_and_release();
    // slot i of part p of a stage
    auto slot = [&](int stage, int p, int i) {
        return ring + ((stage * kParts + p) * NV + i) * threads + threadIdx.x;
    };
    auto fetch = [&](int64_t t, int stage) {
        if (t < a.T) {
            const uint4 *dy = reinterpret_cast<const uint4 *>(elem_at<DT>(a.dy, t * a.lddy));
            const uint4 *x = reinterpret_cast<const uint4 *>(elem_at<DT>(a.x, BITS ? 0 : t * a.ldx));
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (g.tid + i * size < vectors) {
                    copy16(slot(stage, 0, i), dy + g.tid + i * size);
                    if constexpr (BITS == 0) copy16(slot(stage, 1, i), x + g.tid + i * size);
                }
            }
        }
        copies_commit();
    };
    // what does not come in 16-byte copies is loaded a row ahead into registers
    uint32_t lo[BITS ? NV : 1], hi[BITS ? NV : 1];
    float scale[BITS ? NV : 1], mean = 0.0f, rstd = 0.0f;
    auto ahead = [&](int64_t t) {
        if (t >= a.T) return;
        if constexpr (BITS == 0) {
            mean = __ldg(a.mean + t);
            rstd = __ldg(a.rstd + t);
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int j = g.tid + i * size;
                if (j >= vectors) continue;
                const int64_t blk = t * (a.H / kBlock) + j / 16;
                load_chunk<BITS>(static_cast<const uint32_t *>(a.x) + blk * kWords, j & 15, lo[i], hi[i]);
                scale[i] = __ldg(a.scales + blk);
            }
        }
    };
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) fetch(first + s * step, s);
    ahead(first);
    float w[F], dw[F], db[F];
    load_params<DT, NV>(a.w, a.param_f32, vectors, 1.0f, g, w);
#pragma unroll
    for (int i = 0; i < F; ++i) dw[i] = db[i] = 0.0f;
    int stage = 0;
    for (int64_t t = first; t < a.T; t += step) {
        copies_left<kStages - 2>();
        float x[F], d[F];                 // x, then xh; dy
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            uint4 vx = make_uint4(0, 0, 0, 0), vd = vx;
            if (g.tid + i * size < vectors) {
                vd = *slot(stage, 0, i);
                if constexpr (BITS == 0) vx = *slot(stage, 1, i);
                else vx = dequantize_chunk<BITS>(lo[i], hi[i], scale[i]);
            }
            E::unpack(vx, x + i * V);
            E::unpack(vd, d + i * V);
        }
        float mu = mean, r = rstd;
        fetch(t + (kStages - 1) * step, (stage + kStages - 1) % kStages);
        ahead(t + step);
        stage = (stage + 1) % kStages;
        float s0, s1;
        if constexpr (BITS == 0) {
            float s[2] = {0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < F; ++i) {
                x[i] = __fmul_rn(__fsub_rn(x[i], mu), r);
                const float gi = __fmul_rn(d[i], w[i]);
                s[0] = __fadd_rn(s[0], gi);
                s[1] = __fmaf_rn(gi, x[i], s[1]);
            }
            row_sums(s, red[g.id][(t / step) & 1], g);
            s0 = divided(s[0], (float)a.H, inv);
            s1 = divided(s[1], (float)a.H, inv);
        } else {
            float s[2] = {0.0f, 0.0f}, q[2] = {0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < F; ++i) {
                s[0] = __fadd_rn(s[0], x[i]);
                s[1] = __fmaf_rn(d[i], w[i], s[1]);
            }
            row_sums(s, red[g.id][0], g);
            mu = divided(s[0], (float)a.H, inv);
            s0 = divided(s[1], (float)a.H, inv);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const bool in = g.tid + i * size < vectors;
#pragma unroll
                for (int k = i * V; k < (i + 1) * V; ++k) {
                    x[k] = in ? __fsub_rn(x[k], mu) : 0.0f;
                    q[0] = __fmaf_rn(x[k], x[k], q[0]);
                    q[1] = __fmaf_rn(__fmul_rn(d[k], w[k]), x[k], q[1]);
                }
            }
            row_sums(q, red[g.id][1], g);
            const float var = divided(q[0], (float)a.H, inv);
            r = __frcp_rn(__fsqrt_rn(__fadd_rn(var, a.eps)));
            s1 = divided(__fmul_rn(q[1], r), (float)a.H, inv);
#pragma unroll
            for (int i = 0; i < F; ++i) x[i] = __fmul_rn(x[i], r);
        }
        uint4 *out = reinterpret_cast<uint4 *>(elem_at<DT>(a.dx, t * a.lddx));
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (g.tid + i * size >= vectors) continue;
            float o[V];
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const int n = i * V + k;
                o[k] = __fmul_rn(r, __fmaf_rn(-x[n], s1, __fsub_rn(__fmul_rn(d[n], w[n]), s0)));
                dw[n] = __fmaf_rn(d[n], x[n], dw[n]);
                db[n] = __fadd_rn(db[n], d[n]);
            }
            out[g.tid + i * size] = E::pack(o);
        }
    }
    if (!sums) return;
    float *mine = a.workspace + (int64_t)blockIdx.x * 2 * a.H;
    float *joined = reinterpret_cast<float *>(ring);          // [2][H], for several groups
    copies_left<0>();
    for (int who = 0; who < groups; ++who) {
        if (groups > 1) __syncthreads();
        if (g.id != who) continue;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = g.tid + i * size;
            if (j >= vectors) continue;
#pragma unroll
            for (int k = 0; k < V; ++k) {
                float *pw = (groups > 1 ? joined : mine) + j * V + k, *pb = pw + a.H;
                const int n = i * V + k;
                *pw = groups > 1 && who > 0 ? __fadd_rn(*pw, dw[n]) : dw[n];
                *pb = groups > 1 && who > 0 ? __fadd_rn(*pb, db[n]) : db[n];
            }
        }
    }
    if (groups > 1) {
        __syncthreads();
        for (int i = threadIdx.x; i < 2 * (int)a.H; i += threads) mine[i] = joined[i];
    }
}

// dw and db: the P partial rows.  A CTA takes 32 columns; its eight warps add every
// eighth row, and their sums are added in order.
__global__ void __launch_bounds__(kThreads) ln_backward_join_kernel(
    const float *__restrict__ partials, int64_t H, int P, float *__restrict__ dw,
    float *__restrict__ db) {
    pdl_wait_and_release();
    __shared__ float sums[kWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int64_t c0 = (int64_t)blockIdx.x * 32; c0 < 2 * H; c0 += (int64_t)gridDim.x * 32) {
        const int64_t i = c0 + lane;
        float *out = i < H ? dw : db;
        float s = 0.0f;
        if (i < 2 * H && out) {
#pragma unroll 8
            for (int p = warp; p < P; p += kWarps)
                s = __fadd_rn(s, __ldg(partials + (int64_t)p * 2 * H + i));
        }
        sums[warp][lane] = s;
        __syncthreads();
        if (warp == 0 && i < 2 * H && out) {
#pragma unroll
            for (int k = 1; k < kWarps; ++k) s = __fadd_rn(s, sums[k][lane]);
            out[i < H ? i : i - H] = s;
        }
        __syncthreads();
    }
}

int grid_for(int64_t units, int per_sm) {
    const int64_t most = (int64_t)sm_count() * per_sm;
    return (int)(units < most ? (units > 0 ? units : 1) : most);
}

bool on16(const void *p, int64_t ld, int size) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * size % 16 == 0;
}

int threads_for(int64_t units, int per) {
    const int64_t t = (units + per - 1) / per;
    return (int)((t + 31) / 32 * 32);
}

// CTAs of a kernel whose CTAs stay for many units of work: as many as are resident.
template <typename K>
int resident_ctas(K kernel, int threads, size_t smem, int64_t units) {
    int per_sm = 0;
    cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, smem);
    return grid_for(units, per_sm > 0 ? per_sm : 1);
}

// Groups of `size` threads in a CTA: 256 threads, for rows shorter than that.
int groups_of(int size) { return size <= 128 ? 256 / size : 1; }

template <int DT, int BITS, int NV>
cudaError_t forward_rows(const LnForward &a, cudaStream_t st) {
    const int size = threads_for(a.H / Elem<DT>::kVec, NV), groups = groups_of(size);
    const int threads = size * groups;
    const size_t smem = (size_t)kRing<NV> * NV * threads * 16;
    static bool ready[kMaxDevices];
    auto kernel = ln_forward_rows_kernel<DT, BITS, NV>;
    const cudaError_t e =
        allow_shared(kernel, (size_t)kRing<NV> * NV * (NV == 4 ? 1024 : 512) * 16, ready);
    if (e != cudaSuccess) return e;
    const int ctas = resident_ctas(kernel, threads, smem, (a.T + groups - 1) / groups);
    return launch_pdl_clusters(kernel, ctas, threads, 1, smem, st, a, size);
}

template <int DT, int NE>
cudaError_t forward_elems(const LnForward &a, cudaStream_t st) {
    const int threads = threads_for(a.H, NE);
    auto kernel = ln_forward_elems_kernel<DT, NE>;
    return launch_pdl_clusters(kernel, resident_ctas(kernel, threads, 0, a.T), threads, 1, 0, st, a);
}

// Vectors a thread: one for rows of up to 128 vectors (few threads a row wait for one
// another less), two up to 1024 (512 threads), four up to 4096.  0: no row of vectors.
template <int DT>
int row_vectors(int64_t H) {
    constexpr int V = Elem<DT>::kVec;
    if (H % V) return 0;
    const int64_t n = H / V;
    return n <= 128 ? 1 : n <= 1024 ? 2 : n <= 4096 ? 4 : 0;
}

template <int DT, int BITS>
cudaError_t forward_bits(const LnForward &a, cudaStream_t st) {
    if (on16(a.x, a.ldx, Elem<DT>::kSize) && on16(a.y, a.ldy, Elem<DT>::kSize)) {
        switch (row_vectors<DT>(a.H)) {
            case 1: return forward_rows<DT, BITS, 1>(a, st);
            case 2: return forward_rows<DT, BITS, 2>(a, st);
            case 4: return forward_rows<DT, BITS, 4>(a, st);
        }
    }
    if (a.H <= 512) return forward_elems<DT, 4>(a, st);
    if (a.H <= 16384) return forward_elems<DT, 16>(a, st);
    return launch_pdl(ln_forward_kernel<DT>, grid_for(a.T, 8), kThreads, 0, st, a.x, a.ldx, a.w, a.b,
                      a.param_f32, a.T, a.H, a.eps, a.y, a.ldy, a.mean, a.rstd);
}

// Where dw or db is wanted, the partial sums of P CTAs become dw and db.
cudaError_t join(const LnBackward &a, int P, cudaStream_t st) {
    if (!a.dw && !a.db) return cudaSuccess;
    return launch_pdl(ln_backward_join_kernel, grid_for((2 * a.H + 31) / 32, 8), kThreads, 0, st,
                      a.workspace, a.H, P, a.dw, a.db);
}

template <int DT, int BITS, int NV>
cudaError_t backward_rows(const LnBackward &a, cudaStream_t st) {
    const int size = threads_for(a.H / Elem<DT>::kVec, NV), groups = groups_of(size);
    const int threads = size * groups;
    constexpr int kSlots = kRing<NV> * NV * (BITS ? 1 : 2);
    const size_t smem = (size_t)kSlots * threads * 16;
    static bool ready[kMaxDevices];
    auto kernel = ln_backward_rows_kernel<DT, BITS, NV>;
    const cudaError_t e = allow_shared(kernel, (size_t)kSlots * 512 * 16, ready);
    if (e != cudaSuccess) return e;
    int P = resident_ctas(kernel, threads, smem, (a.T + groups - 1) / groups);
    if (P > kLnPartials) P = kLnPartials;
    const cudaError_t r = launch_pdl_clusters(kernel, P, threads, 1, smem, st, a, size);
    return r != cudaSuccess ? r : join(a, P, st);
}

// Elements a thread holds: eight for rows of up to 2048, sixteen up to 8192 (more
// would not leave registers for dw and db).
template <int DT, int BITS>
cudaError_t backward(const Input<DT, BITS> &in, const LnBackward &a, cudaStream_t st) {
    constexpr int kSize = Elem<DT>::kSize, V = Elem<DT>::kVec;
    if ((BITS || on16(a.x, a.ldx, kSize)) && on16(a.dy, a.lddy, kSize) && on16(a.dx, a.lddx, kSize) &&
        a.H % V == 0 && a.H <= 8192)
        return a.H <= 2048 ? backward_rows<DT, BITS, 8 / V>(a, st)
                           : backward_rows<DT, BITS, 16 / V>(a, st);
    const bool sums = a.dw || a.db;
    const int P = sums ? ln_partials(a.T) : grid_for(a.T, 8);
    const cudaError_t e = launch_pdl(ln_backward_kernel<DT, BITS>, P, kThreads, 0, st, in, a.dy,
                                     a.lddy, a.w, a.param_f32, a.mean, a.rstd, a.T, a.H, a.eps,
                                     a.dx, a.lddx, sums ? a.workspace : nullptr);
    return e != cudaSuccess ? e : join(a, P, st);
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
    if (a.dtype == kF32) return forward_bits<kF32, 0>(a, st);
    if (a.dtype == kF16) return forward_bits<kF16, 0>(a, st);
    if (!a.codes) return forward_bits<kBF16, 0>(a, st);
    // y may be x's place: rows that the norm does not quantize are quantized first
    const bool rows = on16(a.x, a.ldx, 2) && on16(a.y, a.ldy, 2) && row_vectors<kBF16>(a.H);
    if (!rows) {
        const cudaError_t e = a.bits == 4   ? codes<4>(a, st)
                              : a.bits == 5 ? codes<5>(a, st)
                              : a.bits == 6 ? codes<6>(a, st)
                                            : codes<8>(a, st);
        return e != cudaSuccess ? e : forward_bits<kBF16, 0>(a, st);
    }
    switch (a.bits) {
        case 4: return forward_bits<kBF16, 4>(a, st);
        case 5: return forward_bits<kBF16, 5>(a, st);
        case 6: return forward_bits<kBF16, 6>(a, st);
        default: return forward_bits<kBF16, 8>(a, st);
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
