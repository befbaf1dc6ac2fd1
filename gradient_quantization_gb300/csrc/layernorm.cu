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
#include <cooperative_groups.h>

#include "agoq_launch.h"
#include "row_units.h"
#include "typed_io.cuh"

namespace agoq {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256, kWarps = kThreads / 32;

// Weight or bias element i (FP32, or the type of the activation), `none` where
// there is no such vector.
template <int DT>
__device__ __forceinline__ float param(const void *p, bool f32, int64_t i, float none) {
    if (!p) return none;
    return f32 ? load_elem<kF32>(p, i) : load_elem<DT>(p, i);
}

// Mean and variance from the sums of a row and of its squares.  They stand where the
// mean is at most one standard deviation: what the difference of the two terms loses
// is then at most a bit.  Elsewhere (and where the squares may have overflowed) the
// row takes a second pass over the differences to its mean.
__device__ __forceinline__ bool moments(float sum, float squares, float inv, float &mu, float &var) {
    mu = __fmul_rn(sum, inv);
    const float second = __fmul_rn(squares, inv);
    var = __fmaf_rn(-mu, mu, second);
    return __fmul_rn(mu, mu) <= var && second < 1e37f;
}

// 1 / sqrt(v): the hardware's approximation, off by less than 2^-22.
__device__ __forceinline__ float inv_sqrt(float v) {
    float r;
    asm("rsqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
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

// ---- rows of vectors ------------------------------------------------------------

// Threads that share a row: the CTA, or for short rows one of several groups in it
// (8, 16 or 32 lanes, or whole warps with a barrier of their own), each with rows of
// its own.
constexpr int kMaxGroups = 8;                 // of more than one warp, in a CTA
struct Group {
    int size, id, tid;            // threads; which of the CTA's groups; thread in the group
    __device__ __forceinline__ explicit Group(int size_)
        : size(size_), id(threadIdx.x / size_), tid(threadIdx.x % size_) {}
    __device__ __forceinline__ void sync() const {
        asm volatile("bar.sync %0, %1;" ::"r"(id + 1), "r"(size) : "memory");
    }
};

// The sums of N = 1, 2, 4 or 8 values over the group (each thread gets them), in a fixed
// order; `red` holds kRed floats a value, 0 where no warp writes, and is free again
// after the group's next barrier.  All threads of a warp call it.  Several values halve
// in number at each of the first exchanges, a half warp (quarter) going on with its
// own: six shuffles for four values, nine for eight.
constexpr int kRed = 32;
template <int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float *red, const Group &g) {
    static_assert(N == 1 || N == 2 || N == 4 || N == 8, "values");
    const int lane = threadIdx.x & 31;
    if (g.size < 32) {
        for (int o = g.size >> 1; o > 0; o >>= 1) {
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = __fadd_rn(v[i], __shfl_xor_sync(0xFFFFFFFFu, v[i], o));
        }
        return;
    }
    float s[N];
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = v[i];
    int o = 16;
#pragma unroll
    for (int m = N / 2; m > 0; m >>= 1) {
        const bool upper = lane & o;
#pragma unroll
        for (int i = 0; i < m; ++i) {
            const float keep = upper ? s[m + i] : s[i], give = upper ? s[i] : s[m + i];
            s[i] = __fadd_rn(keep, __shfl_xor_sync(0xFFFFFFFFu, give, o));
        }
        o >>= 1;
    }
#pragma unroll
    for (; o > 0; o >>= 1) s[0] = __fadd_rn(s[0], __shfl_xor_sync(0xFFFFFFFFu, s[0], o));
    // lane 32 / N * i has the warp's sum of value i in order
    if (g.size == 32) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = __shfl_sync(0xFFFFFFFFu, s[0], 32 / N * i);
        return;
    }
    if (lane % (32 / N) == 0) red[kRed * (lane / (32 / N)) + (g.tid >> 5)] = s[0];
    g.sync();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = 0.0f;
    for (int k = 0; k < g.size; k += 128) {           // four warps' sums
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float4 f = *reinterpret_cast<const float4 *>(red + kRed * i + (k >> 5));
            v[i] = __fadd_rn(v[i], __fadd_rn(__fadd_rn(f.x, f.y), __fadd_rn(f.z, f.w)));
        }
    }
}

// The columns of a CTA: all of a row's or, of long rows, one of the equal parts that the
// CTAs of a cluster take.  CTAs or clusters take the rows `unit`, `unit` + `units`, ...
constexpr int kMaxParts = 8;
struct Columns {
    int first, n, rank, parts, unit, units;
};
template <bool SPLIT>
__device__ __forceinline__ Columns columns_of(int64_t H, int part) {
    if constexpr (!SPLIT) return {0, (int)H, 0, 1, (int)blockIdx.x, (int)gridDim.x};
    const cg::cluster_group cluster = cg::this_cluster();
    const int parts = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    return {rank * part,  min(part, (int)H - rank * part), rank, parts, (int)blockIdx.x / parts,
            (int)gridDim.x / parts};
}

// Before and after a kernel's accesses.  The next launch may take its places from the
// start on, but for clusters, and between their launches, only at the end: CTAs that find
// a place early leave gaps that no whole cluster fits, and the clusters that are left over
// take as long again (backward of 4096 x 8704 back to back: 111 us, 69 so).
template <bool SPLIT>
__device__ __forceinline__ void begin() {
    if constexpr (SPLIT) {
        cg::this_cluster().sync();                               // all of it has begun
        asm volatile("griddepcontrol.wait;" ::: "memory");
    } else {
        pdl_wait_and_release();
    }
}
template <bool SPLIT>
__device__ __forceinline__ void end_rows() {
    if constexpr (SPLIT) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Sums over the CTAs' parts of a row, added in the order of the parts: `box` receives
// them from all, in turn one and the other half, so that one barrier is enough (a CTA
// writes a half again only after the barrier that follows everyone's reading of it).
template <int N>
__device__ __forceinline__ void parts_sums(float (&v)[N], float (&box)[2][kMaxParts * N], int &turn,
                                           const Columns &c) {
    cg::cluster_group cluster = cg::this_cluster();
    float *mine = box[turn];
    turn ^= 1;
    if ((int)threadIdx.x < c.parts) {
        float *to = cluster.map_shared_rank(mine, threadIdx.x) + c.rank * N;
#pragma unroll
        for (int i = 0; i < N; ++i) to[i] = v[i];
    }
    cluster.sync();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = 0.0f;
    for (int k = 0; k < c.parts; ++k) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = __fadd_rn(v[i], mine[k * N + i]);
    }
}

// The i-th of the NV vectors of a row that a thread of a group holds.  16-bit types:
// an octet of lanes holds blocks of 128 elements, lane j their vectors j and j + 8.
template <int DT>
__device__ __forceinline__ int place(const Group &g, int i) {
    if constexpr (DT == kF32) return g.tid + i * g.size;
    else return (g.tid >> 3) * 16 + (g.tid & 7) + 8 * (i & 1) + (i >> 1) * 2 * g.size;
}

// Weight or bias of vector j, in pairs (FP32, or the type of the activation).
template <int DT>
__device__ __forceinline__ void load_params(const void *p, bool f32, int j, float none,
                                            uint64_t *out) {
    constexpr int V = Elem<DT>::kVec;
    float f[V];
    const char *at = static_cast<const char *>(p) + (int64_t)j * V * (f32 ? 4 : Elem<DT>::kSize);
    if (!p) {
#pragma unroll
        for (int k = 0; k < V; ++k) f[k] = none;
    } else if (reinterpret_cast<uintptr_t>(p) & 15u) {
#pragma unroll
        for (int k = 0; k < V; ++k) f[k] = param<DT>(p, f32, (int64_t)j * V + k, none);
    } else if (!f32) {
        Elem<DT>::unpack(__ldg(reinterpret_cast<const uint4 *>(at)), f);
    } else {
#pragma unroll
        for (int k = 0; k < V / 4; ++k)
            Elem<kF32>::unpack(__ldg(reinterpret_cast<const uint4 *>(at) + k), f + 4 * k);
    }
#pragma unroll
    for (int k = 0; k < V / 2; ++k) out[k] = f32x2(f[2 * k], f[2 * k + 1]);
}

// LAAQ codes of a block of 128 BF16 values held by an octet of lanes, lane j having
// vectors j and j + 8; the same codes and scale as agoq_quant_act.  All lanes of
// the warp call it; `valid` gates the stores.
template <int BITS>
__device__ __forceinline__ void quantize_octet(const uint4 &a, const uint4 &b, uint32_t *rec,
                                               float *scale, bool valid) {
    constexpr int kQmax = (1 << (BITS - 1)) - 1;
    constexpr int kBias = BITS < 8 ? 1 << (BITS - 1) : 0;
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    const float s = bf16_div_qmax<kQmax>(octet_max(bf16_absmax<8>(w)));
    const int j = threadIdx.x & 7;
    uint32_t cb[16], lo, hi;
    if (s >= 0x1p-96f) {
        corrected_codes16<kBias>(w, s, cb);
    } else {
        float f[16];
        Elem<kBF16>::unpack(a, f);
        Elem<kBF16>::unpack(b, f + 8);
        integer_codes_n<kQmax, 16, kBias>(f, s, cb);
    }
    __syncwarp();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if constexpr (BITS < 8) pack_biased8<BITS>(cb + 8 * h, lo, hi);
        else pack_fields8<BITS>(cb + 8 * h, lo, hi);
        store_chunk<BITS>(rec, j + 8 * h, lo, hi, valid);
    }
    if (valid && j == 0) *scale = s;
}

// Rows that start at 16-byte boundaries and hold whole vectors: a group of threads R
// rows and step (their sums share the exchanges and the barriers), NV vectors of a row a
// thread.  Copies into a ring of shared memory run kRing - 1 steps ahead; a thread
// reads only what it copied, so the ring needs no barrier, and the row is read from
// there for each of its passes; w and b stay in registers.  BITS: the codes of x too.
// Bound by HBM: 8192 x 4096 BF16 23 us (5.8 TB/s), 4096 x 4096 FP32 22 us (6.1 TB/s).  In
// parts by the exchange, which a step's results wait for: 4096 x 8192 31 us, 2048 x 16384
// 32 us (4.3 and 4.2 TB/s).  With 4-bit codes 8192 x 4096 takes 36 us (4.2 TB/s): half as
// many instructions more (a quotient, a rounding and a field for each element) and 120
// registers, which leave 16 warps an SM; neither HBM (34%) nor issue (62%) is full.
template <int DT>
constexpr int kRows = DT == kF32 ? 1 : 2;
constexpr int kRing = 4;                     // stages

template <int DT, int BITS, bool SPLIT>
__global__ void __launch_bounds__(256, BITS ? 2 : 3)
ln_forward_rows_kernel(const LnForward a, int size, int part) {
    constexpr int V = Elem<DT>::kVec, F = 16, NV = F / V, P = V / 2, R = kRows<DT>;
    constexpr int kStages = kRing;
    extern __shared__ __align__(16) uint4 ring[];
    __shared__ __align__(16) float red[kMaxGroups][2][2 * R * kRed];
    __shared__ float box1[2][kMaxParts * 2 * R], box2[2][kMaxParts * R];
    const Group g(size);
    const Columns c = columns_of<SPLIT>(a.H, part);
    const int vectors = c.n / V, groups = SPLIT ? 1 : blockDim.x / size;
    const int64_t step = (int64_t)c.units * groups * R;
    const float inv = __frcp_rn((float)a.H);
    float (*const mine)[2 * R * kRed] = red[size > 32 ? g.id : 0];
    for (int i = threadIdx.x; i < kMaxGroups * 4 * R * kRed; i += blockDim.x) (&red[0][0][0])[i] = 0.0f;
    __syncthreads();
    // slot i of row r of stage s: shared + s * stage_bytes + (r * NV + i) * slot_bytes
    const uint32_t shared = shared_address(ring + threadIdx.x);
    const uint32_t slot_bytes = blockDim.x * 16, stage_bytes = R * NV * slot_bytes;
    bool in[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        in[i] = place<DT>(g, i) < vectors;
        if (in[i]) continue;
        // beyond the row's end: zeros that no copy overwrites
        for (int k = 0; k < kStages * R; ++k)
            store_shared(shared + (k * NV + i) * slot_bytes, make_uint4(0, 0, 0, 0));
    }
    const int64_t first = (int64_t)c.unit * groups * R;          // of the CTA
    begin<SPLIT>();
    // the next rows to copy, and their pointer
    int64_t tf = first + g.id * R;
    const int64_t x_row = a.ldx * Elem<DT>::kSize, y_row = a.ldy * Elem<DT>::kSize;
    const char *xf = elem_at<DT>(a.x, tf * a.ldx + c.first);
    uint32_t into = shared;
    auto fetch = [&]() {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (tf + r >= a.T) break;
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (in[i])
                    copy16(into + (r * NV + i) * slot_bytes, xf + r * x_row + place<DT>(g, i) * 16);
        }
        copies_commit();
        tf += step;
        xf += step * x_row;
        into = into == shared + (kStages - 1) * stage_bytes ? shared : into + stage_bytes;
    };
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) fetch();
    uint64_t w[F / 2], b[F / 2];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int j = c.first / V + (in[i] ? place<DT>(g, i) : 0);
        load_params<DT>(a.w, a.param_f32, j, 1.0f, w + i * P);
        load_params<DT>(a.b, a.param_f32, j, 0.0f, b + i * P);
    }
    uint32_t from = shared;
    int half = 0, turn1 = 0, turn2 = 0;
    char *out = elem_at<DT>(a.y, (first + g.id * R) * a.ldy + c.first);
    for (int64_t t0 = first; t0 < a.T; t0 += step) {
        const int64_t t = t0 + g.id * R;
        copies_left<kStages - 2>();
        // the row's vector i (beyond T: whatever the slot holds; nothing of it is kept)
        auto load = [&](int r, int i) { return load_shared(from + (r * NV + i) * slot_bytes); };
        bool row[R];
#pragma unroll
        for (int r = 0; r < R; ++r) row[r] = t + r < a.T;
        float s[2 * R], mu[R], var[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f}, squares[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const uint4 v = load(r, i);
                add_elems<DT>(v, sum);
                add_squares<DT>(v, squares);
            }
            s[2 * r] = __fadd_rn(__fadd_rn(sum[0], sum[1]), __fadd_rn(sum[2], sum[3]));
            s[2 * r + 1] = __fadd_rn(__fadd_rn(squares[0], squares[1]), __fadd_rn(squares[2], squares[3]));
        }
        fetch();
        row_sums(s, mine[half], g);
        half ^= 1;
        if constexpr (SPLIT) parts_sums(s, box1, turn1, c);
        // A row takes the second pass for its own moments alone: what shares a step or a warp
        // with it may cost time, but not bits, and slots of rows beyond T (an earlier row's, or
        // never written) count for nothing.  The same for all threads of a group.
        bool stand[R], none = true;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            stand[r] = moments(s[2 * r], s[2 * r + 1], inv, mu[r], var[r]) || !row[r];
            none &= stand[r];
        }
        if (__any_sync(0xFFFFFFFFu, !none)) {
            float q[R];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                uint64_t q0 = 0, q1 = 0;
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    uint64_t d[P];
                    differences<DT>(load(r, i), mu[r], d);
                    if (!in[i]) continue;
#pragma unroll
                    for (int k = 0; k < P; k += 2) {
                        q0 = fma_f32x2(d[k], d[k], q0);
                        q1 = fma_f32x2(d[k + 1], d[k + 1], q1);
                    }
                }
                q[r] = __fadd_rn(sum_pair(q0), sum_pair(q1));
            }
            row_sums(q, mine[half], g);
            half ^= 1;
            if constexpr (SPLIT) parts_sums(q, box2, turn2, c);
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (!stand[r]) var[r] = __fmul_rn(q[r], inv);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float rs = inv_sqrt(__fadd_rn(var[r], a.eps));
            const uint64_t r2 = f32x2(rs, rs);
            uint4 v[NV];
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                v[i] = load(r, i);
                if (!row[r] || !in[i]) continue;
                uint64_t y[P];
                differences<DT>(v[i], mu[r], y);
#pragma unroll
                for (int k = 0; k < P; ++k)
                    y[k] = fma_f32x2(mul_f32x2(y[k], r2), w[i * P + k], b[i * P + k]);
                *reinterpret_cast<uint4 *>(out + r * y_row + place<DT>(g, i) * 16) = pack2<DT>(y);
            }
            if constexpr (BITS != 0) {
#pragma unroll
                for (int i = 0; i < NV; i += 2) {
                    const int64_t blk = (t + r) * (a.H / kBlock) + c.first / kBlock + place<DT>(g, i) / 16;
                    quantize_octet<BITS>(v[i], v[i + 1],
                                         static_cast<uint32_t *>(a.codes) + blk * 4 * BITS,
                                         a.scales + blk, row[r] && in[i]);
                }
            }
            if (g.tid == 0 && c.rank == 0 && row[r]) {
                if (a.mean) a.mean[t + r] = mu[r];
                if (a.rstd) a.rstd[t + r] = rs;
            }
        }
        out += step * y_row;
        from = from == shared + (kStages - 1) * stage_bytes ? shared : from + stage_bytes;
    }
    end_rows<SPLIT>();
}

// ---- rows of any alignment ------------------------------------------------------

// A row of H elements in shared memory as it lies in global memory: vector j at the
// 16-byte boundary before the row's start plus 16 j.
template <int DT>
struct RowCopy {
    using Word = typename Elem<DT>::Word;
    const Word *row;
    int H, skip, from, to, n;     // vectors [from, to) are whole, n in all
    __device__ __forceinline__ RowCopy(const void *row_, int H_)
        : row(static_cast<const Word *>(row_)), H(H_) {
        constexpr int V = Elem<DT>::kVec;
        skip = (int)(reinterpret_cast<uintptr_t>(row_) & 15u) / Elem<DT>::kSize;
        n = (H + skip + V - 1) / V;
        from = skip ? 1 : 0;
        to = max((H + skip) / V, from);
    }
    __device__ __forceinline__ void copy(uint4 *to_shared) const {
        const uint4 *vec = reinterpret_cast<const uint4 *>(row - skip);
        for (int j = from + threadIdx.x; j < to; j += blockDim.x) copy16(to_shared + j, vec + j);
    }
    // The elements in vectors that the row fills in part, at most 16: the i-th's
    // index, or -1.
    __device__ __forceinline__ int edge(int i) const {
        constexpr int V = Elem<DT>::kVec;
        const int head = min(H, from * V - (from ? skip : 0)), tail = max(head, to * V - skip);
        const int e = i < head ? i : tail + i - head;
        return e < H ? e : -1;
    }
};

// The rows of one tensor through a ring of shared memory.  The few elements outside
// whole vectors take a register on their way: loaded with the row's copies and stored
// a row later, so that nothing waits for them.
template <int DT, int STAGES>
struct RowRing {
    using Word = typename Elem<DT>::Word;
    const void *p;
    int64_t ld, T, step;
    int H, vectors;               // of a stage
    uint4 *ring;
    Word held = Word(0);
    int held_at = -1;             // word of the ring where it belongs
    __device__ __forceinline__ void fetch(int64_t t, int stage) {
        settle();
        if (t >= T) return;
        const RowCopy<DT> r(elem_at<DT>(p, t * ld), H);
        r.copy(ring + stage * vectors);
        const int e = threadIdx.x < 16 ? r.edge(threadIdx.x) : -1;
        if (e >= 0) {
            held = r.row[e];
            held_at = stage * vectors * Elem<DT>::kVec + r.skip + e;
        }
    }
    __device__ __forceinline__ void settle() {
        if (held_at >= 0) reinterpret_cast<Word *>(ring)[held_at] = held;
        held_at = -1;
    }
    // The words of row t, which is in `stage`.
    __device__ __forceinline__ const Word *row(int64_t t, int stage) const {
        const int skip = (int)(reinterpret_cast<uintptr_t>(elem_at<DT>(p, t * ld)) & 15u) /
                         Elem<DT>::kSize;
        return reinterpret_cast<const Word *>(ring + stage * vectors) + skip;
    }
};
constexpr int kAnyStages = 3;

// Vectors of a row of H elements that may start anywhere in one.
template <int DT>
__host__ __device__ constexpr int row_slots(int H) {
    return (H + 2 * Elem<DT>::kVec - 2) / Elem<DT>::kVec;
}

// A tensor's rows in the layout of RowCopy: what of it does not change from one row of
// a CTA to the next, because the CTA's rows are a multiple of eight apart.
template <int DT>
struct Place {
    int skip, from, to, n;
    __device__ __forceinline__ Place(const void *row, int H) {
        const RowCopy<DT> r(row, H);
        skip = r.skip, from = r.from, to = r.to, n = r.n;
    }
    // Whether vector j is filled by the row in part, or not at all.
    __device__ __forceinline__ bool part(int j) const { return j < from || j >= to; }
    // Vector j with zeros where the row has no element.
    __device__ __forceinline__ uint4 masked(uint4 v, int j, int H) const {
        constexpr int V = Elem<DT>::kVec;
        typename Elem<DT>::Word e[V];
        __builtin_memcpy(e, &v, 16);
#pragma unroll
        for (int k = 0; k < V; ++k)
            if (j * V - skip + k < 0 || j * V - skip + k >= H) e[k] = 0;
        __builtin_memcpy(&v, e, 16);
        return v;
    }
};

// Writes a row that lies in `mine` in the layout of `in` to `out`, whose boundaries lie
// elsewhere (or, `level`, only its elements in vectors that it fills in part).
template <int DT>
__device__ __forceinline__ void write_any(typename Elem<DT>::Word *out, const Place<DT> &o,
                                          const Place<DT> &in, const uint4 *mine, int H) {
    using Word = typename Elem<DT>::Word;
    constexpr int V = Elem<DT>::kVec;
    if (o.skip != in.skip) {
        uint4 *ovec = reinterpret_cast<uint4 *>(out - o.skip);
        const int shift = ((in.skip - o.skip + V) & (V - 1)) * Elem<DT>::kSize;
        const uint4 *from = mine - (in.skip < o.skip);
        for (int j = o.from + threadIdx.x; j < o.to; j += blockDim.x)
            ovec[j] = bytes_from(from[j], from[j + 1], shift);
    }
    const int e = threadIdx.x < 16 ? RowCopy<DT>(out, H).edge(threadIdx.x) : -1;
    if (e >= 0) out[e] = reinterpret_cast<const Word *>(mine)[in.skip + e];
}

// A CTA a row and step, NV vectors a thread, whatever the alignment of x and y: the row
// is copied in vectors at its own 16-byte boundaries and written in vectors at those of
// y, with shared memory in between where they differ.  The CTAs' steps are multiples of
// eight rows, so that all rows of a CTA start at the same place between boundaries and a
// thread's weights stay in registers.  6151 x 5003 FP16: 36 us (3.4 TB/s); what bounds it
// are the instructions (issue 56%) and the two barriers that a row takes to pass through
// shared memory.
template <int DT, int NV, bool SPLIT>
__global__ void __launch_bounds__(512) ln_forward_any_kernel(const LnForward a, int part) {
    using E = Elem<DT>;
    using Word = typename E::Word;
    constexpr int V = E::kVec, P = V / 2, F = NV * V;
    extern __shared__ __align__(16) uint4 ring[];
    __shared__ __align__(16) float red[2][2 * kRed];
    const Group g(blockDim.x);
    __shared__ float box1[2][kMaxParts * 2], box2[2][kMaxParts];
    const Columns c = columns_of<SPLIT>(a.H, part);
    const int threads = blockDim.x, tid = threadIdx.x, H = c.n, vectors = row_slots<DT>(H);
    const float inv = __frcp_rn((float)a.H);
    const int64_t step = c.units, first = c.unit;
    for (int i = tid; i < 4 * kRed; i += threads) (&red[0][0])[i] = 0.0f;
    RowRing<DT, kAnyStages> x{elem_at<DT>(a.x, c.first), a.ldx, a.T, step, H, vectors, ring};
    uint4 *staged = ring + kAnyStages * vectors;                  // two rows of y
    Word *out = reinterpret_cast<Word *>(elem_at<DT>(a.y, first * a.ldy + c.first));
    const Place<DT> in(elem_at<DT>(x.p, first * a.ldx), H), o(out, H);
    const bool level = o.skip == in.skip;
    begin<SPLIT>();
#pragma unroll
    for (int s = 0; s < kAnyStages - 1; ++s) {
        x.fetch(first + s * step, s);
        copies_commit();
    }
    uint64_t w[F / 2], b[F / 2];
#pragma unroll
    for (int i = 0; i < F; i += 2) {
        float f[4];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int e = (tid + i / V * threads) * V - in.skip + i % V + k;
            const bool has = e >= 0 && e < H;
            f[k] = has ? param<DT>(a.w, a.param_f32, c.first + e, 1.0f) : 0.0f;
            f[2 + k] = has ? param<DT>(a.b, a.param_f32, c.first + e, 0.0f) : 0.0f;
        }
        w[i / 2] = f32x2(f[0], f[1]);
        b[i / 2] = f32x2(f[2], f[3]);
    }
    int stage = 0, half = 0, turn1 = 0, turn2 = 0;
    for (int64_t t = first; t < a.T; t += step) {
        copies_left<kAnyStages - 2>();
        x.settle();
        __syncthreads();                                          // the row is complete
        x.fetch(t + (kAnyStages - 1) * step, stage == 0 ? kAnyStages - 1 : stage - 1);
        copies_commit();
        const uint4 *data = ring + stage * vectors;
        stage = stage + 1 == kAnyStages ? 0 : stage + 1;
        uint4 v[NV];
        float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f}, squares[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = tid + i * threads;
            v[i] = make_uint4(0, 0, 0, 0);
            if (j < in.n) v[i] = data[j];
            if (in.part(j)) v[i] = in.masked(v[i], j, H);
            add_elems<DT>(v[i], sum);
            add_squares<DT>(v[i], squares);
        }
        float s[2] = {__fadd_rn(__fadd_rn(sum[0], sum[1]), __fadd_rn(sum[2], sum[3])),
                      __fadd_rn(__fadd_rn(squares[0], squares[1]), __fadd_rn(squares[2], squares[3]))};
        row_sums(s, red[0], g);
        if constexpr (SPLIT) parts_sums(s, box1, turn1, c);
        float mu, var;
        if (!moments(s[0], s[1], inv, mu, var)) {                 // the same for all threads
            uint64_t q0 = 0;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int j = tid + i * threads;
                uint64_t d[P];
                differences<DT>(v[i], mu, d);
#pragma unroll
                for (int k = 0; k < P; ++k) {
                    const int e = j * V - in.skip + 2 * k;
                    if (in.part(j))
                        d[k] = f32x2(e >= 0 && e < H ? lo_f32(d[k]) : 0.0f,
                                     e + 1 >= 0 && e + 1 < H ? hi_f32(d[k]) : 0.0f);
                    q0 = fma_f32x2(d[k], d[k], q0);
                }
            }
            float q[1] = {sum_pair(q0)};
            row_sums(q, red[1], g);
            if constexpr (SPLIT) parts_sums(q, box2, turn2, c);
            var = __fmul_rn(q[0], inv);
        }
        const float r = inv_sqrt(__fadd_rn(var, a.eps));
        const uint64_t r2 = f32x2(r, r);
        uint4 *mine = staged + half * vectors;
        half ^= 1;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = tid + i * threads;
            if (j >= in.n) continue;
            uint64_t y[P];
            differences<DT>(v[i], mu, y);
#pragma unroll
            for (int k = 0; k < P; ++k)
                y[k] = fma_f32x2(mul_f32x2(y[k], r2), w[i * P + k], b[i * P + k]);
            const uint4 packed = pack2<DT>(y);
            if (level && !in.part(j)) reinterpret_cast<uint4 *>(out - o.skip)[j] = packed;
            else mine[j] = packed;
        }
        __syncthreads();
        write_any<DT>(out, o, in, mine, H);
        out += step * a.ldy;
        if (tid == 0 && c.rank == 0) {
            if (a.mean) a.mean[t] = mu;
            if (a.rstd) a.rstd[t] = r;
        }
    }
    end_rows<SPLIT>();
}

// The codes of x on their own (rows that the kernels above do not quantize): an octet
// of lanes a block, any row distance.
template <int BITS>
__global__ void __launch_bounds__(kThreads) ln_codes_kernel(const void *__restrict__ x, int64_t ldx,
                                                            int64_t T, int64_t H,
                                                            uint32_t *__restrict__ codes,
                                                            float *__restrict__ scales) {
    pdl_wait_and_release();
    const int64_t per_row = H / kBlock, blocks = T * per_row;
    const int j = threadIdx.x & 7;
    const int64_t stride = (int64_t)gridDim.x * (kThreads / 8);
    // every lane of a warp takes the same number of steps
    for (int64_t b0 = (int64_t)blockIdx.x * (kThreads / 8) + (threadIdx.x >> 5) * 4; b0 < blocks;
         b0 += stride) {
        const int64_t blk = b0 + ((threadIdx.x >> 3) & 3);
        const bool valid = blk < blocks;
        uint32_t v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (valid) {
            const uint16_t *p = static_cast<const uint16_t *>(x) + (blk / per_row) * ldx +
                                (blk % per_row) * kBlock + 8 * j;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int e = 2 * i + (i >= 4 ? 56 : 0);
                v[i] = (uint32_t)__ldg(p + e) | ((uint32_t)__ldg(p + e + 1) << 16);
            }
        }
        quantize_octet<BITS>(make_uint4(v[0], v[1], v[2], v[3]), make_uint4(v[4], v[5], v[6], v[7]),
                             codes + blk * 4 * BITS, scales + blk, valid);
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
// x and dy read once, dx written once; R rows a group and step, whose sums share the
// exchanges and the barrier.  The rows are unpacked twice from the ring, once for the
// sums and once for the results: that costs less than the registers that would hold
// them.  A thread adds its columns' terms of dw and db in registers over all rows of
// its group; the groups of a CTA join theirs in order, and the CTA writes one row of the
// partial sums ([grid][2][H]).
// 8192 x 4096 BF16: 40 us, and 2 us for the join (4.7 TB/s); from 4-bit codes 46 us.  HBM
// would allow 30 us: w, dw and db of 16 columns take 48 of a thread's 128 registers, so 16
// warps an SM hide what they can (issue 52% and 63%, 23 and 32 million instructions).
// In parts 2048 x 12288 BF16 51 us, 1024 x 16384 FP32 49 us (3.0 and 4.1 TB/s), which the
// exchange bounds.
template <int DT>
constexpr int kBackRows = DT == kF32 ? 1 : 2;
constexpr int kBackStages = 3;

template <int DT, int BITS, bool SPLIT>
__global__ void __launch_bounds__(512) ln_backward_rows_kernel(const LnBackward a, int size, int part) {
    using E = Elem<DT>;
    constexpr int V = E::kVec, F = 16, NV = F / V, P = V / 2, R = kBackRows<DT>;
    constexpr int kStages = kBackStages, kWords = 4 * BITS;
    constexpr int kParts = BITS ? 1 : 2;             // dy, and x
    extern __shared__ __align__(16) uint4 ring[];
    constexpr int kSums = BITS ? 4 : 2;              // of a row
    __shared__ __align__(16) float red[kMaxGroups][2][kSums * R * kRed];
    __shared__ float box1[2][kMaxParts * kSums * R], box2[2][kMaxParts * 2 * R];
    const Group g(size);
    const Columns c = columns_of<SPLIT>(a.H, part);
    const int threads = blockDim.x, vectors = c.n / V, groups = SPLIT ? 1 : threads / size;
    const int64_t step = (int64_t)c.units * groups * R;
    const float inv = __frcp_rn((float)a.H);
    float (*const mine)[kSums * R * kRed] = red[size > 32 ? g.id : 0];
    for (int i = threadIdx.x; i < kMaxGroups * 2 * kSums * R * kRed; i += threads)
        (&red[0][0][0])[i] = 0.0f;
    __syncthreads();
    // slot i of part p of row r of stage s: shared + s * stage_bytes +
    // ((r * kParts + p) * NV + i) * slot_bytes
    const uint32_t shared = shared_address(ring + threadIdx.x);
    const uint32_t slot_bytes = threads * 16, stage_bytes = R * kParts * NV * slot_bytes;
    bool in[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        in[i] = place<DT>(g, i) < vectors;
        if (in[i]) continue;
        // beyond the row's end: zeros that no copy overwrites
        for (int k = 0; k < kStages * R * kParts; ++k)
            store_shared(shared + (k * NV + i) * slot_bytes, make_uint4(0, 0, 0, 0));
    }
    begin<SPLIT>();
    const int64_t first = (int64_t)c.unit * groups * R;          // of the CTA
    // the next rows to copy, and their pointers
    int64_t tf = first + g.id * R;
    const char *dyf = elem_at<DT>(a.dy, tf * a.lddy + c.first);
    const char *xf = BITS ? nullptr : elem_at<DT>(a.x, tf * a.ldx + c.first);
    const int64_t dy_row = a.lddy * E::kSize, x_row = a.ldx * E::kSize;
    uint32_t into = shared;
    auto fetch = [&]() {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (tf + r >= a.T) break;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (in[i]) {
                    copy16(into + (r * kParts * NV + i) * slot_bytes,
                           dyf + r * dy_row + place<DT>(g, i) * 16);
                    if constexpr (BITS == 0)
                        copy16(into + ((r * kParts + 1) * NV + i) * slot_bytes,
                               xf + r * x_row + place<DT>(g, i) * 16);
                }
            }
        }
        copies_commit();
        tf += step;
        dyf += step * dy_row;
        if constexpr (BITS == 0) xf += step * x_row;
        into = into == shared + (kStages - 1) * stage_bytes ? shared : into + stage_bytes;
    };
    // what does not come in 16-byte copies is loaded a step ahead into registers
    uint32_t lo[R][2], hi[R][2];
    float scale[R], mean[R], rstd[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        scale[r] = mean[r] = rstd[r] = 0.0f;
        lo[r][0] = lo[r][1] = hi[r][0] = hi[r][1] = 0;
    }
    auto ahead = [&](int64_t t) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (t + r >= a.T) return;
            if constexpr (BITS == 0) {
                mean[r] = __ldg(a.mean + t + r);
                rstd[r] = __ldg(a.rstd + t + r);
            } else {
                const int j = place<DT>(g, 0);           // the octet's block
                if (!in[0]) return;
                const int64_t blk = (t + r) * (a.H / kBlock) + c.first / kBlock + j / 16;
                const uint32_t *rec = static_cast<const uint32_t *>(a.x) + blk * kWords;
                load_chunk<BITS>(rec, j & 7, lo[r][0], hi[r][0]);
                load_chunk<BITS>(rec, (j & 7) + 8, lo[r][1], hi[r][1]);
                scale[r] = __ldg(a.scales + blk);
            }
        }
    };
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) fetch();
    ahead(first + g.id * R);
    uint64_t w[F / 2], dw[F / 2], db[F / 2];
#pragma unroll
    for (int i = 0; i < NV; ++i)
        load_params<DT>(a.w, a.param_f32, c.first / V + (in[i] ? place<DT>(g, i) : 0), 1.0f, w + i * P);
#pragma unroll
    for (int i = 0; i < F / 2; ++i) dw[i] = db[i] = 0;
    uint32_t from = shared;
    int half = 0, turn1 = 0, turn2 = 0;
    char *out = elem_at<DT>(a.dx, (first + g.id * R) * a.lddx + c.first);
    const int64_t dx_row = a.lddx * E::kSize;
    for (int64_t t0 = first; t0 < a.T; t0 += step) {
        const int64_t t = t0 + g.id * R;
        copies_left<kStages - 2>();
        float mu[R], rs[R], s0[R], s1[R];
        uint4 vx[R][NV];                  // of codes: the dequantized row
        // the row's vector i of dy and x (beyond T: of an earlier row; nothing of it is kept)
        auto load = [&](int r, int i, uint4 &d, uint4 &x) {
            d = load_shared(from + (r * kParts * NV + i) * slot_bytes);
            if constexpr (BITS == 0) x = load_shared(from + ((r * kParts + 1) * NV + i) * slot_bytes);
            else x = vx[r][i];
        };
        bool row[R];
#pragma unroll
        for (int r = 0; r < R; ++r) row[r] = t + r < a.T;
        if constexpr (BITS != 0) {
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    vx[r][i] = dequantize_chunk<BITS>(lo[r][i & 1], hi[r][i & 1], scale[r]);
        }
        // of a row: sum g and sum g xh; of codes sum g, sum g x, sum x and sum x^2
        float s[kSums * R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            mu[r] = mean[r];
            rs[r] = rstd[r];
            const uint64_t r2 = f32x2(rs[r], rs[r]);
            uint64_t g0 = 0, g1 = 0;
            float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f}, squares[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                uint4 vd, v;
                uint64_t d[P], x[P];
                load(r, i, vd, v);
                unpack2<DT>(vd, d);
                if constexpr (BITS == 0) {
                    differences<DT>(v, mu[r], x);
                } else {
                    unpack2<DT>(v, x);
                    add_elems<DT>(v, sum);
                    add_squares<DT>(v, squares);
                }
#pragma unroll
                for (int k = 0; k < P; ++k) {
                    const uint64_t gk = mul_f32x2(d[k], w[i * P + k]);
                    g0 = add_f32x2(g0, gk);
                    g1 = fma_f32x2(gk, BITS ? x[k] : mul_f32x2(x[k], r2), g1);
                }
            }
            s[kSums * r] = sum_pair(g0);
            s[kSums * r + 1] = sum_pair(g1);
            if constexpr (BITS != 0) {
                s[kSums * r + 2] = __fadd_rn(__fadd_rn(sum[0], sum[1]), __fadd_rn(sum[2], sum[3]));
                s[kSums * r + 3] =
                    __fadd_rn(__fadd_rn(squares[0], squares[1]), __fadd_rn(squares[2], squares[3]));
            }
        }
        fetch();
        ahead(t + step);
        row_sums(s, mine[half], g);
        half ^= 1;
        if constexpr (SPLIT) parts_sums(s, box1, turn1, c);
        bool stand[R], none = true;       // as in the forward pass, of each row by itself
#pragma unroll
        for (int r = 0; r < R; ++r) {
            s0[r] = __fmul_rn(s[kSums * r], inv);
            s1[r] = __fmul_rn(s[kSums * r + 1], inv);
            if constexpr (BITS != 0) {
                // sum g (x - mu) / H; the difference loses no more than the variance's
                float var;
                stand[r] = moments(s[kSums * r + 2], s[kSums * r + 3], inv, mu[r], var) || !row[r];
                none &= stand[r];
                s1[r] = __fmaf_rn(-mu[r], s0[r], s1[r]);
                rs[r] = inv_sqrt(__fadd_rn(var, a.eps));
            }
        }
        if constexpr (BITS != 0) {
            if (__any_sync(0xFFFFFFFFu, !none)) {       // the same for all threads of a group
                float q[2 * R];
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    uint64_t q0 = 0, g1 = 0;
#pragma unroll
                    for (int i = 0; i < NV; ++i) {
                        uint4 vd, v;
                        uint64_t d[P], x[P];
                        load(r, i, vd, v);
                        unpack2<DT>(vd, d);
                        differences<DT>(v, mu[r], x);
                        if (!in[i]) continue;
#pragma unroll
                        for (int k = 0; k < P; ++k) {
                            q0 = fma_f32x2(x[k], x[k], q0);
                            g1 = fma_f32x2(mul_f32x2(d[k], w[i * P + k]), x[k], g1);
                        }
                    }
                    q[2 * r] = sum_pair(q0);
                    q[2 * r + 1] = sum_pair(g1);
                }
                row_sums(q, mine[half], g);
                half ^= 1;
                if constexpr (SPLIT) parts_sums(q, box2, turn2, c);
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    if (stand[r]) continue;
                    rs[r] = inv_sqrt(__fmaf_rn(q[2 * r], inv, a.eps));
                    s1[r] = __fmul_rn(q[2 * r + 1], inv);
                }
            }
#pragma unroll
            for (int r = 0; r < R; ++r) s1[r] = __fmul_rn(s1[r], rs[r]);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const uint64_t r2 = f32x2(rs[r], rs[r]), s02 = f32x2(s0[r], s0[r]),
                           s12 = f32x2(-s1[r], -s1[r]);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (!row[r] || !in[i]) continue;
                uint4 vd, v;
                uint64_t d[P], x[P], o[P];
                load(r, i, vd, v);
                unpack2<DT>(vd, d);
                differences<DT>(v, mu[r], x);
#pragma unroll
                for (int k = 0; k < P; ++k) {
                    const int m = i * P + k;
                    x[k] = mul_f32x2(x[k], r2);
                    o[k] = mul_f32x2(r2, fma_f32x2(x[k], s12, sub_f32x2(mul_f32x2(d[k], w[m]), s02)));
                    dw[m] = fma_f32x2(d[k], x[k], dw[m]);
                    db[m] = add_f32x2(db[m], d[k]);
                }
                *reinterpret_cast<uint4 *>(out + r * dx_row + place<DT>(g, i) * 16) = pack2<DT>(o);
            }
        }
        out += step * dx_row;
        from = from == shared + (kStages - 1) * stage_bytes ? shared : from + stage_bytes;
    }
    end_rows<SPLIT>();
    if (!a.dw && !a.db) return;
    float *partial = a.workspace + (int64_t)c.unit * 2 * a.H + c.first;
    float *joined = reinterpret_cast<float *>(ring);          // [2][H], for several groups
    copies_left<0>();
    // groups of a warp first, then one after another
    for (int o = size; o < 32; o <<= 1) {
#pragma unroll
        for (int i = 0; i < F / 2; ++i) {
            dw[i] = add_f32x2(dw[i], __shfl_xor_sync(0xFFFFFFFFu, dw[i], o));
            db[i] = add_f32x2(db[i], __shfl_xor_sync(0xFFFFFFFFu, db[i], o));
        }
    }
    const int shares = threads / max(size, 32), share = threadIdx.x / max(size, 32);
    for (int who = 0; who < shares; ++who) {
        if (groups > 1) __syncthreads();
        if (share != who || (size < 32 && (threadIdx.x & 31) >= size)) continue;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = place<DT>(g, i);
            if (!in[i]) continue;
            float *pw = (groups > 1 ? joined : partial) + j * V, *pb = pw + a.H;
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const int m = i * P + k / 2;
                const float vw = k & 1 ? hi_f32(dw[m]) : lo_f32(dw[m]);
                const float vb = k & 1 ? hi_f32(db[m]) : lo_f32(db[m]);
                pw[k] = who > 0 ? __fadd_rn(pw[k], vw) : vw;
                pb[k] = who > 0 ? __fadd_rn(pb[k], vb) : vb;
            }
        }
    }
    if (groups > 1) {
        __syncthreads();
        for (int i = threadIdx.x; i < 2 * (int)a.H; i += threads) partial[i] = joined[i];
    }
}

// Rows of any alignment: as the forward pass, x and dy through rings, in the layout of
// dy (x's vectors are cut from two of its own where it lies elsewhere), dx through shared
// memory; dw and db in registers, since a thread's columns stay the same.  6151 x 5003
// BF16 91 us (2.0 TB/s): every element is unpacked twice, cut out of two vectors and
// masked at the row's ends, between three barriers a row.
template <int DT, int LIMIT, bool SPLIT>
__global__ void __launch_bounds__(LIMIT, LIMIT == 320 ? 2 : 1)
ln_backward_any_kernel(const LnBackward a, int part) {
    using E = Elem<DT>;
    using Word = typename E::Word;
    constexpr int V = E::kVec, P = V / 2, F = 16, NV = F / V;
    extern __shared__ __align__(16) uint4 ring[];
    __shared__ __align__(16) float red[2][2 * kRed];
    const Group g(blockDim.x);
    __shared__ float box[2][kMaxParts * 2];
    const Columns c = columns_of<SPLIT>(a.H, part);
    const int threads = blockDim.x, tid = threadIdx.x, H = c.n, vectors = row_slots<DT>(H);
    const float inv = __frcp_rn((float)a.H);
    const int64_t step = c.units, first = c.unit;
    for (int i = tid; i < 4 * kRed; i += threads) (&red[0][0])[i] = 0.0f;
    RowRing<DT, kAnyStages> x{elem_at<DT>(a.x, c.first), a.ldx, a.T, step, H, vectors, ring};
    RowRing<DT, kAnyStages> y{elem_at<DT>(a.dy, c.first), a.lddy, a.T, step, H, vectors,
                              ring + kAnyStages * vectors};
    uint4 *staged = ring + 2 * kAnyStages * vectors;              // two rows of dx
    Word *out = reinterpret_cast<Word *>(elem_at<DT>(a.dx, first * a.lddx + c.first));
    const Place<DT> in(elem_at<DT>(y.p, first * a.lddy), H), ix(elem_at<DT>(x.p, first * a.ldx), H),
        o(out, H);
    const bool level = o.skip == in.skip;
    const int shift = ((ix.skip - in.skip + V) & (V - 1)) * E::kSize, back = ix.skip < in.skip;
    begin<SPLIT>();
#pragma unroll
    for (int s = 0; s < kAnyStages - 1; ++s) {
        x.fetch(first + s * step, s);
        y.fetch(first + s * step, s);
        copies_commit();
    }
    uint64_t w[F / 2], dw[F / 2], db[F / 2];
#pragma unroll
    for (int i = 0; i < F; i += 2) {
        float f[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int e = (tid + i / V * threads) * V - in.skip + i % V + k;
            f[k] = e >= 0 && e < H ? param<DT>(a.w, a.param_f32, c.first + e, 1.0f) : 0.0f;
        }
        w[i / 2] = f32x2(f[0], f[1]);
        dw[i / 2] = db[i / 2] = 0;
    }
    float mean = 0.0f, rstd = 0.0f;
    auto ahead = [&](int64_t t) {
        if (t < a.T) {
            mean = __ldg(a.mean + t);
            rstd = __ldg(a.rstd + t);
        }
    };
    ahead(first);
    int stage = 0, half = 0, turn = 0;
    for (int64_t t = first; t < a.T; t += step) {
        copies_left<kAnyStages - 2>();
        x.settle();
        y.settle();
        __syncthreads();                                          // the rows are complete
        const int into = stage == 0 ? kAnyStages - 1 : stage - 1;
        x.fetch(t + (kAnyStages - 1) * step, into);
        y.fetch(t + (kAnyStages - 1) * step, into);
        copies_commit();
        const float mu = mean, r = rstd;
        ahead(t + step);
        const uint4 *dx = ring + stage * vectors, *dd = dx + kAnyStages * vectors;
        stage = stage + 1 == kAnyStages ? 0 : stage + 1;
        const uint64_t r2 = f32x2(r, r);
        // vector i of dy, and xh: taken from the ring for the sums and again for the results
        auto load = [&](int i, uint64_t *d, uint64_t *xh) {
            const int j = tid + i * threads, k = j - back;
            uint4 vd = make_uint4(0, 0, 0, 0), vx = vd;
            if (j < in.n) {
                vd = dd[j];
                // (beside the row's end one of the two may not be there: masked below)
                if (k >= 0 && k < ix.n) vx = dx[k];
                if (shift) {
                    uint4 next = make_uint4(0, 0, 0, 0);
                    if (k + 1 < ix.n) next = dx[k + 1];
                    vx = bytes_from(vx, next, shift);
                }
            }
            if (in.part(j)) {
                vd = in.masked(vd, j, H);
                vx = in.masked(vx, j, H);
            }
            unpack2<DT>(vd, d);
            differences<DT>(vx, mu, xh);
#pragma unroll
            for (int m = 0; m < P; ++m) xh[m] = mul_f32x2(xh[m], r2);
        };
        uint64_t g0 = 0, g1 = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            uint64_t d[P], xh[P];
            load(i, d, xh);
#pragma unroll
            for (int k = 0; k < P; ++k) {
                const uint64_t gk = mul_f32x2(d[k], w[i * P + k]);
                g0 = add_f32x2(g0, gk);
                g1 = fma_f32x2(gk, xh[k], g1);
            }
        }
        float s[2] = {sum_pair(g0), sum_pair(g1)};
        row_sums(s, red[half], g);
        if constexpr (SPLIT) parts_sums(s, box, turn, c);
        const float s0 = __fmul_rn(s[0], inv), s1 = __fmul_rn(s[1], inv);
        const uint64_t s02 = f32x2(s0, s0), s12 = f32x2(-s1, -s1);
        uint4 *mine = staged + half * vectors;
        half ^= 1;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = tid + i * threads;
            if (j >= in.n) continue;
            uint64_t d[P], xh[P], p[P];
            load(i, d, xh);
#pragma unroll
            for (int k = 0; k < P; ++k) {
                const int m = i * P + k;
                p[k] = mul_f32x2(r2, fma_f32x2(xh[k], s12, sub_f32x2(mul_f32x2(d[k], w[m]), s02)));
                dw[m] = fma_f32x2(d[k], xh[k], dw[m]);
                db[m] = add_f32x2(db[m], d[k]);
            }
            const uint4 packed = pack2<DT>(p);
            if (level && !in.part(j)) reinterpret_cast<uint4 *>(out - o.skip)[j] = packed;
            else mine[j] = packed;
        }
        __syncthreads();
        write_any<DT>(out, o, in, mine, H);
        out += step * a.lddx;
    }
    end_rows<SPLIT>();
    if (!a.dw && !a.db) return;
    float *partial = a.workspace + (int64_t)c.unit * 2 * a.H + c.first;
#pragma unroll
    for (int i = 0; i < F; ++i) {
        const int e = (tid + i / V * threads) * V - in.skip + i % V;
        if (e < 0 || e >= H) continue;
        partial[e] = i & 1 ? hi_f32(dw[i / 2]) : lo_f32(dw[i / 2]);
        partial[a.H + e] = i & 1 ? hi_f32(db[i / 2]) : lo_f32(db[i / 2]);
    }
}

// dw and db: the P partial rows.  A CTA takes 32 columns; its eight warps add every
// eighth row, and their sums are added in order.
template <bool SPLIT>
__global__ void __launch_bounds__(kThreads) ln_backward_join_kernel(
    const float *__restrict__ partials, int64_t H, int P, float *__restrict__ dw,
    float *__restrict__ db) {
    if constexpr (SPLIT) asm volatile("griddepcontrol.wait;" ::: "memory");
    else pdl_wait_and_release();
    __shared__ float sums[kWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int64_t c0 = (int64_t)blockIdx.x * 32; c0 < 2 * H; c0 += (int64_t)gridDim.x * 32) {
        const int64_t i = c0 + lane;
        float *out = i < H ? dw : db;
        float s = 0.0f;
        if (i < 2 * H && out) {
#pragma unroll 19
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
    end_rows<SPLIT>();
}

int grid_for(int64_t units, int per_sm) {
    const int64_t most = (int64_t)sm_count() * per_sm;
    return (int)(units < most ? (units > 0 ? units : 1) : most);
}

bool on16(const void *p, int64_t ld, int size) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * size % 16 == 0;
}

// Threads of a row's group that holds `units` in shares of `per`: 8, 16, or whole warps.
int threads_for(int64_t units, int per) {
    const int64_t t = (units + per - 1) / per;
    return t <= 8 ? 8 : t <= 16 ? 16 : (int)((t + 31) / 32 * 32);
}
// Groups of `size` threads in a CTA: 256 threads, for rows shorter than that.
int groups_of(int size) { return size <= 128 ? 256 / size : 1; }

// CTAs of a kernel whose CTAs stay for many units of work: as many as are resident.
template <typename K>
int resident_ctas(K kernel, int threads, size_t smem, int64_t units) {
    int per_sm = 0;
    cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, smem);
    return grid_for(units, per_sm > 0 ? per_sm : 1);
}

// Most columns of a CTA: what registers hold, 16 elements a thread (32 forward from any
// alignment), and in the kernels for any alignment shared memory (five rows forward,
// eight backward).
constexpr int kForwardRows = 4096, kBackwardRows = 8192;
template <int DT>
constexpr int kForwardAny = DT == kF32 ? 11136 : 16256;
template <int DT>
constexpr int kBackwardAny = DT == kF32 ? 6912 : 8064;
// Beyond that a row is shared by a cluster, in parts of at most as many columns as leave
// room for two or three CTAs an SM (parts of up to 8192 instead of 4096: backward of 2048
// x 12288 54 us, 51 with them; of up to 16256 and 11136 in any alignment: forward of
// 1024 x 16383 46 us, 36 with them; 2000 x 12001 FP32 94 us, 71).  A row that one CTA
// holds is not shared: the cluster's barrier costs more than the room gives (backward
// of 4096 x 8192 55 us, 49 in one; forward of 3000 x 12001 67 us, 49 in one).
constexpr int kForwardPart = 4096, kBackwardPart = 4096;
template <int DT>
constexpr int kAnyPart = DT == kF32 ? 3456 : 4992;

// Long rows: the CTAs of a cluster take parts of `columns` each, a multiple of a block of
// codes (and so of 16 bytes), the last one what is left.
struct Parts {
    int count, columns;
    Parts(int64_t H, int most) {
        count = (int)((H + most - 1) / most);
        columns = (int)((H + count - 1) / count + kBlock - 1) / kBlock * kBlock;
    }
};

// Clusters of a kernel whose CTAs stay: as many as are resident.
template <typename K>
int resident_clusters(K kernel, int threads, size_t smem, int parts, int64_t units) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(parts);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim = {(unsigned)parts, 1, 1};
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1) n = 1;
    return (int)(units < n ? (units > 0 ? units : 1) : n);
}

template <int DT, int BITS>
cudaError_t forward_rows(const LnForward &a, cudaStream_t st) {
    constexpr int NV = 16 / Elem<DT>::kVec, R = kRows<DT>;
    const int size = threads_for(a.H / Elem<DT>::kVec, NV), groups = groups_of(size);
    const int threads = size * groups;
    const size_t smem = (size_t)kRing * R * NV * threads * 16;
    static bool ready[kMaxDevices];
    auto kernel = ln_forward_rows_kernel<DT, BITS, false>;
    const cudaError_t e = allow_shared(kernel, (size_t)kRing * R * NV * 256 * 16, ready);
    if (e != cudaSuccess) return e;
    const int ctas = resident_ctas(kernel, threads, smem, (a.T + groups * R - 1) / (groups * R));
    return launch_pdl_clusters(kernel, ctas, threads, 1, smem, st, a, size, 0);
}

template <int DT, int BITS>
cudaError_t forward_rows_split(const LnForward &a, cudaStream_t st) {
    constexpr int V = Elem<DT>::kVec, NV = 16 / V, R = kRows<DT>;
    const Parts p(a.H, kForwardPart);
    const int threads = threads_for(p.columns / V, NV);
    const size_t smem = (size_t)kRing * R * NV * threads * 16;
    static bool ready[kMaxDevices];
    auto kernel = ln_forward_rows_kernel<DT, BITS, true>;
    const cudaError_t e = allow_shared(kernel, (size_t)kRing * R * NV * 256 * 16, ready);
    if (e != cudaSuccess) return e;
    const int clusters = resident_clusters(kernel, threads, smem, p.count, (a.T + R - 1) / R);
    return launch_pdl_clusters(kernel, clusters * p.count, threads, p.count, smem, st, a, threads,
                               p.columns);
}

// Dynamic shared memory of the kernels for any alignment may reach this.
constexpr size_t kMostShared = 220 * 1024;

// Rows of any alignment, 32 elements a thread (few warps a row: with 16 elements rows of
// 5003 FP16 values took 51 us, with 32 38 us).
template <int DT>
cudaError_t forward_any(const LnForward &a, cudaStream_t st) {
    constexpr int NV = 32 / Elem<DT>::kVec;
    const int slots = row_slots<DT>((int)a.H);
    const int threads = (slots + 32 * NV - 1) / (32 * NV) * 32;
    const size_t smem = (size_t)(kAnyStages + 2) * slots * 16;
    static bool ready[kMaxDevices];
    auto kernel = ln_forward_any_kernel<DT, NV, false>;
    const cudaError_t e = allow_shared(kernel, kMostShared, ready);
    if (e != cudaSuccess) return e;
    const int n = by_eights(resident_ctas(kernel, threads, smem, a.T), a.T, 1 << 20);
    return launch_pdl_clusters(kernel, n, threads, 1, smem, st, a, 0);
}

template <int DT>
cudaError_t forward_any_split(const LnForward &a, cudaStream_t st) {
    constexpr int NV = 32 / Elem<DT>::kVec;
    const Parts p(a.H, kAnyPart<DT>);
    const int slots = row_slots<DT>(p.columns);
    const int threads = (slots + 32 * NV - 1) / (32 * NV) * 32;
    const size_t smem = (size_t)(kAnyStages + 2) * slots * 16;
    static bool ready[kMaxDevices];
    auto kernel = ln_forward_any_kernel<DT, NV, true>;
    const cudaError_t e = allow_shared(kernel, kMostShared, ready);
    if (e != cudaSuccess) return e;
    const int n = by_eights(resident_clusters(kernel, threads, smem, p.count, a.T), a.T, 1 << 20);
    return launch_pdl_clusters(kernel, n * p.count, threads, p.count, smem, st, a, p.columns);
}

// The kernel for the rows: of whole vectors at 16-byte boundaries, of any alignment (each
// in parts where long), else (the longest) element by element.
template <int DT, int BITS>
cudaError_t forward_bits(const LnForward &a, cudaStream_t st) {
    constexpr int V = Elem<DT>::kVec;
    if (on16(a.x, a.ldx, Elem<DT>::kSize) && on16(a.y, a.ldy, Elem<DT>::kSize) && a.H % V == 0) {
        if (a.H <= kForwardRows) return forward_rows<DT, BITS>(a, st);
        if (a.H <= kMaxParts * kForwardPart) return forward_rows_split<DT, BITS>(a, st);
    }
    if (a.H <= kForwardAny<DT>) return forward_any<DT>(a, st);
    if (a.H <= kMaxParts * kAnyPart<DT>) return forward_any_split<DT>(a, st);
    return launch_pdl(ln_forward_kernel<DT>, grid_for(a.T, 8), kThreads, 0, st, a.x, a.ldx, a.w, a.b,
                      a.param_f32, a.T, a.H, a.eps, a.y, a.ldy, a.mean, a.rstd);
}

// Where dw or db is wanted, the partial sums of P CTAs become dw and db.
template <bool SPLIT = false>
cudaError_t join(const LnBackward &a, int P, cudaStream_t st) {
    if (!a.dw && !a.db) return cudaSuccess;
    return launch_pdl(ln_backward_join_kernel<SPLIT>, grid_for((2 * a.H + 31) / 32, 8), kThreads, 0, st,
                      a.workspace, a.H, P, a.dw, a.db);
}

template <int DT, int BITS>
cudaError_t backward_rows(const LnBackward &a, cudaStream_t st) {
    constexpr int NV = 16 / Elem<DT>::kVec, R = kBackRows<DT>;
    // Rows of more than 128 threads pair up in a CTA, for half as many partial sums (8192 x
    // 4096: 42 us, 46 us alone), and CTAs of rows of less than a warp are as large
    // (262144 x 128: 52 us, 64 us with 256 threads; 32768 x 1024: 47 us, 42 us with 256).
    const int size = threads_for(a.H / Elem<DT>::kVec, NV);
    const int groups = size > 256 ? 1 : (size > 128 || size < 32 ? 512 : 256) / size;
    const int threads = size * groups;
    constexpr int kSlots = kBackStages * R * NV * (BITS ? 1 : 2);
    const size_t smem = (size_t)kSlots * threads * 16;
    static bool ready[kMaxDevices];
    auto kernel = ln_backward_rows_kernel<DT, BITS, false>;
    const cudaError_t e = allow_shared(kernel, (size_t)kSlots * 512 * 16, ready);
    if (e != cudaSuccess) return e;
    int P = resident_ctas(kernel, threads, smem, (a.T + groups * R - 1) / (groups * R));
    if (P > ln_partials(a.T, a.H)) P = ln_partials(a.T, a.H);
    const cudaError_t r = launch_pdl_clusters(kernel, P, threads, 1, smem, st, a, size, 0);
    return r != cudaSuccess ? r : join(a, P, st);
}

template <int DT, int BITS>
cudaError_t backward_rows_split(const LnBackward &a, cudaStream_t st) {
    constexpr int V = Elem<DT>::kVec, NV = 16 / V, R = kBackRows<DT>;
    const Parts p(a.H, kBackwardPart);
    const int threads = threads_for(p.columns / V, NV);
    constexpr int kSlots = kBackStages * R * NV * (BITS ? 1 : 2);
    const size_t smem = (size_t)kSlots * threads * 16;
    static bool ready[kMaxDevices];
    auto kernel = ln_backward_rows_kernel<DT, BITS, true>;
    const cudaError_t e = allow_shared(kernel, (size_t)kSlots * 256 * 16, ready);
    if (e != cudaSuccess) return e;
    int P = resident_clusters(kernel, threads, smem, p.count, (a.T + R - 1) / R);
    if (P > ln_partials(a.T, a.H)) P = ln_partials(a.T, a.H);
    const cudaError_t r =
        launch_pdl_clusters(kernel, P * p.count, threads, p.count, smem, st, a, threads, p.columns);
    return r != cudaSuccess ? r : join<true>(a, P, st);
}

template <int DT, int LIMIT>
cudaError_t backward_any(const LnBackward &a, cudaStream_t st) {
    constexpr int NV = 16 / Elem<DT>::kVec;
    const int slots = row_slots<DT>((int)a.H);
    const int threads = (slots + 32 * NV - 1) / (32 * NV) * 32;
    const size_t smem = (size_t)(2 * kAnyStages + 2) * slots * 16;
    static bool ready[kMaxDevices];
    auto kernel = ln_backward_any_kernel<DT, LIMIT, false>;
    const cudaError_t e = allow_shared(kernel, kMostShared, ready);
    if (e != cudaSuccess) return e;
    const int P = by_eights(resident_ctas(kernel, threads, smem, a.T), a.T, ln_partials(a.T, a.H));
    const cudaError_t r = launch_pdl_clusters(kernel, P, threads, 1, smem, st, a, 0);
    return r != cudaSuccess ? r : join(a, P, st);
}

template <int DT>
cudaError_t backward_any_split(const LnBackward &a, cudaStream_t st) {
    constexpr int NV = 16 / Elem<DT>::kVec;
    const Parts p(a.H, kAnyPart<DT>);
    const int slots = row_slots<DT>(p.columns);
    const int threads = (slots + 32 * NV - 1) / (32 * NV) * 32;
    const size_t smem = (size_t)(2 * kAnyStages + 2) * slots * 16;
    static bool ready[kMaxDevices];
    auto kernel = ln_backward_any_kernel<DT, 320, true>;
    const cudaError_t e = allow_shared(kernel, kMostShared, ready);
    if (e != cudaSuccess) return e;
    const int P = by_eights(resident_clusters(kernel, threads, smem, p.count, a.T), a.T,
                            ln_partials(a.T, a.H));
    const cudaError_t r = launch_pdl_clusters(kernel, P * p.count, threads, p.count, smem, st, a, p.columns);
    return r != cudaSuccess ? r : join<true>(a, P, st);
}

// As the forward pass; any alignment from a tensor only (from codes with rows of dy 4099
// elements apart 8192 x 4096 takes 430 us element by element, 48 us aligned).
template <int DT, int BITS>
cudaError_t backward(const Input<DT, BITS> &in, const LnBackward &a, cudaStream_t st) {
    constexpr int kSize = Elem<DT>::kSize, V = Elem<DT>::kVec;
    if ((BITS || on16(a.x, a.ldx, kSize)) && on16(a.dy, a.lddy, kSize) && on16(a.dx, a.lddx, kSize) &&
        a.H % V == 0) {
        if (a.H <= kBackwardRows) return backward_rows<DT, BITS>(a, st);
        if (a.H <= kMaxParts * kBackwardPart) return backward_rows_split<DT, BITS>(a, st);
    }
    if constexpr (BITS == 0) {
        // (rows of up to 4992 leave registers for two CTAs an SM)
        if (a.H <= 4992) return backward_any<DT, 320>(a, st);
        if (a.H <= kBackwardAny<DT>) return backward_any<DT, 512>(a, st);
        if (a.H <= kMaxParts * kAnyPart<DT>) return backward_any_split<DT>(a, st);
    }
    const bool sums = a.dw || a.db;
    const int P = sums ? ln_partials(a.T, a.H) : grid_for(a.T, 8);
    const cudaError_t e = launch_pdl(ln_backward_kernel<DT, BITS>, P, kThreads, 0, st, in, a.dy,
                                     a.lddy, a.w, a.param_f32, a.mean, a.rstd, a.T, a.H, a.eps,
                                     a.dx, a.lddx, sums ? a.workspace : nullptr);
    return e != cudaSuccess ? e : join(a, P, st);
}

template <int BITS>
cudaError_t codes(const LnForward &a, cudaStream_t st) {
    const int64_t blocks = a.T * (a.H / kBlock);
    return launch_pdl(ln_codes_kernel<BITS>, grid_for((blocks + 31) / 32, 8), kThreads, 0, st, a.x,
                      a.ldx, a.T, a.H, static_cast<uint32_t *>(a.codes), a.scales);
}

}  // namespace

cudaError_t launch_ln_forward(const LnForward &a, cudaStream_t st) {
    if (a.dtype == kF32) return forward_bits<kF32, 0>(a, st);
    if (a.dtype == kF16) return forward_bits<kF16, 0>(a, st);
    if (!a.codes) return forward_bits<kBF16, 0>(a, st);
    // y may be x's place: rows that the norm does not quantize are quantized first
    const bool rows = on16(a.x, a.ldx, 2) && on16(a.y, a.ldy, 2) && a.H <= kMaxParts * kForwardPart;
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
