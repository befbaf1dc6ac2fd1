// grad_norm.cu -- the global L2 norm of many gradients at once, and their
// clipping to a norm: FP32, BF16 and FP16 tensors, and the FP8 master gradients
// with block scales ("AGoQ: Activation and Gradient Quantization for
// Memory-Efficient Distributed Training of LLMs", section 2.B), whose clipping
// only multiplies the scales.
//
//   norm = sqrt(sum g^2),  c = min(1, max_norm / (norm + 1e-6)),  g' = R(g c)
//
// Every tensor is cut into chunks of 2048 aligned 16-byte vectors; the CTAs of one
// launch take the chunks of all tensors in turn, a thread loading the eight
// vectors of its part before it uses the first.  The list travels in the kernel's
// parameters (at most kList tensors a launch), so a call copies nothing to the
// device and can be captured in a graph.
//
// Sums: a thread adds the squares of its part of a chunk in binary32 (at most
// 128 of them) and adds that sum to a binary64 one.  Where the binary32 sum is
// zero, so small that squares may have been lost to underflow, or not finite,
// the part is summed again in binary64, so the norm is right over the whole
// range of the types.  Everything after that is binary64, in a fixed order.
//
// Bound by HBM where the list is large: FP8 masters of eight layers (1.7 GB, only their
// scales written) 284 us (6.1 TB/s); 0.8 GB of BF16 gradients 380 us for one reading for the
// norm, one more and a writing for the clipping (6.4 TB/s).  Small lists are bound by the
// launches: 144 FP32 tensors of adapters (3.2 MB) 8 us in a graph.
#include "agoq_launch.h"
#include "typed_io.cuh"

namespace agoq {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kPart = 8;                // vectors of a thread
constexpr int kChunk = kPart * kThreads;
constexpr int kMaxCtas = 1216;          // partial sums of a launch
constexpr int kCtasPerSm = 4;
constexpr int kList = 1000, kMidList = 192, kShortList = 64;

struct Entry {
    const char *data;
    union {
        const float *scales;            // of an FP8 master, for the norm
        char *out;                      // for clipping
    };
    int64_t n;
    int first;                          // index of its first chunk
    int dtype;
};

template <int N>
struct List {
    int count, chunks;
    Entry e[N];
};
static_assert(sizeof(List<kList>) + 64 <= 32764, "kernel parameters hold at most 32,764 bytes");

__host__ __device__ __forceinline__ int elem_bytes(int dtype) {
    return dtype == kF32 ? 4 : dtype == kE4M3 ? 1 : 2;
}
// Elements between the 16-byte boundary before p and p.
__host__ __device__ __forceinline__ int lead(const void *p, int dtype) {
    return (int)(reinterpret_cast<uintptr_t>(p) & 15u) / elem_bytes(dtype);
}

__device__ __forceinline__ double warp_sum_f64(double v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

__device__ __forceinline__ double cta_sum_f64(double v) {
    __shared__ double red[kWarps];
    v = warp_sum_f64(v);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) s += red[i];
    return s;
}

// Whether a binary32 sum of squares stands: no square that mattered was lost.
__device__ __forceinline__ bool sum_stands(float s) { return s >= 0x1p-90f && s < 0x1p+127f; }

// Value of element i of a tensor (AGOQ_E4M3: its code times its scale).
__device__ __forceinline__ float element(const Entry &e, int64_t i) {
    switch (e.dtype) {
        case kF32: return load_elem<kF32>(e.data, i);
        case kBF16: return load_elem<kBF16>(e.data, i);
        case kF16: return load_elem<kF16>(e.data, i);
    }
    float lo, hi;
    e4m3x2_to_f32(static_cast<uint8_t>(__ldg(e.data + i)), lo, hi);
    return __fmul_rn(lo, __ldg(e.scales + i / kBlock));
}

// The chunk's tensor, given one that is not after it: the last entry whose first
// chunk is not after the chunk.
template <int N>
__device__ __forceinline__ int tensor_of(const List<N> &l, int chunk, int t) {
    if (t + 1 >= l.count || l.e[t + 1].first > chunk) return t;
    int lo = t + 1, hi = l.count;       // e[lo].first <= chunk < e[hi].first
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (l.e[mid].first <= chunk) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Add the squares of sixteen E4M3 codes, times that of their block's scale: the sum of
// the codes' squares first.
__device__ __forceinline__ void add_master_squares(const uint4 &v, float scale, float (&acc)[4]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        asm("{\n\t.reg .b16 l, h, a, b;\n\t.reg .b32 p, q;\n\tmov.b32 {l, h}, %4;\n\t"
            "cvt.rn.f16x2.e4m3x2 p, l;\n\tcvt.rn.f16x2.e4m3x2 q, h;\n\t"
            "mov.b32 {a, b}, p;\n\t"
            "fma.rn.f32.f16 %0, a, a, %0;\n\tfma.rn.f32.f16 %1, b, b, %1;\n\t"
            "mov.b32 {a, b}, q;\n\t"
            "fma.rn.f32.f16 %2, a, a, %2;\n\tfma.rn.f32.f16 %3, b, b, %3;\n\t}"
            : "+f"(s[0]), "+f"(s[1]), "+f"(s[2]), "+f"(s[3])
            : "r"(w[i]));
    }
    const float t = __fadd_rn(__fadd_rn(s[0], s[1]), __fadd_rn(s[2], s[3]));
    acc[0] = __fmaf_rn(t, __fmul_rn(scale, scale), acc[0]);
}

// The thread's part of a chunk in binary64, element by element.
__device__ __noinline__ double exact_part(const Entry &e, int64_t v0) {
    const int per = 16 / elem_bytes(e.dtype), skip = lead(e.data, e.dtype);
    double s = 0.0;
    for (int p = 0; p < kPart; ++p) {
        const int64_t at = (v0 + p * kThreads + threadIdx.x) * per - skip;
        for (int i = 0; i < per; ++i) {
            if (at + i < 0 || at + i >= e.n) continue;
            const double x = (double)element(e, at + i);
            s += x * x;
        }
    }
    return s;
}

// The sum of squares of this thread's part of the chunk at vector v0 of the tensor.
template <int DT>
__device__ __forceinline__ double square_part(const Entry &e, int64_t v0) {
    constexpr int kPer = 16 / (DT == kF32 ? 4 : DT == kE4M3 ? 1 : 2);
    const int skip = lead(e.data, DT);
    const uint4 *vec = reinterpret_cast<const uint4 *>(e.data - ((uintptr_t)e.data & 15u)) + v0 +
                       threadIdx.x;
    const int64_t vectors = (e.n + skip + kPer - 1) / kPer;
    uint4 v[kPart];
    float scale[kPart];
    if ((v0 > 0 || skip == 0) && (v0 + kChunk) * kPer <= e.n + skip) {
#pragma unroll
        for (int i = 0; i < kPart; ++i) v[i] = __ldg(vec + i * kThreads);
    } else {
        using E = Elem<DT == kE4M3 ? kF32 : DT>;
#pragma unroll
        for (int i = 0; i < kPart; ++i) {
            const int64_t j = v0 + i * kThreads + threadIdx.x, at = j * kPer - skip;
            v[i] = make_uint4(0, 0, 0, 0);
            if (j >= vectors) continue;
            if (at >= 0 && at + kPer <= e.n) {
                v[i] = __ldg(vec + i * kThreads);
            } else if constexpr (DT != kE4M3) {      // masters are whole vectors
                typename E::Word w[E::kVec];
#pragma unroll
                for (int k = 0; k < E::kVec; ++k)
                    w[k] = at + k >= 0 && at + k < e.n
                               ? __ldg(reinterpret_cast<const typename E::Word *>(e.data) + at + k)
                               : typename E::Word(0);
                __builtin_memcpy(&v[i], w, 16);
            }
        }
    }
    if constexpr (DT == kE4M3) {
#pragma unroll
        for (int i = 0; i < kPart; ++i) {
            const int64_t j = v0 + i * kThreads + threadIdx.x;
            scale[i] = j < vectors ? __ldg(e.scales + j / (kBlock / kPer)) : 0.0f;
        }
    }
    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < kPart; ++i) {
        if constexpr (DT == kE4M3) add_master_squares(v[i], scale[i], acc);
        else add_squares<DT>(v[i], acc);
    }
    const float s = __fadd_rn(__fadd_rn(acc[0], acc[1]), __fadd_rn(acc[2], acc[3]));
    if (sum_stands(s)) return (double)s;
    // nothing but zeros (of either sign) is exact too, unless a scale is not finite, which
    // makes the sum NaN
    uint32_t any = 0;
#pragma unroll
    for (int i = 0; i < kPart; ++i) any |= v[i].x | v[i].y | v[i].z | v[i].w;
    constexpr uint32_t kMagnitude = DT == kF32 ? 0x7FFFFFFFu : DT == kE4M3 ? 0x7F7F7F7Fu : 0x7FFF7FFFu;
    if (s == 0.0f && (any & kMagnitude) == 0) return 0.0;
    return exact_part(e, v0);
}

template <int N>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
square_sum_kernel(const __grid_constant__ List<N> l, double *__restrict__ partials) {
    pdl_wait_and_release();
    double total = 0.0;
    int t = 0;
    for (int chunk = blockIdx.x; chunk < l.chunks; chunk += gridDim.x) {
        t = tensor_of(l, chunk, t);
        const Entry &e = l.e[t];
        const int64_t v0 = (int64_t)(chunk - e.first) * kChunk;
        switch (e.dtype) {
            case kF32: total += square_part<kF32>(e, v0); break;
            case kBF16: total += square_part<kBF16>(e, v0); break;
            case kF16: total += square_part<kF16>(e, v0); break;
            default: total += square_part<kE4M3>(e, v0);
        }
    }
    total = cta_sum_f64(total);
    if (threadIdx.x == 0) partials[blockIdx.x] = total;
}

// The norm from n partial sums (every thread of the CTA gets it).
__device__ __forceinline__ float norm_of(const double *partials, int n) {
    double s = 0.0;
    for (int i = threadIdx.x; i < n; i += kThreads) s += partials[i];
    return (float)sqrt(cta_sum_f64(s));
}

__global__ void __launch_bounds__(kThreads) norm_kernel(const double *__restrict__ partials, int n,
                                                        float *__restrict__ norm) {
    pdl_wait_and_release();
    const float total = norm_of(partials, n);
    if (threadIdx.x == 0) *norm = total;
}

// min(1, max_norm / (norm + 1e-6)); NaN stays NaN.
__device__ __forceinline__ float coefficient(float max_norm, float norm) {
    const float c = __fdiv_rn(max_norm, __fadd_rn(norm, 1e-6f));
    return c > 1.0f ? 1.0f : c;
}

// The clipped values of the chunk at output vector v0: vectors that start at the
// output's 16-byte boundaries, whose input may lie across two.
template <int DT>
__device__ __forceinline__ void clip_part(const Entry &e, int64_t v0, float c) {
    using E = Elem<DT>;
    constexpr int kPer = E::kVec;
    const int oskip = lead(e.out, DT), skip = lead(e.data, DT);
    const int shift = ((skip - oskip + kPer) % kPer) * E::kSize;    // of the input, in bytes
    // input vectors: the one that holds the first element of an output vector, and the next
    const uint4 *vec = reinterpret_cast<const uint4 *>(e.data - skip * E::kSize) - (skip < oskip);
    uint4 *out = reinterpret_cast<uint4 *>(e.out - oskip * E::kSize);
    const int64_t vectors = (e.n + oskip + kPer - 1) / kPer;
    auto scaled = [&](const uint4 &v) {
        float f[kPer];
        E::unpack(v, f);
#pragma unroll
        for (int k = 0; k < kPer; ++k) f[k] = __fmul_rn(f[k], c);
        return E::pack(f);
    };
    const int64_t j0 = v0 + threadIdx.x;
    if (shift == 0 && (v0 > 0 || oskip == 0) && (v0 + kChunk) * kPer <= e.n + oskip) {
        uint4 v[kPart];
#pragma unroll
        for (int i = 0; i < kPart; ++i) v[i] = vec[j0 + i * kThreads];
#pragma unroll
        for (int i = 0; i < kPart; ++i) out[j0 + i * kThreads] = scaled(v[i]);
        return;
    }
#pragma unroll 4
    for (int i = 0; i < kPart; ++i) {
        const int64_t j = j0 + i * kThreads, at = j * kPer - oskip;
        if (j >= vectors) break;
        // both input vectors must lie inside the tensor
        if (at >= kPer && at + 2 * kPer <= e.n) {
            out[j] = scaled(shift ? bytes_from(vec[j], vec[j + 1], shift) : vec[j]);
        } else {
            for (int k = 0; k < kPer; ++k)
                if (at + k >= 0 && at + k < e.n)
                    store_elem<DT>(e.out, at + k, __fmul_rn(load_now<DT>(e.data, at + k), c));
        }
    }
}

// Clip by *norm, or by the norm of the partial sums, which is then also written.
// The chunks go backwards: the last ones that a norm has read are the likeliest to
// be still in the L2 cache.
template <int N>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
clip_kernel(const __grid_constant__ List<N> l, float max_norm, const double *__restrict__ partials,
            int sums, float *norm) {
    pdl_wait_and_release();
    float total;
    if (partials) {
        total = norm_of(partials, sums);
        if (blockIdx.x == 0 && threadIdx.x == 0) *norm = total;
    } else {
        total = *norm;
    }
    const float c = coefficient(max_norm, total);
    int t = 0;
    for (int k = (l.chunks - 1 - (int)blockIdx.x) / (int)gridDim.x; k >= 0; --k) {
        const int chunk = blockIdx.x + k * gridDim.x;
        t = tensor_of(l, chunk, l.e[t].first <= chunk ? t : 0);
        const Entry &e = l.e[t];
        if (c == 1.0f && e.data == e.out) continue;     // in place, nothing to change
        const int64_t v0 = (int64_t)(chunk - e.first) * kChunk;
        switch (e.dtype) {
            case kF32: clip_part<kF32>(e, v0, c); break;
            case kBF16: clip_part<kBF16>(e, v0, c); break;
            default: clip_part<kF16>(e, v0, c);
        }
    }
}

// ---- host -------------------------------------------------------------------------

int ctas_for(int chunks) {
    int most = sm_count() * kCtasPerSm;
    if (most > kMaxCtas) most = kMaxCtas;
    return chunks < most ? chunks : most;
}

// Fill `l` with the tensors from `at` on (at most N); returns the index after the
// last one.  `clip`: what clipping reads and writes (of an FP8 master its scales), cut
// at the boundaries of the output; else what the norm reads.
template <int N>
int fill(List<N> &l, const agoq_grad_tensor *t, int at, int count, bool clip) {
    l.count = 0;
    l.chunks = 0;
    for (; at < count && l.count < N; ++at) {
        if (t[at].n == 0) continue;
        Entry &e = l.e[l.count++];
        const bool scales = clip && t[at].dtype == kE4M3;
        e.data = static_cast<const char *>(scales ? (const void *)t[at].scales : t[at].data);
        if (clip) e.out = static_cast<char *>(t[at].out);
        else e.scales = t[at].scales;
        e.n = scales ? t[at].n / kBlock : t[at].n;
        e.dtype = scales ? kF32 : t[at].dtype;
        e.first = l.chunks;
        const int64_t per = 16 / elem_bytes(e.dtype);
        const int64_t vectors = (e.n + lead(clip ? e.out : e.data, e.dtype) + per - 1) / per;
        l.chunks += (int)((vectors + kChunk - 1) / kChunk);
    }
    return at;
}

// `launch(list, ctas)` for the tensors, N at a time.
template <int N, typename F>
cudaError_t for_lists(const agoq_grad_tensor *t, int count, bool clip, F launch) {
    List<N> l;
    for (int at = 0; at < count;) {
        at = fill(l, t, at, count, clip);
        const cudaError_t e = l.chunks ? launch(l, ctas_for(l.chunks)) : cudaSuccess;
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

template <int N>
cudaError_t norm_sums(const agoq_grad_tensor *t, int count, double *partials, int *used,
                      cudaStream_t st) {
    *used = 0;
    return for_lists<N>(t, count, false, [&](const List<N> &l, int ctas) {
        const cudaError_t r =
            launch_pdl_clusters(square_sum_kernel<N>, ctas, kThreads, 1, 0, st, l, partials + *used);
        *used += ctas;
        return r;
    });
}

template <int N>
cudaError_t clip_lists(const agoq_grad_tensor *t, int count, float max_norm,
                       const double *partials, int sums, float *norm, cudaStream_t st) {
    return for_lists<N>(t, count, true, [&](const List<N> &l, int ctas) {
        return launch_pdl_clusters(clip_kernel<N>, ctas, kThreads, 1, 0, st, l, max_norm, partials,
                                   sums, norm);
    });
}

template <int N>
cudaError_t run_lists(const agoq_grad_tensor *t, int count, bool sum, bool clip, float max_norm,
                      float *norm, double *partials, cudaStream_t st) {
    int used = 0;
    if (sum) {
        const cudaError_t e = norm_sums<N>(t, count, partials, &used, st);
        if (e != cudaSuccess) return e;
        // without clipping, or without anything to clip, a kernel of its own joins the sums
        if (!clip || used == 0) return launch_pdl(norm_kernel, 1, kThreads, 0, st, partials, used, norm);
    }
    return clip_lists<N>(t, count, max_norm, sum ? partials : nullptr, used, norm, st);
}

// The shortest list that holds the tensors: the parameters are copied at each launch.
cudaError_t run(const agoq_grad_tensor *t, int count, bool sum, bool clip, float max_norm,
                float *norm, double *partials, cudaStream_t st) {
    if (count <= kShortList)
        return run_lists<kShortList>(t, count, sum, clip, max_norm, norm, partials, st);
    if (count <= kMidList)
        return run_lists<kMidList>(t, count, sum, clip, max_norm, norm, partials, st);
    return run_lists<kList>(t, count, sum, clip, max_norm, norm, partials, st);
}

}  // namespace

int64_t grad_norm_workspace_bytes(int count) {
    const int64_t launches = count > kList ? (count + kList - 1) / kList : 1;
    return launches * kMaxCtas * (int64_t)sizeof(double);
}

cudaError_t launch_grad_norm(const agoq_grad_tensor *tensors, int count, float *norm,
                             double *workspace, cudaStream_t st) {
    return run(tensors, count, true, false, 0.0f, norm, workspace, st);
}

cudaError_t launch_clip_grads(const agoq_grad_tensor *tensors, int count, float max_norm,
                              const float *norm, cudaStream_t st) {
    return run(tensors, count, false, true, max_norm, const_cast<float *>(norm), nullptr, st);
}

cudaError_t launch_clip_grad_norm(const agoq_grad_tensor *tensors, int count, float max_norm,
                                  float *norm, double *workspace, cudaStream_t st) {
    return run(tensors, count, true, true, max_norm, norm, workspace, st);
}

}  // namespace agoq
