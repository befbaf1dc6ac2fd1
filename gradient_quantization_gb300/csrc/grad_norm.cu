// grad_norm.cu -- the global L2 norm of many gradients at once, and their
// clipping to a norm: FP32, BF16 and FP16 tensors, and the FP8 master gradients
// with block scales ("AGoQ: Activation and Gradient Quantization for
// Memory-Efficient Distributed Training of LLMs", section 2.B), whose clipping
// only multiplies the scales.
//
//   norm = sqrt(sum g^2),  c = min(1, max_norm / (norm + 1e-6)),  g' = R(g c)
//
// Every tensor is cut into chunks; the CTAs of one launch take the chunks of
// all tensors in turn.  The list travels in the kernel's parameters (at most
// kList tensors a launch), so a call copies nothing to the device and can be
// captured in a graph.
//
// Sums: a thread adds the squares of its part of a chunk in binary32 (at most
// 128 of them) and adds that sum to a binary64 one.  Where the binary32 sum is
// zero, so small that squares may have been lost to underflow, or not finite,
// the part is summed again in binary64, so the norm is right over the whole
// range of the types.  Everything after that is binary64, in a fixed order.
#include "agoq_launch.h"
#include "typed_io.cuh"

namespace agoq {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxCtas = 1216;          // rows of partial sums of a launch
constexpr int kList = 800, kShortList = 64;

struct Entry {
    const char *data;
    char *out;
    const float *scales;
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

// Elements of a chunk: 32 KB.
__host__ __device__ constexpr int chunk_elems(int dtype) {
    return dtype == kF32 ? 8192 : dtype == kE4M3 ? 32768 : 16384;
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

// The chunk's tensor: the last entry whose first chunk is not after it
// (`t` never goes back, as a CTA's chunks ascend).
template <int N>
__device__ __forceinline__ void advance(const List<N> &l, int chunk, int &t) {
    while (t + 1 < l.count && l.e[t + 1].first <= chunk) ++t;
}

template <int N>
__global__ void __launch_bounds__(kThreads)
square_sum_kernel(const __grid_constant__ List<N> l, double *__restrict__ partials) {
    pdl_wait_and_release();
    double total = 0.0;
    int t = 0;
    for (int chunk = blockIdx.x; chunk < l.chunks; chunk += gridDim.x) {
        advance(l, chunk, t);
        const Entry &e = l.e[t];
        const int64_t at = (int64_t)(chunk - e.first) * chunk_elems(e.dtype);
        const int64_t end = at + chunk_elems(e.dtype) < e.n ? at + chunk_elems(e.dtype) : e.n;
        float s = 0.0f;
        for (int64_t i = at + threadIdx.x; i < end; i += kThreads) {
            const float v = element(e, i);
            s = __fmaf_rn(v, v, s);
        }
        if (sum_stands(s)) {
            total += (double)s;
        } else {
            for (int64_t i = at + threadIdx.x; i < end; i += kThreads) {
                const double v = (double)element(e, i);
                total += v * v;
            }
        }
    }
    total = cta_sum_f64(total);
    if (threadIdx.x == 0) partials[blockIdx.x] = total;
}

__global__ void __launch_bounds__(kThreads) norm_kernel(const double *__restrict__ partials, int n,
                                                        float *__restrict__ norm) {
    pdl_wait_and_release();
    double s = 0.0;
    for (int i = threadIdx.x; i < n; i += kThreads) s += partials[i];
    s = cta_sum_f64(s);
    if (threadIdx.x == 0) *norm = (float)sqrt(s);
}

// min(1, max_norm / (norm + 1e-6)); NaN stays NaN.
__device__ __forceinline__ float coefficient(float max_norm, float norm) {
    const float c = __fdiv_rn(max_norm, __fadd_rn(norm, 1e-6f));
    return c > 1.0f ? 1.0f : c;
}

template <int N>
__global__ void __launch_bounds__(kThreads)
clip_kernel(const __grid_constant__ List<N> l, float max_norm, const float *__restrict__ norm) {
    pdl_wait_and_release();
    const float c = coefficient(max_norm, *norm);
    int t = 0;
    for (int chunk = blockIdx.x; chunk < l.chunks; chunk += gridDim.x) {
        advance(l, chunk, t);
        const Entry &e = l.e[t];
        const bool fp8 = e.dtype == kE4M3;
        const char *from = fp8 ? reinterpret_cast<const char *>(e.scales) : e.data;
        if (c == 1.0f && from == e.out) continue;   // in place, nothing to change
        const int per = fp8 ? kBlock : 1;           // elements of a value that is written
        const int64_t at = (int64_t)(chunk - e.first) * (chunk_elems(e.dtype) / per);
        const int64_t n = e.n / per, stop = at + chunk_elems(e.dtype) / per;
        const int64_t end = stop < n ? stop : n;
        for (int64_t i = at + threadIdx.x; i < end; i += kThreads) {
            switch (e.dtype) {
                case kBF16: store_elem<kBF16>(e.out, i, __fmul_rn(load_now<kBF16>(from, i), c)); break;
                case kF16: store_elem<kF16>(e.out, i, __fmul_rn(load_now<kF16>(from, i), c)); break;
                default: store_elem<kF32>(e.out, i, __fmul_rn(load_now<kF32>(from, i), c));
            }
        }
    }
}

int norm_ctas() {
    const int n = sm_count() * 8;
    return n < kMaxCtas ? n : kMaxCtas;
}

// Fill `l` with the tensors from `at` on; returns the index after the last one.
template <int N>
int fill(List<N> &l, const agoq_grad_tensor *t, int at, int count) {
    l.count = 0;
    l.chunks = 0;
    for (; at < count && l.count < N; ++at) {
        if (t[at].n == 0) continue;
        Entry &e = l.e[l.count++];
        e.data = static_cast<const char *>(t[at].data);
        e.out = static_cast<char *>(t[at].out);
        e.scales = t[at].scales;
        e.n = t[at].n;
        e.dtype = t[at].dtype;
        e.first = l.chunks;
        l.chunks += (int)((e.n + chunk_elems(e.dtype) - 1) / chunk_elems(e.dtype));
    }
    return at;
}

// `launch(list, ctas)` for the tensors, kList at a time.
template <int N, typename F>
cudaError_t for_lists(const agoq_grad_tensor *t, int count, F launch) {
    List<N> l;
    for (int at = 0; at < count;) {
        at = fill(l, t, at, count);
        const int most = norm_ctas();
        const cudaError_t e = launch(l, l.chunks < most ? l.chunks : most);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

template <int N>
cudaError_t norm_lists(const agoq_grad_tensor *t, int count, float *norm, double *partials,
                       cudaStream_t st) {
    int used = 0;
    const cudaError_t e = for_lists<N>(t, count, [&](const List<N> &l, int ctas) {
        if (ctas == 0) return cudaSuccess;
        const cudaError_t r =
            launch_pdl(square_sum_kernel<N>, ctas, kThreads, 0, st, l, partials + used);
        used += ctas;
        return r;
    });
    if (e != cudaSuccess) return e;
    return launch_pdl(norm_kernel, 1, kThreads, 0, st, partials, used, norm);
}

template <int N>
cudaError_t clip_lists(const agoq_grad_tensor *t, int count, float max_norm, const float *norm,
                       cudaStream_t st) {
    return for_lists<N>(t, count, [&](const List<N> &l, int ctas) {
        if (ctas == 0) return cudaSuccess;
        return launch_pdl(clip_kernel<N>, ctas, kThreads, 0, st, l, max_norm, norm);
    });
}

}  // namespace

int64_t grad_norm_workspace_bytes(int count) {
    const int64_t launches = count > kList ? (count + kList - 1) / kList : 1;
    return launches * kMaxCtas * (int64_t)sizeof(double);
}

cudaError_t launch_grad_norm(const agoq_grad_tensor *tensors, int count, float *norm,
                             double *workspace, cudaStream_t st) {
    return count <= kShortList ? norm_lists<kShortList>(tensors, count, norm, workspace, st)
                               : norm_lists<kList>(tensors, count, norm, workspace, st);
}

cudaError_t launch_clip_grads(const agoq_grad_tensor *tensors, int count, float max_norm,
                              const float *norm, cudaStream_t st) {
    return count <= kShortList ? clip_lists<kShortList>(tensors, count, max_norm, norm, st)
                               : clip_lists<kList>(tensors, count, max_norm, norm, st);
}

}  // namespace agoq
