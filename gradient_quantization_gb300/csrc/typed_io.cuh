// typed_io.cuh -- element types of the operators that accept FP32, BF16 and
// FP16 tensors: loads and stores of single elements and of 16-byte vectors,
// with all arithmetic in binary32.
#pragma once

#include <cuda_fp16.h>

#include "agoq_device.cuh"

namespace agoq {

// Values of agoq_dtype (include/agoq.h).
constexpr int kF32 = 0, kBF16 = 1, kF16 = 2, kE4M3 = 3;

// Type DT: its storage word, its size, and the elements of a 16-byte vector.
template <int DT>
struct Elem;

template <>
struct Elem<kF32> {
    using Word = float;
    static constexpr int kSize = 4, kVec = 4;
    __device__ static __forceinline__ float up(Word v) { return v; }
    __device__ static __forceinline__ Word down(float v) { return v; }
    __device__ static __forceinline__ void unpack(const uint4 &v, float *f) {
        f[0] = __uint_as_float(v.x);
        f[1] = __uint_as_float(v.y);
        f[2] = __uint_as_float(v.z);
        f[3] = __uint_as_float(v.w);
    }
    __device__ static __forceinline__ uint4 pack(const float *f) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                          __float_as_uint(f[3]));
    }
};

template <>
struct Elem<kBF16> {
    using Word = uint16_t;
    static constexpr int kSize = 2, kVec = 8;
    __device__ static __forceinline__ float up(Word v) { return __uint_as_float((uint32_t)v << 16); }
    __device__ static __forceinline__ Word down(float v) { return (Word)pack_bf16x2(v, 0.0f); }
    __device__ static __forceinline__ void unpack(const uint4 &v, float *f) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = bf16_lo(w[i]);
            f[2 * i + 1] = bf16_hi(w[i]);
        }
    }
    __device__ static __forceinline__ uint4 pack(const float *f) {
        return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                          pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
    }
};

template <>
struct Elem<kF16> {
    using Word = uint16_t;
    static constexpr int kSize = 2, kVec = 8;
    __device__ static __forceinline__ float up(Word v) {
        return __half2float(__ushort_as_half(v));
    }
    __device__ static __forceinline__ Word down(float v) {
        return __half_as_ushort(__float2half_rn(v));
    }
    __device__ static __forceinline__ void unpack(const uint4 &v, float *f) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = up((Word)w[i]);
            f[2 * i + 1] = up((Word)(w[i] >> 16));
        }
    }
    __device__ static __forceinline__ uint32_t pair(float lo, float hi) {
        uint32_t r;
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
        return r;
    }
    __device__ static __forceinline__ uint4 pack(const float *f) {
        return make_uint4(pair(f[0], f[1]), pair(f[2], f[3]), pair(f[4], f[5]), pair(f[6], f[7]));
    }
};

// Larger of two vectors' elements, each pair on its own (NaN loses).
template <int DT>
__device__ __forceinline__ uint32_t max_word(uint32_t a, uint32_t b) {
    uint32_t r;
    if constexpr (DT == kF32) {
        r = __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
    } else if constexpr (DT == kBF16) {
        asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    } else {
        asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    }
    return r;
}

// Largest value of a word (one FP32 or two 16-bit values).
template <int DT>
__device__ __forceinline__ float word_max(uint32_t w) {
    if constexpr (DT == kF32) return __uint_as_float(w);
    else return fmaxf(Elem<DT>::up((uint16_t)w), Elem<DT>::up((uint16_t)(w >> 16)));
}

// -infinity in every element of a word.
template <int DT>
constexpr uint32_t kNegInfWord = DT == kF32 ? 0xFF800000u : DT == kBF16 ? 0xFF80FF80u : 0xFC00FC00u;

// The 16 bytes from byte `shift` (0, 2, .. 14) on of the 32 bytes (a, b).
__device__ __forceinline__ uint4 bytes_from(const uint4 &a, const uint4 &b, int shift) {
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    if (shift & 8) {
#pragma unroll
        for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
    }
    if (shift & 4) {
#pragma unroll
        for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
    }
    if (shift & 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// x - ref of a vector's elements, in pairs (one rounding each: the mixed-precision
// addition takes a 16-bit operand as it is, without a conversion).
template <int DT>
__device__ __forceinline__ void differences(const uint4 &v, float ref, uint64_t *d) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if constexpr (DT == kF32) {
        d[0] = sub_f32x2(u32x2(w[0], w[1]), f32x2(ref, ref));
        d[1] = sub_f32x2(u32x2(w[2], w[3]), f32x2(ref, ref));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float lo, hi;
            if constexpr (DT == kBF16)
                asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
                    "add.rn.f32.bf16 %0, a, %3;\n\tadd.rn.f32.bf16 %1, b, %3;\n\t}"
                    : "=f"(lo), "=f"(hi) : "r"(w[i]), "f"(-ref));
            else
                asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
                    "add.rn.f32.f16 %0, a, %3;\n\tadd.rn.f32.f16 %1, b, %3;\n\t}"
                    : "=f"(lo), "=f"(hi) : "r"(w[i]), "f"(-ref));
            d[i] = f32x2(lo, hi);
        }
    }
}

// Add a vector's elements to four sums (one rounding each).
template <int DT>
__device__ __forceinline__ void add_elems(const uint4 &v, float (&acc)[4]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float &lo = acc[(2 * i) & 3], &hi = acc[(2 * i + 1) & 3];
        if constexpr (DT == kF32)
            acc[i] = __fadd_rn(acc[i], __uint_as_float(w[i]));
        else if constexpr (DT == kBF16)
            asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
                "add.rn.f32.bf16 %0, a, %0;\n\tadd.rn.f32.bf16 %1, b, %1;\n\t}"
                : "+f"(lo), "+f"(hi) : "r"(w[i]));
        else
            asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
                "add.rn.f32.f16 %0, a, %0;\n\tadd.rn.f32.f16 %1, b, %1;\n\t}"
                : "+f"(lo), "+f"(hi) : "r"(w[i]));
    }
}

// Add the squares of a vector's elements to four sums.
template <int DT>
__device__ __forceinline__ void add_squares(const uint4 &v, float (&acc)[4]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float &lo = acc[(2 * i) & 3], &hi = acc[(2 * i + 1) & 3];
        if constexpr (DT == kF32) {
            const float x = __uint_as_float(w[i]);
            acc[i] = __fmaf_rn(x, x, acc[i]);
        } else if constexpr (DT == kBF16) {
            asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
                "fma.rn.f32.bf16 %0, a, a, %0;\n\tfma.rn.f32.bf16 %1, b, b, %1;\n\t}"
                : "+f"(lo), "+f"(hi) : "r"(w[i]));
        } else {
            asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
                "fma.rn.f32.f16 %0, a, a, %0;\n\tfma.rn.f32.f16 %1, b, b, %1;\n\t}"
                : "+f"(lo), "+f"(hi) : "r"(w[i]));
        }
    }
}

// A vector's elements as binary32 pairs, and back.  (16-bit types: an addition of -0,
// which changes no value, in place of shifts and masks on the busier integer pipe.)
template <int DT>
__device__ __forceinline__ void unpack2(const uint4 &v, uint64_t *p) {
    if constexpr (DT == kF32) {
        p[0] = u32x2(v.x, v.y);
        p[1] = u32x2(v.z, v.w);
    } else {
        differences<DT>(v, 0.0f, p);
    }
}
template <int DT>
__device__ __forceinline__ uint4 pack2(const uint64_t *p) {
    float f[Elem<DT>::kVec];
#pragma unroll
    for (int i = 0; i < Elem<DT>::kVec / 2; ++i) {
        f[2 * i] = lo_f32(p[i]);
        f[2 * i + 1] = hi_f32(p[i]);
    }
    return Elem<DT>::pack(f);
}
__device__ __forceinline__ float sum_pair(uint64_t p) { return __fadd_rn(lo_f32(p), hi_f32(p)); }

// ---- asynchronous copies of 16 bytes into shared memory -------------------------
__device__ __forceinline__ void copy16(void *to, const void *from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                     static_cast<uint32_t>(__cvta_generic_to_shared(to))),
                 "l"(from)
                 : "memory");
}
__device__ __forceinline__ void copy16(uint32_t to, const void *from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ uint32_t shared_address(const void *p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ uint4 load_shared(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ void store_shared(uint32_t at, const uint4 &v) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z),
                 "r"(v.w)
                 : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_left() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Element i of a tensor of type DT, as binary32.
template <int DT>
__device__ __forceinline__ float load_elem(const void *p, int64_t i) {
    return Elem<DT>::up(__ldg(static_cast<const typename Elem<DT>::Word *>(p) + i));
}

// The same where the kernel may also write the element (in-place calls): an
// ordinary load, not through the read-only path.
template <int DT>
__device__ __forceinline__ float load_now(const void *p, int64_t i) {
    return Elem<DT>::up(static_cast<const typename Elem<DT>::Word *>(p)[i]);
}

// Element i of a tensor of type DT, set to v rounded to nearest even.
template <int DT>
__device__ __forceinline__ void store_elem(void *p, int64_t i, float v) {
    static_cast<typename Elem<DT>::Word *>(p)[i] = Elem<DT>::down(v);
}

// Byte address of element i.
template <int DT>
__device__ __forceinline__ const char *elem_at(const void *p, int64_t i) {
    return static_cast<const char *>(p) + i * Elem<DT>::kSize;
}
template <int DT>
__device__ __forceinline__ char *elem_at(void *p, int64_t i) {
    return static_cast<char *>(p) + i * Elem<DT>::kSize;
}

// Sum over a warp (every lane gets it), in the order of the butterfly.
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
}

// Sum over a CTA of WARPS warps; every thread gets it.  `red` holds WARPS
// floats and may be reused after the next __syncthreads().
template <int WARPS>
__device__ __forceinline__ float cta_sum(float v, float *red) {
    v = warp_sum(v);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < WARPS; ++i) s = __fadd_rn(s, red[i]);
    return s;
}

}  // namespace agoq
