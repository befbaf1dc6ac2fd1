// fp4_format.cuh -- the micro-scaled 4-bit format of the FP4 calls (include/agoq.h):
// sizes and places of codes and scales, and the rounding of a block.
//
// Codes are E2M1 (values 0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign), two to a byte, rows of
// ceil(K / 32) * 16 bytes.  A scale byte stands for 32 elements of a row (MXFP4: E8M0, a power
// of two) or 16 (NVFP4: E4M3, times the tensor's scale).  Scales lie in tiles of 128 rows by
// 4 blocks, 512 bytes: block b of row r at (r % 32) * 16 + (r % 128 / 32) * 4 + b % 4 of tile
// (r / 128, b / 4).  That is how the tensor cores take them: a tile is copied as it is into four
// columns of tensor memory.
#pragma once

#include <cstdint>

namespace agoq {

constexpr int kMx = 0, kNv = 1;                 // agoq_fp4_format

__host__ __device__ constexpr int fp4_block(int fmt) { return fmt == kNv ? 16 : 32; }
// Elements that a scale tile spans.
__host__ __device__ constexpr int fp4_tile_elems(int fmt) { return 4 * fp4_block(fmt); }
__host__ __device__ inline int64_t fp4_row_bytes(int64_t K) { return (K + 31) / 32 * 16; }
// Tiles of a row block: ceil(K / 64) for NVFP4, ceil(K / 128) for MXFP4.
__host__ __device__ inline int64_t fp4_tiles_across(int64_t K, int fmt) {
    return (K + fp4_tile_elems(fmt) - 1) / fp4_tile_elems(fmt);
}
__host__ __device__ inline int64_t fp4_tiles_down(int64_t rows) { return (rows + 127) / 128; }

constexpr int kScaleTile = 512;

#ifdef __CUDACC__
}  // namespace agoq
#include "agoq_device.cuh"
namespace agoq {

constexpr float kE2M1Max = 6.0f;
constexpr float kTensorSpan = 2688.0f;          // 6 * 448
constexpr float kLowestTensorScale = 0x1p-100f; // products with a block's scale stay normal

// The larger and the smaller of two; a NaN stays.
__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ float min_nan(float a, float b) {
    float d;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// A tensor's scale from its largest magnitude.  Of one that is not finite, codes made with it have
// NaN block scales; codes from before may not, so a NaN must stay.
__device__ __forceinline__ float tensor_scale(float amax) {
    return max_nan(__fdiv_rn(amax, kTensorSpan), kLowestTensorScale);
}

__device__ __forceinline__ bool finite_bits(float v) {
    return (__float_as_uint(v) & 0x7F800000u) != 0x7F800000u;
}

// max.NaN(|a|, |b|, |c|): a NaN stays.
__device__ __forceinline__ float max_abs_nan(float a, float b, float c) {
    float d;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// What a thread needs to scale blocks: NVFP4 the tensor's scale, and a table in shared memory of
// the factor fl(1 / fl(s g)) of every scale s that E4M3 has (0 for 0): a look-up takes the place
// of a conversion, a product and a division a block.
struct Scaling {
    float g = 0.0f, six_g = 0.0f, per_six_g = 0.0f;
    bool ok = true;
    const float *table = nullptr;
};
constexpr int kScaleTable = 128;

// By all threads of a CTA (at least kScaleTable); the table may be read after a barrier.
template <int FMT>
__device__ __forceinline__ Scaling scaling_of(const float *amax, float *table) {
    Scaling t;
    if constexpr (FMT == kNv) {
        const float m = __ldg(amax);
        t.g = tensor_scale(m);
        t.six_g = __fmul_rn(t.g, kE2M1Max);
        t.per_six_g = __frcp_rn(t.six_g);
        t.ok = finite_bits(m);
        t.table = table;
        const int i = threadIdx.x;
        if (i < kScaleTable) {
            float lo, hi;
            e4m3x2_to_f32(i, lo, hi);
            table[i] = i ? __frcp_rn(__fmul_rn(lo, t.g)) : 0.0f;
        }
    }
    return t;
}

// Scale byte of a block and the factor of its elements, from its largest magnitude.  A block
// with a NaN or an infinity (or, NVFP4, of a tensor with one) has the NaN of its scale's type
// and codes of 0: the caller masks them with `keep`.
struct BlockScale {
    uint32_t byte;
    float inverse;
    uint32_t keep;
};
template <int FMT>
__device__ __forceinline__ BlockScale block_scale(float top, const Scaling &t) {
    BlockScale s;
    if constexpr (FMT == kMx) {
        // 2^(floor(log2 top) - 2), not below 2^-127: the exponent field less 2
        const int field = (int)(__float_as_uint(top) >> 23) - 2;
        s.keep = finite_bits(top) ? 0xFFFFFFFFu : 0u;
        const uint32_t byte = max(field, 0);
        s.byte = (byte | ~s.keep) & 0xFFu;
        s.inverse = __uint_as_float((254u - byte) << 23);
    } else {
        s.keep = t.ok && finite_bits(top) ? 0xFFFFFFFFu : 0u;
        // top times fl(1 / 6 g) is within 3 * 2^-24 of fl(top / 6 g) (relative; results below
        // binary32's normal range are far below E4M3's): where both sides of it round to one
        // code, that is the quotient's; else, about once in 2^15 blocks, it is divided
        const float q = __fmul_rn(top, t.per_six_g);
        const uint32_t both = e4m3x2_from_f32(__fmul_rn(q, 1.0f - 0x1p-20f), __fmul_rn(q, 1.0f + 0x1p-20f));
        uint32_t byte = both & 0xFFu;
        if (byte != both >> 8) byte = e4m3x2_from_f32(__fdiv_rn(top, t.six_g), 0.0f);
        s.inverse = t.table[byte & 127u];
        s.byte = (byte | ~s.keep) & 127u;
    }
    return s;
}

// Eight values times `inverse`, rounded to E2M1 (to nearest, ties to the even code, beyond 6
// to 6): a word of eight codes.
__device__ __forceinline__ uint32_t e2m1x8(const uint64_t (&p)[4], float inverse) {
    const uint64_t r2 = f32x2(inverse, inverse);
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint64_t q = mul_f32x2(p[i], r2);
        f[2 * i] = lo_f32(q);
        f[2 * i + 1] = hi_f32(q);
    }
    uint32_t w;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(w)
        : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
    return w;
}

// Eight codes to FP16 pairs (exact).
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}

// Value of a scale byte (NaN among them).
template <int FMT>
__device__ __forceinline__ float scale_value(uint32_t byte) {
    // (0: 2^-127, a subnormal; 255: NaN.  Without a comparison: 8192 x 11008 back to BF16 35 us, 46
    // us with.)
    if constexpr (FMT == kMx)
        return __uint_as_float(max(byte << 23, 0x00400000u) | (byte + 1) >> 8 << 22);
    float lo, hi;
    e4m3x2_to_f32(byte, lo, hi);
    return lo;
}

#endif  // __CUDACC__

}  // namespace agoq
