// fp4_quant.cu -- micro-scaled 4-bit quantisation of a matrix along its rows, its columns or
// both, the largest magnitude that NVFP4's tensor scale is taken from, and the way back.
//
// Per block of 32 (MXFP4) or 16 (NVFP4) elements, in binary32:
//   MXFP4: s = 2^e, e = max(floor(log2 absmax) - 2, -127);   code = E2M1(x 2^-e)
//   NVFP4: g = max(fl(amax / 2688), 2^-100); s = E4M3(fl(absmax / fl(6 g)));
//          code = E2M1(fl(x fl(1 / fl(s g)))), 0 where s is 0
// E2M1 and E4M3 round to nearest even and saturate.
#include <cooperative_groups.h>

#include <type_traits>

#include "agoq_launch.h"
#include "fp4_format.cuh"
#include "typed_io.cuh"

namespace agoq {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256;
constexpr int kGroup = 16;                     // elements of a thread's group

// The larger magnitudes of two pairs, NaN before all; the signs are those of the products.
template <int DT>
__device__ __forceinline__ uint32_t larger2(uint32_t a, uint32_t b) {
    uint32_t r;
    if constexpr (DT == kBF16) asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else asm("max.NaN.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

template <int DT>
struct Group {
    static constexpr int kVecs = kGroup * Elem<DT>::kSize / 16;
    uint4 v[kVecs];
    // Elements e .. e + 15 of a row of K (0 beyond it).
    template <typename I>                          // int where rows are short enough
    __device__ __forceinline__ void load(const char *row, I e, I K) {
        using E = Elem<DT>;
        const char *p = row + (int64_t)e * E::kSize;
        const int shift = (int)(reinterpret_cast<uintptr_t>(p) & 15u);
        if (shift == 0 && e + kGroup <= K) {
#pragma unroll
            for (int i = 0; i < kVecs; ++i) v[i] = __ldg(reinterpret_cast<const uint4 *>(p) + i);
            return;
        }
        // the 16-byte vectors around the group, where they lie within the row
        if (p - shift >= row && e + kGroup + (16 - shift) / E::kSize <= K) {
            const uint4 *from = reinterpret_cast<const uint4 *>(p - shift);
            uint4 last = __ldg(from);
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                const uint4 next = __ldg(from + i + 1);
                v[i] = bytes_from(last, next, shift);
                last = next;
            }
            return;
        }
        typename E::Word w[kGroup];
#pragma unroll
        for (int i = 0; i < kGroup; ++i)
            w[i] = e + i < K ? __ldg(reinterpret_cast<const typename E::Word *>(row) + e + i)
                             : typename E::Word(0);
        __builtin_memcpy(v, w, sizeof v);
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < kVecs; ++i) v[i] = make_uint4(0, 0, 0, 0);
    }
    // Largest magnitude; NaN if there is one.
    __device__ __forceinline__ float absmax() const {
        if constexpr (DT == kF32) {
            float m = 0.0f;
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                m = max_abs_nan(m, __uint_as_float(v[i].x), __uint_as_float(v[i].y));
                m = max_abs_nan(m, __uint_as_float(v[i].z), __uint_as_float(v[i].w));
            }
            return m;
        } else {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < kVecs; ++i)
                m = larger2<DT>(m, larger2<DT>(larger2<DT>(v[i].x, v[i].y), larger2<DT>(v[i].z, v[i].w)));
            // magnitudes of 16-bit floats in the order of their bits, NaN last
            const uint32_t lo = m & 0x7FFFu, hi = m >> 16 & 0x7FFFu;
            return Elem<DT>::up((uint16_t)(lo > hi ? lo : hi));
        }
    }
    __device__ __forceinline__ uint2 codes(float inverse) const {
        uint32_t w[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint64_t p[4];
            if constexpr (DT == kF32) {
                unpack2<DT>(v[2 * h], p);
                unpack2<DT>(v[2 * h + 1], p + 2);
            } else {
                unpack2<DT>(v[h], p);
            }
            w[h] = e2m1x8(p, inverse);
        }
        return make_uint2(w[0], w[1]);
    }
};

// Two NaN-keeping magnitudes.
__device__ __forceinline__ float larger(float a, float b) { return max_abs_nan(a, b, 0.0f); }

// The word of four scales that a thread's block belongs to, from the threads of four blocks
// (a block is one thread's group, NVFP4, or two threads', MXFP4).
template <int FMT>
__device__ __forceinline__ uint32_t scale_word(uint32_t byte, int lane) {
    constexpr int kPer = FMT == kMx ? 1 : 0;
    uint32_t w = byte << (8 * ((lane >> kPer) & 3));
    w |= __shfl_xor_sync(0xFFFFFFFFu, w, 1 << kPer);
    w |= __shfl_xor_sync(0xFFFFFFFFu, w, 2 << kPer);
    return w;
}

// Place of the word of blocks 4 t .. 4 t + 3 of a row.
__device__ __forceinline__ int64_t word_at(int64_t row, int64_t t, int64_t across) {
    return ((row >> 7) * across + t) * kScaleTile + (row & 31) * 16 + ((row >> 5) & 3) * 4;
}

// Rows of a 128-row block whose scales share a 32-byte sector of every tile: two neighbours, and
// the same 32, 64 and 96 rows further on.  A CTA takes such eight rows, one a warp, so that a
// sector of scales is read once and written whole.
constexpr int kOctet = 8;
__device__ __forceinline__ int octet_row(int octet, int warp) {       // within the block
    return 2 * octet + (warp & 1) + 32 * (warp >> 1);
}

// ---- rows -------------------------------------------------------------------------
//
// A warp takes PARTS runs of 512 elements of a row, a lane 16 of each.  Rows are padded to whole
// scale words (64 or 128 elements) and to whole tiles of 128, so that every scale byte is
// written (0 where there is no block).  Bound by HBM for MXFP4 and FP32: 8192 x 11008 BF16 to MXFP4
// 33.7 us (6.8 TB/s), 8192 x 8192 FP32 to NVFP4 44.3 us (6.9 TB/s).  BF16 to NVFP4 39.3 us (5.9 TB/s)
// by instruction issue, with a scale every 16 elements.  Eight CTAs an SM (32 registers): with six
// 41 us, with four 45; a lane with one run instead of two (BF16) 51 us.
constexpr int kRun = 32 * kGroup;

template <int DT, int FMT, int PARTS>
__global__ void __launch_bounds__(kThreads, 8) fp4_rows_kernel(const Fp4Quant a, uint32_t chunks) {
    constexpr int kWord = fp4_tile_elems(FMT) / kGroup;        // lanes of a scale word
    constexpr int kWords = 32 / kWord;                         // of a run
    __shared__ uint32_t words[PARTS * kWords][kOctet];
    __shared__ float table[kScaleTable];
    pdl_wait_and_release();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t octet = blockIdx.x / chunks, chunk = blockIdx.x - octet * chunks;
    const int64_t block_row = octet >> 4, row = block_row * 128 + octet_row(octet & 15, warp);
    // (places within a row, of at most 2^24 elements, in 32 bits)
    const int len = (int)a.K, across = (int)fp4_tiles_across(a.K, FMT), row_bytes = (int)fp4_row_bytes(a.K);
    const bool live = row < a.T;
    const char *from = elem_at<DT>(a.x, live ? row * a.ldx : 0);
    const int e0 = (int)chunk * PARTS * kRun + lane * kGroup;
    Group<DT> x[PARTS];
#pragma unroll
    for (int p = 0; p < PARTS; ++p) {
        if (live && e0 + p * kRun < len) x[p].load(from, e0 + p * kRun, len);
        else x[p].clear();
    }
    const Scaling scaling = scaling_of<FMT>(a.amax, table);
    if constexpr (FMT == kNv) __syncthreads();
    uint8_t *codes = a.codes + (live ? row * row_bytes : 0);
#pragma unroll
    for (int p = 0; p < PARTS; ++p) {
        const int e = e0 + p * kRun;
        float top = x[p].absmax();
        if constexpr (FMT == kMx) top = larger(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
        const BlockScale s = block_scale<FMT>(top, scaling);
        uint2 c = x[p].codes(s.inverse);
        c.x &= s.keep;
        c.y &= s.keep;
        if (live && e / 2 < row_bytes) *reinterpret_cast<uint2 *>(codes + e / 2) = c;
        // (no block begins behind the row's end)
        const bool block = live && (FMT == kMx ? e & ~(2 * kGroup - 1) : e) < len;
        const uint32_t w = scale_word<FMT>(block ? s.byte : 0u, lane);
        // (word of the sector: neighbours are 16 bytes apart, the other rows 4)
        if (lane % kWord == 0) words[p * kWords + lane / kWord][(warp & 1) * 4 + (warp >> 1)] = w;
    }
    __syncthreads();
    const int i = threadIdx.x, t = i >> 3;
    const int tile = (int)chunk * PARTS * kWords + t;
    if (t < PARTS * kWords && tile < across)
        *reinterpret_cast<uint32_t *>(a.scales + (block_row * across + tile) * kScaleTile +
                                      2 * (octet & 15) * 16 + (i & 7) * 4) = words[t][i & 7];
}

// ---- columns, and both -------------------------------------------------------------
//
// A CTA copies a tile of 128 columns by 128 rows (FP32: 64) to shared memory; eight threads take a
// row (ROWS), and a thread then takes a block of two neighbouring columns.  The tile's codes of
// the columns and its scale tiles are gathered in shared memory and leave in whole rows.
// 8192 x 11008 BF16: columns 38 us (MXFP4, 6.0 TB/s) and 42 us (NVFP4), both ways 52 us and 60 us (5.3
// and 4.7 TB/s), bound by instruction issue (63% of the slots, the integer pipe 60% busy);
// 8192 x 8192 FP32 to NVFP4 52 us and 60 us (5.8 and 5.7 TB/s).  Five CTAs an SM for MXFP4 (columns
// 41 us with four), four for NVFP4 (columns 47 us with five).  FP32 tiles of 128 rows left room for
// two CTAs: both ways 86 us.
constexpr int kTile = 128;
template <int DT>
struct TileShape {
    static constexpr int kRows = DT == kF32 ? 64 : 128;        // 32 KB of elements
    static constexpr int kCodePitch = kRows / 2 + 8;           // bytes of a column's codes
};

template <int DT, int FMT, bool ROWS>
__global__ void __launch_bounds__(kThreads, FMT == kMx ? 5 : 4) fp4_tiles_kernel(const Fp4Quant a, int64_t tiles_k) {
    using E = Elem<DT>;
    using S = TileShape<DT>;
    constexpr int kPitch = kTile * E::kSize, kRows = S::kRows, kSteps = kRows / 32;
    constexpr int kBlockLen = fp4_block(FMT), kSpan = fp4_tile_elems(FMT);
    constexpr int kTilesK = kTile / kSpan;                     // scale tiles along the columns
    constexpr int kTilesT = kRows > kSpan ? kRows / kSpan : 1; // and along the rows
    extern __shared__ __align__(16) uint8_t tile[];
    uint8_t *out = tile + kRows * kPitch;                      // codes of the columns
    uint8_t *scales = out + kTile * S::kCodePitch;             // their scale tiles
    uint8_t *row_scales = scales + kTilesT * kScaleTile;
    __shared__ float table[kScaleTable];
    pdl_wait_and_release();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t0 = blockIdx.x / tiles_k * kRows, k0 = blockIdx.x % tiles_k * kTile;
    const int64_t row_bytes = fp4_row_bytes(a.K), col_bytes = fp4_row_bytes(a.T);
    const int g = threadIdx.x & 7;
    // Where vector v of a row lies: the vectors of eight threads' groups in eight different places
    // between 128-byte lines.
    auto place = [](int v) { return v ^ (v >> 3 & (Group<DT>::kVecs - 1)); };
    if (a.level) {
        // 16-byte vectors, a warp whole lines of a row
        constexpr int kVecs = kPitch / 16;
        for (int i = threadIdx.x; i < kRows * kVecs; i += kThreads) {
            const int r = i / kVecs, v = i % kVecs;
            const int64_t e = k0 + v * E::kVec;
            uint8_t *to = tile + r * kPitch + place(v) * 16;
            const char *row = elem_at<DT>(a.x, (t0 + r) * a.ldx);
            if (t0 + r < a.T && e + E::kVec <= a.K) {
                copy16(to, row + e * E::kSize);
            } else {
                typename E::Word w[E::kVec];
#pragma unroll
                for (int j = 0; j < E::kVec; ++j)
                    w[j] = t0 + r < a.T && e + j < a.K ? reinterpret_cast<const typename E::Word *>(row)[e + j]
                                                       : typename E::Word(0);
                __builtin_memcpy(to, w, 16);
            }
        }
        copies_commit();
    } else {
        Group<DT> x[kSteps];
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int64_t t = t0 + 32 * i + (threadIdx.x >> 3);
            if (t < a.T && k0 + g * kGroup < a.K)
                x[i].load(elem_at<DT>(a.x, t * a.ldx), (int)k0 + g * kGroup, (int)a.K);
            else
                x[i].clear();
        }
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            uint8_t *to = tile + (32 * i + (threadIdx.x >> 3)) * kPitch;
#pragma unroll
            for (int j = 0; j < Group<DT>::kVecs; ++j)
                *reinterpret_cast<uint4 *>(to + place(g * Group<DT>::kVecs + j) * 16) = x[i].v[j];
        }
    }
    const Scaling scaling = scaling_of<FMT>(a.amax, table);
    copies_left<0>();
    __syncthreads();
    // rows: eight threads a row, 32 rows a step
    if constexpr (ROWS) {
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int r = 32 * i + (threadIdx.x >> 3);
            Group<DT> x;
#pragma unroll
            for (int j = 0; j < Group<DT>::kVecs; ++j)
                x.v[j] = *reinterpret_cast<const uint4 *>(tile + r * kPitch + place(g * Group<DT>::kVecs + j) * 16);
            float top = x.absmax();
            if constexpr (FMT == kMx) top = larger(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
            const BlockScale s = block_scale<FMT>(top, scaling);
            uint2 c = x.codes(s.inverse);
            c.x &= s.keep;
            c.y &= s.keep;
            const int64_t at = k0 / 2 + g * 8;
            if (t0 + r < a.T && at < row_bytes)
                *reinterpret_cast<uint2 *>(a.codes + (t0 + r) * row_bytes + at) = c;
            const bool block = t0 + r < a.T && k0 + (FMT == kMx ? g & ~1 : g) * kGroup < a.K;
            const uint32_t w = scale_word<FMT>(block ? s.byte : 0u, lane);
            constexpr int kWord = FMT == kMx ? 8 : 4;
            if (g % kWord == 0)
                *reinterpret_cast<uint32_t *>(row_scales + g / kWord * kScaleTile + (r & 31) * 16 +
                                              (r >> 5) * 4) = w;
        }
    }
    // columns 2 c and 2 c + 1, blocks of kBlockLen rows
    constexpr int kTasks = kRows / kBlockLen * (kTile / 2);
    for (int task = threadIdx.x; task < kTasks; task += kThreads) {
        const int c = task & 63, b = task >> 6;
        constexpr int kPairs = 8 / E::kSize;           // column pairs of a vector
        const int at_c = place(c / kPairs) * 16 + c % kPairs * 2 * E::kSize;
        // the two columns' elements as they lie in the tile
        using Pair = typename std::conditional<DT == kF32, float2, uint32_t>::type;
        Pair v[kBlockLen];
        float top[2] = {0.0f, 0.0f};
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < kBlockLen; ++i)
            v[i] = *reinterpret_cast<const Pair *>(tile + (b * kBlockLen + i) * kPitch + at_c);
        if constexpr (DT == kF32) {
#pragma unroll
            for (int i = 0; i < kBlockLen; i += 2) {
                top[0] = max_abs_nan(top[0], v[i].x, v[i + 1].x);
                top[1] = max_abs_nan(top[1], v[i].y, v[i + 1].y);
            }
        } else {
#pragma unroll
            for (int i = 0; i < kBlockLen; ++i) m = larger2<DT>(m, v[i]);
            top[0] = E::up((uint16_t)(m & 0x7FFFu));
            top[1] = E::up((uint16_t)(m >> 16 & 0x7FFFu));
        }
#pragma unroll
        for (int side = 0; side < 2; ++side) {
            const BlockScale s = block_scale<FMT>(top[side], scaling);
            const int col = 2 * c + side;
            auto element = [&](int i) {
                if constexpr (DT == kF32) return side ? v[i].y : v[i].x;
                else return E::up((uint16_t)(side ? v[i] >> 16 : v[i]));
            };
#pragma unroll
            for (int h = 0; h < kBlockLen / 16; ++h) {
                uint32_t w[2];
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    uint64_t p[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int at = 16 * h + 8 * q + 2 * i;
                        p[i] = f32x2(element(at), element(at + 1));
                    }
                    w[q] = e2m1x8(p, s.inverse) & s.keep;
                }
                *reinterpret_cast<uint2 *>(out + col * S::kCodePitch + b * (kBlockLen / 2) + 8 * h) =
                    make_uint2(w[0], w[1]);
            }
            scales[(b >> 2) * kScaleTile + (col & 31) * 16 + (col >> 5) * 4 + (b & 3)] =
                (uint8_t)(k0 + col < a.K && t0 + b * kBlockLen < a.T ? s.byte : 0u);
        }
    }
    __syncthreads();
    // codes: kRows / 16 threads a column
    constexpr int kPer = kRows / 16;
    const int j = threadIdx.x % kPer;
    for (int col = threadIdx.x / kPer; col < kTile; col += kThreads / kPer) {
        const int64_t at = t0 / 2 + j * 8;
        if (k0 + col < a.K && at < col_bytes)
            *reinterpret_cast<uint2 *>(a.codes_t + (k0 + col) * col_bytes + at) =
                *reinterpret_cast<const uint2 *>(out + col * S::kCodePitch + j * 8);
    }
    // Scale tiles, a warp each.  A tile of 64 rows fills half of a scale tile's rows, and of MXFP4
    // half of its blocks; where no rows follow, it clears the other half.
    const int64_t down_t = fp4_tiles_across(a.T, FMT), across = fp4_tiles_across(a.K, FMT);
    const bool second = kRows == 64 && (t0 & 64), last = kRows == 64 && !second && t0 + 64 >= a.T;
    if (warp < kTilesT) {
        const int64_t at = t0 / kSpan + warp;
        uint8_t *to = a.scales_t + ((k0 >> 7) * down_t + at) * kScaleTile + lane * 16;
        const uint4 v = *reinterpret_cast<const uint4 *>(scales + warp * kScaleTile + lane * 16);
        if (at < down_t) {
            if constexpr (kRows >= kSpan) {
                *reinterpret_cast<uint4 *>(to) = v;
            } else {
                const uint32_t w[4] = {v.x & 0xFFFFu, v.y & 0xFFFFu, v.z & 0xFFFFu, v.w & 0xFFFFu};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (last) reinterpret_cast<uint32_t *>(to)[i] = w[i];
                    else reinterpret_cast<uint16_t *>(to)[2 * i + second] = (uint16_t)w[i];
                }
            }
        }
    } else if (ROWS && warp < kTilesT + kTilesK) {
        const int w = warp - kTilesT;
        const int64_t at = k0 / kSpan + w;
        uint8_t *to = a.scales + ((t0 >> 7) * across + at) * kScaleTile + lane * 16;
        const uint4 v = *reinterpret_cast<const uint4 *>(row_scales + w * kScaleTile + lane * 16);
        if (at < across) {
            if constexpr (kRows == 128) *reinterpret_cast<uint4 *>(to) = v;
            else if (last) *reinterpret_cast<uint4 *>(to) = make_uint4(v.x, v.y, 0, 0);
            else reinterpret_cast<uint2 *>(to)[second] = make_uint2(v.x, v.y);
        }
    }
}

// ---- the largest magnitude -----------------------------------------------------------

// Magnitudes as binary32 bits are in the order of their values, NaN last.  Bound by HBM: 8192 x 11008
// BF16 29.7 us (6.1 TB/s); 16 x 4096 by one cluster 2.1 us.
template <int DT>
__device__ __forceinline__ uint32_t absmax_of(const void *x, int64_t ldx, int64_t T, int64_t K,
                                              int64_t first, int64_t step) {
    uint32_t m = 0;
    if (T == 1) {
        // one long row: whole lines a warp; single elements before and behind its 16-byte vectors
        using Word = typename Elem<DT>::Word;
        constexpr int N = Elem<DT>::kVec;
        const Word *row = static_cast<const Word *>(x);
        const int64_t skip = (16 - (reinterpret_cast<uintptr_t>(x) & 15u)) % 16 / Elem<DT>::kSize;
        const int64_t head = skip < K ? skip : K, n = (K - head) / N;
        const uint4 *vec = reinterpret_cast<const uint4 *>(row + head);
        float top = 0.0f;
        uint32_t two = 0;
        auto add = [&](const uint4 &v) {
            if constexpr (DT == kF32) {
                top = max_abs_nan(top, __uint_as_float(v.x), __uint_as_float(v.y));
                top = max_abs_nan(top, __uint_as_float(v.z), __uint_as_float(v.w));
            } else {
                two = larger2<DT>(two, larger2<DT>(larger2<DT>(v.x, v.y), larger2<DT>(v.z, v.w)));
            }
        };
        int64_t i = first;
        for (; i + 3 * step < n; i += 4 * step) {
            uint4 v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = __ldg(vec + i + j * step);
#pragma unroll
            for (int j = 0; j < 4; ++j) add(v[j]);
        }
        for (; i < n; i += step) add(__ldg(vec + i));
        if constexpr (DT != kF32) {
            const uint32_t lo = two & 0x7FFFu, hi = two >> 16 & 0x7FFFu;
            top = Elem<DT>::up((uint16_t)(lo > hi ? lo : hi));
        }
        const int64_t tail = K - head - n * N;
        if (first < head) top = larger(top, Elem<DT>::up(__ldg(row + first)));
        if (first < tail) top = larger(top, Elem<DT>::up(__ldg(row + head + n * N + first)));
        return __float_as_uint(top);
    }
    const int64_t per_row = (K + kGroup - 1) / kGroup;
    int64_t row = first / per_row, g = first % per_row;
    const int64_t rows_step = step / per_row, g_step = step % per_row;
    while (row < T) {
        Group<DT> v;
        v.load(elem_at<DT>(x, row * ldx), g * kGroup, K);
        m = max(m, __float_as_uint(v.absmax()));
        row += rows_step;
        g += g_step;
        if (g >= per_row) {
            g -= per_row;
            ++row;
        }
    }
    return m;
}

__device__ __forceinline__ uint32_t cta_largest(uint32_t m, uint32_t *red, int warps) {
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
    __syncthreads();
    m = (int)(threadIdx.x & 31) < warps ? red[threadIdx.x & 31] : 0u;
    return __reduce_max_sync(0xFFFFFFFFu, m);
}

template <int DT>
__global__ void __launch_bounds__(kThreads) amax_kernel(const void *x, int64_t ldx, int64_t T,
                                                        int64_t K, uint32_t *amax) {
    __shared__ uint32_t red[kThreads / 32];
    pdl_wait_and_release();
    uint32_t m = absmax_of<DT>(x, ldx, T, K, (int64_t)blockIdx.x * kThreads + threadIdx.x,
                               (int64_t)gridDim.x * kThreads);
    m = cta_largest(m, red, kThreads / 32);
    if (threadIdx.x == 0) atomicMax(amax, m);      // whole numbers: in any order the same
}

// One cluster over the whole tensor: no initial value in memory, no second launch.
constexpr int kSmallCluster = 8, kSmallThreads = 512;
template <int DT>
__global__ void __launch_bounds__(kSmallThreads) amax_small_kernel(const void *x, int64_t ldx,
                                                                   int64_t T, int64_t K,
                                                                   uint32_t *amax) {
    __shared__ uint32_t red[kSmallThreads / 32], mine;
    cg::cluster_group cluster = cg::this_cluster();
    pdl_wait_and_release();
    uint32_t m = absmax_of<DT>(x, ldx, T, K, (int64_t)blockIdx.x * kSmallThreads + threadIdx.x,
                               (int64_t)kSmallCluster * kSmallThreads);
    m = cta_largest(m, red, kSmallThreads / 32);
    if (threadIdx.x == 0) mine = m;
    cluster.sync();
    if (blockIdx.x == 0 && threadIdx.x < 32) {
        m = threadIdx.x < kSmallCluster ? *cluster.map_shared_rank(&mine, threadIdx.x) : 0u;
        m = __reduce_max_sync(0xFFFFFFFFu, m);
        if (threadIdx.x == 0) *amax = m;
    }
    cluster.sync();
}

// ---- the way back ----------------------------------------------------------------------
//
// y = R(fl(fl(code s) g)); code s is exact.  A lane takes a 16-byte vector of the output at a
// time, so that a warp writes whole lines whatever the rows' alignment; of rows that do not begin
// at such a boundary (SHIFTED) a vector's codes begin anywhere and may belong to two blocks.  Bound
// by HBM: 8192 x 11008 to BF16 35 us (MXFP4, 6.5 TB/s) and 35 us (NVFP4); 1021 x 5003 to FP32 rows
// of any alignment 6.0 us (a group of 16 a lane, element by element: 21 us).
template <int DT, int FMT, bool SHIFTED, int PARTS>
__global__ void __launch_bounds__(kThreads, 8)
fp4_dequant_kernel(const uint8_t *codes, const uint8_t *scales, const float *amax, int64_t T,
                   int64_t K, void *y, int64_t ldy, uint32_t chunks) {
    using E = Elem<DT>;
    constexpr int N = E::kVec, kLen = fp4_block(FMT);
    pdl_wait_and_release();
    const float g = FMT == kNv ? tensor_scale(__ldg(amax)) : 1.0f;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t octet = blockIdx.x / chunks, chunk = blockIdx.x - octet * chunks;
    const int64_t row = (int64_t)(octet >> 4) * 128 + octet_row(octet & 15, warp);
    if (row >= T) return;
    // (places within a row, of at most 2^24 elements, in 32 bits)
    const int len = (int)K, row_bytes = (int)fp4_row_bytes(K);
    const uint8_t *from = codes + row * row_bytes;
    const uint8_t *scale = scales + word_at(row, 0, fp4_tiles_across(K, FMT));
    char *out = elem_at<DT>(y, row * ldy);
    const int skip = SHIFTED ? (int)(reinterpret_cast<uintptr_t>(out) & 15u) / E::kSize : 0;
    auto step_of = [&](int e) {                 // value of the scale of element e's block
        const uint32_t b = (uint32_t)e / kLen;
        return scale_value<FMT>(__ldg(scale + (b >> 2) * kScaleTile + (b & 3)));
    };
    const int e0 = ((int)chunk * PARTS * 32 + lane) * N - skip;
    uint32_t w[PARTS];
    float lo[PARTS], hi[PARTS];
#pragma unroll
    for (int p = 0; p < PARTS; ++p) {
        const int e = e0 + 32 * N * p;
        w[p] = 0;
        lo[p] = hi[p] = 0.0f;
        if (e >= len || e + N <= 0) continue;
        if constexpr (!SHIFTED) {
            if constexpr (N == 8) w[p] = __ldg(reinterpret_cast<const uint32_t *>(from + e / 2));
            else w[p] = __ldg(reinterpret_cast<const uint16_t *>(from + e / 2));
            lo[p] = step_of(e);
        } else {
            // eight codes from e on out of two words (before the row's first: none)
            const int at = e < 0 ? 0 : e & ~7;
            const uint32_t a0 = __ldg(reinterpret_cast<const uint32_t *>(from + at / 2));
            const uint32_t a1 = at / 2 + 4 < row_bytes ? __ldg(reinterpret_cast<const uint32_t *>(from + at / 2 + 4)) : 0u;
            w[p] = e < 0 ? a0 << (-4 * e) : __funnelshift_r(a0, a1, 4 * (e & 7));
            lo[p] = step_of(e < 0 ? 0 : e);
            hi[p] = step_of(e + N - 1 < len ? e + N - 1 : len - 1);
        }
    }
#pragma unroll
    for (int p = 0; p < PARTS; ++p) {
        const int e = e0 + 32 * N * p;
        if (e >= len || e + N <= 0) continue;
        uint32_t h[4];
        e2m1x8_to_f16(w[p], h);
        const int border = SHIFTED ? kLen - (e & (kLen - 1)) : N;   // elements of the first block
        float f[N];
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const float2 v = __half22float2(*reinterpret_cast<__half2 *>(&h[i]));
            const uint64_t s2 = SHIFTED ? f32x2(2 * i < border ? lo[p] : hi[p], 2 * i + 1 < border ? lo[p] : hi[p])
                                        : f32x2(lo[p], lo[p]);
            uint64_t q = mul_f32x2(f32x2(v.x, v.y), s2);
            if constexpr (FMT == kNv) q = mul_f32x2(q, f32x2(g, g));
            f[2 * i] = lo_f32(q);
            f[2 * i + 1] = hi_f32(q);
        }
        char *to = out + (int64_t)e * E::kSize;
        if (e >= 0 && e + N <= len) {
            *reinterpret_cast<uint4 *>(to) = E::pack(f);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (e + i >= 0 && e + i < len) store_elem<DT>(to, i, f[i]);
        }
    }
}

// ---- launches ------------------------------------------------------------------------------

// Rows of a launch whose octets take `chunks` CTAs each: CTA numbers stay within 31 bits.
int64_t rows_a_launch(int64_t chunks) { return ((1ll << 30) / chunks / 16 + 1) * 128; }
int octets(int64_t rows) { return (int)fp4_tiles_down(rows) * 16; }

template <int DT, int FMT>
cudaError_t launch_rows(const Fp4Quant &all, cudaStream_t st) {
    constexpr int kParts = DT == kF32 ? 1 : 2;             // 64 bytes a lane in flight
    // whole scale words
    const int64_t width = fp4_tiles_across(all.K, FMT) * fp4_tile_elems(FMT);
    const int64_t chunks = (width + kParts * kRun - 1) / (kParts * kRun), step = rows_a_launch(chunks);
    for (int64_t r = 0; r < all.T; r += step) {
        Fp4Quant a = all;
        a.T = all.T - r < step ? all.T - r : step;
        a.x = static_cast<const char *>(all.x) + r * all.ldx * Elem<DT>::kSize;
        a.codes += r * fp4_row_bytes(all.K);
        a.scales += r / 128 * fp4_tiles_across(all.K, FMT) * kScaleTile;
        const cudaError_t e = launch_pdl(fp4_rows_kernel<DT, FMT, kParts>, octets(a.T) * (int)chunks,
                                         kThreads, 0, st, a, (uint32_t)chunks);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

template <int DT, int FMT, bool ROWS>
cudaError_t launch_tiles(const Fp4Quant &a, cudaStream_t st) {
    static bool ready[kMaxDevices];
    using S = TileShape<DT>;
    constexpr int kSpan = fp4_tile_elems(FMT);
    constexpr int kScaleTiles = kTile / kSpan + (S::kRows > kSpan ? S::kRows / kSpan : 1);
    constexpr size_t bytes = S::kRows * kTile * Elem<DT>::kSize + kTile * S::kCodePitch +
                             kScaleTiles * kScaleTile;
    auto kernel = fp4_tiles_kernel<DT, FMT, ROWS>;
    const cudaError_t e = allow_shared(kernel, bytes, ready);
    if (e != cudaSuccess) return e;
    const int64_t tiles_k = (a.K + kTile - 1) / kTile, tiles = (a.T + S::kRows - 1) / S::kRows * tiles_k;
    if (tiles > 0x7FFFFFFFll) return cudaErrorInvalidValue;
    Fp4Quant b = a;
    b.level = reinterpret_cast<uintptr_t>(a.x) % 16 == 0 && (a.T == 1 || a.ldx * Elem<DT>::kSize % 16 == 0);
    return launch_pdl(kernel, (int)tiles, kThreads, bytes, st, b, tiles_k);
}

template <int DT, int FMT>
cudaError_t launch_quant(const Fp4Quant &a, cudaStream_t st) {
    if (!a.codes_t) return launch_rows<DT, FMT>(a, st);
    return a.codes ? launch_tiles<DT, FMT, true>(a, st) : launch_tiles<DT, FMT, false>(a, st);
}

template <int DT, int FMT, bool SHIFTED>
cudaError_t launch_dequant_rows(const uint8_t *codes, const uint8_t *scales, const float *amax,
                                int64_t T, int64_t K, char *y, int64_t ldy, cudaStream_t st) {
    constexpr int kParts = 4, N = Elem<DT>::kVec;
    const int64_t vectors = (K + N - 1 + (SHIFTED ? N - 1 : 0)) / N;
    const int64_t chunks = (vectors + 32 * kParts - 1) / (32 * kParts), step = rows_a_launch(chunks);
    for (int64_t r = 0; r < T; r += step) {
        const int64_t n = T - r < step ? T - r : step;
        const cudaError_t e = launch_pdl(
            fp4_dequant_kernel<DT, FMT, SHIFTED, kParts>, octets(n) * (int)chunks, kThreads, 0, st,
            codes + r * fp4_row_bytes(K), scales + r / 128 * fp4_tiles_across(K, FMT) * kScaleTile,
            amax, n, K, static_cast<void *>(y + r * ldy * Elem<DT>::kSize), ldy, (uint32_t)chunks);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

template <int DT, int FMT>
cudaError_t launch_dequant(const uint8_t *codes, const uint8_t *scales, const float *amax,
                           int64_t T, int64_t K, void *y, int64_t ldy, cudaStream_t st) {
    const bool level = reinterpret_cast<uintptr_t>(y) % 16 == 0 && (T == 1 || ldy * Elem<DT>::kSize % 16 == 0);
    return level ? launch_dequant_rows<DT, FMT, false>(codes, scales, amax, T, K, static_cast<char *>(y), ldy, st)
                 : launch_dequant_rows<DT, FMT, true>(codes, scales, amax, T, K, static_cast<char *>(y), ldy, st);
}

template <int DT>
cudaError_t launch_amax_type(const void *x, int64_t ldx, int64_t T, int64_t K, float *amax,
                             cudaStream_t st) {
    if (T == 0 || K == 0) {
        T = 1;
        K = 0;
    } else if (ldx == K) {                     // one long row
        K *= T;
        T = 1;
    }
    uint32_t *to = reinterpret_cast<uint32_t *>(amax);
    if (T * K <= (1 << 20))
        return launch_pdl_clusters(amax_small_kernel<DT>, kSmallCluster, kSmallThreads,
                                   kSmallCluster, 0, st, x, ldx, T, K, to);
    cudaError_t e = cudaMemsetAsync(amax, 0, 4, st);
    if (e != cudaSuccess) return e;
    const int64_t ctas = (T * ((K + kGroup - 1) / kGroup) + kThreads - 1) / kThreads;
    const int64_t most = 6ll * sm_count();
    return launch_pdl(amax_kernel<DT>, (int)(ctas < most ? ctas : most), kThreads, 0, st, x, ldx,
                      T, K, to);
}

}  // namespace

cudaError_t launch_amax(const void *x, int64_t ldx, int64_t T, int64_t K, int dtype, float *amax,
                        cudaStream_t st) {
    return dtype == kF32    ? launch_amax_type<kF32>(x, ldx, T, K, amax, st)
           : dtype == kBF16 ? launch_amax_type<kBF16>(x, ldx, T, K, amax, st)
                            : launch_amax_type<kF16>(x, ldx, T, K, amax, st);
}

cudaError_t launch_fp4_quant(const Fp4Quant &a, cudaStream_t st) {
    if (a.fmt == kMx)
        return a.dtype == kF32    ? launch_quant<kF32, kMx>(a, st)
               : a.dtype == kBF16 ? launch_quant<kBF16, kMx>(a, st)
                                  : launch_quant<kF16, kMx>(a, st);
    return a.dtype == kF32    ? launch_quant<kF32, kNv>(a, st)
           : a.dtype == kBF16 ? launch_quant<kBF16, kNv>(a, st)
                              : launch_quant<kF16, kNv>(a, st);
}

cudaError_t launch_fp4_dequant(const uint8_t *codes, const uint8_t *scales, const float *amax,
                               int64_t T, int64_t K, int fmt, void *y, int64_t ldy, int dtype,
                               cudaStream_t st) {
    auto pick = [&](auto mx, auto nv) {
        return fmt == kMx ? mx(codes, scales, amax, T, K, y, ldy, st)
                          : nv(codes, scales, amax, T, K, y, ldy, st);
    };
    return dtype == kF32    ? pick(launch_dequant<kF32, kMx>, launch_dequant<kF32, kNv>)
           : dtype == kBF16 ? pick(launch_dequant<kBF16, kMx>, launch_dequant<kBF16, kNv>)
                            : pick(launch_dequant<kF16, kMx>, launch_dequant<kF16, kNv>);
}

}  // namespace agoq
