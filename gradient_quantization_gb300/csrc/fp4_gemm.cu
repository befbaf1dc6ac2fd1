// fp4_gemm.cu -- the product of two operands in the micro-scaled 4-bit format
// (fp4_format.cuh), both K-major:
//   D[m][n] = R(gA gB sum_k a[m][k] b[n][k]),   a, b = E2M1 code times block scale
// on the block-scaled tensor cores: tcgen05.mma kind::mxf4 (MXFP4, a scale for 32 elements) and
// kind::mxf4nvf4 (NVFP4, a scale for 16) take packed codes from shared memory and the scales
// from tensor memory and add in binary32, so nothing is ever dequantised.
//
// The operand that fills the 128 lanes of an MMA is called P here, the one along its columns Q.
//   warp 0      TMA: a stage is 256 elements of K: 128-byte rows of codes of P and Q with the
//               128-byte swizzle, and the scale tiles of those rows, which lie in memory one
//               after another, by plain bulk copies;
//   warp 1      copies the stage's scale tiles to tensor memory (tcgen05.cp) and issues an MMA
//               for every 64 elements of K that the operands have (the last stage of a K that
//               is no multiple of 256 has fewer: what lies behind them is never read);
//   the others  the epilogue, a row of D a thread.
// Every stage has scale columns of its own, so a copy never overwrites scales that an MMA may
// still read.  Every wait is time-limited (gemm_common.cuh).
#include <algorithm>

#include "agoq_launch.h"
#include "fp4_format.cuh"
#include "gemm_common.cuh"
#include "typed_io.cuh"

namespace agoq {
namespace {

using namespace gemm;

__device__ unsigned g_fp4_status;

constexpr int BM = 128, BK = 256;                   // P rows of a CTA, elements of a stage
constexpr int kRowBytes = BK / 2;                   // 128: the swizzle's span
constexpr int kThreadsMma = 64;                     // warps 0 and 1

struct Fp4Args {
    const uint8_t *p_scales, *q_scales;
    const float *p_amax, *q_amax;
    int P, Q, K;                                    // rows of P and Q
    int across, p_down, q_down;                     // scale tiles
    void *d;
    int64_t ldd;
    int dtype;
    bool swapped;                                   // P is B: D[q][p]
    bool vectors;                                   // rows of D at 16-byte boundaries
};

// ---- instructions -----------------------------------------------------------------------
template <int GROUP>
__device__ __forceinline__ void scale_copy(uint32_t tmem, uint64_t desc) {
    if constexpr (GROUP == 2)
        asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
    else
        asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
}

#define AGOQ_FP4_MMA(GROUP, KIND)                                                                   \
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"                                  \
                 "tcgen05.mma.cta_group::" GROUP ".kind::" KIND " [%0], %1, %2, %3, [%5], [%6], p;" \
                 "\n\t}" ::"r"(d), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb) \
                 : "memory")
template <int FMT, int GROUP>
__device__ __forceinline__ void mma_fp4(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                        uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
    if constexpr (FMT == kNv && GROUP == 1) AGOQ_FP4_MMA("1", "mxf4nvf4.block_scale.scale_vec::4X");
    if constexpr (FMT == kNv && GROUP == 2) AGOQ_FP4_MMA("2", "mxf4nvf4.block_scale.scale_vec::4X");
    if constexpr (FMT == kMx && GROUP == 1) AGOQ_FP4_MMA("1", "mxf4.block_scale.scale_vec::2X");
    if constexpr (FMT == kMx && GROUP == 2) AGOQ_FP4_MMA("2", "mxf4.block_scale.scale_vec::2X");
}
#undef AGOQ_FP4_MMA

__device__ __forceinline__ void commit_one(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                     smem_u32(bar))
                 : "memory");
}

// A scale tile in shared memory: 32 rows of 16 bytes without swizzle, 8-row groups 128 bytes
// apart.
__device__ __forceinline__ uint64_t scale_desc(uint32_t saddr) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
    d |= static_cast<uint64_t>(128u >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    return d;
}

__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
            smem_u32(dst)),
        "l"(src), "r"(bytes), "r"(smem_u32(bar))
        : "memory");
}

// ---- shapes of a variant ------------------------------------------------------------------
//
// BN columns of D a tile.  PAIR: the two CTAs of a cluster share an MMA over 256 rows of P and
// BN of Q, half of whose codes each of them loads (the scales of all BN both need).  SPLIT: the
// CTAs of a cluster each take a part of K of one tile and join their sums.
template <int FMT, int BN_, bool PAIR_, bool SPLIT_>
struct Shape {
    static constexpr int BN = BN_;
    static constexpr bool PAIR = PAIR_, SPLIT = SPLIT_;
    static constexpr int kCtas = PAIR ? 2 : 1;
    static constexpr int kTileRows = BM * kCtas;
    static constexpr int kQRows = BN / kCtas;
    static constexpr int kQTiles = (BN + 127) / 128;            // row blocks of Q's scales
    static constexpr int kTiles = BK / fp4_tile_elems(FMT);     // scale tiles of a stage
    static constexpr int kPBytes = BM * kRowBytes, kQBytes = kQRows * kRowBytes;
    static constexpr int kPScales = kTiles * kScaleTile, kQScales = kQTiles * kTiles * kScaleTile;
    static constexpr int kStages = SPLIT ? (BN > 32 ? 3 : 4) : 5;
    static constexpr int kEpiWarps = SPLIT ? 4 : 8;
    static constexpr int kThreads = kThreadsMma + 32 * kEpiWarps;
    static constexpr int kBuffers = !SPLIT && BN <= 128 ? 2 : 1;   // accumulators
    static constexpr int kScaleCols = 4 * kTiles * (1 + kQTiles);
    static constexpr int kUsedCols = kBuffers * BN + kStages * kScaleCols;
    static constexpr int kTmemCols = kUsedCols <= 256 ? 256 : 512;
    static constexpr int kOffQ = kStages * kPBytes;
    static constexpr int kOffPS = kOffQ + kStages * kQBytes;
    static constexpr int kOffQS = kOffPS + kStages * kPScales;
    static constexpr int kOffRows = kOffQS + kStages * kQScales;
    static constexpr int kPitch = 17;                           // staged rows of 16 values
    static constexpr int kRowsBytes = SPLIT ? 0 : kEpiWarps * 32 * kPitch * 4;
    static constexpr int kOffBar = kOffRows + kRowsBytes;
    static constexpr int kBars = 3 * kStages + 2 * kBuffers + 1;
    static constexpr int kOffMisc = kOffBar + 8 * kBars;
    static constexpr int kSmem = kOffMisc + 16 + 1024;
    static constexpr uint32_t kIdesc = (1u << 7) | (1u << 10) | ((uint32_t)(BN >> 3) << 17) |
                                       (FMT == kMx ? 1u << 23 : 0u) |
                                       ((uint32_t)(kTileRows >> 4) << 24);
    static_assert(kUsedCols <= 512, "tensor memory");
    static_assert(kSmem <= 232448, "shared memory");
    static_assert(!SPLIT || BM * BN * 4 <= kStages * kPBytes, "the sums take the stages' place");
};

// Tiles in bands of kBand along Q: the CTAs at work share a few rows of both operands.
constexpr int kBand = 16;
__device__ __forceinline__ void tile_at(int tile, int num_p, int num_q, int &tp, int &tq) {
    const int band = tile / (kBand * num_p);
    const int nb = min(kBand, num_q - band * kBand);
    const int r = tile - band * kBand * num_p;
    tp = r / nb;
    tq = band * kBand + r % nb;
}

// 32 columns of D's row, as vectors.
__device__ __forceinline__ void store32(void *row, int64_t col, int dtype, const float *v) {
    if (dtype == kF32) {
        uint4 *to = reinterpret_cast<uint4 *>(static_cast<float *>(row) + col);
#pragma unroll
        for (int i = 0; i < 8; ++i) to[i] = Elem<kF32>::pack(v + 4 * i);
    } else if (dtype == kBF16) {
        uint4 *to = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(row) + col);
#pragma unroll
        for (int i = 0; i < 4; ++i) to[i] = Elem<kBF16>::pack(v + 8 * i);
    } else {
        uint4 *to = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(row) + col);
#pragma unroll
        for (int i = 0; i < 4; ++i) to[i] = Elem<kF16>::pack(v + 8 * i);
    }
}
__device__ __forceinline__ void store1(void *d, int64_t i, int dtype, float v) {
    if (dtype == kF32) store_elem<kF32>(d, i, v);
    else if (dtype == kBF16) store_elem<kBF16>(d, i, v);
    else store_elem<kF16>(d, i, v);
}

template <int FMT, class S>
__global__ void __launch_bounds__(S::kThreads, 1)
fp4_gemm_kernel(const __grid_constant__ CUtensorMap map_p, const __grid_constant__ CUtensorMap map_q,
                const Fp4Args a) {
    constexpr int NS = S::kStages, BN = S::BN, kGroup = S::PAIR ? 2 : 1;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t *sp = smem, *sq = smem + S::kOffQ, *sps = smem + S::kOffPS, *sqs = smem + S::kOffQS;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + S::kOffBar);
    uint64_t *full = bars, *empty = bars + NS, *ready = bars + 2 * NS, *tfull = bars + 3 * NS,
             *tempty = tfull + S::kBuffers, *drain = tempty + S::kBuffers;
    uint32_t *tmem_addr = reinterpret_cast<uint32_t *>(smem + S::kOffMisc);
    volatile int *abort = reinterpret_cast<volatile int *>(smem + S::kOffMisc + 4);
    unsigned *status = &g_fp4_status;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = S::PAIR || S::SPLIT ? (int)cluster_ctarank() : 0;
    const int pair_rank = S::PAIR ? rank : 0;
    uint32_t csize = 1;
    if constexpr (S::PAIR || S::SPLIT) asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(csize));
    const int C = (int)csize;
    const int cid = (int)blockIdx.x / C, ncl = (int)gridDim.x / C;
    const int num_p = (a.P + S::kTileRows - 1) / S::kTileRows, num_q = (a.Q + BN - 1) / BN;
    const int num_tiles = num_p * num_q;
    const int kall = (a.K + BK - 1) / BK;
    int kb0 = 0, kb1 = kall;                         // stages of this CTA
    if constexpr (S::SPLIT) {
        const int per = (kall + C - 1) / C;
        kb0 = min(rank * per, kall);
        kb1 = min(kb0 + per, kall);
    }

    if (threadIdx.x == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
            mbar_init(&ready[s], 1);
        }
        for (int b = 0; b < S::kBuffers; ++b) {
            mbar_init(&tfull[b], 1);
            mbar_init(&tempty[b], S::kEpiWarps * S::kCtas);
        }
        mbar_init(drain, 1);
        *abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        if constexpr (S::PAIR) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                             smem_u32(tmem_addr)), "r"(S::kTmemCols) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                             smem_u32(tmem_addr)), "r"(S::kTmemCols) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if constexpr (S::PAIR) cluster_sync_all();       // the peer's barriers are initialised
    const uint32_t tmem = *tmem_addr;
    // (after the allocation: a following launch may start and allocate only once every CTA of
    // this one has its columns)
    pdl_wait_and_release();

    if (warp == 0) {
        if (lane == 0) {
            uint32_t it = 0;
            bool ok = true;
            for (int tile = cid; ok && tile < num_tiles; tile += ncl) {
                int tp, tq;
                tile_at(tile, num_p, num_q, tp, tq);
                const int p0 = tp * S::kTileRows + BM * pair_rank, q0 = tq * BN;
                const int p_block = p0 / 128, q_block = q0 / 128;
                for (int kb = kb0; kb < kb1; ++kb, ++it) {
                    const int s = it % NS;
                    if (!wait_bar(&empty[s], ((it / NS) & 1u) ^ 1u, abort, status)) {
                        ok = false;
                        break;
                    }
                    // the scale tiles that exist
                    const uint32_t bytes = min(S::kTiles, a.across - kb * S::kTiles) * kScaleTile;
                    uint32_t all = S::kPBytes + S::kQBytes;
                    if (p_block < a.p_down) all += bytes;
#pragma unroll
                    for (int i = 0; i < S::kQTiles; ++i)
                        if (q_block + i < a.q_down) all += bytes;
                    mbar_expect_tx(&full[s], all);
                    tma_load_2d(sp + s * S::kPBytes, &map_p, &full[s], kb * kRowBytes, p0);
                    tma_load_2d(sq + s * S::kQBytes, &map_q, &full[s], kb * kRowBytes,
                                q0 + S::kQRows * pair_rank);
                    if (p_block < a.p_down)
                        bulk_load(sps + s * S::kPScales,
                                  a.p_scales + ((int64_t)p_block * a.across + kb * S::kTiles) * kScaleTile,
                                  bytes, &full[s]);
#pragma unroll
                    for (int i = 0; i < S::kQTiles; ++i)
                        if (q_block + i < a.q_down)
                            bulk_load(sqs + s * S::kQScales + i * S::kTiles * kScaleTile,
                                      a.q_scales + ((int64_t)(q_block + i) * a.across + kb * S::kTiles) * kScaleTile,
                                      bytes, &full[s]);
                }
            }
            for (int d = 0; d < NS && d < (int)it; ++d) {
                const uint32_t last = it - 1 - d;
                wait_bar(&full[last % NS], (last / NS) & 1u, abort, status, true);
            }
        }
    } else if (warp == 1) {
        if (lane == 0 && pair_rank == 0) {
            uint32_t it = 0, t = 0;
            bool ok = true, issued = false;
            for (int tile = cid; ok && tile < num_tiles; tile += ncl, ++t) {
                const int buf = t % S::kBuffers;
                if (!wait_bar(&tempty[buf], ((t / S::kBuffers) & 1u) ^ 1u, abort, status)) break;
                tc_fence_after();
                const uint32_t d = tmem + buf * BN;
                for (int kb = kb0; kb < kb1; ++kb, ++it) {
                    const int s = it % NS;
                    if (!wait_bar(&full[s], (it / NS) & 1u, abort, status) ||
                        (S::PAIR && !wait_bar(&ready[s], (it / NS) & 1u, abort, status))) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t cols = tmem + S::kBuffers * BN + s * S::kScaleCols;
                    const uint32_t qcols = cols + 4 * S::kTiles;
                    const uint32_t ps = smem_u32(sps + s * S::kPScales), qs = smem_u32(sqs + s * S::kQScales);
                    const int tiles = min(S::kTiles, a.across - kb * S::kTiles);
                    const int steps = min(4, (a.K - kb * BK + 63) / 64);
                    for (int j = 0; j < tiles; ++j) {
                        scale_copy<kGroup>(cols + 4 * j, scale_desc(ps + j * kScaleTile));
#pragma unroll
                        for (int i = 0; i < S::kQTiles; ++i)
                            scale_copy<kGroup>(qcols + 4 * (j * S::kQTiles + i),
                                               scale_desc(qs + (i * S::kTiles + j) * kScaleTile));
                    }
                    const uint64_t pd = sw128_kmajor_desc(smem_u32(sp + s * S::kPBytes));
                    const uint64_t qd = sw128_kmajor_desc(smem_u32(sq + s * S::kQBytes));
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        if (kk >= steps) break;
                        // a step is 32 bytes of a row; MXFP4: two scales of a tile's four
                        const int j = FMT == kNv ? kk : kk >> 1;
                        const uint32_t id = FMT == kNv ? 0 : 2 * (kk & 1);
                        mma_fp4<FMT, kGroup>(d, pd + 2 * kk, qd + 2 * kk,
                                             S::kIdesc | (id << 29) | (id << 4), cols + 4 * j,
                                             qcols + 4 * j * S::kQTiles, kb > kb0 || kk > 0);
                    }
                    issued = true;
                    if constexpr (S::PAIR) umma_commit_pair_multicast(&empty[s], 3);
                    else commit_one(&empty[s]);
                }
                if (!ok) break;
                if constexpr (S::PAIR) umma_commit_pair_multicast(&tfull[buf], 3);
                else if (kb0 < kb1) commit_one(&tfull[buf]);
            }
            if (issued) {
                if constexpr (S::PAIR) umma_commit_pair(drain);
                else commit_one(drain);
                wait_bar(drain, 0u, abort, status, true);
            }
        } else if (S::PAIR && lane == 0) {
            // CTA 1: each landed stage is announced to CTA 0
            const uint32_t ready0 = mapa_shared(smem_u32(ready), 0);
            uint32_t it = 0;
            bool ok = true;
            for (int tile = cid; ok && tile < num_tiles; tile += ncl) {
                for (int kb = kb0; kb < kb1; ++kb, ++it) {
                    const int s = it % NS;
                    if (!wait_bar(&full[s], (it / NS) & 1u, abort, status)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_remote(ready0 + (uint32_t)s * 8u);
                }
            }
        }
    } else if constexpr (!S::SPLIT) {
        // lane quarter of tensor memory: warp % 4; columns: half of the tile's
        const int q = warp & 3, half = (warp - 2) >> 2;
        constexpr int CW = BN / (S::kEpiWarps / 4);
        float *rows = reinterpret_cast<float *>(smem + S::kOffRows) + (warp - 2) * 32 * S::kPitch;
        const uint32_t tempty0 = S::PAIR ? mapa_shared(smem_u32(tempty), 0) : 0u;
        // the smaller tensor scale first: no overflow or underflow on the way
        float g0 = 1.0f, g1 = 1.0f;
        if constexpr (FMT == kNv) {
            const float gp = tensor_scale(__ldg(a.p_amax)), gq = tensor_scale(__ldg(a.q_amax));
            g0 = fminf(gp, gq);
            g1 = fmaxf(gp, gq);
        }
        const int es = a.dtype == kF32 ? 4 : 2;
        uint32_t t = 0;
        for (int tile = cid; tile < num_tiles; tile += ncl, ++t) {
            const int buf = t % S::kBuffers;
            if (!warp_wait(&tfull[buf], (t / S::kBuffers) & 1u, abort, status)) break;
            tc_fence_after();
            int tp, tq;
            tile_at(tile, num_p, num_q, tp, tq);
            const uint32_t from = tmem + ((uint32_t)(32 * q) << 16) + buf * BN + half * CW;
            float v[CW];
#pragma unroll
            for (int c = 0; c < CW; c += 32) {
                uint32_t w[32];
                tmem_ld32(from + c, w);
#pragma unroll
                for (int i = 0; i < 32; ++i) v[c + i] = __uint_as_float(w[i]);
            }
            // the accumulator is free as soon as it has been read
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (S::PAIR && rank != 0) mbar_arrive_remote(tempty0 + (uint32_t)buf * 8u);
                else mbar_arrive(&tempty[buf]);
            }
            if constexpr (FMT == kNv) {
#pragma unroll
                for (int i = 0; i < CW; ++i) v[i] = __fmul_rn(__fmul_rn(v[i], g0), g1);
            }
            const int r0 = tp * S::kTileRows + BM * pair_rank + 32 * q, row = r0 + lane;
            const int c0 = tq * BN + half * CW;
            if (a.swapped) {
#pragma unroll
                for (int i = 0; i < CW; ++i)
                    if (c0 + i < a.Q && row < a.P) store1(a.d, (int64_t)(c0 + i) * a.ldd + row, a.dtype, v[i]);
                continue;
            }
            char *out = static_cast<char *>(a.d) + (int64_t)row * a.ldd * es;
#pragma unroll
            for (int c = 0; c < CW; c += 32) {
                if (a.vectors && c0 + c + 32 <= a.Q) {
                    if (row < a.P) store32(out, c0 + c, a.dtype, v + c);
                    continue;
                }
                // rows that no vector fits: two rows of 16 values a step
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 16; ++i) rows[lane * S::kPitch + i] = v[c + 16 * h + i];
                    __syncwarp();
                    const int col = c0 + c + 16 * h + (lane & 15);
                    for (int r = lane >> 4; r < 32; r += 2)
                        if (r0 + r < a.P && col < a.Q)
                            store1(a.d, (int64_t)(r0 + r) * a.ldd + col, a.dtype,
                                   rows[r * S::kPitch + (lane & 15)]);
                }
            }
        }
    } else {
        // this CTA's part of the sums, as [column][row], in the stages' place
        const int q = warp & 3;
        float *sums = reinterpret_cast<float *>(smem);
        const bool any = kb0 < kb1;
        bool ok = true;
        if (any) {
            ok = warp_wait(&tfull[0], 0u, abort, status);
            tc_fence_after();
        }
        if (ok) {
#pragma unroll
            for (int c = 0; c < BN; c += 32) {
                uint32_t w[32];
                if (any) {
                    __syncwarp();
                    tmem_ld32(tmem + ((uint32_t)(32 * q) << 16) + c, w);
                }
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    sums[(c + i) * BM + 32 * q + lane] = any ? __uint_as_float(w[i]) : 0.0f;
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if constexpr (S::SPLIT) {
        cluster_sync_all();                          // all parts are there
        if (warp >= 2) {
            float g0 = 1.0f, g1 = 1.0f;
            if constexpr (FMT == kNv) {
                const float gp = tensor_scale(__ldg(a.p_amax)), gq = tensor_scale(__ldg(a.q_amax));
                g0 = fminf(gp, gq);
                g1 = fmaxf(gp, gq);
            }
            int tp, tq;
            tile_at(cid, num_p, num_q, tp, tq);
            const int r = (warp - 2) * 32 + lane, row = tp * BM + r;
            const uint32_t mine = smem_u32(smem);
            for (int c = rank; c < BN; c += C) {
                const int col = tq * BN + c;
                if (col >= a.Q) break;
                float v = 0.0f;
                for (int k = 0; k < C; ++k) {
                    float part;
                    asm volatile("ld.shared::cluster.f32 %0, [%1];"
                                 : "=f"(part)
                                 : "r"(mapa_shared(mine + (c * BM + r) * 4, k))
                                 : "memory");
                    v = __fadd_rn(v, part);
                }
                if constexpr (FMT == kNv) v = __fmul_rn(__fmul_rn(v, g0), g1);
                if (row < a.P)
                    store1(a.d, a.swapped ? (int64_t)col * a.ldd + row : (int64_t)row * a.ldd + col,
                           a.dtype, v);
            }
        }
    }
    // No CTA of a cluster frees tensor memory or exits while another may arrive on its barriers,
    // read its shared memory or have a shared MMA run on it.
    if constexpr (S::PAIR || S::SPLIT) cluster_sync_all();
    if (warp == 1) {
        __syncwarp();
        if constexpr (S::PAIR)
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                         "r"(S::kTmemCols) : "memory");
        else
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                         "r"(S::kTmemCols) : "memory");
    }
}

// ---- launches ---------------------------------------------------------------------------------
bool encode_codes(CUtensorMap *map, const uint8_t *codes, int64_t rows, int64_t K, int box_rows) {
    const uint64_t bytes = (uint64_t)fp4_row_bytes(K);
    return encode_2d(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, codes, bytes, (uint64_t)rows, bytes,
                     kRowBytes, (uint32_t)box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int FMT, class S>
cudaError_t launch_shape(const Fp4Args &a, const uint8_t *p_codes, const uint8_t *q_codes, int split,
                         cudaStream_t st) {
    CUtensorMap mp, mq;
    if (!encode_codes(&mp, p_codes, a.P, a.K, BM) || !encode_codes(&mq, q_codes, a.Q, a.K, S::kQRows))
        return cudaErrorInvalidValue;
    auto kernel = fp4_gemm_kernel<FMT, S>;
    static bool ready[kMaxDevices];
    const cudaError_t e = allow_shared(kernel, S::kSmem, ready);
    if (e != cudaSuccess) return e;
    const int cluster = S::PAIR ? 2 : split;
    const int64_t tiles = ((int64_t)a.P + S::kTileRows - 1) / S::kTileRows * (((int64_t)a.Q + S::BN - 1) / S::BN);
    int64_t clusters = tiles;
    if (!S::SPLIT) clusters = std::min<int64_t>(tiles, sm_count() / cluster);   // persistent
    if (tiles * S::kCtas > 0x3FFFFFFF || clusters * cluster > 0x3FFFFFFF) return cudaErrorInvalidValue;
    return launch_pdl_clusters(kernel, (int)clusters * cluster, S::kThreads, cluster, S::kSmem, st,
                               mp, mq, a);
}

template <int FMT>
cudaError_t launch_fmt(const Fp4Operand &A, const Fp4Operand &B, int64_t M, int64_t N, int64_t K,
                       void *d, int64_t ldd, int dtype, cudaStream_t st) {
    const int64_t small = std::min(M, N);
    // The 128 lanes take the operand with more rows where the other has few; else A.
    const bool swapped = small <= 64 && N > M;
    const Fp4Operand &p = swapped ? B : A, &q = swapped ? A : B;
    Fp4Args a{};
    a.p_scales = p.scales, a.q_scales = q.scales, a.p_amax = p.amax, a.q_amax = q.amax;
    a.P = (int)(swapped ? N : M), a.Q = (int)(swapped ? M : N), a.K = (int)K;
    a.across = (int)fp4_tiles_across(K, FMT);
    a.p_down = (int)fp4_tiles_down(a.P), a.q_down = (int)fp4_tiles_down(a.Q);
    a.d = d, a.ldd = ldd, a.dtype = dtype, a.swapped = swapped;
    const int es = dtype == kF32 ? 4 : 2;
    a.vectors = reinterpret_cast<uintptr_t>(d) % 16 == 0 && (ldd * es) % 16 == 0;
    if (small <= 64) {
        // the CTAs of a tile: as many as the GPU has room for, with two stages each at least
        const int64_t tiles = fp4_tiles_down(a.P), stages = (K + BK - 1) / BK;
        int split = 1;
        while (split < 8 && tiles * split * 2 <= 2 * sm_count() && stages >= split * 4) split *= 2;
        return small <= 32 ? launch_shape<FMT, Shape<FMT, 32, false, true>>(a, p.codes, q.codes, split, st)
                           : launch_shape<FMT, Shape<FMT, 64, false, true>>(a, p.codes, q.codes, split, st);
    }
    // tiles of 256 x 256 by CTA pairs where they fill the GPU
    const int64_t pairs = (M + 255) / 256 * ((N + 255) / 256);
    if (pairs * 2 >= sm_count())
        return launch_shape<FMT, Shape<FMT, 256, true, false>>(a, p.codes, q.codes, 1, st);
    return launch_shape<FMT, Shape<FMT, 128, false, false>>(a, p.codes, q.codes, 1, st);
}

}  // namespace

cudaError_t launch_fp4_gemm(const Fp4Operand &a, const Fp4Operand &b, int64_t M, int64_t N,
                            int64_t K, int fmt, void *d, int64_t ldd, int dtype, cudaStream_t st) {
    return fmt == kMx ? launch_fmt<kMx>(a, b, M, N, K, d, ldd, dtype, st)
                      : launch_fmt<kNv>(a, b, M, N, K, d, ldd, dtype, st);
}

// Read and clear the status word (the caller has synchronised).
cudaError_t read_and_clear_fp4_status(unsigned *status) {
    unsigned v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_fp4_status, sizeof v);
    if (e != cudaSuccess) return e;
    if (v) {
        const unsigned zero = 0;
        e = cudaMemcpyToSymbol(g_fp4_status, &zero, sizeof zero);
        if (e != cudaSuccess) return e;
    }
    *status = v;
    return cudaSuccess;
}

}  // namespace agoq
