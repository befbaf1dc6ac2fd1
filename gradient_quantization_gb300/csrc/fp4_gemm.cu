// fp4_gemm.cu -- the product of two operands in the micro-scaled 4-bit format
// (fp4_format.cuh), both K-major:
//   D[m][n] = R(gA gB sum_k a[m][k] b[n][k]),   a, b = E2M1 code times block scale
// on the block-scaled tensor cores: tcgen05.mma kind::mxf4 (MXFP4, a scale for 32 elements) and
// kind::mxf4nvf4 (NVFP4, a scale for 16) take packed codes from shared memory and the scales
// from tensor memory and add in binary32, so nothing is ever dequantised.
//
// The operand that fills the 128 lanes of an MMA is called P here, the one along its columns Q.
//   warp 0      TMA: a stage is 256 elements of K: 128-byte rows of codes of P and Q with the
//               128-byte swizzle;
//   warp 2      the scale tiles of those rows, which lie in memory one after another, by plain
//               bulk copies into a ring of their own that runs ahead of the codes;
//   warps 4-7   write a stage's scales to tensor memory, each to the lanes that it reaches: the
//               MMA wants them in all four lane quarters;
//   warp 1      issues an MMA for every 64 elements of K that the operands have (the last stage
//               of a K that is no multiple of 256 has fewer: what lies behind is never used);
//   the others  the epilogue (SPLIT: warps 4-7).
// Every stage has scale columns of its own, so that a write never meets an MMA that still reads.
//
// Measured (in a graph, inputs warm): 8192^3 NVFP4 to BF16 163 us (6.7 PFLOP/s), 8192 x 11008 x 4096
// 124 us (6.0), 11008 x 4096 x 8192 MXFP4 to FP32 118 us (6.3); 1 x 11008 x 4096 8.1 us (3.1 TB/s of
// operands).  Products one after another for a second, with operands that change, or on another GPU of
// the same kind, take up to 16% longer, by the clock (8192 x 11008 x 4096 123 to 139 us).  The MMAs of a
// pair for 256 x 256 x 64, two of 128 columns, take 128 cycles together, which is 10.2 PFLOP/s at 2.05
// GHz; a stage of four such steps takes 542 (MXFP4) or 584 (NVFP4) where its operands come from the L2
// cache, by one pair or by all, and about 730 at 4096 x 4864 x 16384 on all pairs, by the traffic of the
// L2 (584 again where the same number of tiles read the same rows).  (The chip's nominal rate, 13.5, is
// that of an MMA of 96 elements of K, which is not used here: where all pairs read rows of their own, the
// L2's traffic is the nearer bound.)  The rest at large sizes: the end of a tile, 1.3 us
// before its halves were ordered apart (below: kHold; 129, 121 and 167 us without), as the two CTAs' 256
// columns are the only accumulator (tensor memory has no room for a second one beside the scales); the
// last round (8192 x 11008 is 18.1 rounds of 76 pairs); and the clock, which falls from 2070 MHz to
// 1750 in a second of such products.  What bounded it before: the thread that issues MMAs, whose two
// waits, four MMAs and commit took 940 cycles a stage with operands in ordinary registers (now one wait
// of the whole warp and an elected lane); scale tiles by tcgen05.cp, 50 to 110 cycles of the MMAs' own
// pipe for each of a stage's twelve (266 us for 8192 x 11008 x 4096); clusters of two pairs that share Q by multicast, of which
// 36 fit the GPU (72 of 76 pairs) and which moved less without being faster (81 us for 4096 x 4864 x
// 8192, 67 us then by pairs).  Few rows are bound by latency: a call of one tile and one stage takes
// 4.7 us, of which the loads are 1.1, the scales' way to tensor memory 0.7, the MMAs and their
// commit 0.8, and the sums' way out 1.0.
//
// Every wait is time-limited (gemm_common.cuh).
#include <algorithm>

#include "agoq_launch.h"
#include "fp4_format.cuh"
#include "fp4_split.h"
#include "gemm_common.cuh"
#include "typed_io.cuh"

namespace agoq {
namespace {

using namespace gemm;

__device__ unsigned g_fp4_status;

constexpr int BM = 128, BK = 256;                   // P rows of a CTA, elements of a stage
constexpr int kRowBytes = BK / 2;                   // 128: the swizzle's span
// Warps of a role make up whole warpgroups, whose registers can be shared out.
constexpr int kTmaWarp = 0, kMmaWarp = 1, kScaleTmaWarp = 2, kScaleWarp0 = 4;

struct Fp4Args {
    const uint8_t *p_scales, *q_scales;
    const float *p_amax, *q_amax;
    int P, Q, K;                                    // rows of P and Q
    int across, p_down, q_down;                     // scale tiles
    void *d;
    int64_t ldd;
    int dtype;
    bool swapped;                                   // P is B: D[q][p]
    bool vectors, whole;                            // rows of D begin, and end, at 16-byte boundaries
};

// ---- instructions -----------------------------------------------------------------------
#define AGOQ_FP4_MMA(GROUP, KIND)                                                                   \
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"                                  \
                 "tcgen05.mma.cta_group::" GROUP ".kind::" KIND " [%0], %1, %2, %3, [%5], [%6], p;" \
                 "\n\t}" ::"r"(d), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb) \
                 : "memory")
template <int FMT, bool PAIR>
__device__ __forceinline__ void mma_fp4(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                        uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
    if constexpr (FMT == kNv && !PAIR) AGOQ_FP4_MMA("1", "mxf4nvf4.block_scale.scale_vec::4X");
    if constexpr (FMT == kNv && PAIR) AGOQ_FP4_MMA("2", "mxf4nvf4.block_scale.scale_vec::4X");
    if constexpr (FMT == kMx && !PAIR) AGOQ_FP4_MMA("1", "mxf4.block_scale.scale_vec::2X");
    if constexpr (FMT == kMx && PAIR) AGOQ_FP4_MMA("2", "mxf4.block_scale.scale_vec::2X");
}
#undef AGOQ_FP4_MMA

__device__ __forceinline__ void commit_one(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                     smem_u32(bar))
                 : "memory");
}

__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
            smem_u32(dst)),
        "l"(src), "r"(bytes), "r"(smem_u32(bar))
        : "memory");
}
// A tile load of one CTA of a pair whose bytes count on a barrier of either (`bar`: its address
// in the cluster).
__device__ __forceinline__ void tma_load_2d_pair(void *dst, const CUtensorMap *map, uint32_t bar, int x,
                                                 int y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
        : "memory");
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap *map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}
__device__ __forceinline__ void tma_store_2d(const CUtensorMap *map, const void *src, int x, int y) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(smem_u32(src)), "r"(x), "r"(y)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// Wait until none of this thread's stores still reads shared memory.
__device__ __forceinline__ void stores_read() {
    asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t *v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
                 "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t *v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
        "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}

// ---- shapes of a variant ------------------------------------------------------------------
//
// BN columns of D a tile.  PAIR: the two CTAs of a cluster share an MMA over 256 rows of P and
// BN of Q, half of whose codes each of them holds (the scales of all BN both need).  SPLIT: the
// CTAs of a cluster each take a part of K of one tile and join their sums.
template <int FMT, int BN_, bool PAIR_, bool SPLIT_>
struct Shape {
    static constexpr int BN = BN_;
    static constexpr bool PAIR = PAIR_, SPLIT = SPLIT_;
    static constexpr int kCluster = PAIR ? 2 : 1;               // (SPLIT: given at launch)
    static constexpr int kTileRows = BM * kCluster;             // of a cluster
    static constexpr int kQRows = BN / kCluster;
    static constexpr int kQTiles = (BN + 127) / 128;            // row blocks of Q's scales
    static constexpr int kTiles = BK / fp4_tile_elems(FMT);     // scale tiles of a stage
    static constexpr int kPBytes = BM * kRowBytes, kQBytes = kQRows * kRowBytes;
    static constexpr int kPScales = kTiles * kScaleTile, kQScales = kQTiles * kTiles * kScaleTile;
    static constexpr int kStages = !SPLIT ? 5 : BN == 64 ? 3 : 4;    // (SPLIT, BN < 128: two CTAs an SM)
    static constexpr int kScaleWarps = 4, kEpiWarps = SPLIT ? 0 : 8;
    static constexpr int kThreads = 32 * (kScaleWarp0 + kScaleWarps + kEpiWarps);
    static constexpr int kBuffers = !SPLIT && BN <= 128 ? 2 : 1;   // accumulators
    // A pair's accumulator is two halves of its columns, each with MMAs and barriers of its own.
    static constexpr int kHalves = PAIR ? 2 : 1;
    static constexpr int kAccs = kBuffers * kHalves, kAccCols = BN / kHalves;
    static constexpr int kScaleCols = 4 * kTiles * (1 + kQTiles);
    static constexpr int kUsedCols = kBuffers * BN + kStages * kScaleCols;
    static constexpr int kTmemCols = kUsedCols <= 256 ? 256 : 512;
    static constexpr int kOffQ = kStages * kPBytes;
    static constexpr int kOffOut = kOffQ + kStages * kQBytes;
    static constexpr int kOutBytes = 4096;                      // an epilogue warp's buffer
    static constexpr int kOffPS = kOffOut + kEpiWarps * kOutBytes;
    static constexpr int kOffQS = kOffPS + kStages * kPScales;
    static constexpr int kOffBar = kOffQS + kStages * kQScales;
    static constexpr int kBars = 4 * kStages + 2 * kAccs + 1;
    static constexpr int kOffMisc = kOffBar + 8 * kBars;
    static constexpr int kSmem = kOffMisc + 16 + 1024;
    static constexpr uint32_t kIdesc = (1u << 7) | (1u << 10) | ((uint32_t)(kAccCols >> 3) << 17) |
                                       (FMT == kMx ? 1u << 23 : 0u) |
                                       ((uint32_t)(kTileRows >> 4) << 24);
    static_assert(kUsedCols <= 512, "tensor memory");
    static_assert(kSmem <= 232448, "shared memory");
    static_assert(!SPLIT || BM * BN * 4 <= kStages * kPBytes, "the sums take the stages' place");
};

// The wait of a whole warp, all lanes at once.  A phase that is complete, as most are in a loop
// that runs behind its producers, costs one test (with a lane that waits and tells the others,
// 250 cycles of a stage's 500).  Returns false as wait_bar does.
__device__ __forceinline__ bool mbar_test(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool warp_wait_all(uint64_t *bar, uint32_t parity, volatile int *abort,
                                              unsigned *status, uint32_t hint_ns) {
    if (__all_sync(0xFFFFFFFFu, mbar_test(bar, parity))) return true;
    return warp_wait(bar, parity, abort, status, hint_ns);
}
// One lane of a converged warp; what runs under it keeps its operands in uniform registers.
__device__ __forceinline__ bool elect_one() {
    uint32_t is;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(is));
    return is != 0;
}

// A place in a ring of NS stages and the parity of its use.
template <int NS>
struct Ring {
    int s = 0;
    uint32_t parity = 0;
    __device__ __forceinline__ void next() {
        if (++s == NS) {
            s = 0;
            parity ^= 1u;
        }
    }
};

// Waits that are long as a rule let the thread sleep: a poll takes an issue slot and a cycle of
// the shared memory that the MMAs read from.
constexpr uint32_t kSleepNs = 20000;

// Stages of a pair whose MMAs are ordered by halves of the accumulator at a tile's end and the next
// one's begin: the first half is read while the second half's last MMAs run, and the second while
// the next tile's first MMAs run in the first.  They are held until the second half's MMAs are done.
// 8192 x 11008 x 4096: 124 us with three, 125 with two, 129 without; four 2% slower than three.
constexpr int kHold = 3;
static_assert(kHold >= 1 && kHold < 5, "stages held, of five");

// Tiles in bands of kBand along Q: the CTAs at work share a few rows of both operands.
constexpr int kBand = 16;
__device__ __forceinline__ void tile_at(int tile, int num_p, int num_q, int &tp, int &tq) {
    const int band = tile / (kBand * num_p);
    const int nb = min(kBand, num_q - band * kBand);
    const int r = tile - band * kBand * num_p;
    tp = r / nb;
    tq = band * kBand + r % nb;
}

__device__ __forceinline__ void store1(void *d, int64_t i, int dtype, float v) {
    if (dtype == kF32) store_elem<kF32>(d, i, v);
    else if (dtype == kBF16) store_elem<kBF16>(d, i, v);
    else store_elem<kF16>(d, i, v);
}

// 32 rows of 128 bytes, 16-byte vectors swizzled (`buf`), to rows of D that lie anywhere: a row
// at a time, its 16-bit values in aligned pairs.
template <int DT>
__device__ __forceinline__ void store_lines(const uint8_t *buf, char *out, int64_t row_step, int rows, int cols,
                                            int lane) {
    auto at = [&](int r, int e) {
        constexpr int kVec = Elem<DT>::kVec;
        return buf + r * 128 + (((e / kVec) ^ (r & 7)) << 4) + e % kVec * Elem<DT>::kSize;
    };
#pragma unroll 4
    for (int r = 0; r < rows; ++r, out += row_step) {
        if constexpr (DT == kF32) {
            if (lane < cols) reinterpret_cast<float *>(out)[lane] = *reinterpret_cast<const float *>(at(r, lane));
        } else {
            uint16_t *to = reinterpret_cast<uint16_t *>(out);
            const int odd = (int)(reinterpret_cast<uintptr_t>(out) >> 1) & 1, e = 2 * lane + odd;
            if (e < cols) {
                const uint32_t lo = *reinterpret_cast<const uint16_t *>(at(r, e));
                if (e + 1 < cols) {
                    const uint32_t hi = *reinterpret_cast<const uint16_t *>(at(r, e + 1));
                    *reinterpret_cast<uint32_t *>(to + e) = lo | hi << 16;
                } else {
                    to[e] = (uint16_t)lo;
                }
            }
            if (odd && lane == 0) to[0] = *reinterpret_cast<const uint16_t *>(at(r, 0));
        }
    }
}

// An epilogue warp's 32 rows x CW columns, by way of 128-byte wide boxes in shared memory, swizzled
// so that the lanes' 16-byte stores meet no bank twice: by TMA, or where D's rows do not lie at
// 16-byte boundaries line by line.  `free_acc` is called as soon as the accumulator has been read:
// the next tile's MMAs have five stages to run through and so make up for a short pause.
template <int FMT, int DT, int CW, class F>
__device__ __forceinline__ void store_tile(const CUtensorMap *map, uint8_t *buf, uint32_t from, int row,
                                           int col, const Fp4Args &a, float g0, float g1, int lane,
                                           F free_acc) {
    constexpr int kCols = DT == kF32 ? 32 : 64, kBoxes = CW / kCols;
    // (a box across the end of rows that are no whole 16-byte vectors would write up to the next
    // vector's end)
    const bool boxes = a.vectors && (a.whole || col + CW <= a.Q);
    auto put = [&](int c, const uint4 (&o)[8]) {
        if (lane == 0) stores_read();
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i)
            *reinterpret_cast<uint4 *>(buf + lane * 128 + ((i ^ (lane & 7)) << 4)) = o[i];
        const int at = col + c * kCols;
        if (boxes) {
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0 && row < a.P && at < a.Q) tma_store_2d(map, buf, at, row);
        } else {
            __syncwarp();
            constexpr int kSize = Elem<DT>::kSize;
            if (at < a.Q)
                store_lines<DT>(buf, static_cast<char *>(a.d) + ((int64_t)row * a.ldd + at) * kSize,
                                a.ldd * kSize, min(32, a.P - row), min(kCols, a.Q - at), lane);
            __syncwarp();
        }
    };
    // all loads of the accumulator in flight at once
    uint32_t w[CW / 16][16];
#pragma unroll
    for (int c = 0; c < CW / 16; ++c) tmem_ld16_nowait(from + 16 * c, w[c]);
    tmem_wait_ld();
    free_acc();
#pragma unroll
    for (int c = 0; c < kBoxes; ++c) {
        uint4 o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float v[Elem<DT>::kVec];
#pragma unroll
            for (int j = 0; j < Elem<DT>::kVec; ++j) {
                const int at = c * kCols + i * Elem<DT>::kVec + j;
                v[j] = __uint_as_float(w[at / 16][at % 16]);
                if constexpr (FMT == kNv) v[j] = __fmul_rn(__fmul_rn(v[j], g0), g1);
            }
            o[i] = Elem<DT>::pack(v);
        }
        put(c, o);
    }
}

template <int FMT, class S>
__global__ void __launch_bounds__(S::kThreads, 1)
fp4_gemm_kernel(const __grid_constant__ CUtensorMap map_p, const __grid_constant__ CUtensorMap map_q,
                const __grid_constant__ CUtensorMap map_d, const Fp4Args a) {
    constexpr int NS = S::kStages, BN = S::BN;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t *sp = smem, *sq = smem + S::kOffQ, *sps = smem + S::kOffPS, *sqs = smem + S::kOffQS;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + S::kOffBar);
    uint64_t *full = bars, *empty = bars + NS, *sfull = bars + 2 * NS, *sempty = bars + 3 * NS,
             *tfull = bars + 4 * NS, *tempty = tfull + S::kAccs,
             *drain = tempty + S::kAccs;
    uint32_t *tmem_addr = reinterpret_cast<uint32_t *>(smem + S::kOffMisc);
    volatile int *abort = reinterpret_cast<volatile int *>(smem + S::kOffMisc + 4);
    unsigned *status = &g_fp4_status;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = S::PAIR || S::SPLIT ? (int)cluster_ctarank() : 0;
    const int side = S::PAIR ? rank : 0;
    uint32_t csize = 1;
    if constexpr (S::PAIR || S::SPLIT) asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(csize));
    const int C = (int)csize;
    const int cid = (int)blockIdx.x / C, ncl = (int)gridDim.x / C;
    const int num_p = (a.P + S::kTileRows - 1) / S::kTileRows, num_q = (a.Q + BN - 1) / BN;
    const int num_tiles = num_p * num_q;
    const int kall = (a.K + BK - 1) / BK;
    int kb0 = 0, kb1 = kall;                         // stages of this CTA
    if constexpr (S::SPLIT) {
        const int per = (kall + C - 1) / C;          // (fp4_split.h: every CTA has stages)
        kb0 = rank * per;
        kb1 = min(kb0 + per, kall);
    }

    if (threadIdx.x == 32 * kScaleTmaWarp) {         // (their first use would wait for them)
        prefetch_map(&map_p);
        prefetch_map(&map_q);
        if (!S::SPLIT && a.vectors) prefetch_map(&map_d);
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(&full[s], 1 + S::kScaleWarps * S::kCluster);   // codes, and scales written
            mbar_init(&empty[s], 1);
            mbar_init(&sfull[s], 1);
            mbar_init(&sempty[s], S::kScaleWarps);
        }
        for (int b = 0; b < S::kAccs; ++b) {
            mbar_init(&tfull[b], 1);
            mbar_init(&tempty[b], S::SPLIT ? 1 : S::kEpiWarps * S::kCluster / S::kHalves);
        }
        mbar_init(drain, 1);
        *abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kMmaWarp) {
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
    if constexpr (S::PAIR) cluster_sync_all();       // the others' barriers are initialised
    const uint32_t tmem = *tmem_addr;
    const uint32_t scale_cols = tmem + S::kBuffers * BN;
    // (after the allocation: a following launch may start and allocate only once every CTA of
    // this one has its columns)
    pdl_wait_and_release();
    // (long before they are needed.  The smaller tensor scale is multiplied first: no overflow or
    // underflow on the way.)
    float g0 = 1.0f, g1 = 1.0f;
    if (FMT == kNv && (S::SPLIT || warp >= kScaleWarp0)) {
        const float gp = tensor_scale(__ldg(a.p_amax)), gq = tensor_scale(__ldg(a.q_amax));
        g0 = min_nan(gp, gq);
        g1 = max_nan(gp, gq);
    }
    // The epilogue holds 128 columns of a row.  512 threads were launched with 128 registers each:
    // 2 * 80 + 2 * 176 a thread of the four warpgroups is 4 * 128.
    if (warp < kScaleWarp0) {
        if constexpr (!S::SPLIT) asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
        if (warp == kTmaWarp) {
            if (lane == 0) {
                // A pair's codes all count on the barrier of its CTA 0, which issues the MMAs; so do the
                // warps that write scales.
                const uint32_t full0 = S::PAIR ? mapa_shared(smem_u32(full), 0) : 0u;
                uint32_t it = 0;
                bool ok = true;
                Ring<NS> ring;
                for (int tile = cid; ok && tile < num_tiles; tile += ncl) {
                    int tp, tq;
                    tile_at(tile, num_p, num_q, tp, tq);
                    const int p0 = tp * S::kTileRows + BM * side, q0 = tq * BN + S::kQRows / S::kHalves * side;
                    for (int kb = kb0; kb < kb1; ++kb, ++it, ring.next()) {
                        const int s = ring.s;
                        if (!wait_bar(&empty[s], ring.parity ^ 1u, abort, status, false, kSleepNs)) {
                            ok = false;
                            break;
                        }
                        if (side == 0) mbar_expect_tx(&full[s], (S::kPBytes + S::kQBytes) * S::kCluster);
                        if constexpr (S::PAIR) {
                            tma_load_2d_pair(sp + s * S::kPBytes, &map_p, full0 + 8u * s, kb * kRowBytes, p0);
                            // (an MMA of one half of the columns takes half of them from each CTA)
#pragma unroll
                            for (int h = 0; h < S::kHalves; ++h)
                                tma_load_2d_pair(sq + s * S::kQBytes + h * (S::kQBytes / S::kHalves), &map_q,
                                                 full0 + 8u * s, kb * kRowBytes, q0 + h * S::kAccCols);
                        } else {
                            tma_load_2d(sp + s * S::kPBytes, &map_p, &full[s], kb * kRowBytes, p0);
                            tma_load_2d(sq + s * S::kQBytes, &map_q, &full[s], kb * kRowBytes, q0);
                        }
                    }
                }
                // (CTA 1 of a pair leaves the wait for its copies to CTA 0, which sees both's: neither
                // exits before the other)
                for (int d = 0; side == 0 && d < NS && d < (int)it; ++d) {
                    const uint32_t last = it - 1 - d;
                    wait_bar(&full[last % NS], (last / NS) & 1u, abort, status, true);
                }
            }
        } else if (warp == kScaleTmaWarp) {
            if (lane == 0) {
                uint32_t it = 0;
                bool ok = true;
                Ring<NS> ring;
                for (int tile = cid; ok && tile < num_tiles; tile += ncl) {
                    int tp, tq;
                    tile_at(tile, num_p, num_q, tp, tq);
                    const int p_block = (tp * S::kTileRows) / 128 + side, q_block = tq * BN / 128;
                    const uint8_t *ps = a.p_scales + (int64_t)p_block * a.across * kScaleTile;
                    const uint8_t *qs = a.q_scales + (int64_t)q_block * a.across * kScaleTile;
                    for (int kb = kb0; kb < kb1; ++kb, ++it, ring.next()) {
                        const int s = ring.s;
                        if (!wait_bar(&sempty[s], ring.parity ^ 1u, abort, status, false, kSleepNs)) {
                            ok = false;
                            break;
                        }
                        // the scale tiles that exist
                        const uint32_t bytes = min(S::kTiles, a.across - kb * S::kTiles) * kScaleTile;
                        const int64_t at = (int64_t)kb * S::kTiles * kScaleTile;
                        uint32_t all = p_block < a.p_down ? bytes : 0u;
#pragma unroll
                        for (int i = 0; i < S::kQTiles; ++i) all += q_block + i < a.q_down ? bytes : 0u;
                        mbar_expect_tx(&sfull[s], all);
                        if (p_block < a.p_down) bulk_load(sps + s * S::kPScales, ps + at, bytes, &sfull[s]);
#pragma unroll
                        for (int i = 0; i < S::kQTiles; ++i)
                            if (q_block + i < a.q_down)
                                bulk_load(sqs + s * S::kQScales + i * S::kTiles * kScaleTile,
                                          qs + (int64_t)i * a.across * kScaleTile + at, bytes, &sfull[s]);
                    }
                }
                for (int d = 0; d < NS && d < (int)it; ++d) {
                    const uint32_t last = it - 1 - d;
                    wait_bar(&sfull[last % NS], (last / NS) & 1u, abort, status, true);
                }
            }
        } else if (warp == kMmaWarp) {
            if (side == 0) {
                // the whole warp runs the loop, one lane issues
                uint32_t t = 0;
                bool ok = true, issued = false;
                Ring<NS> ring, second;               // stages of the first half's MMAs and the second's
                const uint64_t pd0 = sw128_kmajor_desc(smem_u32(sp)), qd0 = sw128_kmajor_desc(smem_u32(sq));
                for (int tile = cid; ok && tile < num_tiles; tile += ncl, ++t) {
                    const int buf = t % S::kBuffers;
                    const uint32_t free_parity = ((t / S::kBuffers) & 1u) ^ 1u;
                    if (!S::SPLIT && !warp_wait_all(&tempty[buf], free_parity, abort, status, 0)) break;
                    tc_fence_after();
                    const uint32_t d = tmem + buf * BN;
                    // Waits for the ring's stage, which is issued next: from then on MMAs may be in flight,
                    // however the loop ends, and the drain below waits for them.
                    auto stage_there = [&] {
                        if (!warp_wait_all(&full[ring.s], ring.parity, abort, status, 0)) return false;
                        tc_fence_after();
                        issued = true;
                        return true;
                    };
                    // the MMAs of stage kb, in place s, for halves h0 .. h1 - 1
                    auto issue = [&](int s, int kb, int h0, int h1) {
                        const int left = a.K - kb * BK;          // elements of K from this stage on
                        const uint32_t cols = scale_cols + s * S::kScaleCols, qcols = cols + 4 * S::kTiles;
                        const uint64_t pd = pd0 + (uint32_t)s * (S::kPBytes >> 4);
                        const uint64_t qd = qd0 + (uint32_t)s * (S::kQBytes >> 4);
                        auto step = [&](int kk, uint32_t accumulate) {
                            // a step is 32 bytes of a row; MXFP4: two scales of a tile's four
                            const int j = FMT == kNv ? kk : kk >> 1;
                            const uint32_t id = FMT == kNv ? 0 : 2 * (kk & 1);
#pragma unroll
                            for (int h = 0; h < S::kHalves; ++h)
                                if (h >= h0 && h < h1)
                                    mma_fp4<FMT, S::PAIR>(d + h * S::kAccCols, pd + 2 * kk,
                                                          qd + h * (S::kQBytes / S::kHalves >> 4) + 2 * kk,
                                                          S::kIdesc | (id << 29) | (id << 4), cols + 4 * j,
                                                          qcols + 4 * (j * S::kQTiles + h), accumulate);
                        };
                        step(0, kb > kb0);
                        if (left > 192) {
                            step(1, 1);
                            step(2, 1);
                            step(3, 1);
                        } else {
                            if (left > 64) step(1, 1);
                            if (left > 128) step(2, 1);
                        }
                    };
                    if constexpr (S::PAIR) {
                        // kHold stages at a tile's begin and its end: all MMAs of the first half, then those
                        // of the second.  Between them both halves of a stage at a time.
                        int kb = 0;
                        auto by_halves = [&](bool begin, bool end, int some) {
                            for (int i = 0; i < some; ++i, ring.next()) {
                                if (!stage_there()) return false;
                                if (elect_one()) {
                                    issue(ring.s, kb + i, 0, 1);
                                    if (end && i == some - 1) umma_commit_pair_multicast(&tfull[0], 3);
                                }
                                __syncwarp();
                            }
                            if (begin) {
                                if (!warp_wait_all(&tempty[1], free_parity, abort, status, 0)) return false;
                                tc_fence_after();
                            }
                            for (int i = 0; i < some; ++i, ++kb, second.next()) {
                                if (elect_one()) {
                                    issue(second.s, kb, 1, 2);
                                    umma_commit_pair_multicast(&empty[second.s], 3);
                                    if (end && i == some - 1) umma_commit_pair_multicast(&tfull[1], 3);
                                }
                                __syncwarp();
                            }
                            return true;
                        };
                        // (at the first tile no accumulator is being read)
                        const int held = t > 0 ? min(kHold, kall) : 0;
                        ok = by_halves(true, held == kall, held);
                        for (; ok && kb < kall - kHold; ++kb, ring.next()) {
                            ok = stage_there();
                            if (!ok) break;
                            if (elect_one()) {
                                issue(ring.s, kb, 0, 2);
                                umma_commit_pair_multicast(&empty[ring.s], 3);
                            }
                            __syncwarp();
                        }
                        second = ring;
                        if (ok && kb < kall) ok = by_halves(false, true, kall - kb);
                    } else {
                        for (int kb = kb0; kb < kb1; ++kb, ring.next()) {
                            const int s = ring.s;
                            ok = stage_there();
                            if (!ok) break;
                            if (elect_one()) {
                                issue(s, kb, 0, 1);
                                commit_one(&empty[s]);
                            }
                            __syncwarp();
                        }
                        // (a condition among the stage's own instructions: 512 x 4096 x 4096 9.3 us, 8.7 here)
                        if (ok) {
                            if (elect_one()) commit_one(&tfull[buf]);
                            __syncwarp();
                        }
                    }
                    if (!ok) break;
                }
                // (elect_one names the same lane each time: the commits are of the thread that issued)
                if (issued) {
                    if (elect_one()) {
                        if constexpr (S::PAIR) umma_commit_pair(drain);
                        else commit_one(drain);
                        wait_bar(drain, 0u, abort, status, true);
                    }
                    __syncwarp();
                }
            }
        }
    } else if (warp < kScaleWarp0 + S::kScaleWarps) {
        if constexpr (!S::SPLIT) asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
        // scales: P's tiles, then Q's, four columns each
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t full0 = S::PAIR ? mapa_shared(smem_u32(full), 0) : 0u;
        bool ok = true;
        Ring<NS> ring;
        for (int tile = cid; ok && tile < num_tiles; tile += ncl) {
            for (int kb = kb0; kb < kb1; ++kb, ring.next()) {
                const int s = ring.s;
                if (!warp_wait_all(&sfull[s], ring.parity, abort, status, kSleepNs)) {
                    ok = false;
                    break;
                }
                uint32_t w[S::kScaleCols];
#pragma unroll
                for (int j = 0; j < S::kTiles; ++j) {
                    const uint4 v = *reinterpret_cast<const uint4 *>(sps + s * S::kPScales + j * kScaleTile + lane * 16);
                    w[4 * j] = v.x, w[4 * j + 1] = v.y, w[4 * j + 2] = v.z, w[4 * j + 3] = v.w;
                }
#pragma unroll
                for (int j = 0; j < S::kTiles; ++j) {
#pragma unroll
                    for (int i = 0; i < S::kQTiles; ++i) {
                        const uint4 v = *reinterpret_cast<const uint4 *>(
                            sqs + s * S::kQScales + (i * S::kTiles + j) * kScaleTile + lane * 16);
                        const int c = 4 * (S::kTiles + j * S::kQTiles + i);
                        w[c] = v.x, w[c + 1] = v.y, w[c + 2] = v.z, w[c + 3] = v.w;
                    }
                }
                // the MMAs that used these columns are done
                if (!warp_wait_all(&empty[s], ring.parity ^ 1u, abort, status, kSleepNs)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t to = scale_cols + s * S::kScaleCols + lanes;
#pragma unroll
                for (int c = 0; c + 16 <= S::kScaleCols; c += 16) tmem_st16(to + c, w + c);
                if constexpr (S::kScaleCols % 16 != 0) tmem_st8(to + S::kScaleCols / 16 * 16, w + S::kScaleCols / 16 * 16);
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (S::PAIR && side != 0) mbar_arrive_remote(full0 + (uint32_t)s * 8u);
                    else mbar_arrive(&full[s]);
                    // Released only now: the values are in tensor memory, so that no load of this stage
                    // can still be in flight when the next bulk copy overwrites it.  (An arrival does not
                    // wait for the loads before it, and the copies are not ordered behind them: released
                    // after the loads, one product in about 30000 of 1 x 11008 x 4096, with others in five
                    // streams beside it, used scales of a later stage in 32 rows.)
                    mbar_arrive(&sempty[s]);
                }
            }
        }
        if constexpr (S::SPLIT) {
            // this CTA's part of the sums, as [column][row], in the stages' place
            float *sums = reinterpret_cast<float *>(smem);
            int tile_p, tile_q;
            tile_at(cid, num_p, num_q, tile_p, tile_q);
            ok = ok && warp_wait(&tfull[0], 0u, abort, status, kSleepNs);
            tc_fence_after();
            if (ok) {
#pragma unroll
                for (int c = 0; c < BN; c += 32) {
                    if (tile_q * BN + c >= a.Q) break;
                    uint32_t w[32];
                    __syncwarp();
                    tmem_ld32(tmem + lanes + c, w);
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        sums[(c + i) * BM + 32 * (warp & 3) + lane] = __uint_as_float(w[i]);
                }
            }
        }
    } else if constexpr (!S::SPLIT) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
        // lane quarter of tensor memory: warp % 4; columns: half of the tile's
        const int q = warp & 3, e = warp - kScaleWarp0 - S::kScaleWarps, half = e >> 2;
        constexpr int CW = BN / 2;
        uint8_t *buf_out = smem + S::kOffOut + e * S::kOutBytes;
        const uint32_t tempty0 = S::PAIR ? mapa_shared(smem_u32(tempty), 0) : 0u;
        uint32_t t = 0;
        for (int tile = cid; tile < num_tiles; tile += ncl, ++t) {
            const int buf = t % S::kBuffers, acc = S::PAIR ? half : buf;
            if (!warp_wait_all(&tfull[acc], (t / S::kBuffers) & 1u, abort, status, 500)) break;
            tc_fence_after();
            int tp, tq;
            tile_at(tile, num_p, num_q, tp, tq);
            const uint32_t from = tmem + ((uint32_t)(32 * q) << 16) + buf * BN + half * CW;
            const int row = tp * S::kTileRows + BM * side + 32 * q, col = tq * BN + half * CW;
            // the accumulator is free as soon as it has been read
            auto free_acc = [&] {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (S::PAIR && side != 0) mbar_arrive_remote(tempty0 + (uint32_t)acc * 8u);
                    else mbar_arrive(&tempty[acc]);
                }
            };
            if (a.dtype == kF32) store_tile<FMT, kF32, CW>(&map_d, buf_out, from, row, col, a, g0, g1, lane, free_acc);
            else if (a.dtype == kBF16) store_tile<FMT, kBF16, CW>(&map_d, buf_out, from, row, col, a, g0, g1, lane, free_acc);
            else store_tile<FMT, kF16, CW>(&map_d, buf_out, from, row, col, a, g0, g1, lane, free_acc);
        }
        asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if constexpr (S::SPLIT) {
        if (C > 1) cluster_sync_all();               // all parts are there
        int tp, tq;
        tile_at(cid, num_p, num_q, tp, tq);
        const uint32_t mine = smem_u32(smem);
        const int cols = min(BN, a.Q - tq * BN), rows_left = a.P - tp * BM;
        auto out_of = [&](float v) { return FMT == kNv ? __fmul_rn(__fmul_rn(v, g0), g1) : v; };
        if (a.swapped) {
            // a warp a column of the tile (a row of D), four values a lane
            for (int c = rank + C * warp; c < cols; c += C * (S::kThreads / 32)) {
                float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
                for (int k = 0; k < C; ++k) {
                    float p[4];
                    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                                 : "=f"(p[0]), "=f"(p[1]), "=f"(p[2]), "=f"(p[3])
                                 : "r"(mapa_shared(mine + (c * BM + 4 * lane) * 4, k))
                                 : "memory");
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[i] = __fadd_rn(v[i], p[i]);
                }
                const int64_t at = (int64_t)(tq * BN + c) * a.ldd + tp * BM + 4 * lane;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (4 * lane + i < rows_left) store1(a.d, at + i, a.dtype, out_of(v[i]));
            }
        } else {
            // a thread a row of D, eight values at a time
            constexpr int kGroups = S::kThreads / BM;
            const int r = threadIdx.x % BM;
            for (int c = 8 * (rank + C * (threadIdx.x / BM)); c < cols; c += 8 * C * kGroups) {
                float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
                for (int k = 0; k < C; ++k) {
                    const uint32_t from = mapa_shared(mine + (c * BM + r) * 4, k);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        float p;
                        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(p) : "r"(from + i * BM * 4) : "memory");
                        v[i] = __fadd_rn(v[i], p);
                    }
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = out_of(v[i]);
                if (r >= rows_left) continue;
                const int64_t at = (int64_t)(tp * BM + r) * a.ldd + tq * BN + c;
                if (a.vectors && c + 8 <= cols) {
                    if (a.dtype == kF32) {
                        uint4 *to = reinterpret_cast<uint4 *>(static_cast<float *>(a.d) + at);
                        to[0] = Elem<kF32>::pack(v);
                        to[1] = Elem<kF32>::pack(v + 4);
                    } else {
                        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.d) + at) =
                            a.dtype == kBF16 ? Elem<kBF16>::pack(v) : Elem<kF16>::pack(v);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (c + i < cols) store1(a.d, at + i, a.dtype, v[i]);
                }
            }
        }
    }
    // No CTA of a cluster frees tensor memory or exits while another may arrive on its barriers,
    // read or write its shared memory or have a shared MMA run on it.
    if (S::PAIR || (S::SPLIT && C > 1)) cluster_sync_all();
    if (warp == kMmaWarp) {
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

// Clusters that can be resident at once (once a device).
template <class K>
int resident_clusters(K kernel, int cluster, int threads, size_t smem, int *cache) {
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= kMaxDevices) dev = 0;
    if (cache[dev] == 0) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(sm_count() / cluster * cluster);
        cfg.blockDim = dim3(threads);
        cfg.dynamicSmemBytes = smem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim = {(unsigned)cluster, 1, 1};
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n <= 0)
            n = std::max(1, sm_count() / cluster);
        cache[dev] = n;
    }
    return cache[dev];
}

template <int FMT, class S>
cudaError_t launch_shape(const Fp4Args &a, const uint8_t *p_codes, const uint8_t *q_codes, int split,
                         cudaStream_t st) {
    CUtensorMap mp, mq, md{};
    if (!encode_codes(&mp, p_codes, a.P, a.K, BM) || !encode_codes(&mq, q_codes, a.Q, a.K, S::kQRows / S::kHalves))
        return cudaErrorInvalidValue;
    if (!S::SPLIT && a.vectors) {
        const int es = a.dtype == kF32 ? 4 : 2;
        const CUtensorMapDataType dt = a.dtype == kF32    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                       : a.dtype == kBF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                          : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
        if (!encode_2d(&md, dt, a.d, (uint64_t)a.Q, (uint64_t)a.P, (uint64_t)a.ldd * es, 128 / es, 32,
                       CU_TENSOR_MAP_SWIZZLE_128B))
            return cudaErrorInvalidValue;
    }
    auto kernel = fp4_gemm_kernel<FMT, S>;
    static bool ready[kMaxDevices];
    const cudaError_t e = allow_shared(kernel, S::kSmem, ready);
    if (e != cudaSuccess) return e;
    const int cluster = S::SPLIT ? split : S::kCluster;
    const int64_t tiles = ((int64_t)a.P + S::kTileRows - 1) / S::kTileRows * (((int64_t)a.Q + S::BN - 1) / S::BN);
    int64_t clusters = tiles;
    if (!S::SPLIT) {                           // persistent
        static int resident[kMaxDevices];
        clusters = std::min<int64_t>(tiles, resident_clusters(kernel, cluster, S::kThreads, S::kSmem, resident));
    }
    if (tiles > 0x3FFFFFFF || clusters * cluster > 0x3FFFFFFF) return cudaErrorInvalidValue;
    return launch_pdl_clusters(kernel, (int)clusters * cluster, S::kThreads, cluster, S::kSmem, st,
                               mp, mq, md, a);
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
    // (a tensor map's rows are less than 2^40 bytes apart)
    a.vectors = reinterpret_cast<uintptr_t>(d) % 16 == 0 && (ldd * es) % 16 == 0 && ldd < 1ll << 37;
    a.whole = (N * es) % 16 == 0;
    if (small <= 64) {
        const int split = fp4_split_few_rows((K + BK - 1) / BK, fp4_tiles_down(a.P), sm_count());
        return small <= 32 ? launch_shape<FMT, Shape<FMT, 32, false, true>>(a, p.codes, q.codes, split, st)
                           : launch_shape<FMT, Shape<FMT, 64, false, true>>(a, p.codes, q.codes, split, st);
    }
    const int64_t tiles = fp4_tiles_down(M) * fp4_tiles_down(N), stages = (K + BK - 1) / BK;
    const int split = fp4_split_few_tiles(stages, tiles, sm_count());
    if (split > 2)
        return launch_shape<FMT, Shape<FMT, 128, false, true>>(a, p.codes, q.codes, split, st);
    // Tiles of 256 x 256 by CTA pairs, or of 128 x 128 by single CTAs, by what their rounds take: a
    // pair's 0.27 us a stage and 1.8 for its end, a single CTA's 0.34 a stage and 0.2 (its second
    // accumulator hides the rest), but 1.6 at least for its stores.  What a call takes beside its
    // rounds (launch, first loads, last stores) is 5.8 us for pairs and 3.8 for single CTAs.  Below in
    // tenths of a microsecond (a stage in hundredths, divided).  From 36 sizes
    // timed both ways, of which it misses five by 6% at most (pairs, then single CTAs): 4096 x 4096 x
    // 2048 20.5 and 23.8 us, 700 x 11008 x 4096 18.0 and 23.7, 300 x 11008 x 4096 16.6 and 14.1,
    // 517 x 5003 x 1999 16.7 and 14.8, 2500 x 2504 x 500 to FP32 10.2 and 8.5.
    const int64_t pair_tiles = (M + 255) / 256 * ((N + 255) / 256), pairs = sm_count() / 2;
    const int64_t pair_time = 58 + (pair_tiles + pairs - 1) / pairs * (27 * stages / 10 + 18);
    const int64_t single_time = 38 + (tiles + sm_count() - 1) / sm_count() * std::max<int64_t>(34 * stages / 10 + 2, 16);
    if (pair_time <= single_time)
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
