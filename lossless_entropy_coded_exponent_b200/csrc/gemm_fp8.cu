// gemm_fp8.cu -- Y = X W^T with X and W in e4m3 and a power-of-two scale for each 128 values
// of a token's row and each 128 x 128 block of W; one matrix, or one per expert with the
// expert's own run of X's rows.
//
// The scales go into the tensor cores with the values: tcgen05.mma kind::mxf8f6f4 multiplies
// by e8m0 scale bytes held in tensor memory, one per row and 32 values of K, so the four MMAs
// of a 128-value block name the same byte and the whole sum over K stays in one FP32
// accumulator: no step that takes it out, scales and adds.
//
// W's rows are the MMA's M (a tile is 128 rows: one row of scale blocks), tokens its N: 16 to
// kCap columns, chosen per unit, so one token and thousands run through the same code (up to eight
// tokens and a small matrix leave it to stream_fp8.cu).  An MMA of
// K = 32 takes some 120 cycles for any N (measured with the copies left out), so a unit costs
// the cores the same for one token and for 240; with tokens as M and 240 rows of W as N one token
// would cost half, but the weights of a decoding step streamed 15 to 20 % slower that way.
// A unit is one expert's 128 rows (256 for a pair) by a run of its tokens.  Shapes:
//   up to 32 and up to 128 tokens on one CTA.  Bound by DRAM: 128 rows to 128 experts of
//     2048 x 4096 in 112 to 117 us (6.0 to 6.25 TB/s, 93 to 97 % of the measured copy rate).
//     Where units are few, the CTAs of a cluster share a unit's K and add their sums up through
//     distributed shared memory, in the order of K's parts: one token through 4096 x 14336 in
//     14.5 us (29 unsplit), 16 tokens through 4096 x 4096 in 7.2 us;
//   up to 240 (256) tokens on a pair of CTAs (cta_group::2), each holding 128 rows of W and half of
//     the tokens, which halves the shared-memory traffic of a product that the cores bound:
//     8192 tokens through 14336 x 4096 take some 500 thousand cycles (27 waves of 32 blocks, 577 a
//     block, of which the MMAs take 490): 362 us in a short run (2.66 PFLOP/s), 431 us once the
//     power limit holds the clock at 1.16 GHz (the MMAs alone without copies or stores: 260 us).
// A persistent CTA (pair) takes units in turn.  Warps:
//   0     brings the tiles in by TMA (128-byte swizzle), kStages deep;
//   1     issues the MMAs and copies each group of four blocks' scale bytes from shared to
//         tensor memory; owns the tensor memory.  The whole warp runs the loop and one elected
//         lane issues: a lone lane took some 870 cycles a block;
//   2     lays out the scale bytes in shared memory: byte j of word (32 i + l) of a 512-byte
//         tile is the scale of row 32 i + l and block 4 g + j (row l's four words are
//         neighbours), which tcgen05.cp spreads over the lanes;
//   4-7, 4-11 for up to 128 tokens: read the accumulator (lane = row of W) and write Y, while the
//         next unit's MMAs run into the other accumulator.
// Every wait is bounded: one that runs out sets DFX_STATUS_TIMEOUT and the CTA's warps leave their
// loops.  On every way out the copies and MMAs in flight are waited for before the tensor memory is freed.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include "dfx_common.cuh"
#include "experts.cuh"
#include "launch.cuh"
#include "tcgen05.cuh"
#include "vec.cuh"

namespace dfx {
namespace {

constexpr uint32_t kTileRows = 128;                       // rows of W per tile: the MMA's M
constexpr uint32_t kTileK = 128;                          // values of K per stage: one scale block
constexpr uint32_t kABytes = kTileRows * kTileK;          // 16 KiB
constexpr uint32_t kScaleTile = 512;                      // scale bytes of 128 rows x 4 blocks
constexpr uint32_t kGroup = 4;                            // blocks of K per scale tile
constexpr uint32_t kChunkGroups = 4;                      // scale tiles whose words are loaded at once
constexpr uint32_t kMaxSplit = 8;                         // CTAs that share a unit's K
constexpr uint32_t kTmemColumns = 512;                    // one CTA per SM: all of it

// kCap: most tokens of a tile; kBox: tokens of one TMA copy; kPair: the two CTAs of a cluster
// multiply 256 rows of W together, each holding its own 128 rows and half of the tokens
template <uint32_t CAP, bool PAIR>
struct Shape {
    static constexpr uint32_t kCap = CAP;
    static constexpr bool kPair = PAIR;
    static constexpr uint32_t kCtas = PAIR ? 2 : 1;
    // Warps that write Y, from warp 4 on.  Eight (two to a quarter of the lanes) where 128 tokens
    // are written when nothing is left to multiply: 123 tokens through 5619 x 4007 in 14.4 us, with
    // four 16.6.  Beside a pair's MMAs eight are in the way: 8192 tokens take 3 % longer.
    static constexpr uint32_t kEpilogueWarps = CAP == 128 ? 8 : 4, kColumnStep = 4 * kEpilogueWarps;
    static constexpr int kThreads = 32 * (4 + kEpilogueWarps);
    static constexpr uint32_t kHeld = CAP / kCtas;                     // tokens in one CTA's memory
    static constexpr uint32_t kUnitRows = kCtas * kTileRows;
    static constexpr uint32_t kBox = CAP == 256 ? 64 : PAIR ? 40 : 32;
    static constexpr uint32_t kStages = CAP == 32 ? 9 : 6;
    static constexpr uint32_t kSumBytes = CAP * kTileRows * 4;         // a split unit's sums, in the stages
    static constexpr uint32_t kStageBytes = kABytes + kHeld * kTileK;
    static constexpr uint32_t kSlots = 4;                              // scale groups in shared memory
    static constexpr uint32_t kCopies = 2;                             // and in tensor memory
    static constexpr uint32_t kBTiles = (CAP + 127) / 128;             // scale tiles of the tokens
    static constexpr uint32_t kSlotBytes = (1 + kBTiles) * kScaleTile;
    static constexpr uint32_t kSlotColumns = 4 * (1 + kBTiles);        // tensor memory of a slot
    // two accumulators, but of 256 columns one: the scales need room behind them
    static constexpr uint32_t kAccs = CAP == 256 ? 1 : 2, kScaleColumn = kAccs * CAP;
    static_assert(CAP % 16 == 0 && kHeld % kBox == 0 && kBox % 8 == 0, "whole MMA columns and swizzle groups");
    static_assert(kStageBytes % 1024 == 0, "the swizzle pattern starts every 1024 bytes");
    static_assert(kScaleColumn + kCopies * kSlotColumns <= kTmemColumns, "tensor memory");
    static_assert(PAIR || kStages * kStageBytes >= kSumBytes, "the stages hold a split unit's sums");
    static constexpr size_t kSmem = 1024 + kStages * kStageBytes + kSlots * kSlotBytes;
    static_assert(kSmem + 8192 <= 227 * 1024, "shared memory");
};

// Instruction descriptor of kind::mxf8f6f4: FP32 accumulator, e4m3 A and B, K-major, e8m0
// scales, N = n (a multiple of 16), M = 128 per CTA; | sf_id(j): byte j of each scale word.
__device__ __forceinline__ uint32_t idesc_e4m3(uint32_t n, uint32_t ctas) {
    return ((n >> 3) << 17) | (1u << 23) | (ctas << 27);
}
__device__ __forceinline__ constexpr uint32_t sf_id(uint32_t j) { return (j << 4) | (j << 29); }

template <bool PAIR>
__device__ __forceinline__ void mma_e4m3(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                         uint32_t acc) {
    if constexpr (PAIR)
        asm volatile(
            "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
            " tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc)
            : "memory");
    else
        asm volatile(
            "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
            " tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc)
            : "memory");
}
// 512 bytes of shared memory, 32 rows of 16 bytes, to four columns of 32 tensor-memory lanes,
// repeated in each quarter of the lanes (of both CTAs of a pair, each from its own shared
// memory); MMAs this thread issues later see them
template <bool PAIR>
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint32_t saddr) {
    // no swizzle, 8-row groups 128 bytes apart, descriptor version 1
    const uint64_t desc = (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)(128 >> 4) << 32) | ((uint64_t)1 << 46);
    if constexpr (PAIR) asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;\n" ::"r"(taddr), "l"(desc) : "memory");
    else asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n" ::"r"(taddr), "l"(desc) : "memory");
}
// arrives on `bar` (of both CTAs of a pair) when what this thread issued has completed
template <bool PAIR>
__device__ __forceinline__ void commit(unsigned long long* bar) {
    if constexpr (PAIR)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n" ::"r"(
                smem_addr(bar)),
            "h"((uint16_t)3)
            : "memory");
    else mma_commit(bar);
}
// a box of `map` at (x, y) to this CTA's shared memory; x is a multiple of 128.  The bytes
// count on `bar`, of a pair the first CTA's.
template <bool PAIR>
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, uint32_t x, uint32_t y, uint32_t bar) {
    if constexpr (PAIR)
        asm volatile(
            "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
            "%3}], [%4];\n" ::"r"(dst),
            "l"(map), "r"(x), "r"(y), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n" ::"r"(
                dst),
            "l"(map), "r"(x), "r"(y), "r"(bar)
            : "memory");
}
__device__ __forceinline__ void expect_bytes(unsigned long long* bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n" ::"r"(smem_addr(bar)), "r"(bytes) : "memory");
}
// the same place in the shared memory of the cluster's CTA `rank`
__device__ __forceinline__ uint32_t in_cta(uint32_t addr, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(a) : "r"(addr), "r"(rank));
    return a;
}
// the address of `bar` in the first CTA of a pair
template <bool PAIR>
__device__ __forceinline__ uint32_t first_cta(unsigned long long* bar) {
    return PAIR ? in_cta(smem_addr(bar), 0) : smem_addr(bar);
}
// arrives at a barrier of this CTA, or of another of the cluster
template <bool CLUSTER>
__device__ __forceinline__ void arrive(uint32_t bar) {
    if constexpr (CLUSTER) asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];\n" ::"r"(bar) : "memory");
    else asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void sync_ctas(bool cluster) {
    if (cluster)
        asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
    else __syncthreads();
}
// one lane of a warp that is together
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(one));
    return one != 0;
}

struct KernelArgs {
    GemmFp8Args g;
    uint32_t row_tiles, blocks;  // 128-row tiles of a matrix, 128-value blocks of K
    uint32_t row_units;          // tiles, or pairs of tiles, of a matrix
    uint32_t wide_sx, wide_sw;   // rows of scales in 16-byte pieces
    uint32_t wide_y;             // rows of Y in 16-byte pieces
    uint32_t split;              // CTAs (of a cluster) that share a unit's K; 1 for pairs.  Above 1 there
                                 // is a cluster for every unit
};

// One unit of work
struct Unit {
    uint32_t expert, row_unit;
    uint32_t first, n;   // its tokens
    uint32_t columns;    // n rounded up to the MMA's 16
};

// Units in order: experts; then groups of kRunGroup runs of tokens; in a group the rows of W, so
// that units near each other in time share W's rows and a few runs of X, and both come from L2.
constexpr uint32_t kRunGroup = 8;
struct Walk {
    const KernelArgs& a;
    const uint32_t* start;  // units of the experts before
    const uint32_t* edge;   // first row of X of each expert, and one past the last
    uint32_t e = 0;
    __device__ __forceinline__ Walk(const KernelArgs& a_, const uint32_t* s, const uint32_t* x) : a(a_), start(s), edge(x) {}
    __device__ __forceinline__ Unit at(uint32_t u) {
        while (u >= start[e + 1]) e++;
        const uint32_t runs = (start[e + 1] - start[e]) / a.row_units, tokens = edge[2 * e + 1] - edge[2 * e];
        const uint32_t local = u - start[e], group = local / (kRunGroup * a.row_units);
        const uint32_t in_group = local - group * kRunGroup * a.row_units, wide = min(kRunGroup, runs - group * kRunGroup);
        const uint32_t run = group * kRunGroup + in_group % wide;
        // the expert's tokens in `runs` runs of nearly equal length
        const uint32_t size = ((tokens + runs - 1) / runs + 15) & ~15u;
        Unit w;
        w.expert = e;
        w.row_unit = in_group / wide;
        w.first = edge[2 * e] + min(tokens, run * size);
        w.n = min(size, tokens - min(tokens, run * size));
        w.columns = max(16u, (w.n + 15) & ~15u);
        return w;
    }
    // the same for a warp that is together, in registers the compiler knows to be uniform
    __device__ __forceinline__ Unit uniform(uint32_t u) {
        Unit w = at(u);
        w.expert = __shfl_sync(kFull, w.expert, 0);
        w.row_unit = __shfl_sync(kFull, w.row_unit, 0);
        w.first = __shfl_sync(kFull, w.first, 0);
        w.columns = __shfl_sync(kFull, w.columns, 0);
        return w;
    }
};

// The scale words of four groups of blocks: W's row of scale blocks, and the rows of X that are
// this lane's (lane, lane + 32, ...).
template <class S>
struct ScaleChunk {
    static constexpr uint32_t kRows = (S::kCap + 31) / 32;
    uint32_t w[kChunkGroups], x[4 * S::kBTiles][kChunkGroups];
    // four words at p, of which those before `blocks` are there
    static __device__ __forceinline__ void words(uint32_t (&v)[kChunkGroups], const uint8_t* p, bool whole, uint32_t blocks) {
        if (whole) {
            const uint4 q = *reinterpret_cast<const uint4*>(p);
            v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
        } else {
#pragma unroll
            for (uint32_t g = 0; g < kChunkGroups; g++)
                v[g] = kGroup * g < blocks ? *reinterpret_cast<const uint32_t*>(p + kGroup * g) : 0u;
        }
    }
    __device__ __forceinline__ void load(const KernelArgs& a, const Unit& u, uint32_t row_tile, uint32_t kb, uint32_t lane) {
        // a pair's second tile may lie past W's last: its rows are not stored
        const uint32_t t = min(row_tile, a.row_tiles - 1);
        words(w, a.g.sw + ((uint64_t)u.expert * a.row_tiles + t) * a.g.ld_sw + kb, a.wide_sw && kb % 16 == 0, a.blocks - kb);
#pragma unroll
        for (uint32_t i = 0; i < 4 * S::kBTiles; i++) {
            const uint32_t r = 32 * i + lane;
            if (i < kRows && r < u.n) {
                words(x[i], a.g.sx + (uint64_t)(u.first + r) * a.g.ld_sx + kb, a.wide_sx && kb % 16 == 0,
                      a.blocks - kb);
            } else {
#pragma unroll
                for (uint32_t g = 0; g < kChunkGroups; g++) x[i][g] = 0;
            }
        }
    }
};

// A unit's columns (tokens) of this lane's row of W to Y (y: the first token's element of the row),
// 16 from c0 on and from every kColumnStep behind it
template <class S, class T>
__device__ __forceinline__ void store_columns(T* y, uint64_t ld, uint32_t taddr, uint32_t c0, const Unit& w, bool inside) {
#pragma unroll 1
    for (uint32_t c = c0; c < w.columns; c += S::kColumnStep) {
        uint32_t v[16];
        tmem_ld16(taddr + c, v);
        if (inside) {
            T* d = y + c * ld;
#pragma unroll
            for (uint32_t j = 0; j < 16; j++, d += ld)
                if (c + j < w.n) store_one(d, __uint_as_float(v[j]));
        }
        __syncwarp();
    }
}

// up to four sums, of which the row of Y has room for n
__device__ __forceinline__ void store_four(float* d, bool whole, const float (&v)[4], uint32_t n) {
    if (whole && n >= 4) {
        *reinterpret_cast<float4*>(d) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
        for (uint32_t j = 0; j < 4; j++)
            if (j < n) d[j] = v[j];
    }
}
__device__ __forceinline__ void store_four(__nv_bfloat16* d, bool whole, const float (&v)[4], uint32_t n) {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(v[0], v[1]), hi = __floats2bfloat162_rn(v[2], v[3]);
    if (whole && n >= 4) {
        *reinterpret_cast<uint2*>(d) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    } else {
        const __nv_bfloat16 h[4] = {lo.x, lo.y, hi.x, hi.y};
#pragma unroll
        for (uint32_t j = 0; j < 4; j++)
            if (j < n) d[j] = h[j];
    }
}

template <class S>
__global__ void __launch_bounds__(S::kThreads, 1)
    k_gemm_fp8(const __grid_constant__ KernelArgs a, const __grid_constant__ CUtensorMap map_x,
               const __grid_constant__ CUtensorMap map_w) {
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    constexpr bool P = S::kPair;
    __shared__ __align__(8) unsigned long long bar_full[S::kStages], bar_free[S::kStages], bar_scale[S::kSlots],
        bar_scale_free[S::kSlots], bar_acc[2], bar_acc_free[2], bar_part;
    __shared__ uint32_t tmem_slot;
    extern __shared__ __align__(16) uint8_t dyn_smem[];
    const uint32_t dyn0 = smem_addr(dyn_smem), pad = (1024u - (dyn0 & 1023u)) & 1023u;
    const uint32_t tiles = dyn0 + pad, scales = tiles + S::kStages * S::kStageBytes;
    uint8_t* scales_ptr = dyn_smem + pad + S::kStages * S::kStageBytes;
    // behind the tiles: the experts' rows and first units
    uint32_t* edge = reinterpret_cast<uint32_t*>(dyn_smem + S::kSmem);  // 2 per expert
    uint32_t* start = edge + 2 * a.g.experts;                           // experts + 1

    const uint32_t warp = __shfl_sync(kFull, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    // of a pair: which half; of a split unit: which part of K
    const uint32_t ctas = P ? S::kCtas : a.split, in_cluster = blockIdx.x % ctas, rank = P ? in_cluster : 0;
    const uint32_t first = blockIdx.x / ctas, step = gridDim.x / ctas;
    const uint32_t kb_begin = P ? 0 : in_cluster * a.blocks / ctas, kb_end = P ? a.blocks : (in_cluster + 1) * a.blocks / ctas;
    if (warp == 1) {
        if constexpr (P) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(smem_addr(&tmem_slot)),
                         "r"(kTmemColumns)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;\n" ::: "memory");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(smem_addr(&tmem_slot)),
                         "r"(kTmemColumns)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
        }
    } else if (threadIdx.x == 0) {
        for (uint32_t i = 0; i < S::kStages; i++) mbar_init_count(&bar_full[i], 1), mbar_init_count(&bar_free[i], 1);
        for (uint32_t i = 0; i < S::kSlots; i++)
            mbar_init_count(&bar_scale[i], S::kCtas), mbar_init_count(&bar_scale_free[i], 1);
        for (uint32_t i = 0; i < 2; i++) mbar_init_count(&bar_acc[i], 1), mbar_init_count(&bar_acc_free[i], S::kEpilogueWarps * S::kCtas);
        mbar_init_count(&bar_part, S::kEpilogueWarps * ctas);
        fence_mbar_init();
    }
    wait_prior_grid();
    uint32_t err = 0;
    // the experts' rows, clamped to X, and their units
    if (a.g.offsets) {
        for (uint32_t e = threadIdx.x; e < a.g.experts; e += S::kThreads) {
            const int32_t o0 = a.g.offsets[e], o1 = a.g.offsets[e + 1];
            const uint32_t lo = (uint32_t)min(max(o0, 0), (int32_t)a.g.tokens);
            const uint32_t hi = (uint32_t)min(max(o1, (int32_t)lo), (int32_t)a.g.tokens);
            if ((int32_t)lo != o0 || (int32_t)hi != o1) err |= DFX_STATUS_INDEX;
            edge[2 * e] = lo;
            edge[2 * e + 1] = hi;
        }
        __syncthreads();
        if (warp == 0) {
            uint32_t carry = 0;
            for (uint32_t e0 = 0; e0 < a.g.experts; e0 += 32) {
                const uint32_t e = e0 + lane;
                const uint32_t n = e < a.g.experts ? edge[2 * e + 1] - edge[2 * e] : 0;
                const uint32_t v = (n + S::kCap - 1) / S::kCap * a.row_units;
                uint32_t incl = v;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const uint32_t y = __shfl_up_sync(kFull, incl, d);
                    if (lane >= (uint32_t)d) incl += y;
                }
                if (e < a.g.experts) start[e] = carry + incl - v;
                carry += __shfl_sync(kFull, incl, 31);
            }
            if (lane == 0) start[a.g.experts] = carry;
            __syncwarp();
        }
    } else if (threadIdx.x == 0) {
        edge[0] = 0;
        edge[1] = a.g.tokens;
        start[0] = 0;
        start[1] = (a.g.tokens + S::kCap - 1) / S::kCap * a.row_units;
    }
    __syncwarp();
    tc_fence_before();
    sync_ctas(ctas > 1);
    tc_fence_after();
    // all of the tensor memory is this CTA's, from column 0 (tmem_slot) on
    constexpr uint32_t tmem = 0;
    // (of a split, one unit to a cluster: offsets out of order could count rows twice)
    const uint32_t all_units = __shfl_sync(kFull, start[a.g.experts], 0), units = ctas > S::kCtas ? min(all_units, step) : all_units;
    // Every warp waits together and leaves together.  A wait that runs out ends its warp's loop;
    // the other warps' waits then run out too.
    auto wait = [&](unsigned long long* bar, uint32_t parity) {
        if (__all_sync(kFull, mbar_poll<P>(bar, parity))) return true;
        if (__all_sync(kFull, mbar_wait<P>(bar, parity))) return true;
        err |= DFX_STATUS_TIMEOUT;
        return false;
    };
    Walk walk(a, start, edge);

    if (warp == 0) {
        // ------------------------------------------------------------ tiles
        uint32_t st = 0, ph = 0, issued = 0;
        bool ok = true;
        // test hook: the copies from the middle of the first unit on are left out
        const uint32_t kb_stop = a.g.inject ? (kb_begin + kb_end) / 2 : kb_end;
        for (uint32_t u = first; ok && u < units; u += step) {
            const Unit w = walk.uniform(u);
            // this CTA's tokens: all, or its half of the columns
            const uint32_t held = w.columns / S::kCtas, token = w.first + rank * held;
            const uint32_t boxes = (held + S::kBox - 1) / S::kBox;
            const uint32_t row = w.expert * a.g.rows + (w.row_unit * S::kCtas + rank) * kTileRows;
            for (uint32_t kb = kb_begin; kb < kb_stop; kb++) {
                if (issued >= S::kStages && !(ok = wait(&bar_free[st], ph ^ 1u))) break;
                const uint32_t sA = tiles + st * S::kStageBytes, sB = sA + kABytes;
                const uint32_t bar = first_cta<P>(&bar_full[st]);
                if (elect_one()) {
                    if (rank == 0) expect_bytes(&bar_full[st], S::kCtas * (kABytes + boxes * S::kBox * kTileK));
                    tma_load<P>(sA, &map_w, kb * kTileK, row, bar);
                    for (uint32_t b = 0; b < boxes; b++)
                        tma_load<P>(sB + b * S::kBox * kTileK, &map_x, kb * kTileK, token + b * S::kBox, bar);
                }
                __syncwarp();
                issued++;
                if (++st == S::kStages) st = 0, ph ^= 1u;
            }
            ok = ok && kb_stop == kb_end;
        }
        // The copies in flight land before the CTA ends, also when it was another warp that gave up:
        // those of each stage's last use (of a pair both CTAs', which end together).
        if (rank == 0)
            for (uint32_t i = 0; i < S::kStages && i < issued; i++) {
                const uint32_t last = issued - 1 - i;
                mbar_wait(&bar_full[last % S::kStages], (last / S::kStages) & 1u);
            }
        // of a pair that stopped half-way one CTA may have begun copies that the other did not expect:
        // a millisecond is a thousand times what they take
        if (P && !ok) {
            const long long begin = clock64();
            for (uint32_t i = 0; i < (1u << 20) && clock64() - begin < 2000000; i++) __nanosleep(1000);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMAs
        if (rank == 0) {
            uint32_t st = 0, ph = 0, slot = 0, slot_ph = 0, acc = 0, acc_ph = 0, unit = 0, group = 0;
            bool ok = true;
            const uint64_t descA = smem_desc_sw128(tiles), descB = smem_desc_sw128(tiles + kABytes);
            for (uint32_t u = first; ok && u < units; u += step, unit++) {
                const Unit w = walk.uniform(u);
                const uint32_t d = tmem + acc * S::kCap, idesc = idesc_e4m3(w.columns, S::kCtas);
                if (unit >= S::kAccs) ok = wait(&bar_acc_free[acc], acc_ph ^ 1u);
                for (uint32_t kb0 = kb_begin & ~(kGroup - 1); ok && kb0 < kb_end; kb0 += kGroup) {
                    // the group before last read the same columns of scales: its MMAs have completed
                    const uint32_t sf = tmem + S::kScaleColumn + (group % S::kCopies) * S::kSlotColumns;
                    if (group >= S::kCopies) {
                        const uint32_t before = group - S::kCopies;
                        if (!(ok = wait(&bar_scale_free[before % S::kSlots], (before / S::kSlots) & 1u))) break;
                    }
                    group++;
                    if (!(ok = wait(&bar_scale[slot], slot_ph))) break;
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (uint32_t i = 0; i < 1 + S::kBTiles; i++)
                            copy_scales<P>(sf + 4 * i, scales + slot * S::kSlotBytes + i * kScaleTile);
                    }
                    __syncwarp();
#pragma unroll
                    for (uint32_t j = 0; j < kGroup; j++) {
                        if (!ok || kb0 + j >= kb_end) break;
                        if (!P && kb0 + j < kb_begin) continue;
                        if (!(ok = wait(&bar_full[st], ph))) break;
                        tc_fence_after();
                        if (elect_one()) {
                            const uint64_t at = (uint64_t)(st * (S::kStageBytes >> 4));
#pragma unroll
                            for (uint32_t k = 0; k < kTileK / 32; k++)
                                mma_e4m3<P>(d, descA + at + 2 * k, descB + at + 2 * k, idesc | sf_id(j), sf, sf + 4,
                                            kb0 + j != kb_begin || k != 0);
                            commit<P>(&bar_free[st]);
                        }
                        __syncwarp();
                        if (++st == S::kStages) st = 0, ph ^= 1u;
                    }
                    if (elect_one()) commit<P>(&bar_scale_free[slot]);
                    __syncwarp();
                    if (++slot == S::kSlots) slot = 0, slot_ph ^= 1u;
                }
                // the accumulator is ready
                if (elect_one()) commit<P>(&bar_acc[acc]);
                __syncwarp();
                if (++acc == S::kAccs) acc = 0, acc_ph ^= 1u;
            }
            // what was issued completes before the tensor memory is freed, also when the warps that read it
            // have given up
            if (unit) mbar_wait(&bar_acc[acc ? acc - 1 : S::kAccs - 1], acc ? acc_ph : acc_ph ^ 1u);
        }
    } else if (warp == 2) {
        // ------------------------------------------------------------ scales
        // chunks of four groups, one ahead of the group being laid out: a chunk's loads take a
        // microsecond or more, a group's MMAs less
        uint32_t slot = 0, slot_ph = 0, issued = 0;
        ScaleChunk<S> now, next;
        const uint32_t kb_first = kb_begin & ~(kGroup - 1);
        uint32_t u = first, kb = kb_first;
        Unit w;
        if (u < units) {
            w = walk.at(u);
            next.load(a, w, w.row_unit * S::kCtas + rank, kb, lane);
        }
        bool ok = true;
        while (ok && u < units) {
            now = next;
            const uint32_t groups = (min(kb_end - kb, kGroup * kChunkGroups) + kGroup - 1) / kGroup;
            kb += kGroup * kChunkGroups;
            if (kb >= kb_end) {
                kb = kb_first;
                u += step;
                if (u < units) w = walk.at(u);
            }
            if (u < units) next.load(a, w, w.row_unit * S::kCtas + rank, kb, lane);
#pragma unroll
            for (uint32_t g = 0; g < kChunkGroups; g++) {
                if (g >= groups) break;
                if (issued >= S::kSlots && !(ok = wait(&bar_scale_free[slot], slot_ph ^ 1u))) break;
                uint4* dst = reinterpret_cast<uint4*>(scales_ptr + slot * S::kSlotBytes);
                const uint32_t aw = now.w[g];
                dst[lane] = make_uint4(aw, aw, aw, aw);
#pragma unroll
                for (uint32_t i = 0; i < S::kBTiles; i++)
                    dst[32 * (i + 1) + lane] =
                        make_uint4(now.x[4 * i][g], now.x[4 * i + 1][g], now.x[4 * i + 2][g], now.x[4 * i + 3][g]);
                fence_proxy_async();  // read by tcgen05.cp
                __syncwarp();
                const uint32_t bar = first_cta<P>(&bar_scale[slot]);
                if (lane == 0) arrive<P>(bar);
                issued++;
                if (++slot == S::kSlots) slot = 0, slot_ph ^= 1u;
            }
        }
    } else if (warp >= 4) {
        // ------------------------------------------------------------ epilogue
        // tensor-memory lanes 32 quarter .. + 31; of eight warps every second 16 columns
        const uint32_t quarter = warp % 4, c0 = (warp - 4) / 4 * 16;
        uint32_t acc = 0, acc_ph = 0;
        for (uint32_t u = first; u < units; u += step) {
            const Unit w = walk.at(u);
            if (!wait(&bar_acc[acc], acc_ph)) break;
            tc_fence_after();
            const uint32_t in_tile = 32 * quarter + lane, row = (w.row_unit * S::kCtas + rank) * kTileRows + in_tile;
            const uint32_t taddr = tmem + acc * S::kCap + ((32 * quarter) << 16);
            if (P || a.split == 1) {
                if (a.g.y_f32) store_columns<S>((float*)a.g.y + (uint64_t)w.first * a.g.ld_y + row, a.g.ld_y, taddr, c0, w, row < a.g.rows);
                else store_columns<S>((__nv_bfloat16*)a.g.y + (uint64_t)w.first * a.g.ld_y + row, a.g.ld_y, taddr, c0, w, row < a.g.rows);
            } else {
                // Every CTA lays its sums out in its tile memory, which its MMAs have read, as
                // [token][row].  Then every CTA of the cluster adds up its share of them, four rows
                // at a time, in the order of K's parts.
                for (uint32_t c = c0; c < w.n; c += S::kColumnStep) {
                    uint32_t v[16];
                    tmem_ld16(taddr + c, v);
#pragma unroll
                    for (uint32_t j = 0; j < 16; j++)
                        if (c + j < w.n)
                            asm volatile("st.shared.u32 [%0], %1;\n" ::"r"(tiles + ((c + j) * kTileRows + in_tile) * 4), "r"(v[j])
                                         : "memory");
                }
                __syncwarp();
                if (lane < a.split) arrive<true>(in_cta(smem_addr(&bar_part), lane));
                __syncwarp();
                if (!__all_sync(kFull, mbar_wait<true>(&bar_part, 0))) {
                    err |= DFX_STATUS_TIMEOUT;
                    break;
                }
                constexpr uint32_t kFours = kTileRows / 4;
                const uint32_t share = (w.n * kFours + a.split - 1) / a.split;
                const uint32_t last = min(w.n * kFours, (in_cluster + 1) * share);
                for (uint32_t i = in_cluster * share + threadIdx.x - 128; i < last; i += 32 * S::kEpilogueWarps) {
                    const uint32_t t = i / kFours, r = w.row_unit * kTileRows + 4 * (i % kFours);
                    if (r >= a.g.rows) continue;
                    float4 q[kMaxSplit];
#pragma unroll
                    for (uint32_t from = 0; from < kMaxSplit; from++) {
                        if (from >= a.split) break;
                        asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];\n"
                                     : "=f"(q[from].x), "=f"(q[from].y), "=f"(q[from].z), "=f"(q[from].w)
                                     : "r"(in_cta(tiles + i * 16, from))
                                     : "memory");
                    }
                    float sum[4] = {};
#pragma unroll
                    for (uint32_t from = 0; from < kMaxSplit; from++) {
                        if (from >= a.split) break;
                        sum[0] += q[from].x, sum[1] += q[from].y, sum[2] += q[from].z, sum[3] += q[from].w;
                    }
                    const uint64_t at = (uint64_t)(w.first + t) * a.g.ld_y + r;
                    if (a.g.y_f32) store_four((float*)a.g.y + at, a.wide_y, sum, a.g.rows - r);
                    else store_four((__nv_bfloat16*)a.g.y + at, a.wide_y, sum, a.g.rows - r);
                }
            }
            tc_fence_before();
            const uint32_t bar = first_cta<P>(&bar_acc_free[acc]);
            if (lane == 0) arrive<P>(bar);
            if (++acc == S::kAccs) acc = 0, acc_ph ^= 1u;
        }
    }
    __syncwarp();
    if (err) atomicOr(a.g.status, err);
    __syncwarp();
    tc_fence_before();
    sync_ctas(ctas > 1);
    if (warp == 1) {
        tc_fence_after();
        if constexpr (P)
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(kTmemColumns) : "memory");
        else
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(kTmemColumns) : "memory");
    }
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// the driver's call, looked up once (the library links no driver library)
EncodeTiled encode_tiled() {
    static EncodeTiled fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            p = nullptr;
        return (EncodeTiled)p;
    }();
    return fn;
}

// rows x cols bytes, `ld` apart, in boxes of box_rows x 128; what lies past cols or rows reads 0
bool make_map(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols, uint64_t ld, uint32_t box_rows) {
    const EncodeTiled fn = encode_tiled();
    if (!fn) return false;
    const cuuint64_t dims[2] = {cols, rows}, strides[1] = {ld};
    const cuuint32_t box[2] = {kTileK, box_rows}, steps[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, steps,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Runs of tokens of all experts, at most (an expert's last run may be short).
template <class S>
uint64_t most_runs(const GemmFp8Args& g) {
    return g.offsets ? (uint64_t)g.tokens / S::kCap + (g.experts < g.tokens ? g.experts : g.tokens)
                     : ((uint64_t)g.tokens + S::kCap - 1) / S::kCap;
}

// Clusters of a shape that the device holds at once (a GPC's SMs need not be a multiple of the
// cluster: of 4 CTAs the B200 holds 33, of 8 it holds 15), asked once per device.
template <class S>
cudaError_t cluster_slots(uint32_t split, int sms, uint64_t* slots) {
    static int known[64][kMaxSplit + 1] = {};
    static bool attr_set[64] = {};
    constexpr size_t most = S::kSmem + (3 * kMaxGemmExperts + 1) * sizeof(uint32_t);
    static_assert(most + 1024 <= 227 * 1024, "shared memory");
    const cudaError_t e = allow_smem(k_gemm_fp8<S>, most, attr_set);
    if (e != cudaSuccess) return e;
    const uint32_t ctas = S::kCtas * split;
    int dev = 0, n = 0;
    if (ctas == 1 || cudaGetDevice(&dev) != cudaSuccess || dev >= 64) {
        *slots = (uint64_t)sms / ctas;
        return cudaSuccess;
    }
    if (known[dev][split] == 0) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(ctas);
        cfg.blockDim = dim3(S::kThreads);
        cfg.dynamicSmemBytes = most;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim = {ctas, 1, 1};
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        const cudaError_t q = cudaOccupancyMaxActiveClusters(&n, k_gemm_fp8<S>, &cfg);
        if (q != cudaSuccess) return q;
        known[dev][split] = n > 0 ? n : 1;
    }
    *slots = (uint64_t)known[dev][split];
    return cudaSuccess;
}

template <class S>
cudaError_t launch(const GemmFp8Args& g, uint32_t split, uint64_t slots, cudaStream_t s) {
    KernelArgs a;
    memset(&a, 0, sizeof(a));
    a.g = g;
    a.row_units = (g.rows + S::kUnitRows - 1) / S::kUnitRows;
    a.row_tiles = (g.rows + kTileRows - 1) / kTileRows;
    a.blocks = (g.cols + kTileK - 1) / kTileK;
    a.wide_sx = g.ld_sx % 16 == 0;
    a.wide_sw = g.ld_sw % 16 == 0;
    a.wide_y = g.ld_y * (g.y_f32 ? 4 : 2) % 16 == 0;
    a.split = split;
    CUtensorMap mx, mw;
    if (!make_map(&mx, g.x, g.tokens, g.cols, g.ld_x, S::kBox) ||
        !make_map(&mw, g.w, (uint64_t)g.experts * g.rows, g.cols, g.ld_w, kTileRows))
        return cudaErrorInvalidValue;
    const uint32_t ctas = S::kCtas * split;
    const uint64_t units = most_runs<S>(g) * a.row_units;
    const int grid = (int)((units < slots || split > 1 ? units : slots) * ctas);
    return launch_clusters(k_gemm_fp8<S>, grid, ctas, S::kThreads, S::kSmem + (3 * g.experts + 1) * sizeof(uint32_t), s, a, mx,
                           mw);
}

// Cycles of a kernel: waves of units, each its blocks and what it costs to begin and to write Y.
// A block costs its four MMAs (some 500 cycles; more where shared memory bounds them: 128 tokens
// on one CTA), or its CTA's share of the DRAM rate if the weights are not reused.
template <class S>
double estimate(const GemmFp8Args& g, uint32_t split, uint64_t slots, int sms) {
    const uint64_t row_units = (g.rows + S::kUnitRows - 1) / S::kUnitRows, blocks = (g.cols + kTileK - 1) / kTileK;
    // an expert's usual tokens; its runs
    const uint64_t mean = (g.tokens + g.experts - 1) / g.experts, runs = (mean + S::kCap - 1) / S::kCap;
    const uint64_t units = runs * row_units * (g.experts < g.tokens ? g.experts : g.tokens);
    const double waves = (double)((units + slots - 1) / slots);
    const double busy = (double)(units < slots ? units : slots) * split * S::kCtas / sms;
    const double mma = S::kPair ? 620 : 540, dram = 5.6 * kTileRows * busy / (double)runs;
    // with one accumulator the tensor cores wait while it is read
    const double block = mma > dram ? mma : dram, unit = S::kAccs == 1 ? 2500 : 700;
    return waves * ((double)((blocks + split - 1) / split) * block + unit) + (split > 1 ? 1500 : 0);
}

// The shape and the split of K that the estimate favours.
struct Choice {
    double time = 1e300;
    int shape = 0;
    uint32_t split = 1;
    uint64_t slots = 1;
};
template <class S>
cudaError_t consider(Choice* best, int shape, uint32_t split, const GemmFp8Args& g, int sms) {
    uint64_t slots = 1;
    const cudaError_t e = cluster_slots<S>(split, sms, &slots);
    if (e != cudaSuccess) return e;
    // a split needs a cluster for every unit at once, and a block of K for every CTA
    const uint64_t row_units = (g.rows + S::kUnitRows - 1) / S::kUnitRows, blocks = (g.cols + kTileK - 1) / kTileK;
    if (split > 1 && (split > blocks || most_runs<S>(g) * row_units > slots)) return cudaSuccess;
    const double t = estimate<S>(g, split, slots, sms);
    if (t < best->time * 0.99) *best = {t, shape, split, slots};
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_gemm_fp8(const GemmFp8Args& g, int sms, cudaStream_t s) {
    using Few = Shape<32, false>;
    using Middle = Shape<128, false>;
    using Pair = Shape<240, true>;
    using PairLong = Shape<256, true>;  // of one matrix: powers of two of tokens in fewer runs (512 by
                                        // 14336 x 4096: 37 us, against 43)
    // an injected failure is one of the tiles'
    if (!g.inject && stream_fp8_takes(g, sms)) return launch_stream_fp8(g, sms, s);
    const uint64_t mean = (g.tokens + g.experts - 1) / g.experts;
    Choice best;
    cudaError_t e = cudaSuccess;
    for (uint32_t split = 1; split <= kMaxSplit && e == cudaSuccess; split *= 2) {
        if (mean <= 64) e = consider<Few>(&best, 0, split, g, sms);
        if (mean > 32 && e == cudaSuccess) e = consider<Middle>(&best, 1, split, g, sms);
    }
    if (mean > 128 && e == cudaSuccess) e = consider<Pair>(&best, 2, 1, g, sms);
    if (mean > 240 && g.experts == 1 && e == cudaSuccess) e = consider<PairLong>(&best, 3, 1, g, sms);
    if (e != cudaSuccess) return e;
    switch (best.shape) {
        case 0: return launch<Few>(g, best.split, best.slots, s);
        case 1: return launch<Middle>(g, best.split, best.slots, s);
        case 2: return launch<Pair>(g, 1, best.slots, s);
        default: return launch<PairLong>(g, 1, best.slots, s);
    }
}

}  // namespace dfx
