// stream_fp8.cu -- Y = X W^T in 8 bits for up to eight tokens and one matrix of up to 16 MiB, held
// in the registers of the whole device at once.
//
// Y[t, r] = sum over the blocks b of 2^(sx[t, b] + sw[r / 128, b] - 254) sum over k in b of
// x[t, k] w[r, k].  A matrix that small takes less time to read than tiles take to set up (tensor
// memory, descriptors, barriers, clusters), so a warp multiplies 16 rows by one block of K straight
// from registers: e4m3 becomes f16 exactly, mma.sync (M = 16 rows, N = 8 tokens) adds a block's
// products up in FP32, and a block's sum is scaled as it leaves.  Any order of K inside a block
// will do, so a lane loads 16 bytes at a time and its words are fragments as they lie.
// Every SM has the same number of rows (not of tiles), cut into (16 rows, block) items of which
// each of its warps takes one or two, with all of their loads in flight at once.  The items' sums
// meet in shared memory and are added in the order of the blocks.
//
// Bound by latency: the launch, W, X behind it, the joining of the sums.  On the device, W from
// DRAM, one token (beside it gemm_fp8.cu's tiles): 1024 x 1024 in 3.0 us (4.7), 2048 x 2048 3.7
// (5.4), 1024 x 4096 4.1 (5.7), 4096 x 4096 6.5 (8.1); eight tokens 2 to 6 % more.  Larger matrices
// need several rounds of items, each a memory latency and a joining: 8192 x 4096 in 11.7 us with
// a prefetch of one item, against 10.7 with tiles, whose copies never pause.  16 warps of four items
// each: 1024 x 4096 in 4.7 us, 4096 x 4096 in 7.4.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include "dfx_common.cuh"
#include "experts.cuh"
#include "launch.cuh"
#include "vec.cuh"

namespace dfx {
namespace {

constexpr uint32_t kWarps = 32;
constexpr uint32_t kItems = 2;        // most items of a warp: both fit its registers
constexpr uint32_t kItemRows = 16;    // rows of an item: the mma's M
constexpr uint32_t kBlock = 128;      // its columns: one scale block
constexpr uint32_t kMostTiles = 8;    // most 16-row tiles of a CTA
constexpr uint64_t kMostBytes = 16ull << 20;
constexpr uint32_t kTokenStride = 20;  // floats from token to token of a sum: no bank twice in a store

struct StreamArgs {
    GemmFp8Args g;
    uint32_t blocks;
    uint32_t share;   // rows of a CTA
};

// the 16 bytes at p, of which n are inside the matrix (n <= 0: none); the others are 0.  keep: other
// warps of the SM read them too
__device__ __forceinline__ uint4 load_bytes(const uint8_t* p, int32_t n, bool keep) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (n >= 16) {
        if (keep) v = *reinterpret_cast<const uint4*>(p);
        else
            asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];\n"
                         : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                         : "l"(p));
    } else if (n > 0) {
        uint32_t w[4] = {};
#pragma unroll
        for (int32_t i = 0; i < 15; i++)
            if (i < n) w[i / 4] |= (uint32_t)p[i] << (8 * (i % 4));
        v = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return v;
}

// four e4m3 values as two pairs of f16 (every e4m3 value is one of f16)
__device__ __forceinline__ void to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

// c += 16 rows x 16 columns of W by as many columns of 8 tokens; one word of a row and of a token
// holds a lane's four columns
__device__ __forceinline__ void mma_word(float (&c)[4], uint32_t w_low, uint32_t w_high, uint32_t x) {
    uint32_t a0, a1, a2, a3, b0, b1;
    to_f16(w_low, a0, a2);
    to_f16(w_high, a1, a3);
    to_f16(x, b0, b1);
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// the value of an e8m0 byte (255: NaN)
__device__ __forceinline__ float scale_value(uint32_t e) {
    return __uint_as_float(e == 255 ? 0x7fffffffu : e == 0 ? 0x00400000u : e << 23);
}

// part * 2^(a + b - 254): one product where the factor is an ordinary float, else two with factors of
// half the exponent each, so that the first does not leave FP32's range before the result does
__device__ __forceinline__ float scaled(float part, uint32_t a, uint32_t b) {
    const uint32_t e = a + b;
    if (max(a, b) == 255) return scale_value(255);
    if (e - 128u < 254u) return part * __uint_as_float((e - 127u) << 23);
    return part * scale_value(e / 2) * scale_value(e - e / 2);
}

// a lane's part of an item: two rows (g and g + 8 of the tile) of 32 bytes, and their scales
struct Item {
    uint4 low[2], high[2];
    uint32_t sw_low, sw_high;
    __device__ __forceinline__ void load(const StreamArgs& a, uint32_t row, uint32_t last, uint32_t kb, uint32_t q) {
        const uint32_t at = kb * kBlock + 16 * q;
        const int32_t left = (int32_t)(a.g.cols - at);
        const uint8_t* p = a.g.w + (uint64_t)row * a.g.ld_w + at;
        const bool in_low = row < last, in_high = row + 8 < last;
        low[0] = load_bytes(p, in_low ? left : 0, false);
        low[1] = load_bytes(p + 64, in_low ? left - 64 : 0, false);
        p += 8 * a.g.ld_w;
        high[0] = load_bytes(p, in_high ? left : 0, false);
        high[1] = load_bytes(p + 64, in_high ? left - 64 : 0, false);
        sw_low = in_low ? a.g.sw[(uint64_t)(row / kBlock) * a.g.ld_sw + kb] : 127;
        sw_high = in_high ? a.g.sw[(uint64_t)((row + 8) / kBlock) * a.g.ld_sw + kb] : 127;
    }
};

__global__ void __launch_bounds__(32 * kWarps, 1) k_stream_fp8(const StreamArgs a) {
    extern __shared__ float sums[];  // [item][token][row], kTokenStride a token
    asm volatile("griddepcontrol.launch_dependents;\n");
    const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, q = lane % 4;
    const uint32_t first = blockIdx.x * a.share, last = min(a.g.rows, first + a.share);
    const uint32_t tiles = (last - first + kItemRows - 1) / kItemRows, items = tiles * a.blocks;
    const uint32_t item_floats = a.g.tokens * kTokenStride;
    wait_prior_grid();
    Item item[kItems];
#pragma unroll
    for (uint32_t i = 0; i < kItems; i++) {
        const uint32_t n = warp + i * kWarps;
        if (n < items) item[i].load(a, first + n / a.blocks * kItemRows + g, last, n % a.blocks, q);
    }
#pragma unroll
    for (uint32_t i = 0; i < kItems; i++) {
        const uint32_t n = warp + i * kWarps;
        if (n >= items) break;
        const uint32_t kb = n % a.blocks, at = kb * kBlock + 16 * q;
        const int32_t left = g < a.g.tokens ? (int32_t)(a.g.cols - at) : 0;
        const uint8_t* px = a.g.x + (uint64_t)g * a.g.ld_x + at;
        const uint8_t* ps = a.g.sx + (uint64_t)(2 * q) * a.g.ld_sx + kb;
        const uint32_t even = 2 * q < a.g.tokens ? ps[0] : 127, odd = 2 * q + 1 < a.g.tokens ? ps[a.g.ld_sx] : 127;
        float part[4] = {};
#pragma unroll
        for (uint32_t h = 0; h < 2; h++) {
            const uint4 x = load_bytes(px + 64 * h, left - (int32_t)(64 * h), true);
            mma_word(part, item[i].low[h].x, item[i].high[h].x, x.x);
            mma_word(part, item[i].low[h].y, item[i].high[h].y, x.y);
            mma_word(part, item[i].low[h].z, item[i].high[h].z, x.z);
            mma_word(part, item[i].low[h].w, item[i].high[h].w, x.w);
        }
        float* d = sums + n * item_floats + 2 * q * kTokenStride + g;
        if (2 * q < a.g.tokens) {
            d[0] = scaled(part[0], item[i].sw_low, even);
            d[8] = scaled(part[2], item[i].sw_high, even);
        }
        if (2 * q + 1 < a.g.tokens) {
            d[kTokenStride] = scaled(part[1], item[i].sw_low, odd);
            d[kTokenStride + 8] = scaled(part[3], item[i].sw_high, odd);
        }
    }
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < tiles * kItemRows * a.g.tokens; i += 32 * kWarps) {
        const uint32_t r = i % kItemRows, t = i / kItemRows % a.g.tokens, tile = i / kItemRows / a.g.tokens;
        const uint32_t row = first + tile * kItemRows + r;
        if (row >= last) continue;
        const float* s = sums + tile * a.blocks * item_floats + t * kTokenStride + r;
        float v = 0;
#pragma unroll 8
        for (uint32_t kb = 0; kb < a.blocks; kb++) v += s[kb * item_floats];
        const uint64_t at = t * a.g.ld_y + row;
        if (a.g.y_f32) store_one((float*)a.g.y + at, v);
        else store_one((__nv_bfloat16*)a.g.y + at, v);
    }
}

StreamArgs stream_args(const GemmFp8Args& g, int sms) {
    StreamArgs a;
    memset(&a, 0, sizeof(a));
    a.g = g;
    a.blocks = (g.cols + kBlock - 1) / kBlock;
    a.share = (g.rows + (uint32_t)sms - 1) / (uint32_t)sms;
    return a;
}

}  // namespace

// One matrix, every row, and no more of it on an SM than its warps take at once.  At the limits: 4096 x
// 4096 (64 items) 6.5 us, with tiles 8.1; 18944 x 512 (8 tiles) 4.2 and 5.5; 2368 x 7000 7.1 and 9.2.
// Behind them: 18944 x 1000 8.1 and 7.3; 2384 x 7000 (110 items, two rounds of loads) 10.5 and 9.2.
bool stream_fp8_takes(const GemmFp8Args& g, int sms) {
    const StreamArgs a = stream_args(g, sms);
    const uint64_t tiles = (a.share + kItemRows - 1) / kItemRows;
    return g.tokens <= kStreamTokens && !g.offsets && (uint64_t)g.rows * g.cols <= kMostBytes && tiles <= kMostTiles &&
           tiles * a.blocks <= kWarps * kItems;
}

cudaError_t launch_stream_fp8(const GemmFp8Args& g, int sms, cudaStream_t s) {
    const StreamArgs a = stream_args(g, sms);
    const uint32_t tiles = (a.share + kItemRows - 1) / kItemRows;
    const size_t smem = (size_t)tiles * a.blocks * g.tokens * kTokenStride * sizeof(float);
    static_assert(kWarps * kItems * kStreamTokens * kTokenStride * sizeof(float) <= 48 * 1024, "shared memory");
    return launch_programmatic(k_stream_fp8, (int)((g.rows + a.share - 1) / a.share), 32 * (int)kWarps, smem, s, a);
}

}  // namespace dfx
