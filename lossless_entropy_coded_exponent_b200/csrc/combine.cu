// combine.cu -- y[t] = sum over k of weight[t, k] z[slot[t, k]]: a token's rows come back from
// the experts it was sent to, weighted by the router.
//
// Each thread owns eight columns of one token and adds its topk rows in the order of k in FP32, so
// the result does not depend on the launch; the sum is rounded once, to the output's type.  A
// token's slots and weights are read by every thread of its row (one broadcast load each).
// k_combine, for rows in whole 16-byte pieces: eight neighbouring columns, the rows of up to eight k
// loaded before the first is added.  Bound by the DRAM reads of z: 8191 tokens' 8 rows of 4096 BF16
// in 92 us (6.3 TB/s, 97 % of the measured copy rate).
// k_combine_any, for all others: a lane's columns are 32 apart, so that a warp's loads and stores of
// single values are 64 or 128 neighbouring bytes wherever a row starts; with eight neighbours a
// lane, loaded one by one or shifted together from aligned pieces, 4093 columns took 167 and 271 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "experts.cuh"
#include "launch.cuh"
#include "vec.cuh"

namespace dfx {
namespace {

constexpr int kCombineThreads = 256;

// The slot of a token's k-th row, or -1: none, or (flagged) outside z.
__device__ __forceinline__ int64_t slot_of(const CombineArgs& a, const int32_t* slots, uint32_t k) {
    const int64_t slot = k < a.topk ? slots[k] : -1;
    if (slot < (int64_t)a.z_rows) return slot;
    atomicOr(a.status, DFX_STATUS_INDEX);
    return -1;
}

// The token and the piece of work number u (32-bit where it fits: a 64-bit division is some 100
// instructions).
__device__ __forceinline__ uint64_t token_of(uint64_t u, uint32_t pieces) {
    return u >> 32 ? u / pieces : (uint64_t)((uint32_t)u / pieces);
}

// BATCH: rows of z in flight per thread
template <class TZ, class TY, uint32_t BATCH>
__global__ void __launch_bounds__(kCombineThreads) k_combine(const CombineArgs a, const uint32_t pieces) {
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    wait_prior_grid();
    const uint64_t u = (uint64_t)blockIdx.x * kCombineThreads + threadIdx.x;
    const uint64_t t = token_of(u, pieces);
    if (t >= a.tokens) return;
    const uint64_t c = (u - t * pieces) * 8;
    const int32_t* slots = a.slots + t * a.topk;
    const float* weights = a.weights + t * a.topk;
    float acc[8] = {};
    for (uint32_t k0 = 0; k0 < a.topk; k0 += BATCH) {
        float w[BATCH];
        Eight<TZ> p[BATCH];
#pragma unroll
        for (uint32_t i = 0; i < BATCH; i++) {
            w[i] = 0.0f;
            p[i].zero();
            const int64_t slot = slot_of(a, slots, k0 + i);
            if (slot < 0) continue;  // neither its weight nor a row counts
            w[i] = weights[k0 + i];
            p[i].load((const TZ*)a.z + (uint64_t)slot * a.ld_z + c);
        }
#pragma unroll
        for (uint32_t i = 0; i < BATCH; i++) {
            float v[8];
            p[i].get(v);
#pragma unroll
            for (int j = 0; j < 8; j++) acc[j] = fmaf(w[i], v[j], acc[j]);
        }
    }
    store_eight((TY*)a.y + t * a.ld_y + c, acc);
}

template <class TZ, class TY>
__global__ void __launch_bounds__(kCombineThreads) k_combine_any(const CombineArgs a, const uint32_t pieces) {
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    wait_prior_grid();
    constexpr uint32_t kBatch = 4;  // rows in flight
    const uint64_t u = (uint64_t)blockIdx.x * (kCombineThreads / 32) + threadIdx.x / 32;
    const uint64_t t = token_of(u, pieces);
    if (t >= a.tokens) return;
    const uint64_t c = (u - t * pieces) * 256 + threadIdx.x % 32;  // and c + 32, c + 64, ...
    const uint32_t n = c < a.cols ? (uint32_t)min((uint64_t)8, (a.cols - c + 31) / 32) : 0;
    const int32_t* slots = a.slots + t * a.topk;
    const float* weights = a.weights + t * a.topk;
    float acc[8] = {};
    for (uint32_t k0 = 0; k0 < a.topk; k0 += kBatch) {
        float w[kBatch];
        TZ p[kBatch][8];
#pragma unroll
        for (uint32_t i = 0; i < kBatch; i++) {
            const int64_t slot = slot_of(a, slots, k0 + i);
            w[i] = slot < 0 ? 0.0f : weights[k0 + i];
            const TZ* s = (const TZ*)a.z + (uint64_t)(slot < 0 ? 0 : slot) * a.ld_z + c;
#pragma unroll
            for (uint32_t j = 0; j < 8; j++) p[i][j] = slot >= 0 && j < n ? s[32 * j] : TZ(0.0f);
        }
#pragma unroll
        for (uint32_t i = 0; i < kBatch; i++)
#pragma unroll
            for (int j = 0; j < 8; j++) acc[j] = fmaf(w[i], as_f32(p[i][j]), acc[j]);
    }
    TY* d = (TY*)a.y + t * a.ld_y + c;
#pragma unroll
    for (uint32_t j = 0; j < 8; j++)
        if (j < n) store_one(d + 32 * j, acc[j]);
}

template <class TZ, class TY>
cudaError_t launch(const CombineArgs& a, cudaStream_t s) {
    const bool whole = a.cols % 8 == 0 && a.ld_z * sizeof(TZ) % 16 == 0 && a.ld_y * sizeof(TY) % 16 == 0;
    const uint64_t pieces = whole ? a.cols / 8 : (a.cols + 255) / 256;  // of a row: a thread's, or a warp's
    const uint64_t per_cta = whole ? kCombineThreads : kCombineThreads / 32;
    const uint64_t grid = (a.tokens * pieces + per_cta - 1) / per_cta;
    if (grid > 0x7fffffffull) return cudaErrorInvalidValue;
    auto go = [&](auto* k) { return launch_programmatic(k, (int)grid, kCombineThreads, 0, s, a, (uint32_t)pieces); };
    if (!whole) return go(k_combine_any<TZ, TY>);
    // a batch that few rows leave empty costs registers: one row of 4096 in 54 us with a batch of 8
    return a.topk <= 2 ? go(k_combine<TZ, TY, 2>) : a.topk <= 4 ? go(k_combine<TZ, TY, 4>) : go(k_combine<TZ, TY, 8>);
}

}  // namespace

cudaError_t launch_combine(const CombineArgs& a, cudaStream_t s) {
    if (a.z_bf16) return a.y_bf16 ? launch<__nv_bfloat16, __nv_bfloat16>(a, s) : launch<__nv_bfloat16, float>(a, s);
    return a.y_bf16 ? launch<float, __nv_bfloat16>(a, s) : launch<float, float>(a, s);
}

}  // namespace dfx
