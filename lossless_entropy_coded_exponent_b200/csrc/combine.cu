// combine.cu -- y[t] = sum over k of weight[t, k] z[slot[t, k]]: a token's rows come back from
// the experts it was sent to, weighted by the router.
//
// Each thread owns eight neighbouring columns of one token and adds its topk rows in the order
// of k in FP32, so the result does not depend on the launch; the sum is rounded once, to the
// output's type.  A token's slots and weights are read by every thread of its row (one
// broadcast load each).  The rows of up to eight k are loaded before the first is added: the
// kernel is bound by the DRAM reads of z, which are gathered in pieces of a whole row.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "experts.cuh"
#include "launch.cuh"
#include "vec.cuh"

namespace dfx {
namespace {

constexpr int kCombineThreads = 256;
constexpr uint32_t kCombineBatch = 8;  // rows of z in flight per thread

template <class TZ, class TY, bool VEC>
__global__ void __launch_bounds__(kCombineThreads) k_combine(const CombineArgs a, const uint32_t pieces) {
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    wait_prior_grid();
    const uint64_t u = (uint64_t)blockIdx.x * kCombineThreads + threadIdx.x;
    const uint64_t t = u / pieces;
    if (t >= a.tokens) return;
    const uint64_t c = (u - t * pieces) * 8;
    const uint32_t n = (uint32_t)min((uint64_t)8, a.cols - c);
    const int32_t* slots = a.slots + t * a.topk;
    const float* weights = a.weights + t * a.topk;
    float acc[8] = {};
    for (uint32_t k0 = 0; k0 < a.topk; k0 += kCombineBatch) {
        float w[kCombineBatch];
        Eight<TZ> p[kCombineBatch];
#pragma unroll
        for (uint32_t i = 0; i < kCombineBatch; i++) {
            w[i] = 0.0f;
            p[i].zero();
            const int64_t slot = k0 + i < a.topk ? *(slots + k0 + i) : -1;
            if (slot < 0) continue;  // not sent anywhere: neither its weight nor a row counts
            if ((uint64_t)slot >= a.z_rows) {
                atomicOr(a.status, DFX_STATUS_INDEX);
                continue;
            }
            w[i] = *(weights + k0 + i);
            const TZ* s = (const TZ*)a.z + (uint64_t)slot * a.ld_z + c;
            if constexpr (VEC) {
                p[i].load(s);
            } else {
                float v[8];
                load_some(s, n, v);
#pragma unroll
                for (int j = 0; j < 8; j++) acc[j] = fmaf(w[i], v[j], acc[j]);
            }
        }
        if constexpr (VEC) {
#pragma unroll
            for (uint32_t i = 0; i < kCombineBatch; i++) {
                float v[8];
                p[i].get(v);
#pragma unroll
                for (int j = 0; j < 8; j++) acc[j] = fmaf(w[i], v[j], acc[j]);
            }
        }
    }
    TY* d = (TY*)a.y + t * a.ld_y + c;
    if constexpr (VEC) {
        store_eight(d, acc);
    } else {
#pragma unroll
        for (uint32_t j = 0; j < 8; j++)
            if (j < n) store_one(d + j, acc[j]);
    }
}

template <class TZ, class TY>
cudaError_t launch(const CombineArgs& a, cudaStream_t s) {
    // 16-byte pieces when every row of z and y starts on one and holds a whole number of them
    const bool vec = a.cols % 8 == 0 && a.ld_z * sizeof(TZ) % 16 == 0 && a.ld_y * sizeof(TY) % 16 == 0;
    const uint64_t pieces = (a.cols + 7) / 8;
    const uint64_t grid = (a.tokens * pieces + kCombineThreads - 1) / kCombineThreads;
    if (grid > 0x7fffffffull) return cudaErrorInvalidValue;
    return vec ? launch_programmatic(k_combine<TZ, TY, true>, (int)grid, kCombineThreads, 0, s, a, (uint32_t)pieces)
               : launch_programmatic(k_combine<TZ, TY, false>, (int)grid, kCombineThreads, 0, s, a, (uint32_t)pieces);
}

}  // namespace

cudaError_t launch_combine(const CombineArgs& a, cudaStream_t s) {
    if (a.z_bf16) return a.y_bf16 ? launch<__nv_bfloat16, __nv_bfloat16>(a, s) : launch<__nv_bfloat16, float>(a, s);
    return a.y_bf16 ? launch<float, __nv_bfloat16>(a, s) : launch<float, float>(a, s);
}

}  // namespace dfx
