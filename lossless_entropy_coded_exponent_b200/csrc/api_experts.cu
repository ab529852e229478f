// api_experts.cu -- the C entry points of a mixture-of-experts layer declared in include/dfx.h:
// argument checks and launches of dfx_route, dfx_quantize_fp8, dfx_gemm_fp8 and dfx_combine.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "dfx.h"
#include "experts.cuh"
#include "plan.cuh"

using dfx::aligned16;
using dfx::check_device;

namespace {

bool float_type(uint32_t t) { return t == DFX_F32 || t == DFX_BF16; }

int launched(cudaError_t e) {
    if (e == cudaSuccess) return DFX_OK;
    cudaGetLastError();
    return DFX_ERR_CUDA;
}

int check_route(uint64_t tokens, uint32_t experts, const dfx_route_params* p) {
    if (!p || experts == 0 || p->topk == 0 || p->topk > experts) return DFX_ERR_ARG;
    if (p->score != DFX_SCORE_SOFTMAX && p->score != DFX_SCORE_SIGMOID) return DFX_ERR_ARG;
    if (p->groups > 1) {
        if (experts % p->groups != 0 || p->top_groups == 0 || p->top_groups > p->groups) return DFX_ERR_ARG;
        if (p->group_best > 2 || (uint64_t)p->top_groups * (experts / p->groups) < p->topk) return DFX_ERR_ARG;
    }
    if (p->renormalize > 1 || !isfinite(p->scale)) return DFX_ERR_ARG;
    if (experts > dfx::kMaxExperts || p->topk > dfx::kMaxTopk || p->groups > dfx::kMaxRouteGroups)
        return DFX_ERR_UNSUPPORTED;
    if (tokens > 0x7fffffffull / p->topk) return DFX_ERR_TOO_LARGE;  // slots are 32-bit
    return DFX_OK;
}

}  // namespace

extern "C" {

int dfx_route_workspace(uint64_t tokens, uint32_t experts, const dfx_route_params* params, size_t* bytes) {
    if (!bytes) return DFX_ERR_ARG;
    const int rc = check_route(tokens, experts, params);
    if (rc) return rc;
    *bytes = (size_t)dfx::route_workspace_bytes(tokens, experts);
    return DFX_OK;
}

int dfx_route(dfx_plan_t plan, const void* d_logits, uint32_t logits_type, uint64_t ld_logits, uint64_t tokens,
              uint32_t experts, const float* d_bias, const dfx_route_params* params, int32_t* d_ids, float* d_weights,
              int32_t* d_offsets, int32_t* d_rows, int32_t* d_slots, void* d_workspace, size_t workspace_bytes,
              cudaStream_t stream) {
    if (!plan) return DFX_ERR_ARG;
    int rc = check_route(tokens, experts, params);
    if (rc) return rc;
    if (!float_type(logits_type) || ld_logits < experts) return DFX_ERR_ARG;
    const bool lists = d_offsets || d_rows || d_slots;
    if (lists && !d_offsets) return DFX_ERR_ARG;
    if (tokens && (!d_logits || !d_ids || !d_weights || (lists && (!d_rows || !d_slots)))) return DFX_ERR_ARG;
    if (!aligned16(d_logits) || !aligned16(d_bias) || !aligned16(d_ids) || !aligned16(d_weights) ||
        !aligned16(d_offsets) || !aligned16(d_rows) || !aligned16(d_slots))
        return DFX_ERR_ARG;
    if (lists) {
        if (!d_workspace || !aligned16(d_workspace)) return DFX_ERR_ARG;
        if (workspace_bytes < dfx::route_workspace_bytes(tokens, experts)) return DFX_ERR_CAPACITY;
    }
    rc = check_device(plan);
    if (rc) return rc;
    if (tokens == 0 && !lists) return DFX_OK;
    dfx::RouteArgs a;
    memset(&a, 0, sizeof(a));
    a.logits = d_logits;
    a.bias = d_bias;
    a.ld = ld_logits;
    a.tokens = (uint32_t)tokens;
    a.experts = experts;
    a.topk = params->topk;
    a.groups = params->groups ? params->groups : 1;
    a.top_groups = params->top_groups;
    a.group_best = params->group_best ? params->group_best : 1;
    a.sigmoid = params->score == DFX_SCORE_SIGMOID;
    a.renormalize = params->renormalize;
    a.bf16 = logits_type == DFX_BF16;
    a.scale = params->scale == 0.0f ? 1.0f : params->scale;
    a.ids = d_ids;
    a.weights = d_weights;
    a.offsets = d_offsets;
    a.rows = d_rows;
    a.slots = d_slots;
    a.counts = (uint16_t*)d_workspace;
    return launched(dfx::launch_route(a, stream));
}

int dfx_quantize_fp8(dfx_plan_t plan, const void* d_x, uint32_t x_type, uint64_t ld_x, uint64_t x_rows,
                     const int32_t* d_index, uint64_t rows, uint64_t cols, uint32_t block_rows, uint32_t flags,
                     void* d_q, uint64_t ld_q, void* d_scales, uint64_t ld_scales, cudaStream_t stream) {
    if (!plan || !float_type(x_type) || (flags & ~(uint32_t)DFX_QUANT_SWIGLU)) return DFX_ERR_ARG;
    if (block_rows != 1 && block_rows != dfx::kScaleBlock) return DFX_ERR_ARG;
    if (block_rows != 1 && (d_index || flags)) return DFX_ERR_UNSUPPORTED;
    if (cols == 0 || rows >= (1ull << 31) || x_rows >= (1ull << 31) || cols >= (1ull << 31)) return DFX_ERR_ARG;
    const uint64_t width = (flags & DFX_QUANT_SWIGLU) ? 2 * cols : cols;
    const uint64_t blocks = (cols + dfx::kScaleBlock - 1) / dfx::kScaleBlock;
    if (ld_x < width || ld_q < cols || ld_q % 16 != 0 || ld_scales < blocks || ld_scales % 4 != 0) return DFX_ERR_ARG;
    if (!d_index && rows > x_rows) return DFX_ERR_ARG;
    if (!aligned16(d_x) || !aligned16(d_index) || !aligned16(d_q) || !aligned16(d_scales)) return DFX_ERR_ARG;
    if (rows && ((!d_x && x_rows) || !d_q || !d_scales)) return DFX_ERR_ARG;
    const int rc = check_device(plan);
    if (rc || rows == 0) return rc;
    dfx::QuantizeArgs a;
    memset(&a, 0, sizeof(a));
    a.x = d_x;
    a.ld_x = ld_x;
    a.x_rows = x_rows;
    a.index = d_index;
    a.rows = rows;
    a.cols = cols;
    a.q = (uint8_t*)d_q;
    a.ld_q = ld_q;
    a.scales = (uint8_t*)d_scales;
    a.ld_s = ld_scales;
    a.status = plan->d_status;
    a.bf16 = x_type == DFX_BF16;
    a.swiglu = (flags & DFX_QUANT_SWIGLU) != 0;
    a.block_rows = block_rows;
    return launched(dfx::launch_quantize_fp8(a, stream));
}

int dfx_gemm_fp8(dfx_plan_t plan, const void* d_x, uint64_t ld_x, const void* d_x_scales, uint64_t ld_x_scales,
                 uint64_t tokens, const void* d_w, uint64_t ld_w, const void* d_w_scales, uint64_t ld_w_scales,
                 uint64_t rows, uint64_t cols, uint32_t experts, const int32_t* d_offsets, void* d_y, uint32_t y_type,
                 uint64_t ld_y, cudaStream_t stream) {
    if (!plan || !float_type(y_type) || experts == 0 || cols == 0) return DFX_ERR_ARG;
    if (experts > 1 && !d_offsets) return DFX_ERR_ARG;
    if (experts > dfx::kMaxGemmExperts) return DFX_ERR_UNSUPPORTED;
    if (tokens >= (1ull << 31) || cols > dfx::kMaxGemmCols || rows >= (1ull << 31) || rows * experts >= (1ull << 31))
        return DFX_ERR_TOO_LARGE;
    const uint64_t blocks = (cols + dfx::kScaleBlock - 1) / dfx::kScaleBlock;
    if (ld_x < cols || ld_x % 16 != 0 || ld_w < cols || ld_w % 16 != 0 || ld_y < rows) return DFX_ERR_ARG;
    if (ld_x_scales < blocks || ld_x_scales % 4 != 0 || ld_w_scales < blocks || ld_w_scales % 4 != 0) return DFX_ERR_ARG;
    if (!aligned16(d_x) || !aligned16(d_x_scales) || !aligned16(d_w) || !aligned16(d_w_scales) || !aligned16(d_offsets) ||
        !aligned16(d_y))
        return DFX_ERR_ARG;
    if (tokens && rows && (!d_x || !d_x_scales || !d_w || !d_w_scales || !d_y)) return DFX_ERR_ARG;
    const int rc = check_device(plan);
    if (rc || tokens == 0 || rows == 0) return rc;
    dfx::GemmFp8Args a;
    memset(&a, 0, sizeof(a));
    a.x = (const uint8_t*)d_x;
    a.sx = (const uint8_t*)d_x_scales;
    a.w = (const uint8_t*)d_w;
    a.sw = (const uint8_t*)d_w_scales;
    a.offsets = d_offsets;
    a.y = d_y;
    a.ld_x = ld_x;
    a.ld_sx = ld_x_scales;
    a.ld_w = ld_w;
    a.ld_sw = ld_w_scales;
    a.ld_y = ld_y;
    a.tokens = (uint32_t)tokens;
    a.rows = (uint32_t)rows;
    a.cols = (uint32_t)cols;
    a.experts = experts;
    a.y_f32 = y_type == DFX_F32;
    a.inject = dfx::g_inject & DFX_INJECT_SKIP_TILE_COPY;
    a.status = plan->d_status;
    return launched(dfx::launch_gemm_fp8(a, plan->sms, stream));
}

int dfx_combine(dfx_plan_t plan, const void* d_z, uint32_t z_type, uint64_t ld_z, uint64_t z_rows, uint64_t cols,
                const int32_t* d_slots, const float* d_weights, uint64_t tokens, uint32_t topk, void* d_y,
                uint32_t y_type, uint64_t ld_y, cudaStream_t stream) {
    if (!plan || !float_type(z_type) || !float_type(y_type) || cols == 0 || topk == 0) return DFX_ERR_ARG;
    if (topk > dfx::kMaxTopk) return DFX_ERR_UNSUPPORTED;
    if (cols >= (1ull << 31) || tokens >= (1ull << 31) || z_rows >= (1ull << 31)) return DFX_ERR_TOO_LARGE;
    if (ld_z < cols || ld_y < cols) return DFX_ERR_ARG;
    if (!aligned16(d_z) || !aligned16(d_slots) || !aligned16(d_weights) || !aligned16(d_y)) return DFX_ERR_ARG;
    if (tokens && ((!d_z && z_rows) || !d_slots || !d_weights || !d_y)) return DFX_ERR_ARG;
    const int rc = check_device(plan);
    if (rc || tokens == 0) return rc;
    dfx::CombineArgs a;
    memset(&a, 0, sizeof(a));
    a.z = d_z;
    a.ld_z = ld_z;
    a.z_rows = z_rows;
    a.slots = d_slots;
    a.weights = d_weights;
    a.y = d_y;
    a.ld_y = ld_y;
    a.tokens = tokens;
    a.cols = cols;
    a.topk = topk;
    a.z_bf16 = z_type == DFX_BF16;
    a.y_bf16 = y_type == DFX_BF16;
    a.status = plan->d_status;
    return launched(dfx::launch_combine(a, stream));
}

}  // extern "C"
