// experts.cuh -- what the kernels of a mixture-of-experts layer share: launch arguments and
// the launchers the C entry points (api_experts.cu) call.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "dfx.h"

namespace dfx {

constexpr uint32_t kScaleBlock = 128;        // values of a row that share a scale (and rows, for weights)
constexpr uint32_t kMaxExperts = 512;        // of a router
constexpr uint32_t kMaxTopk = 32;            // experts per token
constexpr uint32_t kMaxRouteGroups = 32;     // groups of experts
constexpr uint32_t kMaxGemmExperts = 1024;   // matrices of one grouped product
// columns of a product: a sum over 2^25 of them takes 0.1 s and more, and the warps that wait for it give up
// after some 0.35 s
constexpr uint64_t kMaxGemmCols = 1ull << 25;

struct RouteArgs {
    const void* logits;
    const float* bias;      // or NULL
    uint64_t ld;            // elements between rows of logits
    uint32_t tokens, experts, topk;
    uint32_t groups, top_groups, group_best;
    uint32_t sigmoid, renormalize, bf16;
    float scale;
    int32_t* ids;           // tokens x topk
    float* weights;         // tokens x topk
    int32_t* offsets;       // experts + 1, or NULL: no assignment lists
    int32_t* rows;          // tokens * topk
    int32_t* slots;         // tokens x topk
    uint16_t* counts;       // workspace: chunks rows of `row` counts (16-byte pieces)
    uint32_t chunk;         // tokens per CTA
    uint32_t chunks, row;
    uint32_t whole;         // every lane has its share of experts, in pieces that are aligned
};

struct QuantizeArgs {
    const void* x;
    uint64_t ld_x;          // elements between rows of x
    uint64_t x_rows, shifted_rows;
    const int32_t* index;   // row of x of each row of q, or NULL
    uint64_t rows, cols;
    uint8_t* q;
    uint64_t ld_q;          // bytes between rows of q
    uint8_t* scales;
    uint64_t ld_s;          // bytes between rows of scales
    uint32_t* status;
    uint32_t bf16, swiglu, block_rows;
};

struct GemmFp8Args {
    const uint8_t* x;
    const uint8_t* sx;
    const uint8_t* w;
    const uint8_t* sw;
    const int32_t* offsets;  // experts + 1, or NULL (one matrix, every token)
    void* y;
    uint64_t ld_x, ld_sx, ld_w, ld_sw, ld_y;
    uint32_t tokens, rows, cols, experts;
    uint32_t y_f32;
    uint32_t inject;         // test hook (dfx_debug_inject), normally 0
    uint32_t* status;
};

struct CombineArgs {
    const void* z;
    uint64_t ld_z, z_rows;
    const int32_t* slots;    // tokens x topk, negative: none
    const float* weights;    // tokens x topk
    void* y;
    uint64_t ld_y;
    uint64_t tokens, cols;
    uint32_t topk, z_bf16, y_bf16;
    uint32_t* status;
};

uint64_t route_workspace_bytes(uint64_t tokens, uint32_t experts);
cudaError_t launch_route(RouteArgs a, cudaStream_t s);
cudaError_t launch_quantize_fp8(const QuantizeArgs& a, cudaStream_t s);
cudaError_t launch_gemm_fp8(const GemmFp8Args& a, int sms, cudaStream_t s);
constexpr uint32_t kStreamTokens = 8;  // most tokens of launch_stream_fp8
bool stream_fp8_takes(const GemmFp8Args& a, int sms);
cudaError_t launch_stream_fp8(const GemmFp8Args& a, int sms, cudaStream_t s);
cudaError_t launch_combine(const CombineArgs& a, cudaStream_t s);

}  // namespace dfx
