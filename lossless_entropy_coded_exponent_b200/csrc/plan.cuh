// plan.cuh -- what a dfx_plan_t points at, shared by the C entry points (api.cu,
// api_experts.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "dfx_common.cuh"

struct dfx_plan_s {
    uint64_t n;
    uint32_t K, G, max_len;
    uint32_t coder, table_log;  // exponent coder; tANS table log (coder 1)
    uint32_t decode_flags;      // DFX_DECODE_*
    dfx::Layout L;
    uint64_t max_bytes;
    uint64_t ws_bytes;
    uint32_t* d_status;
    int device;
    int sms;  // streaming multiprocessors of the device
    int decode_grid;
    int resident_ctas;  // decode CTAs that fit on the device at once
    // events ordering dfx_decode_host's copies before the decode of their slices,
    // created on first use
    static constexpr uint32_t kHostSlicesMax = 64;
    cudaEvent_t slice_done[kHostSlicesMax];
    // recorded on the decode stream when dfx_decode_host starts: its copies into the
    // staging buffer wait for the decoding already queued there (an earlier call's
    // slices may still be reading the buffer)
    cudaEvent_t decode_idle;
    bool events_made;
};

namespace dfx {

extern uint32_t g_inject;  // dfx_debug_inject

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

// a plan's calls run on the device it was made on
inline int check_device(const dfx_plan_s* plan) {
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) return DFX_ERR_CUDA;
    return dev == plan->device ? DFX_OK : DFX_ERR_ARG;
}

}  // namespace dfx
