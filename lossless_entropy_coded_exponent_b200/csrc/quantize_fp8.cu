// quantize_fp8.cu -- BF16 or FP32 values to e4m3 with a power-of-two scale for each block of
// 1 x 128 (activations) or 128 x 128 (weights) values.
//
// For a block with the largest finite magnitude m the scale is 2^e, the smallest power of two
// with m / 2^e <= 448 (e4m3's largest value), held as the byte e + 127 (e8m0, what the tensor
// cores take).  Dividing by a power of two is exact, so a value is rounded once, to nearest
// even, by the conversion itself.  448 = 1.75 * 2^8, so e follows from m's exponent and one
// comparison of its mantissa.  NaN and infinities become e4m3's NaN and have no part in m: they
// stay visible in a product instead of being clipped to a number.
//
// 1 x 128: 16 lanes hold a block, 8 values each; the maximum is four shuffles.  A warp takes 8
// neighbouring blocks of one row and has all their loads in flight before it uses the first:
// the kernel is bound by DRAM.  With `index`, output row r is row index[r] of x (rows sent to
// experts, in the experts' order).  With SwiGLU a row of x holds cols gates, then cols values,
// and silu(gate) * value is quantized, in FP32 without a rounding in between.
// 128 x 128: a CTA holds a block in registers, 64 values per thread.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "dfx_common.cuh"
#include "experts.cuh"
#include "launch.cuh"
#include "vec.cuh"

namespace dfx {
namespace {

constexpr int kQuantThreads = 256;
constexpr uint32_t kUnits = 4;                    // blocks of a half warp
constexpr uint32_t kWarpBlocks = 2 * kUnits;      // neighbouring blocks of a warp
constexpr uint32_t kTallRows = 8;                 // rows of a 128 x 128 block per thread
constexpr uint32_t kBorder = 0x600000;            // mantissa of 1.75

// the scale byte of a block whose largest magnitude has these FP32 bits
__device__ __forceinline__ uint32_t scale_byte(uint32_t m) {
    if (m == 0) return 127;
    const int e = (int)(m >> 23) - 8 + ((m & 0x7fffffu) > kBorder);
    return (uint32_t)max(e, 0);  // at most 247: FP32's largest exponent is 254
}
// 1 / scale: 2^(127 - byte), an FP32 normal for the bytes scale_byte gives
__device__ __forceinline__ float inverse_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// FP32 bits of the largest finite magnitude of eight values; what is not finite becomes NaN
__device__ __forceinline__ uint32_t magnitude(float (&v)[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const uint32_t b = __float_as_uint(v[i]) & 0x7fffffffu;
        if (b >= 0x7f800000u) v[i] = __uint_as_float(0x7fffffffu);
        else m = max(m, b);
    }
    return m;
}

__device__ __forceinline__ uint2 to_e4m3(const float (&v)[8], float inv) {
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; i++)
        h[i] = __nv_cvt_float2_to_fp8x2(make_float2(v[2 * i] * inv, v[2 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
    return make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
}

// up to 8 bytes at d (8-byte aligned)
__device__ __forceinline__ void store_bytes(uint8_t* d, uint2 q, uint32_t n) {
    if (n == 8) {
        *reinterpret_cast<uint2*>(d) = q;
    } else {
        for (uint32_t i = 0; i < n; i++) d[i] = (uint8_t)((i < 4 ? q.x : q.y) >> (8 * (i & 3)));
    }
}

__device__ __forceinline__ float silu_times(float g, float u) {
    // fast exponential and division (a few units in the last place) where they are in range
    if (fabsf(g) < 80.0f) return __fdividef(g, 1.0f + __expf(-g)) * u;
    return g / (1.0f + expf(-g)) * u;
}
__device__ __forceinline__ double silu_times_64(float g, float u) { return (double)g / (1.0 + exp(-(double)g)) * (double)u; }

template <class T, bool VEC, bool SWIGLU>
__global__ void __launch_bounds__(kQuantThreads) k_quantize_rows(const QuantizeArgs a, const uint32_t col_warps) {
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    wait_prior_grid();
    const uint32_t lane = threadIdx.x & 31, q = lane & 15, half = lane >> 4;
    const uint64_t gw = (uint64_t)blockIdx.x * (kQuantThreads / 32) + (threadIdx.x >> 5);
    const uint64_t row = gw / col_warps;
    if (row >= a.rows) return;
    const uint32_t b0 = (uint32_t)(gw - row * col_warps) * kWarpBlocks + half;  // blocks b0, b0 + 2, ...
    int64_t from = (int64_t)row;
    if (a.index) {
        from = *(a.index + row);
        if (from < 0) return;  // a row that stays as it is
        if ((uint64_t)from >= a.x_rows) {
            if (lane == 0) atomicOr(a.status, DFX_STATUS_INDEX);
            return;
        }
    }
    const T* x = (const T*)a.x + (uint64_t)from * a.ld_x;
    const unsigned mask = half ? 0xffff0000u : 0x0000ffffu;
    constexpr int P = SWIGLU ? 2 : 1;
    Eight<T> p[VEC ? kUnits : 1][P];
    if constexpr (VEC) {
#pragma unroll
        for (uint32_t i = 0; i < kUnits; i++) {
            const uint64_t c = (uint64_t)(b0 + 2 * i) * kScaleBlock + 8 * q;
#pragma unroll
            for (int j = 0; j < P; j++) {
                if (c < a.cols) p[i][j].load(x + j * a.cols + c);
                else p[i][j].zero();
            }
        }
    }
#pragma unroll
    for (uint32_t i = 0; i < kUnits; i++) {
        const uint32_t b = b0 + 2 * i;
        const uint64_t c = (uint64_t)b * kScaleBlock + 8 * q;
        const uint32_t n = c < a.cols ? (uint32_t)min((uint64_t)8, a.cols - c) : 0;
        float v[8], u[8];
        if constexpr (VEC) {
            p[i][0].get(v);
            if constexpr (SWIGLU) p[i][1].get(u);
        } else {
            load_some(x + c, n, v);
            if constexpr (SWIGLU) load_some(x + a.cols + c, n, u);
        }
        float g[SWIGLU ? 8 : 1];
        if constexpr (SWIGLU) {
#pragma unroll
            for (int j = 0; j < 8; j++) {
                g[j] = v[j];
                v[j] = silu_times(v[j], u[j]);
            }
        }
        uint32_t m = magnitude(v);
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) m = max(m, __shfl_xor_sync(mask, m, d));
        uint32_t byte = scale_byte(m);
        if constexpr (SWIGLU) {
            // within 2^-16 of the border the scale is settled in 64 bits, so that it does not
            // hang on the exponential's last places (one block in some 30 thousand)
            const int d = (int)(m & 0x7fffffu) - (int)kBorder;
            if (d > -256 && d < 256 && m >= 0x00800000u) {
                double w = 0.0;
#pragma unroll
                for (int j = 0; j < 8; j++)
                    if (isfinite(v[j])) w = fmax(w, fabs(silu_times_64(g[j], u[j])));
#pragma unroll
                for (int e = 8; e > 0; e >>= 1) w = fmax(w, __shfl_xor_sync(mask, w, e));
                const long long bits = __double_as_longlong(w);
                const int e = (int)(bits >> 52) - 1023 + 127 - 8 + ((bits & 0xfffffffffffffll) > (0xcll << 48));
                byte = (uint32_t)max(e, 0);
            }
        }
        if (n == 0) continue;  // past the row's end (a lane; its shuffles are done)
        store_bytes(a.q + row * a.ld_q + c, to_e4m3(v, inverse_scale(byte)), n);
        if (q == 0) a.scales[row * a.ld_s + b] = (uint8_t)byte;
    }
}

template <class T, bool VEC>
__global__ void __launch_bounds__(kQuantThreads) k_quantize_tall(const QuantizeArgs a, const uint32_t col_blocks) {
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    wait_prior_grid();
    __shared__ uint32_t warp_max[kQuantThreads / 32];
    const uint32_t q = threadIdx.x & 15, r0 = threadIdx.x >> 4;  // rows r0, r0 + 16, ...
    const uint64_t rb = blockIdx.x / col_blocks;
    const uint32_t cb = blockIdx.x - (uint32_t)rb * col_blocks;
    const uint64_t c = (uint64_t)cb * kScaleBlock + 8 * q;
    const uint32_t n = c < a.cols ? (uint32_t)min((uint64_t)8, a.cols - c) : 0;
    float v[kTallRows][8];
    if constexpr (VEC) {
        Eight<T> p[kTallRows];
#pragma unroll
        for (uint32_t i = 0; i < kTallRows; i++) {
            const uint64_t r = rb * kScaleBlock + r0 + 16 * i;
            if (r < a.rows && n) p[i].load((const T*)a.x + r * a.ld_x + c);
            else p[i].zero();
        }
#pragma unroll
        for (uint32_t i = 0; i < kTallRows; i++) p[i].get(v[i]);
    } else {
#pragma unroll
        for (uint32_t i = 0; i < kTallRows; i++) {
            const uint64_t r = rb * kScaleBlock + r0 + 16 * i;
            load_some((const T*)a.x + r * a.ld_x + c, r < a.rows ? n : 0, v[i]);
        }
    }
    uint32_t m = 0;
#pragma unroll
    for (uint32_t i = 0; i < kTallRows; i++) m = max(m, magnitude(v[i]));
    m = __reduce_max_sync(kFull, m);
    if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kQuantThreads / 32; i++) m = max(m, warp_max[i]);
    const uint32_t byte = scale_byte(m);
    const float inv = inverse_scale(byte);
#pragma unroll
    for (uint32_t i = 0; i < kTallRows; i++) {
        const uint64_t r = rb * kScaleBlock + r0 + 16 * i;
        if (r < a.rows && n) store_bytes(a.q + r * a.ld_q + c, to_e4m3(v[i], inv), n);
    }
    if (threadIdx.x == 0) a.scales[rb * a.ld_s + cb] = (uint8_t)byte;
}

template <class T>
cudaError_t launch(const QuantizeArgs& a, cudaStream_t s) {
    // 16-byte pieces when every row (and a row's values behind its gates) starts on one and a
    // row holds a whole number of eights
    const bool vec = a.cols % 8 == 0 && a.ld_x * sizeof(T) % 16 == 0;
    const uint64_t blocks = (a.cols + kScaleBlock - 1) / kScaleBlock;
    uint64_t grid;
    if (a.block_rows == 1) {
        const uint64_t col_warps = (blocks + kWarpBlocks - 1) / kWarpBlocks;
        grid = (a.rows * col_warps + kQuantThreads / 32 - 1) / (kQuantThreads / 32);
        if (grid > 0x7fffffffull) return cudaErrorInvalidValue;
        auto* k = a.swiglu ? (vec ? k_quantize_rows<T, true, true> : k_quantize_rows<T, false, true>)
                           : (vec ? k_quantize_rows<T, true, false> : k_quantize_rows<T, false, false>);
        return launch_programmatic(k, (int)grid, kQuantThreads, 0, s, a, (uint32_t)col_warps);
    }
    grid = (a.rows + kScaleBlock - 1) / kScaleBlock * blocks;
    if (grid > 0x7fffffffull) return cudaErrorInvalidValue;
    auto* k = vec ? k_quantize_tall<T, true> : k_quantize_tall<T, false>;
    return launch_programmatic(k, (int)grid, kQuantThreads, 0, s, a, (uint32_t)blocks);
}

}  // namespace

cudaError_t launch_quantize_fp8(const QuantizeArgs& a, cudaStream_t s) {
    return a.bf16 ? launch<__nv_bfloat16>(a, s) : launch<float>(a, s);
}

}  // namespace dfx
