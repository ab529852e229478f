// vec.cuh -- eight neighbouring BF16 or FP32 values of a row as FP32, loaded and stored in
// 16-byte pieces where the row's alignment allows it and one by one where it does not.  Plain
// loads: the kernel before, in whose last moments these kernels start, may have written them.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace dfx {
namespace {

__device__ __forceinline__ float as_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float as_f32(float v) { return v; }

__device__ __forceinline__ void unpack_bf16(uint32_t w, float& lo, float& hi) {
    lo = __uint_as_float(w << 16);
    hi = __uint_as_float(w & 0xffff0000u);
}

// The 16-byte pieces of eight values, as they are loaded: kept apart from their conversion
// so that a thread can have several loads in flight.
template <class T>
struct Eight;
template <>
struct Eight<__nv_bfloat16> {
    uint4 p;
    __device__ __forceinline__ void load(const __nv_bfloat16* s) { p = *reinterpret_cast<const uint4*>(s); }
    __device__ __forceinline__ void zero() { p = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        unpack_bf16(p.x, v[0], v[1]);
        unpack_bf16(p.y, v[2], v[3]);
        unpack_bf16(p.z, v[4], v[5]);
        unpack_bf16(p.w, v[6], v[7]);
    }
    // n (0 .. 8) values one by one, the others zero
    __device__ __forceinline__ void load_some(const __nv_bfloat16* s, uint32_t n) {
        const uint16_t* h = reinterpret_cast<const uint16_t*>(s);
        uint32_t w[8];
#pragma unroll
        for (uint32_t i = 0; i < 8; i++) w[i] = i < n ? h[i] : 0u;
        p = make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
    }
};
template <>
struct Eight<float> {
    float4 p, q;
    __device__ __forceinline__ void load(const float* s) {
        p = reinterpret_cast<const float4*>(s)[0];
        q = reinterpret_cast<const float4*>(s)[1];
    }
    __device__ __forceinline__ void zero() { p = q = make_float4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        v[0] = p.x, v[1] = p.y, v[2] = p.z, v[3] = p.w;
        v[4] = q.x, v[5] = q.y, v[6] = q.z, v[7] = q.w;
    }
    __device__ __forceinline__ void load_some(const float* s, uint32_t n) {
        float v[8];
#pragma unroll
        for (uint32_t i = 0; i < 8; i++) v[i] = i < n ? s[i] : 0.0f;
        p = make_float4(v[0], v[1], v[2], v[3]);
        q = make_float4(v[4], v[5], v[6], v[7]);
    }
};

// n (0 .. 8) values at s one by one, the others zero
template <class T>
__device__ __forceinline__ void load_some(const T* s, uint32_t n, float (&v)[8]) {
#pragma unroll
    for (uint32_t i = 0; i < 8; i++) v[i] = i < n ? as_f32(s[i]) : 0.0f;
}

// FP32 to BF16 rounds to nearest, ties to even
__device__ __forceinline__ void store_eight(__nv_bfloat16* d, const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&p);
    }
    *reinterpret_cast<uint4*>(d) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store_eight(float* d, const float (&v)[8]) {
    reinterpret_cast<float4*>(d)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(d)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store_one(__nv_bfloat16* d, float v) { *d = __float2bfloat16_rn(v); }
__device__ __forceinline__ void store_one(float* d, float v) { *d = v; }

}  // namespace
}  // namespace dfx
