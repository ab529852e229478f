// vec.cuh -- eight neighbouring BF16 or FP32 values of a row, loaded in 16-byte pieces: the row's
// own where they are aligned, else the aligned pieces that hold the values, shifted together (a row
// of an odd length starts anywhere).  Plain loads: the kernel before, in whose last moments these
// kernels start, may have written the values.
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

// v[i] = v[i + by], by 0 .. 3; the last ones are of no use then
template <int N>
__device__ __forceinline__ void shift_words(uint32_t (&v)[N], uint32_t by) {
#pragma unroll
    for (int i = 0; i + 2 < N; i++) v[i] = by & 2 ? v[i + 2] : v[i];
#pragma unroll
    for (int i = 0; i + 1 < N; i++) v[i] = by & 1 ? v[i + 1] : v[i];
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
    // The first n (0 .. 8) values at s, the others zero: shifted together from the aligned pieces they
    // are in, of which up to kShiftedSpan bytes from s on are read ...
    __device__ __forceinline__ void load_shifted(const __nv_bfloat16* s, uint32_t n) {
        const uint32_t off = (uint32_t)(uintptr_t)s & 15u;
        const uint4* q = reinterpret_cast<const uint4*>((uintptr_t)s - off);
        const uint4 lo = q[0], hi = q[1];
        uint32_t v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
        shift_words(v, off >> 2);
#pragma unroll
        for (int i = 0; i < 4; i++) v[i] = __funnelshift_r(v[i], v[i + 1], 8 * (off & 3u));
        auto keep = [&](uint32_t w, uint32_t i) { return n >= i + 2 ? w : n > i ? w & 0xffffu : 0u; };
        p = make_uint4(keep(v[0], 0), keep(v[1], 2), keep(v[2], 4), keep(v[3], 6));
    }
    // ... or one by one
    __device__ __forceinline__ void load_each(const __nv_bfloat16* s, uint32_t n) {
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
    __device__ __forceinline__ void load_shifted(const float* s, uint32_t n) {
        const uint32_t off = (uint32_t)(uintptr_t)s & 15u;
        const uint4* at = reinterpret_cast<const uint4*>((uintptr_t)s - off);
        uint32_t w[12];
#pragma unroll
        for (int i = 0; i < 3; i++) {
            const uint4 four = at[i];
            w[4 * i] = four.x, w[4 * i + 1] = four.y, w[4 * i + 2] = four.z, w[4 * i + 3] = four.w;
        }
        shift_words(w, off >> 2);
        float v[8];
#pragma unroll
        for (uint32_t i = 0; i < 8; i++) v[i] = i < n ? __uint_as_float(w[i]) : 0.0f;
        p = make_float4(v[0], v[1], v[2], v[3]);
        q = make_float4(v[4], v[5], v[6], v[7]);
    }
    __device__ __forceinline__ void load_each(const float* s, uint32_t n) {
        float v[8];
#pragma unroll
        for (uint32_t i = 0; i < 8; i++) v[i] = i < n ? s[i] : 0.0f;
        p = make_float4(v[0], v[1], v[2], v[3]);
        q = make_float4(v[4], v[5], v[6], v[7]);
    }
};

constexpr uint64_t kShiftedSpan = 48;
// Rows of a matrix (of `rows`, ld elements apart) from which load_shifted of any value before `cols`
// stays inside the matrix: kShiftedSpan bytes behind the row there are still rows.
inline uint64_t shifted_rows(uint64_t rows, uint64_t ld, uint64_t element_bytes) {
    const uint64_t last = (kShiftedSpan + ld * element_bytes - 1) / (ld * element_bytes);
    return rows > last ? rows - last : 0;
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
