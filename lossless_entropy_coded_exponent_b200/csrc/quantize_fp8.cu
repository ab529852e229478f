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
// 1 x 128: 8 lanes hold a block, 16 values each, and the maximum is three shuffles; a lane has 8
// loads in flight before it uses the first.  With `index`, output row r is row index[r] of x
// (rows sent to experts, in the experts' order).  With SwiGLU a row of x holds cols gates, then
// cols values, and silu(gate) * value is quantized, in FP32 without a rounding in between.
// Plain rows are bound by DRAM.  With SwiGLU the instructions count too: 16 values a lane, paired
// arithmetic and 32-bit indices brought 8195 x 14320 values from 184 to 111 us (5.3 TB/s, 82 % of
// the measured copy rate); 8 values a lane took 124 us, more CTAs per SM with fewer registers
// 113 to 150 us.
// 128 x 128: a CTA holds a block as it was loaded in registers, 64 values per thread, so four CTAs
// are resident and one's loads overlap another's stores: 14336 x 4096 BF16 values in 30 us
// (5.9 TB/s, 91 %), against 83 us with the block held as FP32 (one CTA per SM).
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
constexpr int kQuantCtas = 4;                     // per SM: 64 registers a thread
constexpr uint32_t kTallRows = 8;                 // rows of a 128 x 128 block per thread
constexpr uint32_t kBorder = 0x600000;            // mantissa of 1.75

constexpr uint32_t kRowLanes = 8;                 // lanes of a 1 x 128 block: 16 values each
constexpr uint32_t kRowBlocks = 32 / kRowLanes;   // blocks of a warp side by side

// runs of kRowBlocks blocks of a warp: 8 loads of 16 bytes in flight per lane
template <class T, bool SWIGLU>
__host__ __device__ constexpr uint32_t units() { return 4 / (sizeof(T) / 2) / (SWIGLU ? 2 : 1); }

// the scale byte of a block whose largest magnitude has these FP32 bits
__device__ __forceinline__ uint32_t scale_byte(uint32_t m) {
    if (m == 0) return 127;
    const int e = (int)(m >> 23) - 8 + ((m & 0x7fffffu) > kBorder);
    return (uint32_t)max(e, 0);  // at most 247: FP32's largest exponent is 254
}
// 1 / scale: 2^(127 - byte), an FP32 normal for the bytes scale_byte gives
__device__ __forceinline__ float inverse_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// Largest magnitude: NaN has no part in it, an infinity is the largest of all (the block is
// then looked at again, without infinities: finite_magnitude).
__device__ __forceinline__ float magnitude(const float (&v)[8], float m) {
#pragma unroll
    for (int i = 0; i < 8; i++) m = fmaxf(m, fabsf(v[i]));
    return m;
}
__device__ __forceinline__ float magnitude(const Eight<float>& p, float m) {
    float v[8];
    p.get(v);
    return magnitude(v, m);
}
__device__ __forceinline__ float magnitude(const Eight<__nv_bfloat16>& p, float m) {
    auto pair = [](const uint32_t& w) { return __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w)); };
    const float2 f = __bfloat1622float2(__hmax2(__hmax2(pair(p.p.x), pair(p.p.y)), __hmax2(pair(p.p.z), pair(p.p.w))));
    return fmaxf(m, fmaxf(f.x, f.y));
}
// the same over finite values only; infinities become NaN
__device__ __forceinline__ float finite_magnitude(float (&v)[8], float m) {
#pragma unroll
    for (int i = 0; i < 8; i++) {
        if (fabsf(v[i]) < INFINITY) m = fmaxf(m, fabsf(v[i]));
        else v[i] = __uint_as_float(0x7fffffffu);
    }
    return m;
}

// two FP32 operations in one instruction
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 c;
    asm("{\n .reg .b64 a, b, c;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mul.rn.f32x2 c, a, b;\n mov.b64 {%0, %1}, c;\n}\n"
        : "=f"(c.x), "=f"(c.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return c;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 c;
    asm("{\n .reg .b64 a, b, c;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n add.rn.f32x2 c, a, b;\n mov.b64 {%0, %1}, c;\n}\n"
        : "=f"(c.x), "=f"(c.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return c;
}

__device__ __forceinline__ uint2 to_e4m3(const float (&v)[8], float inv) {
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; i++)
        h[i] = __nv_cvt_float2_to_fp8x2(mul2(make_float2(v[2 * i], v[2 * i + 1]), make_float2(inv, inv)), __NV_SATFINITE,
                                        __NV_E4M3);
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

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float reciprocal_fast(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}

// gate / (1 + exp(-gate)) * value of eight neighbours: with the approximate power of two and
// reciprocal (together within 2^-22 + |gate| 2^-24) unless a gate is so low that 1 + exp(-gate)
// leaves the reciprocal's range.  Below -88.7 it leaves FP32's, where a large value still makes a product
// that FP32 holds: from -80 down the quotient is gate * exp(-80) * exp(gate + 80), of which the
// last factor comes in two halves behind the value (within 2^-20)
__device__ __forceinline__ void swiglu(const float (&g)[8], const float (&u)[8], float (&v)[8]) {
    float low = g[0];
#pragma unroll
    for (int i = 1; i < 8; i++) low = fminf(low, g[i]);
    if (low > -80.0f) {
        constexpr float kLog2e = 1.4426950408889634f;
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const float2 g2 = make_float2(g[i], g[i + 1]);
            float2 t = mul2(g2, make_float2(-kLog2e, -kLog2e));
            t = add2(make_float2(exp2_fast(t.x), exp2_fast(t.y)), make_float2(1.0f, 1.0f));
            t = mul2(mul2(g2, make_float2(reciprocal_fast(t.x), reciprocal_fast(t.y))), make_float2(u[i], u[i + 1]));
            v[i] = t.x, v[i + 1] = t.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++) {
            constexpr float kExpMinus80 = 1.8048513878454153e-35f;
            const float half = expf(0.5f * fminf(g[i] + 80.0f, 0.0f));
            v[i] = (g[i] > -80.0f ? g[i] / (1.0f + expf(-g[i])) : g[i] * kExpMinus80) * u[i] * half * half;
        }
    }
}
__device__ __forceinline__ double silu_times_64(float g, float u) { return (double)g / (1.0 + exp(-(double)g)) * (double)u; }

// maximum over the lanes of a block
__device__ __forceinline__ float block_max(unsigned mask, float m) {
#pragma unroll
    for (int d = kRowLanes / 2; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(mask, m, d));
    return m;
}

// Within 2^-15 of the border the scale is settled in 64 bits, so that it does not hang on the
// exponential's last places (one block in some 16 thousand); the n gates and values of this lane
// are read again.  The FP32 maximum is next to a border, at most 1.75 * 2^127, so what is above 1.875 *
// 2^127 is a product that FP32 did not hold: it became NaN and has no part in the scale.
template <class T>
__device__ __noinline__ uint32_t swiglu_scale_64(unsigned mask, const T* gates, const T* values, uint32_t n) {
    double w = 0.0;
    for (uint32_t j = 0; j < n; j++) {
        const double v = fabs(silu_times_64(as_f32(gates[j]), as_f32(values[j])));
        if (v < 0x1.ep127) w = fmax(w, v);
    }
#pragma unroll
    for (int e = kRowLanes / 2; e > 0; e >>= 1) w = fmax(w, __shfl_xor_sync(mask, w, e));
    const long long bits = __double_as_longlong(w);
    const int e = (int)(bits >> 52) - 1023 + 127 - 8 + ((bits & 0xfffffffffffffll) > (0xcll << 48));
    return (uint32_t)max(e, 0);
}

template <class T, bool VEC, bool SWIGLU>
__global__ void __launch_bounds__(kQuantThreads, kQuantCtas) k_quantize_rows(const QuantizeArgs a, const uint32_t col_warps) {
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    wait_prior_grid();
    constexpr uint32_t kUnits = units<T, SWIGLU>();
    const uint32_t lane = threadIdx.x & 31, q = lane % kRowLanes, part = lane / kRowLanes;
    // 32-bit indices within the row; the launcher sees to it that the warps fit 32 bits
    const uint32_t gw = blockIdx.x * (kQuantThreads / 32) + (threadIdx.x >> 5), row = gw / col_warps;
    if (row >= a.rows) return;
    const uint32_t b0 = (gw - row * col_warps) * (kRowBlocks * kUnits) + part;  // blocks b0, b0 + 4, ...
    const uint32_t cols = (uint32_t)a.cols;
    int64_t from = row;
    if (a.index) {
        from = a.index[row];
        if (from < 0) return;  // a row that stays as it is
        if ((uint64_t)from >= a.x_rows) {
            if (lane == 0) atomicOr(a.status, DFX_STATUS_INDEX);
            return;
        }
    }
    const T* x = (const T*)a.x + (uint64_t)from * a.ld_x;
    uint8_t *out = a.q + row * a.ld_q, *out_s = a.scales + row * a.ld_s;
    const unsigned mask = ((1u << kRowLanes) - 1u) << (kRowLanes * part);
    constexpr int P = SWIGLU ? 2 : 1;
    Eight<T> p[kUnits][2][P];
    auto load = [&](auto how) {
#pragma unroll
        for (uint32_t i = 0; i < kUnits; i++)
#pragma unroll
            for (uint32_t h = 0; h < 2; h++) {
                const uint32_t c = (b0 + kRowBlocks * i) * kScaleBlock + 16 * q + 8 * h;
#pragma unroll
                for (int j = 0; j < P; j++) {
                    if (c < cols) how(p[i][h][j], x + j * cols + c, min(8u, cols - c));
                    else p[i][h][j].zero();
                }
            }
    };
    if constexpr (VEC) load([](Eight<T>& e, const T* s, uint32_t) { e.load(s); });
    else if ((uint64_t)from < a.shifted_rows) load([](Eight<T>& e, const T* s, uint32_t n) { e.load_shifted(s, n); });
    else load([](Eight<T>& e, const T* s, uint32_t n) { e.load_each(s, n); });  // the last row or rows
#pragma unroll
    for (uint32_t i = 0; i < kUnits; i++) {
        const uint32_t b = b0 + kRowBlocks * i, c0 = b * kScaleBlock + 16 * q;
        const uint32_t n = c0 < cols ? min(16u, cols - c0) : 0;
        float v[2][8];
        float m = 0.0f;
#pragma unroll
        for (uint32_t h = 0; h < 2; h++) {
            float g[8], u[8];
            p[i][h][0].get(SWIGLU ? g : v[h]);
            if constexpr (SWIGLU) {
                p[i][h][1].get(u);
                swiglu(g, u, v[h]);
            }
            m = magnitude(v[h], m);
        }
        m = block_max(mask, m);
        if (m == INFINITY) m = block_max(mask, finite_magnitude(v[1], finite_magnitude(v[0], 0.0f)));
        uint32_t byte = scale_byte(__float_as_uint(m));
        if constexpr (SWIGLU) {
            const int d = (int)(__float_as_uint(m) & 0x7fffffu) - (int)kBorder;
            if (d > -256 && d < 256 && m >= 0x1p-126f) byte = swiglu_scale_64(mask, x + c0, x + cols + c0, n);
        }
        if (n == 0) continue;  // past the row's end (a lane; its shuffles are done)
        const float inv = inverse_scale(byte);
        const uint2 lo = to_e4m3(v[0], inv), hi = to_e4m3(v[1], inv);
        if (n == 16) {
            *reinterpret_cast<uint4*>(out + c0) = make_uint4(lo.x, lo.y, hi.x, hi.y);
        } else {
            store_bytes(out + c0, lo, min(n, 8u));
            if (n > 8) store_bytes(out + c0 + 8, hi, n - 8);
        }
        if (q == 0) out_s[b] = (uint8_t)byte;
    }
}

template <class T, bool VEC>
__global__ void __launch_bounds__(kQuantThreads, sizeof(T) == 2 ? kQuantCtas : 2)
    k_quantize_tall(const QuantizeArgs a, const uint32_t col_blocks) {
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    wait_prior_grid();
    __shared__ float warp_max[kQuantThreads / 32];
    const uint32_t q = threadIdx.x & 15, r0 = threadIdx.x >> 4;  // rows r0, r0 + 16, ...
    const uint64_t rb = blockIdx.x / col_blocks;
    const uint32_t cb = blockIdx.x - (uint32_t)rb * col_blocks;
    const uint64_t c = (uint64_t)cb * kScaleBlock + 8 * q;
    const uint32_t n = c < a.cols ? (uint32_t)min((uint64_t)8, a.cols - c) : 0;
    const uint64_t first = rb * kScaleBlock + r0;
    const T* x = (const T*)a.x + first * a.ld_x + c;
    const bool shifted = (rb + 1) * kScaleBlock <= a.shifted_rows;
    // the block stays in registers as it was loaded
    Eight<T> p[kTallRows];
#pragma unroll
    for (uint32_t i = 0; i < kTallRows; i++) {
        if (first + 16 * i >= a.rows || n == 0) p[i].zero();
        else if constexpr (VEC) p[i].load(x + 16 * i * a.ld_x);
        else if (shifted) p[i].load_shifted(x + 16 * i * a.ld_x, n);
        else p[i].load_each(x + 16 * i * a.ld_x, n);
    }
    auto block_of = [&](float m) {
        m = __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(m)));  // magnitudes: bits in order
        if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = m;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kQuantThreads / 32; i++) m = fmaxf(m, warp_max[i]);
        return m;
    };
    float m = 0.0f;
#pragma unroll
    for (uint32_t i = 0; i < kTallRows; i++) m = magnitude(p[i], m);
    m = block_of(m);
    const bool infinite = m == INFINITY;  // the same for the whole CTA
    if (infinite) {
        m = 0.0f;
#pragma unroll
        for (uint32_t i = 0; i < kTallRows; i++) {
            float v[8];
            p[i].get(v);
            m = finite_magnitude(v, m);
        }
        __syncthreads();
        m = block_of(m);
    }
    const uint32_t byte = scale_byte(__float_as_uint(m));
    const float inv = inverse_scale(byte);
    uint8_t* out = a.q + first * a.ld_q + c;
#pragma unroll
    for (uint32_t i = 0; i < kTallRows; i++) {
        float v[8];
        p[i].get(v);
        if (infinite) finite_magnitude(v, 0.0f);
        if (first + 16 * i < a.rows && n) store_bytes(out + 16 * i * a.ld_q, to_e4m3(v, inv), n);
    }
    if (threadIdx.x == 0) a.scales[rb * a.ld_s + cb] = (uint8_t)byte;
}

template <class T>
cudaError_t launch(QuantizeArgs a, cudaStream_t s) {
    a.shifted_rows = shifted_rows(a.x_rows, a.ld_x, sizeof(T));
    // 16-byte pieces when every row (and a row's values behind its gates) starts on one and a
    // row holds a whole number of eights
    const bool vec = a.cols % 8 == 0 && a.ld_x * sizeof(T) % 16 == 0;
    const uint64_t blocks = (a.cols + kScaleBlock - 1) / kScaleBlock;
    uint64_t grid;
    if (a.block_rows == 1) {
        const uint64_t per_warp = kRowBlocks * (a.swiglu ? units<T, true>() : units<T, false>());
        const uint64_t col_warps = (blocks + per_warp - 1) / per_warp;
        if (a.rows * col_warps >= (1ull << 32) - kQuantThreads / 32) return cudaErrorInvalidValue;  // terabytes of x
        grid = (a.rows * col_warps + kQuantThreads / 32 - 1) / (kQuantThreads / 32);
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
