// route.cu -- a mixture-of-experts router: each token's best experts and their weights, and the
// assignments sorted by expert.
//
// Scores are s = softmax(l) or 1 / (1 + exp(-l)) of the gate's logits l.  An expert is open to
// a token if its logit is above -inf and not NaN (and its bias, where there is one).  The
// choice goes by s + bias among open experts, of the best groups only where there are groups;
// the weights are the scores without the bias.  Without a bias the order of s is the order of
// l, so the logits themselves are compared.  Where s + bias or a sum of scores decides, it is
// formed in FP64: two experts whose choices are nearer than FP32's rounding would otherwise
// come in an order that hangs on how a sum was formed.  Ties go to the lowest index.
//
// k_route: a warp per token.  Lane i holds the experts i * KPL .. i * KPL + KPL - 1 as unsigned
// integers in the order of their values (0: not open), so the best is a maximum over the warp
// (redux), and the lowest lane that has it holds the lowest index.  A CTA takes a chunk of
// neighbouring tokens and counts its assignments per expert.
// k_place: each CTA sums the counts of the chunks before its own and of all lower experts,
// then ranks its chunk's assignments: within 32 of them by a match of equal experts, across
// warps by counts, always in the order of the tokens, so the result does not depend on timing.
// Up to kOneChunk tokens one CTA does both in one launch.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "dfx_common.cuh"
#include "experts.cuh"
#include "launch.cuh"

namespace dfx {
namespace {

constexpr int kRouteThreads = 512;
constexpr uint32_t kRouteWarps = kRouteThreads / 32;
constexpr uint32_t kOneChunk = 64;       // tokens that one CTA routes and sorts in one launch
constexpr uint32_t kChunks = 296;        // chunks of a longer batch: two per SM
constexpr uint32_t kMaxChunk = 1u << 15; // tokens of a chunk: its counts are 16 bits wide

// unsigned integers in the order of the values; -0 and +0 are the same
__device__ __forceinline__ uint32_t ordered(float v) {
    const uint32_t b = __float_as_uint(v + 0.0f);
    return (b >> 31) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ uint64_t ordered(double v) {
    const uint64_t b = (uint64_t)__double_as_longlong(v + 0.0);
    return (b >> 63) ? ~b : b | (1ull << 63);
}
__device__ __forceinline__ double value_of(uint64_t key) {
    return __longlong_as_double((long long)((key >> 63) ? key & ~(1ull << 63) : ~key));
}
__device__ __forceinline__ uint32_t warp_max(uint32_t v) { return __reduce_max_sync(kFull, v); }
__device__ __forceinline__ uint64_t warp_max(uint64_t v) {
    const uint32_t hi = __reduce_max_sync(kFull, (uint32_t)(v >> 32));
    const uint32_t lo = __reduce_max_sync(kFull, (uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
    return (uint64_t)hi << 32 | lo;
}
__device__ __forceinline__ float warp_max(float v) {
    const uint32_t k = __reduce_max_sync(kFull, ordered(v));
    return __uint_as_float((k >> 31) ? k & 0x7fffffffu : ~k);
}
template <class F>
__device__ __forceinline__ F warp_sum(F v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(kFull, v, d);
    return v;
}
// exp(x - m) with m the row's largest value, which may be infinite
__device__ __forceinline__ float shifted_exp(float x, float m) { return x == m ? 1.0f : expf(x - m); }
__device__ __forceinline__ double shifted_exp64(float x, float m) { return x == m ? 1.0 : exp((double)x - (double)m); }

__device__ __forceinline__ float logit(const RouteArgs& a, uint64_t i) {
    return a.bf16 ? __bfloat162float(((const __nv_bfloat16*)a.logits)[i]) : ((const float*)a.logits)[i];
}

// One token by one warp: ids and weights.  counts: the CTA's assignments per expert, in shared
// memory, or NULL.
template <int KPL, bool WIDE>
__device__ __forceinline__ void route_token(const RouteArgs& a, uint32_t t, uint32_t* counts) {
    using Key = typename std::conditional<WIDE, uint64_t, uint32_t>::type;
    const uint32_t lane = threadIdx.x & 31, e0 = lane * KPL;
    constexpr float kNone = -INFINITY;
    float x[KPL];
    bool open[KPL];
    float top = kNone;
#pragma unroll
    for (int j = 0; j < KPL; j++) {
        x[j] = e0 + j < a.experts ? logit(a, t * a.ld + e0 + j) : kNone;
        open[j] = x[j] > kNone;
        if (open[j]) top = fmaxf(top, x[j]);
    }
    if (!a.sigmoid) top = warp_max(top);
    Key key[KPL];
    double denominator = 0.0;
    if constexpr (WIDE) {
        double s[KPL];
        double sum = 0.0;
#pragma unroll
        for (int j = 0; j < KPL; j++) {
            s[j] = 0.0;
            if (open[j]) s[j] = a.sigmoid ? 1.0 / (1.0 + exp(-(double)x[j])) : shifted_exp64(x[j], top);
            sum += s[j];
        }
        if (!a.sigmoid) {
            denominator = warp_sum(sum);
#pragma unroll
            for (int j = 0; j < KPL; j++) s[j] = open[j] ? s[j] / denominator : 0.0;
        }
#pragma unroll
        for (int j = 0; j < KPL; j++) {
            if (a.bias && open[j]) {
                const float b = *(a.bias + e0 + j);
                open[j] = b > kNone;
                s[j] += (double)b;
            }
            key[j] = open[j] ? ordered(s[j]) : 0;
        }
    } else {
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < KPL; j++) key[j] = open[j] ? ordered(x[j]) : 0;
        if (!a.sigmoid && !a.renormalize) {
#pragma unroll
            for (int j = 0; j < KPL; j++) sum += open[j] ? shifted_exp(x[j], top) : 0.0f;
            denominator = (double)warp_sum(sum);
        }
    }

    if (a.groups > 1) {
        // lane g gets group g's score: its best key, or the sum of its best two choices
        const uint32_t per = a.experts / a.groups;
        Key mine = 0;
        for (uint32_t g = 0; g < a.groups; g++) {
            Key m = 0;
#pragma unroll
            for (int j = 0; j < KPL; j++)
                if ((e0 + j) / per == g && key[j] > m) m = key[j];
            const Key best = warp_max(m);
            Key score = best;
            if constexpr (WIDE) {
                if (a.group_best == 2 && best != 0) {
                    // the same again without the first that has it
                    const uint32_t first = __ffs((int)__ballot_sync(kFull, m == best)) - 1;
                    Key m2 = 0;
                    bool dropped = lane != first;
#pragma unroll
                    for (int j = 0; j < KPL; j++) {
                        if ((e0 + j) / per != g) continue;
                        if (!dropped && key[j] == best) dropped = true;
                        else if (key[j] > m2) m2 = key[j];
                    }
                    const Key second = warp_max(m2);
                    if (second != 0) score = ordered(value_of(best) + value_of(second));
                }
            }
            if (lane == g) mine = score;
        }
        uint32_t above = 0;  // groups that come before lane's
        for (uint32_t g = 0; g < a.groups; g++) {
            const Key other = __shfl_sync(kFull, mine, g);
            above += other > mine || (other == mine && g < lane);
        }
        const uint32_t kept = __ballot_sync(kFull, lane < a.groups && above < a.top_groups);
#pragma unroll
        for (int j = 0; j < KPL; j++)
            if (e0 + j < a.experts && !((kept >> ((e0 + j) / per)) & 1u)) key[j] = 0;
    }

    int id = -1;         // of pick number `lane`
    float chosen = 0.0f; // its logit
    for (uint32_t k = 0; k < a.topk; k++) {
        Key m = 0;
#pragma unroll
        for (int j = 0; j < KPL; j++) m = max(m, key[j]);
        const Key best = warp_max(m);
        if (best == 0) break;
        const uint32_t winner = __ffs((int)__ballot_sync(kFull, m == best)) - 1;
        int e = -1;
        float l = 0.0f;
        if (lane == winner) {
#pragma unroll
            for (int j = KPL - 1; j >= 0; j--)
                if (key[j] == best) e = j, l = x[j];
#pragma unroll
            for (int j = 0; j < KPL; j++)
                if (j == e) key[j] = 0;
            e += e0;
        }
        e = __shfl_sync(kFull, e, winner);
        l = __shfl_sync(kFull, l, winner);
        if (lane == k) id = e, chosen = l;
    }

    // the weights, in FP64 and rounded once: one value per lane
    double w = 0.0;
    if (id >= 0) w = a.sigmoid ? 1.0 / (1.0 + exp(-(double)chosen)) : shifted_exp64(chosen, top);
    if (a.renormalize) denominator = warp_sum(w);
    if (a.renormalize || !a.sigmoid) w = denominator > 0.0 ? w / denominator : 0.0;
    if (lane < a.topk) {
        const uint64_t o = (uint64_t)t * a.topk + lane;
        a.ids[o] = id;
        a.weights[o] = (float)(w * (double)a.scale);
        if (counts && id >= 0) atomicAdd(counts + id, 1u);
    }
}

// Slots of the assignments [first, first + n) of a chunk by this CTA, in shared memory
// base[experts]: the slot of each expert's first assignment of the chunk; warp_base:
// kRouteWarps x experts, scratch.  Ends with the CTA's warps unsynchronised.
__device__ __forceinline__ void place_chunk(const RouteArgs& a, uint32_t first, uint32_t n, const uint32_t* base,
                                            uint16_t* warp_base) {
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // warp w takes the assignments [w * span, (w + 1) * span)
    const uint32_t span = ((n + kRouteWarps - 1) / kRouteWarps + 31) & ~31u;
    const uint32_t lo = min(n, warp * span), hi = min(n, lo + span);
    uint16_t* mine = warp_base + warp * a.experts;
    for (uint32_t e = lane; e < a.experts; e += 32) mine[e] = 0;
    __syncwarp();
    for (int pass = 0; pass < 2; pass++) {
        for (uint32_t i0 = lo; i0 < hi; i0 += 32) {
            const uint32_t i = i0 + lane;
            const int e = i < hi ? a.ids[first + i] : -1;
            const uint32_t peers = __match_any_sync(kFull, e);
            const uint32_t before = __popc(peers & ((1u << lane) - 1u));
            uint32_t at = 0;
            if (e >= 0) at = mine[e];
            __syncwarp();
            if (e >= 0 && before == 0) mine[e] = (uint16_t)(at + __popc(peers));
            __syncwarp();
            if (pass == 1 && i < hi) {
                int slot = -1;
                if (e >= 0) {
                    slot = (int)(base[e] + at + before);
                    a.rows[slot] = (int32_t)((first + i) / a.topk);
                }
                a.slots[first + i] = slot;
            }
        }
        if (pass == 0) {
            // counts of the warps before each, per expert
            __syncthreads();
            for (uint32_t e = threadIdx.x; e < a.experts; e += kRouteThreads) {
                uint32_t sum = 0;
                for (uint32_t w = 0; w < kRouteWarps; w++) {
                    const uint32_t c = warp_base[w * a.experts + e];
                    warp_base[w * a.experts + e] = (uint16_t)sum;
                    sum += c;
                }
            }
            __syncthreads();
        }
    }
}

// Exclusive sum over the experts of total[] (shared, experts <= 512) into offset[experts + 1];
// every thread calls it.
__device__ __forceinline__ void scan_experts(const uint32_t* total, uint32_t* offset, uint32_t experts) {
    const uint32_t lane = threadIdx.x & 31;
    if (threadIdx.x < 32) {
        uint32_t carry = 0;
        for (uint32_t e0 = 0; e0 < experts; e0 += 32) {
            const uint32_t v = e0 + lane < experts ? total[e0 + lane] : 0;
            uint32_t incl = v;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const uint32_t y = __shfl_up_sync(kFull, incl, d);
                if (lane >= (uint32_t)d) incl += y;
            }
            if (e0 + lane < experts) offset[e0 + lane] = carry + incl - v;
            carry += __shfl_sync(kFull, incl, 31);
        }
        if (lane == 0) offset[experts] = carry;
    }
    __syncthreads();
}

// rows[] past the last assignment
__device__ __forceinline__ void clear_unused(const RouteArgs& a, uint32_t used, uint32_t thread, uint32_t threads) {
    for (uint64_t i = (uint64_t)used + thread; i < (uint64_t)a.tokens * a.topk; i += threads) a.rows[i] = -1;
}

template <int KPL, bool WIDE>
__global__ void __launch_bounds__(kRouteThreads) k_route(const RouteArgs a) {
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    __shared__ uint32_t counts[kMaxExperts], offset[kMaxExperts + 1];
    extern __shared__ __align__(16) uint16_t warp_base[];
    for (uint32_t e = threadIdx.x; e < a.experts; e += kRouteThreads) counts[e] = 0;
    wait_prior_grid();
    __syncthreads();
    const uint32_t first = blockIdx.x * a.chunk, last = min(a.tokens, first + a.chunk);
    for (uint32_t t = first + (threadIdx.x >> 5); t < last; t += kRouteWarps)
        route_token<KPL, WIDE>(a, t, a.offsets ? counts : nullptr);
    if (!a.offsets) return;
    __syncthreads();
    if (a.chunks > 1) {
        for (uint32_t e = threadIdx.x; e < a.experts; e += kRouteThreads)
            a.counts[(uint64_t)blockIdx.x * a.experts + e] = counts[e];
        return;
    }
    scan_experts(counts, offset, a.experts);
    for (uint32_t e = threadIdx.x; e <= a.experts; e += kRouteThreads) a.offsets[e] = (int32_t)offset[e];
    place_chunk(a, 0, a.tokens * a.topk, offset, warp_base);
    clear_unused(a, offset[a.experts], threadIdx.x, kRouteThreads);
}

__global__ void __launch_bounds__(kRouteThreads) k_place(const RouteArgs a) {
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    __shared__ uint32_t total[kMaxExperts], before[kMaxExperts], offset[kMaxExperts + 1];
    extern __shared__ __align__(16) uint16_t warp_base[];
    for (uint32_t e = threadIdx.x; e < a.experts; e += kRouteThreads) total[e] = before[e] = 0;
    __syncthreads();
    wait_prior_grid();
    // every chunk's counts: thread (e, part) sums a part of the chunks of expert e
    const uint32_t parts = max(1u, kRouteThreads / a.experts);
    if (threadIdx.x < parts * a.experts) {
        const uint32_t e = threadIdx.x % a.experts, part = threadIdx.x / a.experts;
        uint32_t all = 0, prior = 0;
#pragma unroll 8
        for (uint32_t c = part; c < a.chunks; c += parts) {
            const uint32_t v = a.counts[(uint64_t)c * a.experts + e];
            all += v;
            if (c < blockIdx.x) prior += v;
        }
        atomicAdd(total + e, all);
        atomicAdd(before + e, prior);
    }
    __syncthreads();
    scan_experts(total, offset, a.experts);
    if (blockIdx.x == 0)
        for (uint32_t e = threadIdx.x; e <= a.experts; e += kRouteThreads) a.offsets[e] = (int32_t)offset[e];
    for (uint32_t e = threadIdx.x; e < a.experts; e += kRouteThreads) before[e] += offset[e];
    __syncthreads();
    const uint32_t first = blockIdx.x * a.chunk, last = min(a.tokens, first + a.chunk);
    place_chunk(a, first * a.topk, (last - first) * a.topk, before, warp_base);
    clear_unused(a, offset[a.experts], blockIdx.x * kRouteThreads + threadIdx.x, gridDim.x * kRouteThreads);
}

uint32_t chunk_tokens(uint64_t tokens) {
    if (tokens <= kOneChunk) return kOneChunk;
    const uint64_t per = (tokens + kChunks - 1) / kChunks;
    const uint64_t chunk = (per + kRouteWarps - 1) / kRouteWarps * kRouteWarps;
    return (uint32_t)(chunk < kMaxChunk ? chunk : kMaxChunk);
}

template <bool WIDE>
cudaError_t launch(const RouteArgs& a, size_t smem, cudaStream_t s) {
    const int grid = (int)a.chunks;
    auto go = [&](auto* k, bool* attr_set) {
        const cudaError_t e = allow_smem(k, kRouteWarps * kMaxExperts * sizeof(uint16_t), attr_set);
        return e != cudaSuccess ? e : launch_programmatic(k, grid, kRouteThreads, smem, s, a);
    };
    static bool set[5][64] = {};
    if (a.experts <= 32) return go(k_route<1, WIDE>, set[0]);
    if (a.experts <= 64) return go(k_route<2, WIDE>, set[1]);
    if (a.experts <= 128) return go(k_route<4, WIDE>, set[2]);
    if (a.experts <= 256) return go(k_route<8, WIDE>, set[3]);
    return go(k_route<16, WIDE>, set[4]);
}

}  // namespace

uint64_t route_workspace_bytes(uint64_t tokens, uint32_t experts) {
    const uint64_t chunk = chunk_tokens(tokens), chunks = (tokens + chunk - 1) / chunk;
    return align16(4 * (chunks > 1 ? chunks * experts : 4));
}

cudaError_t launch_route(RouteArgs a, cudaStream_t s) {
    a.chunk = chunk_tokens(a.tokens);
    a.chunks = (a.tokens + a.chunk - 1) / a.chunk;
    if (a.chunks == 0) a.chunks = 1;  // no token: the offsets are still written
    const size_t smem = kRouteWarps * a.experts * sizeof(uint16_t);
    // FP64 choices where a bias or a sum decides; else the logits' own order
    const bool wide = a.bias || (a.groups > 1 && a.group_best == 2);
    cudaError_t e = wide ? launch<true>(a, a.chunks == 1 ? smem : 0, s) : launch<false>(a, a.chunks == 1 ? smem : 0, s);
    if (e != cudaSuccess || !a.offsets || a.chunks == 1) return e;
    static bool set[64] = {};
    e = allow_smem(k_place, kRouteWarps * kMaxExperts * sizeof(uint16_t), set);
    return e != cudaSuccess ? e : launch_programmatic(k_place, (int)a.chunks, kRouteThreads, smem, s, a);
}

}  // namespace dfx
