// route.cu -- a mixture-of-experts router: each token's best experts and their weights, and the
// assignments sorted by expert.
//
// Scores are s = softmax(l) or 1 / (1 + exp(-l)) of the gate's logits l.  An expert is open to
// a token if its logit is above -inf and not NaN (and its bias, where there is one).  The
// choice goes by s + bias among open experts, of the best groups only where there are groups;
// the weights are the scores without the bias.  Without a bias the order of s is the order of
// l, so the logits themselves are compared.  Where s + bias or a sum of scores decides, the order is
// that of FP64: two experts whose choices are nearer than FP32's rounding would otherwise come in
// an order that hangs on how a sum was formed.  The picks are made in FP32, and again in FP64 where
// two that decide are too near (quick_picks).  Ties go to the lowest index.
//
// k_route: a warp per token, a few tokens after one another.  Lane i holds the experts
// i * KPL .. i * KPL + KPL - 1 as unsigned integers in the order of their values (0: not open), so
// the best is a maximum over the warp (redux).  Where the logits decide, an expert's index stands
// in the low bits of its key and the maximum names it; FP64 choices fill their 64 bits, and the
// lowest lane that has the maximum holds the lowest index.  A warp keeps the picks of 32 / topk
// tokens, one to a lane, and forms their weights together.  A CTA takes a chunk of neighbouring
// tokens and counts its assignments per expert.
// k_place: each CTA sums the counts of the chunks before its own and of all lower experts,
// then ranks its chunk's assignments: within 32 of them by a match of equal experts, across
// warps by counts, always in the order of the tokens, so the result does not depend on timing.
// Up to kOneChunk tokens one CTA does both in one launch.
//
// Bound by instructions and their latency, not by memory: 32749 tokens over 128 experts, 8 each, in
// 25 us (2 us for their bytes), of which k_route takes 14.6; 4096 over 256 in 8 groups with a bias in
// 20.6 (13.3; 29 with every choice in FP64).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "dfx_common.cuh"
#include "experts.cuh"
#include "launch.cuh"
#include "vec.cuh"

namespace dfx {
namespace {

constexpr uint32_t kOneChunk = 64;       // tokens that one CTA routes and sorts in one launch
constexpr uint32_t kChunks = 148;        // chunks of a longer batch: one per SM
constexpr uint32_t kMinChunk = 16;       // tokens of a chunk, at least
constexpr uint32_t kMaxChunk = 1u << 15; // and at most: its counts are 16 bits wide
constexpr int kPlaceThreads = 512;
constexpr uint32_t kPlaceWarps = kPlaceThreads / 32;  // warps that rank assignments

// What decides between experts: the logits (BF16 or FP32), or FP64 choices.
enum Mode { kBf16Logits, kF32Logits, kChoices };
// A warp's tokens are a chain of dependent steps, so the SM wants many warps: with 512 threads and no
// spills 4096 tokens over 256 experts took 22.8 us, with 1024 they take 20.5.
constexpr int kRouteThreads = 1024;

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

// The logits of a token: KPL neighbours per lane, -inf past the last expert.
template <int KPL>
__device__ __forceinline__ void load_logits(const RouteArgs& a, uint32_t t, uint32_t e0, float (&x)[KPL]) {
    const uint64_t at = (uint64_t)t * a.ld + e0;
    if (a.whole) {  // 32 * KPL experts, rows in whole pieces
        if (a.bf16) {
            const __nv_bfloat16* p = (const __nv_bfloat16*)a.logits + at;
            if constexpr (KPL == 1) {
                x[0] = __bfloat162float(p[0]);
            } else if constexpr (KPL == 2) {
                unpack_bf16(*(const uint32_t*)p, x[0], x[1]);
            } else if constexpr (KPL == 4) {
                const uint2 v = *(const uint2*)p;
                unpack_bf16(v.x, x[0], x[1]), unpack_bf16(v.y, x[2], x[3]);
            } else {
#pragma unroll
                for (int j = 0; j < KPL; j += 8) {
                    const uint4 v = *(const uint4*)(p + j);
                    unpack_bf16(v.x, x[j], x[j + 1]), unpack_bf16(v.y, x[j + 2], x[j + 3]);
                    unpack_bf16(v.z, x[j + 4], x[j + 5]), unpack_bf16(v.w, x[j + 6], x[j + 7]);
                }
            }
        } else {
            const float* p = (const float*)a.logits + at;
            if constexpr (KPL == 1) {
                x[0] = p[0];
            } else if constexpr (KPL == 2) {
                const float2 v = *(const float2*)p;
                x[0] = v.x, x[1] = v.y;
            } else {
#pragma unroll
                for (int j = 0; j < KPL; j += 4) {
                    const float4 v = *(const float4*)(p + j);
                    x[j] = v.x, x[j + 1] = v.y, x[j + 2] = v.z, x[j + 3] = v.w;
                }
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < KPL; j++) x[j] = e0 + j < a.experts ? logit(a, at + j) : -INFINITY;
    }
}

template <int MODE>
struct KeyOf { using type = uint64_t; };
template <>
struct KeyOf<kBf16Logits> { using type = uint32_t; };

// the key of a logit x of expert e where the logits decide; a larger key for a lower index
__device__ __forceinline__ void logit_key(float x, uint32_t e, uint32_t& key) { key = (ordered(x) & 0xffff0000u) | (0xffffu - e); }
__device__ __forceinline__ void logit_key(float x, uint32_t e, uint64_t& key) { key = (uint64_t)ordered(x) << 32 | (0xffffu - e); }

// The best two keys of the experts of a group: those whose place from `at` on (of this lane's first
// expert, from the group's first) is below `per`.
template <int KPL, class Key>
__device__ __forceinline__ void best_of_group(const Key (&key)[KPL], uint32_t at, uint32_t per, Key& best, Key& second) {
    Key m = 0, m2 = 0;  // the lane's own
#pragma unroll
    for (int j = 0; j < KPL; j++) {
        const Key k = at + j < per ? key[j] : 0;
        m2 = max(m2, min(m, k));
        m = max(m, k);
    }
    best = warp_max(m);
    const uint32_t first = __ffs((int)__ballot_sync(kFull, m == best)) - 1;
    second = warp_max((threadIdx.x & 31) == first ? m2 : m);
}
// Lane g gets the best two keys of group g (0: none; the second only where it counts).
template <int KPL, class Key>
__device__ __forceinline__ void best_of_groups(const RouteArgs& a, const Key (&key)[KPL], uint32_t e0, Key& best, Key& second) {
    const uint32_t lane = threadIdx.x & 31, per = a.experts / a.groups, lanes = per / KPL;
    best = second = 0;
    if (per % KPL == 0 && (lanes & (lanes - 1)) == 0) {
        // a group is `lanes` whole lanes: their best two, then an exchange among them
#pragma unroll
        for (int j = 0; j < KPL; j++) {
            second = max(second, min(best, key[j]));
            best = max(best, key[j]);
        }
        for (uint32_t d = 1; d < lanes; d <<= 1) {
            const Key other = __shfl_xor_sync(kFull, best, d), other2 = __shfl_xor_sync(kFull, second, d);
            second = max(min(best, other), max(second, other2));
            best = max(best, other);
        }
        best = __shfl_sync(kFull, best, lane * lanes);  // wraps for lanes past the groups
        if (a.group_best == 2) second = __shfl_sync(kFull, second, lane * lanes);
    } else {
        for (uint32_t g = 0; g < a.groups; g++) {
            Key b, c;
            best_of_group<KPL>(key, e0 - g * per, per, b, c);
            if (lane == g) best = b, second = c;
        }
    }
}
// The mask of the best top_groups groups by the scores that the first lanes hold.
template <class Key>
__device__ __forceinline__ uint32_t kept_groups(const RouteArgs& a, Key mine) {
    const uint32_t lane = threadIdx.x & 31;
    uint32_t above = 0;  // groups that come before lane's
    for (uint32_t g = 0; g < a.groups; g++) {
        const Key other = __shfl_sync(kFull, mine, g);
        above += other > mine || (other == mine && g < lane);
    }
    return __ballot_sync(kFull, lane < a.groups && above < a.top_groups);
}
// keys outside the groups of the mask `kept` become 0
template <int KPL, class Key>
__device__ __forceinline__ void drop_groups(const RouteArgs& a, Key (&key)[KPL], uint32_t e0, uint32_t kept) {
    const uint32_t per = a.experts / a.groups;
    for (uint32_t g = 0; g < a.groups; g++) {
        if ((kept >> g) & 1u) continue;
#pragma unroll
        for (int j = 0; j < KPL; j++)
            if (e0 + j - g * per < per) key[j] = 0;
    }
}

// One token by one warp: the keys of its experts, those outside its best groups 0.
// top, denominator: what its softmax needs.
template <int KPL, int MODE, class Key>
__device__ __forceinline__ void token_keys(const RouteArgs& a, const float (&x)[KPL], uint32_t e0, Key (&key)[KPL], float& top,
                                           double& denominator) {
    constexpr float kNone = -INFINITY;
    top = kNone;
    denominator = 0.0;
    if (!a.sigmoid) {
#pragma unroll
        for (int j = 0; j < KPL; j++) top = fmaxf(top, x[j]);  // NaN has no part in it
        top = warp_max(top);
    }
    if constexpr (MODE == kChoices) {
        double s[KPL];
        double sum = 0.0;
#pragma unroll
        for (int j = 0; j < KPL; j++) {
            s[j] = 0.0;
            if (x[j] > kNone) s[j] = a.sigmoid ? 1.0 / (1.0 + exp(-(double)x[j])) : shifted_exp64(x[j], top);
            sum += s[j];
        }
        if (!a.sigmoid) {
            denominator = warp_sum(sum);
#pragma unroll
            for (int j = 0; j < KPL; j++) s[j] = x[j] > kNone ? s[j] / denominator : 0.0;
        }
#pragma unroll
        for (int j = 0; j < KPL; j++) {
            bool open = x[j] > kNone;
            if (a.bias && e0 + j < a.experts) {
                const float b = a.bias[e0 + j];
                open = open && b > kNone;
                s[j] += (double)b;
            }
            key[j] = open ? ordered(s[j]) : 0;
        }
    } else {
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < KPL; j++) {
            logit_key(x[j], e0 + j, key[j]);
            if (!(x[j] > kNone)) key[j] = 0;
        }
        if (!a.sigmoid && !a.renormalize) {
#pragma unroll
            for (int j = 0; j < KPL; j++) sum += x[j] > kNone ? shifted_exp(x[j], top) : 0.0f;
            denominator = (double)warp_sum(sum);
        }
    }

    if (a.groups <= 1) return;
    // lane g: group g's score, its best key or the sum of its best two choices
    Key mine, second;
    best_of_groups<KPL>(a, key, e0, mine, second);
    if constexpr (MODE == kChoices)
        if (a.group_best == 2 && second != 0) mine = ordered(value_of(mine) + value_of(second));
    drop_groups<KPL>(a, key, e0, kept_groups(a, mine));
}

__device__ __forceinline__ float value_of(uint32_t key) {
    return __uint_as_float((key >> 31) ? key & 0x7fffffffu : ~key);
}

// The picks of one token whose choices are sums, in FP32: true if no two choices (or groups) that
// decide are nearer than their rounding.  The error of a choice c: of its score at most 2^-21 for a
// sigmoid (exponential 2^-22, sum and quotient 2^-24 each), 2^-19 for a softmax (up to 21 additions of
// 2^-24 more); 2^-24 |c| from adding the bias; and the key's last bits, given to its place in the lane,
// (KPL - 1) 2^-23 |c|, which is below 2^-19 |c|.  Two neighbours are trusted from a difference of
// 2^-18 (2^-16 for a softmax) times 1 + |c| on: their errors together are at most 2^-20 (2^-18) and 31
// of the 32 parts of 2^-23 |c|.  A group's score, of one choice or of two, is off by at most 2^-18
// (2^-16) times 1 + its choices' magnitudes: the sum of their errors and its own rounding, 2^-24.
// Lane first_lane + k gets pick k in id.
template <int KPL>
__device__ __forceinline__ bool quick_picks(const RouteArgs& a, const float (&x)[KPL], uint32_t e0, uint32_t first_lane, float& top,
                                            double& denominator, int& id) {
    const uint32_t lane = threadIdx.x & 31;
    constexpr float kNone = -INFINITY;
    const float tolerance = a.sigmoid ? 0x1p-18f : 0x1p-16f;
    uint32_t key[KPL];
    float sum = 0.0f;
    top = kNone;
    if (!a.sigmoid) {
#pragma unroll
        for (int j = 0; j < KPL; j++) top = fmaxf(top, x[j]);
        top = warp_max(top);
#pragma unroll
        for (int j = 0; j < KPL; j++) sum += x[j] > kNone ? shifted_exp(x[j], top) : 0.0f;
        sum = warp_sum(sum);
    }
    denominator = (double)sum;
#pragma unroll
    for (int j = 0; j < KPL; j++) {
        bool open = x[j] > kNone;
        float c = a.sigmoid ? 1.0f / (1.0f + expf(-x[j])) : shifted_exp(x[j], top) / sum;
        if (a.bias && e0 + j < a.experts) {
            const float b = a.bias[e0 + j];
            open = open && b > kNone;
            c += b;
        }
        // the last bits name the key within its lane
        key[j] = open ? (ordered(c) & ~(uint32_t)(KPL - 1)) | (KPL - 1 - j) : 0;
    }
    bool sure = true;
    if (a.groups > 1) {
        uint32_t best, second;
        best_of_groups<KPL>(a, key, e0, best, second);
        const bool two = a.group_best == 2 && second != 0;
        const float first_choice = value_of(best), second_choice = two ? value_of(second) : 0.0f;
        const float score = first_choice + second_choice;
        const uint32_t mine = two ? ordered(score) : best, kept = kept_groups(a, mine);
        // A score is off by its terms' errors, which go by the terms: a sum may cancel.  The kept
        // groups' lowest possible scores have to be above the others' highest.
        const float error = tolerance * (1.0f + fabsf(first_choice) + fabsf(second_choice));
        const bool counts = lane < a.groups && mine != 0, keep = (kept >> lane) & 1u;
        const uint32_t low = __reduce_min_sync(kFull, counts && keep ? ordered(score - error) : 0xffffffffu);
        const uint32_t high = warp_max(counts && !keep ? ordered(score + error) : 0u);
        sure = __all_sync(kFull, !counts || error < INFINITY) && low > high;
        drop_groups<KPL>(a, key, e0, kept);
    }
    float last = 0.0f;
    for (uint32_t k = 0; k <= a.topk; k++) {  // one more than is picked: the last must stand clear too
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < KPL; j++) m = max(m, key[j]);
        const uint32_t best = warp_max(m);
        if (best == 0) break;
        const float c = value_of(best);
        const uint32_t who = __ballot_sync(kFull, m == best);
        sure = sure && (who & (who - 1)) == 0 && (k == 0 || last - c > tolerance * (1.0f + fabsf(c)));
        last = c;
#pragma unroll
        for (int j = 0; j < KPL; j++)
            if (key[j] == best) key[j] = 0;
        const int e = (__ffs((int)who) - 1) * KPL + (KPL - 1 - (int)(best & (KPL - 1)));
        if (k < a.topk && lane == first_lane + k) id = e;
    }
    return sure;
}

// `n` (at most 32 / topk) tokens from t0 on by one warp: ids and weights.  counts: the CTA's
// assignments per expert, in shared memory, or NULL.
template <int KPL, int MODE>
__device__ __forceinline__ void route_tokens(const RouteArgs& a, uint32_t t0, uint32_t n, uint32_t my_token, uint32_t* counts) {
    using Key = typename KeyOf<MODE>::type;
    const uint32_t lane = threadIdx.x & 31, e0 = lane * KPL;
    int id = -1;  // this lane's pick: number lane % topk of token lane / topk
    float my_top = 0.0f;
    double my_denominator = 0.0;
    float x[KPL];
    load_logits<KPL>(a, t0, e0, x);
    for (uint32_t i = 0; i < n; i++) {
        Key key[KPL];
        float top;
        double denominator;
        if constexpr (MODE == kChoices) {
            if (quick_picks<KPL>(a, x, e0, i * a.topk, top, denominator, id)) {
                if (i + 1 < n) load_logits<KPL>(a, t0 + i + 1, e0, x);
                if (my_token == i) my_top = top, my_denominator = denominator;
                continue;
            }
            if (my_token == i) id = -1;
        }
        token_keys<KPL, MODE>(a, x, e0, key, top, denominator);
        if (i + 1 < n) load_logits<KPL>(a, t0 + i + 1, e0, x);
        if (my_token == i) my_top = top, my_denominator = denominator;
        for (uint32_t k = 0; k < a.topk; k++) {
            Key m = 0;
#pragma unroll
            for (int j = 0; j < KPL; j++) m = max(m, key[j]);
            const Key best = warp_max(m);
            if (best == 0) break;
            int e;
            if constexpr (MODE == kChoices) {
                const uint32_t winner = __ffs((int)__ballot_sync(kFull, m == best)) - 1;
                uint32_t at = 0;
#pragma unroll
                for (int j = KPL - 1; j >= 0; j--)
                    if (key[j] == best) at = j;
#pragma unroll
                for (int j = 0; j < KPL; j++)
                    if (lane == winner && at == (uint32_t)j) key[j] = 0;
                e = (int)(winner * KPL + __shfl_sync(kFull, at, winner));
            } else {
                e = 0xffff - (int)((uint32_t)best & 0xffffu);
#pragma unroll
                for (int j = 0; j < KPL; j++)
                    if (key[j] == best) key[j] = 0;
            }
            if (lane == i * a.topk + k) id = e;
        }
    }

    // The weights, in FP64 and rounded once: one value per lane.  Where a softmax over all logits is the
    // denominator, it is an FP32 sum of FP32 exponentials, within 2^-18 (exponentials of every expert in
    // FP64 are what makes the choices in FP64 half as slow again); for a token whose choices were made in
    // FP64 it is their sum.
    double w = 0.0;
    if (id >= 0) {
        const float chosen = logit(a, (uint64_t)(t0 + my_token) * a.ld + id);
        w = a.sigmoid ? 1.0 / (1.0 + exp(-(double)chosen)) : shifted_exp64(chosen, my_top);
    }
    if (a.renormalize) {
        my_denominator = 0.0;
        for (uint32_t k = 0; k < a.topk; k++) my_denominator += __shfl_sync(kFull, w, my_token * a.topk + k);
    }
    if (a.renormalize || !a.sigmoid) w = my_denominator > 0.0 ? w / my_denominator : 0.0;
    if (lane < n * a.topk) {
        const uint64_t o = (uint64_t)t0 * a.topk + lane;
        a.ids[o] = id;
        a.weights[o] = (float)(w * (double)a.scale);
        if (counts && id >= 0) atomicAdd(counts + id, 1u);
    }
}

// The ranking of a chunk's assignments [first, first + n) by the CTA's first kPlaceWarps warps, warp
// w those of its span.  count() ranks each among the warp's of the same expert and leaves the
// warp's counts in warp_base (a row of experts for each warp with a span); place() turns the
// counts into starts and writes the slots, from base[experts], the slot of each expert's first
// assignment of the chunk.  Every thread of the CTA calls both, with a barrier in between.
struct Ranking {
    static constexpr uint32_t kHeld = 8;  // rounds of 32 whose ranks stay in registers
    const RouteArgs& a;
    uint32_t first, n, warps, lo, hi;
    uint32_t held[kHeld];  // expert << 16 | rank
    __device__ __forceinline__ Ranking(const RouteArgs& a_, uint32_t first_, uint32_t n_) : a(a_), first(first_), n(n_) {
        const uint32_t warp = threadIdx.x >> 5, span = ((n + kPlaceWarps - 1) / kPlaceWarps + 31) & ~31u;
        warps = n ? (n + span - 1) / span : 0;
        lo = min(n, warp * span);
        hi = min(n, lo + span);
    }
    __device__ __forceinline__ uint32_t rank(uint32_t i, uint16_t* mine) {
        const uint32_t lane = threadIdx.x & 31;
        const int e = i < hi ? a.ids[first + i] : -1;
        const uint32_t peers = __match_any_sync(kFull, e), before = __popc(peers & ((1u << lane) - 1u));
        uint32_t at = 0;
        if (e >= 0) at = mine[e];
        __syncwarp();
        if (e >= 0 && before == 0) mine[e] = (uint16_t)(at + __popc(peers));
        __syncwarp();
        return e >= 0 ? (uint32_t)e << 16 | (at + before) : 0xffffffffu;
    }
    __device__ __forceinline__ void count(uint16_t* warp_base) {
        const uint32_t lane = threadIdx.x & 31;
        uint16_t* mine = warp_base + (threadIdx.x >> 5) * a.experts;
        if (lo >= hi) return;  // the same for the warp
        for (uint32_t e = lane; e < a.experts; e += 32) mine[e] = 0;
        __syncwarp();
#pragma unroll
        for (uint32_t k = 0; k < kHeld; k++)
            if (lo + 32 * k < hi) held[k] = rank(lo + 32 * k + lane, mine);
        for (uint32_t i = lo + 32 * kHeld + lane; i - lane < hi; i += 32) {
            const uint32_t r = rank(i, mine);
            if (i < hi) a.slots[first + i] = (int32_t)r;  // kept there for place()
        }
    }
    __device__ __forceinline__ void write(uint32_t i, uint32_t r, const uint32_t* base, const uint16_t* mine) {
        if (i >= hi) return;
        int slot = -1;
        if (r != 0xffffffffu) {
            slot = (int)(base[r >> 16] + mine[r >> 16] + (r & 0xffffu));
            a.rows[slot] = (int32_t)((first + i) / a.topk);
        }
        a.slots[first + i] = slot;
    }
    __device__ __forceinline__ void place(const uint32_t* base, uint16_t* warp_base) {
        for (uint32_t e = threadIdx.x; e < a.experts; e += blockDim.x) {
            uint32_t sum = 0;
#pragma unroll 4
            for (uint32_t w = 0; w < warps; w++) {
                const uint32_t c = warp_base[w * a.experts + e];
                warp_base[w * a.experts + e] = (uint16_t)sum;
                sum += c;
            }
        }
        __syncthreads();
        const uint32_t lane = threadIdx.x & 31;
        const uint16_t* mine = warp_base + (threadIdx.x >> 5) * a.experts;
#pragma unroll
        for (uint32_t k = 0; k < kHeld; k++)
            if (lo + 32 * k < hi) write(lo + 32 * k + lane, held[k], base, mine);
        for (uint32_t i = lo + 32 * kHeld + lane; i < hi; i += 32) write(i, (uint32_t)a.slots[first + i], base, mine);
    }
};

// Exclusive sum over the experts of total[] (shared, experts <= 512, the CTA at least as wide) into
// offset[experts + 1]; every thread calls it, between barriers of its own.
__device__ __forceinline__ void scan_experts(const uint32_t* total, uint32_t* offset, uint32_t experts) {
    __shared__ uint32_t warp_sum[kMaxExperts / 32];
    const uint32_t e = threadIdx.x, lane = e & 31;
    const uint32_t v = e < experts ? total[e] : 0;
    uint32_t incl = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint32_t y = __shfl_up_sync(kFull, incl, d);
        if (lane >= (uint32_t)d) incl += y;
    }
    if (lane == 31 && e < kMaxExperts) warp_sum[e / 32] = incl;
    __syncthreads();
    if (e < experts) {
        uint32_t before = 0;
        for (uint32_t w = 0; w < e / 32; w++) before += warp_sum[w];
        offset[e] = before + incl - v;
        if (e + 1 == experts) offset[experts] = before + incl;
    }
    __syncthreads();
}

// rows[] past the last assignment
__device__ __forceinline__ void clear_unused(const RouteArgs& a, uint32_t used, uint32_t thread, uint32_t threads) {
    for (uint64_t i = (uint64_t)used + thread; i < (uint64_t)a.tokens * a.topk; i += threads) a.rows[i] = -1;
}

template <int KPL, int MODE>
__global__ void __launch_bounds__(kRouteThreads, 1) k_route(const RouteArgs a) {
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    __shared__ uint32_t counts[kMaxExperts], offset[kMaxExperts + 1];
    extern __shared__ __align__(16) uint16_t warp_base[];
    constexpr uint32_t kWarps = kRouteThreads / 32;
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31, my_token = lane / a.topk;
    for (uint32_t e = threadIdx.x; e < a.experts; e += blockDim.x) counts[e] = 0;
    wait_prior_grid();
    __syncthreads();
    const uint32_t first = blockIdx.x * a.chunk, last = min(a.tokens, first + a.chunk);
    // tokens of a warp at a time: their picks fit its lanes, and every warp has some
    const uint32_t at_once = min(32 / a.topk, (last - first + kWarps - 1) / kWarps);
    for (uint32_t t = first + warp * at_once; t < last; t += kWarps * at_once)
        route_tokens<KPL, MODE>(a, t, min(at_once, last - t), my_token, a.offsets ? counts : nullptr);
    if (!a.offsets) return;
    __syncthreads();
    if (a.chunks > 1) {
        for (uint32_t e = threadIdx.x; e < a.row; e += blockDim.x)
            a.counts[(uint64_t)blockIdx.x * a.row + e] = (uint16_t)(e < a.experts ? counts[e] : 0);
        return;
    }
    Ranking ranking(a, 0, a.tokens * a.topk);
    ranking.count(warp_base);
    scan_experts(counts, offset, a.experts);
    for (uint32_t e = threadIdx.x; e <= a.experts; e += blockDim.x) a.offsets[e] = (int32_t)offset[e];
    ranking.place(offset, warp_base);
    clear_unused(a, offset[a.experts], threadIdx.x, blockDim.x);
}

__global__ void __launch_bounds__(kPlaceThreads) k_place(const RouteArgs a) {
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    __shared__ uint32_t total[kMaxExperts], before[kMaxExperts], offset[kMaxExperts + 1];
    extern __shared__ __align__(16) uint16_t warp_base[];
    for (uint32_t e = threadIdx.x; e < kMaxExperts; e += kPlaceThreads) total[e] = before[e] = 0;
    __syncthreads();
    wait_prior_grid();
    // every chunk's counts, 8 experts to a 16-byte piece: a thread sums some chunks' piece.  The
    // loads of the first are on their way while the chunk's assignments are ranked.
    const uint32_t pieces = a.row / 8, parts = kPlaceThreads / pieces;
    const uint32_t piece = threadIdx.x % pieces, part = threadIdx.x / pieces;
    const uint16_t* counts = a.counts + 8 * piece;
    constexpr uint32_t kEarly = 8;
    uint4 early[kEarly];
#pragma unroll
    for (uint32_t i = 0; i < kEarly; i++) {
        const uint32_t c = part + i * parts;
        early[i] = part < parts && c < a.chunks ? *reinterpret_cast<const uint4*>(counts + (uint64_t)c * a.row) : make_uint4(0, 0, 0, 0);
    }
    const uint32_t first = blockIdx.x * a.chunk, last = min(a.tokens, first + a.chunk);
    Ranking ranking(a, first * a.topk, (last - first) * a.topk);
    ranking.count(warp_base);
    if (part < parts) {
        uint32_t all[8] = {}, prior[8] = {};
        auto add = [&](const uint4& v, uint32_t c) {
            const uint32_t w[4] = {v.x, v.y, v.z, v.w}, mine = c < blockIdx.x ? 0xffffffffu : 0u;
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const uint32_t n = (w[j / 2] >> (16 * (j & 1))) & 0xffffu;
                all[j] += n;
                prior[j] += n & mine;
            }
        };
#pragma unroll
        for (uint32_t i = 0; i < kEarly; i++) add(early[i], part + i * parts);
#pragma unroll 4
        for (uint32_t c = part + kEarly * parts; c < a.chunks; c += parts)
            add(*reinterpret_cast<const uint4*>(counts + (uint64_t)c * a.row), c);
#pragma unroll
        for (int j = 0; j < 8; j++) {
            if (all[j]) atomicAdd(total + 8 * piece + j, all[j]);
            if (prior[j]) atomicAdd(before + 8 * piece + j, prior[j]);
        }
    }
    __syncthreads();
    scan_experts(total, offset, a.experts);
    if (blockIdx.x == 0)
        for (uint32_t e = threadIdx.x; e <= a.experts; e += kPlaceThreads) a.offsets[e] = (int32_t)offset[e];
    for (uint32_t e = threadIdx.x; e < a.experts; e += kPlaceThreads) before[e] += offset[e];
    __syncthreads();
    ranking.place(before, warp_base);
    clear_unused(a, offset[a.experts], blockIdx.x * kPlaceThreads + threadIdx.x, gridDim.x * kPlaceThreads);
}

uint32_t chunk_tokens(uint64_t tokens) {
    if (tokens <= kOneChunk) return kOneChunk;
    const uint64_t chunk = (tokens + kChunks - 1) / kChunks;
    return (uint32_t)(chunk < kMinChunk ? kMinChunk : chunk < kMaxChunk ? chunk : kMaxChunk);
}
uint32_t count_row(uint32_t experts) { return (experts + 7) & ~7u; }

template <int MODE>
cudaError_t launch(const RouteArgs& a, size_t smem, cudaStream_t s) {
    const int grid = (int)a.chunks;
    static bool set[5][64] = {};
    auto go = [&](auto* k, bool* attr_set) {
        const cudaError_t e = allow_smem(k, kPlaceWarps * kMaxExperts * sizeof(uint16_t), attr_set);
        return e != cudaSuccess ? e : launch_programmatic(k, grid, kRouteThreads, smem, s, a);
    };
    if (a.experts <= 32) return go(k_route<1, MODE>, set[0]);
    if (a.experts <= 64) return go(k_route<2, MODE>, set[1]);
    if (a.experts <= 128) return go(k_route<4, MODE>, set[2]);
    if (a.experts <= 256) return go(k_route<8, MODE>, set[3]);
    return go(k_route<16, MODE>, set[4]);
}

}  // namespace

uint64_t route_workspace_bytes(uint64_t tokens, uint32_t experts) {
    const uint64_t chunk = chunk_tokens(tokens), chunks = (tokens + chunk - 1) / chunk;
    return align16(2 * (chunks > 1 ? chunks * count_row(experts) : 8));
}

cudaError_t launch_route(RouteArgs a, cudaStream_t s) {
    a.chunk = chunk_tokens(a.tokens);
    a.chunks = (a.tokens + a.chunk - 1) / a.chunk;
    if (a.chunks == 0) a.chunks = 1;  // no token: the offsets are still written
    a.row = count_row(a.experts);
    const uint32_t lane_experts = (a.experts + 31) / 32, bytes = a.bf16 ? 2 : 4;
    a.whole = a.experts % 32 == 0 && (lane_experts & (lane_experts - 1)) == 0 && a.ld * bytes % 16 == 0;
    const size_t smem = kPlaceWarps * a.experts * sizeof(uint16_t), first = a.chunks == 1 && a.offsets ? smem : 0;
    // FP64 choices where a bias or a sum decides; else the logits' own order
    cudaError_t e = a.bias || (a.groups > 1 && a.group_best == 2) ? launch<kChoices>(a, first, s)
                    : a.bf16                                      ? launch<kBf16Logits>(a, first, s)
                                                                  : launch<kF32Logits>(a, first, s);
    if (e != cudaSuccess || !a.offsets || a.chunks == 1) return e;
    static bool set[64] = {};
    e = allow_smem(k_place, kPlaceWarps * kMaxExperts * sizeof(uint16_t), set);
    return e != cudaSuccess ? e : launch_programmatic(k_place, (int)a.chunks, kPlaceThreads, smem, s, a);
}

}  // namespace dfx
