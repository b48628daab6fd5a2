// routing.cu -- which experts a token goes to and with what weight, forward and
// backward, and the plan of the rows that follow from it.

#include <cuda_fp16.h>

#include "common.cuh"
#include "host_common.h"
#include "../../include/mxrouting.h"

namespace mx {

// ---------------------------------------------------------------- routing
struct RouteParams {
    const void* logits;
    const float* bias;
    int32_t* experts;
    float* weights;
    float* dense;
    const float* dweights;  // the backward only
    void* dlogits;
    int64_t T;
    int32_t type, E, top_k, score, groups, top_groups, group_max, renormalize;
    int32_t group_size, group_lanes;  // group_lanes: of the route kernel, where a group is a power of two of them; else 0
    float scale;
};

constexpr int kRouteWarps = 4;  // tokens of a CTA, a warp each
constexpr uint32_t kFull = 0xffffffffu;

__device__ __forceinline__ float logit(const float* p) { return *p; }
__device__ __forceinline__ float logit(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float logit(const __half* p) { return __half2float(*p); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void put(__half* p, float v) { *p = __float2half_rn(v); }

__device__ __forceinline__ float logit_at(const RouteParams& p, int64_t t, int e) {
    const int64_t i = t * p.E + e;
    if (p.type == MX_LOGITS_FP32) return logit(static_cast<const float*>(p.logits) + i);
    if (p.type == MX_LOGITS_BF16) return logit(static_cast<const __nv_bfloat16*>(p.logits) + i);
    return logit(static_cast<const __half*>(p.logits) + i);
}

__device__ __forceinline__ float exp2_approx(float x) {  // within 2 ulp
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp_approx(float x) {  // within 1 ulp
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Integers that order as the values do: NaN above everything, -0 as +0.  No value's is 0, which stands for "none".
__device__ __forceinline__ uint32_t order_of(float v) {
    if (v != v) return 0xffffffffu;
    const uint32_t u = __float_as_uint(v + 0.0f);
    return u >> 31 ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t o) {
    return o == 0xffffffffu ? __uint_as_float(0x7fc00000u) : __uint_as_float(o >> 31 ? o & 0x7fffffffu : ~o);
}
__device__ __forceinline__ unsigned long long order_of(double v) {
    if (v != v) return ~0ull;
    const unsigned long long u = (unsigned long long)__double_as_longlong(v + 0.0);
    return u >> 63 ? ~u : u | (1ull << 63);
}
__device__ __forceinline__ double value_of(unsigned long long o) {
    if (o == ~0ull) return __longlong_as_double(0x7ff8000000000000ll);
    return __longlong_as_double((long long)(o >> 63 ? o & ~(1ull << 63) : ~o));
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int d = 16; d; d >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, d));
    return v;
}
template <typename F>
__device__ __forceinline__ F warp_sum(F v) {
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(kFull, v, d);
    return v;
}

// The two largest of group `lane` among the integers in shared memory (kept as integers, so that a NaN counts).
template <typename O>
__device__ __forceinline__ void group_top2(const O* keys, const RouteParams& p, int lane, O& top, O& second) {
    const int size = p.group_size;
    top = second = 0;
    if (lane >= p.groups) return;
    int at = lane % size;  // lanes start apart, so that they do not meet in a bank
    for (int i = 0; i < size; ++i) {
        const O v = keys[lane * size + at];
        if (++at == size) at = 0;
        second = max(second, min(top, v));
        top = max(top, v);
    }
}
// Whether a bias that is the same for all tells groups apart: it counts once for each of a group's two largest keys, so not
// where all groups have two experts to select, or one.  The whole warp asks, every lane for its group (0, 0: none).
template <typename O>
__device__ __forceinline__ bool uneven_groups(const RouteParams& p, O top, O second) {
    return p.bias != nullptr && __any_sync(kFull, second != 0) && __any_sync(kFull, top != 0 && second == 0);
}
// Which groups stay, where lane g holds what group g is worth: bit g.
template <typename O>
__device__ __forceinline__ uint32_t best_groups(O worth, const RouteParams& p, int lane) {
    int rank = 0;
    for (int g = 0; g < p.groups; ++g) {
        const O other = __shfl_sync(kFull, worth, g);
        rank += other > worth || (other == worth && g < lane);
    }
    return __ballot_sync(kFull, lane < p.groups && worth && rank < p.top_groups);
}

// The maximum of a token's logits and the sum of their exponentials above it, in 64 bits (softmax over all experts).
__device__ __forceinline__ void softmax_64(const RouteParams& p, int64_t t, int lane, double& top, double& sum) {
    float m = -INFINITY;
    for (int e = lane; e < p.E; e += 32) m = fmaxf(m, logit_at(p, t, e));
    top = warp_max(m);
    sum = 0.0;
    for (int e = lane; e < p.E; e += 32) sum += exp((double)logit_at(p, t, e) - top);
    sum = warp_sum(sum);
}
__device__ __forceinline__ double score_64(const RouteParams& p, double l, double top, double sum) {
    if (p.score == MX_SCORE_SOFTMAX_ALL) return exp(l - top) / sum;
    if (p.score == MX_SCORE_SIGMOID) return 1.0 / (1.0 + exp(-l));
    return l;
}
// The integer that orders as expert e's key does, from 64 bits; 0: not to be selected.
__device__ __forceinline__ unsigned long long key_64(const RouteParams& p, int64_t t, int e, double top, double sum) {
    const float l = logit_at(p, t, e), bias = p.bias[e];  // asked by themselves: a NaN score's key would not tell
    return l == -INFINITY || bias == -INFINITY ? 0ull : order_of(score_64(p, l, top, sum) + (double)bias);
}

// The selection in 64 bits, for a token whose order 32 bits leave open.  by_logits: the experts rank by their logits.  Lane
// j returns the j-th expert, -1: none.
__device__ __noinline__ int select_64(const RouteParams& p, int64_t t, bool by_logits, unsigned long long* keys, int lane) {
    double top = 0.0, sum = 1.0;
    if (p.score == MX_SCORE_SOFTMAX_ALL) softmax_64(p, t, lane, top, sum);
    for (int e = lane; e < p.E; e += 32) {
        const float l = logit_at(p, t, e);
        keys[e] = !by_logits ? key_64(p, t, e, top, sum) : l == -INFINITY ? 0ull : order_of((double)l);
    }
    __syncwarp();
    if (p.groups > 1) {
        unsigned long long first, second, worth;
        group_top2(keys, p, lane, first, second);
        worth = first;
        const double common = by_logits && !p.group_max && uneven_groups(p, first, second) ? (double)*p.bias : 0.0;
        if (!p.group_max && first) {
            double v = by_logits ? score_64(p, value_of(first), top, sum) + common : value_of(first);
            if (second) v += by_logits ? score_64(p, value_of(second), top, sum) + common : value_of(second);
            worth = order_of(v);
        }
        const uint32_t stay = best_groups(worth, p, lane);
        for (int e = lane; e < p.E; e += 32)
            if (!(stay >> (e / p.group_size) & 1u)) keys[e] = 0ull;
        __syncwarp();
    }
    int mine = -1;
    for (int j = 0; j < p.top_k; ++j) {
        unsigned long long best = 0;
        int at = p.E;
        for (int e = lane; e < p.E; e += 32)
            if (keys[e] > best) {
                best = keys[e];
                at = e;
            }
#pragma unroll
        for (int d = 16; d; d >>= 1) {
            const unsigned long long o = __shfl_xor_sync(kFull, best, d);
            const int i = __shfl_xor_sync(kFull, at, d);
            if (o > best || (o == best && i < at)) {
                best = o;
                at = i;
            }
        }
        if (best == 0) break;
        if (lane == j) mine = at;
        __syncwarp();
        if (lane == 0) keys[at] = 0ull;
        __syncwarp();
    }
    return mine;
}

// Where a lane holds a selected expert's logit (`in`): its share of the weights, unscaled.  m and sum: the maximum of
// the token's logits and the sum of their exponentials above it (softmax over all, not renormalised).
__device__ __forceinline__ float weight_of(const RouteParams& p, bool in, float l, float m, float sum) {
    if (p.score == MX_SCORE_SIGMOID) {
        const float a = expf(-fabsf(l));
        float s = l >= 0.0f ? 1.0f : a;
        if (p.renormalize) {
            // s_j / sum s with every s_j times e^-c, c the largest logit where that is negative: where all logits are far
            // below 0 the scores themselves would underflow, and their quotients be lost
            if (!__any_sync(kFull, in && !(l < 0.0f))) s = expf(l - warp_max(in ? l : -INFINITY));
        }
        s = in ? (l == l ? s / (1.0f + a) : l) : 0.0f;
        if (!p.renormalize) return s;
        const float total = warp_sum(s);
        return in ? s / total : 0.0f;
    }
    if (p.score == MX_SCORE_SOFTMAX_ALL && !p.renormalize) return in ? expf(l - m) / sum : 0.0f;
    const float top = warp_max(in ? l : -INFINITY);
    const float s = in ? expf(l - top) : 0.0f;
    const float total = warp_sum(s);
    return in ? s / total : 0.0f;
}

// VPL neighbouring values of a row of n from lane * VPL on, `fill` past its end; by vectors where the row's start allows.
template <typename L, int VPL>
__device__ __forceinline__ void load_row(const L* row, const void* base, int n, int lane, float fill, float (&out)[VPL]) {
    constexpr int V = VPL * sizeof(L) < 16 ? VPL : 16 / (int)sizeof(L);
    if (n % V == 0 && (reinterpret_cast<uintptr_t>(base) & (V * sizeof(L) - 1)) == 0) {
#pragma unroll
        for (int c = 0; c < VPL / V; ++c) {
            struct alignas(V * sizeof(L)) Vec { L v[V]; } u;
            const int e = lane * VPL + c * V;
            if (e < n) u = *reinterpret_cast<const Vec*>(row + e);
#pragma unroll
            for (int i = 0; i < V; ++i) out[c * V + i] = e < n ? logit(u.v + i) : fill;
        }
    } else {
#pragma unroll
        for (int i = 0; i < VPL; ++i) out[i] = lane * VPL + i < n ? logit(row + lane * VPL + i) : fill;
    }
}
template <int VPL>
__device__ __forceinline__ void load_logits(const RouteParams& p, int64_t t, int lane, float (&l)[VPL]) {
    if (p.type == MX_LOGITS_FP32) {
        load_row<float, VPL>(static_cast<const float*>(p.logits) + t * p.E, p.logits, p.E, lane, -INFINITY, l);
    } else if (p.type == MX_LOGITS_BF16) {
        load_row<__nv_bfloat16, VPL>(static_cast<const __nv_bfloat16*>(p.logits) + t * p.E, p.logits, p.E, lane, -INFINITY, l);
    } else {
        load_row<__half, VPL>(static_cast<const __half*>(p.logits) + t * p.E, p.logits, p.E, lane, -INFINITY, l);
    }
}

// Keys: the logits themselves (exact), logit + bias, or a score + bias.  Without a bias, and with one that is the same for
// all, experts rank by their logits, which order as their scores do; then a score is only needed of a group's two best.
enum RouteKeys : int { kKeysLogits = 0, kKeysBias = 1, kKeysSigmoid = 2, kKeysSoftmax = 3 };

__device__ __forceinline__ float sigmoid_approx(float l) { return rcp_approx(1.0f + exp2_approx(l * -1.4426950408889634f)); }

// How far a score s computed in 32 bits may be off, in units of 2^-24:
//   sigmoid_approx  e^-l: its exponent is a product with a rounded constant (1.5 |l|, times e^-l / (1 + e^-l), so that it only
//                   counts below 0), its value good to 2 ulp (4); the sum 1; the reciprocal 2 (1 ulp): s (7 + 1.5 max(0, -l)),
//                   at most s (7 + 1.5 ln(1/s)), which grows with s
//   softmax         the exponent's difference d, which is rounded, here and (7, the entropy, at most) in the sum; two expf of
//                   4; 5 + VPL sums; the quotient: s (d + 21 + VPL), where s <= e^-d
// and what subnormals lose.  `at` is l or d.
template <int KEYS, int VPL>
__device__ __forceinline__ float score_error(float s, float at) {
    const float units = KEYS == kKeysSigmoid ? 9.0f + 1.5f * fminf(fmaxf(-at, 0.0f), 128.0f) : 24.0f + VPL + fminf(at, 200.0f);
    return s * units * 0x1p-24f + 0x1p-125f;
}

// The same where the groups are settled and the experts that come into question are few: lane i's is e, -1: none.
__device__ __noinline__ int select_64_among(const RouteParams& p, int64_t t, int e, int total, uint2* shared, int lane) {
    double top = 0.0, sum = 1.0;
    if (p.score == MX_SCORE_SOFTMAX_ALL) softmax_64(p, t, lane, top, sum);
    const unsigned long long key = e >= 0 ? key_64(p, t, e, top, sum) : 0ull;
    int rank = 0;
    for (int j = 0; j < total; ++j) {
        const unsigned long long other = __shfl_sync(kFull, key, j);
        const int expert = __shfl_sync(kFull, e, j);
        rank += other > key || (other == key && expert < e);
    }
    if (lane < total) shared[rank].y = (uint32_t)e;
    __syncwarp();
    return lane < min(total, p.top_k) ? (int)shared[lane].y : -1;
}

// A warp a token: lane i holds VPL neighbouring experts.
//
// The largest top_k (and one more, for the doubts below): with few experts a lane they leave one by one, each by a maximum
// over the warp (one instruction on 32-bit integers).  With more, the (top_k + 1)-th largest of the lanes' own
// maxima bounds them from below; what reaches it, rarely more than a dozen, is gathered in shared memory, one a lane, and
// ranked by counting.  (More than 32 such candidates: one by one.)
//
// Keys with a score or a bias are sums of rounded terms, and experts are told apart by them all the same: a key's
// error has a bound, and where two neighbours in the order, or the groups on both sides of the cut, are no further
// apart than their bounds, the token is done again in 64 bits: among the candidates (that come within four bounds of the
// least, so that the exact largest are there), one a lane, or, where the groups are in doubt, from the start.  The keys can
// then be made of the approximate exponential and reciprocal; weights are not.
//
// Bound by its instructions: 32768 tokens, 8 of 256 experts in 8 groups, 34.7 us (10 for the bytes of this and the
// backward, which takes 9.6); about a dozen of those tokens are done again.  Registers for 11 CTAs an SM (10 where a lane has
// two experts at most, which is bound by latency): 36.4 us with as many as the compiler likes.
template <int VPL, int KEYS>
__global__ void __launch_bounds__(kRouteWarps * 32, VPL <= 2 ? 10 : VPL <= 8 ? 11 : 1) route_kernel(const RouteParams p) {
    extern __shared__ unsigned long long route_smem[];
    constexpr bool kCandidates = VPL > 2;
    __shared__ __align__(8) uint2 candidates[kCandidates ? kRouteWarps : 1][32];  // ~expert, key: as 64 bits the order
    __shared__ int filled[kRouteWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * kRouteWarps + warp;
    if (t >= p.T) return;
    if (kCandidates && lane == 0) filled[warp] = 0;  // (before any of the exchanges below)
    unsigned long long* keys = route_smem + (size_t)warp * p.E;  // this warp's, where there are groups or doubts
    constexpr float kUlp = 0x1p-24f;

    float l[VPL];
    load_logits(p, t, lane, l);
    float m = 0.0f, sum = 1.0f;
    if (KEYS == kKeysSoftmax || (KEYS <= kKeysBias && p.score == MX_SCORE_SOFTMAX_ALL && !p.renormalize)) {
        float top = l[0];
#pragma unroll
        for (int i = 1; i < VPL; ++i) top = fmaxf(top, l[i]);
        m = warp_max(top);
        float part = 0.0f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) part += expf(l[i] - m);
        sum = warp_sum(part);
    }

    uint32_t ord[VPL];
    float err = 0.0f;  // of a key at most
    bool by_logits = KEYS == kKeysLogits || p.bias == nullptr;
    float b[KEYS == kKeysLogits ? 1 : VPL];
    if constexpr (KEYS != kKeysLogits) {
        if (p.bias != nullptr) {
            load_row<float, VPL>(p.bias, p.bias, p.E, lane, 0.0f, b);
            const float first = __shfl_sync(kFull, b[0], 0);
            bool same = fabsf(first) < INFINITY;
#pragma unroll
            for (int i = 0; i < VPL; ++i) same = same && (b[i] == first || lane * VPL + i >= p.E);
            by_logits = __all_sync(kFull, same);
        }
    }
    if (by_logits) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) ord[i] = l[i] == -INFINITY ? 0u : order_of(l[i]);
    } else if constexpr (KEYS != kKeysLogits) {
        float top = -INFINITY, largest = 0.0f;  // the largest logit, the largest |key|
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            float key = l[i];
            if constexpr (KEYS == kKeysSigmoid) {
                top = fmaxf(top, key);
                key = sigmoid_approx(key);
            } else if constexpr (KEYS == kKeysSoftmax) {
                key = expf(l[i] - m) / sum;
            }
            key += b[i];
            // (a finite logit and a finite bias may add up to an infinite key: its bound is infinite, and 64 bits tell)
            const bool out = l[i] == -INFINITY || b[i] == -INFINITY;
            if (!out) largest = fmaxf(largest, fabsf(key));
            ord[i] = out ? 0u : order_of(key);
        }
        // (bounds: score_error, at the largest score, as they grow with it)
        if constexpr (KEYS == kKeysSigmoid) {
            top = value_of(__reduce_max_sync(kFull, order_of(top)));
            err = score_error<KEYS, VPL>(sigmoid_approx(top) * 1.001f, fminf(top, 0.0f));
        } else if constexpr (KEYS == kKeysSoftmax) {
            err = score_error<KEYS, VPL>(fminf(1.001f / sum, 1.0f), 1.0f);  // d e^-d < 1
        }
        err += kUlp * __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(largest)));
    }
    bool doubt = false;

    if (p.groups > 1) {
        const int size = p.group_size, lanes = p.group_lanes;
        uint32_t top, second;  // of a group: every of its lanes, or lane g
        if (lanes) {
            // a group is a power of two of neighbouring lanes: its two largest by exchanges between them
            top = ord[0];
            second = 0u;
#pragma unroll
            for (int i = 1; i < VPL; ++i) {
                second = max(second, min(top, ord[i]));
                top = max(top, ord[i]);
            }
            for (int d = 1; d < lanes; d <<= 1) {
                const uint32_t t2 = __shfl_xor_sync(kFull, top, d), s2 = __shfl_xor_sync(kFull, second, d);
                second = max(min(top, t2), max(second, s2));
                top = max(top, t2);
            }
        } else {
            uint32_t* k32 = reinterpret_cast<uint32_t*>(keys);
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                if (lane * VPL + i < p.E) k32[lane * VPL + i] = ord[i];
            __syncwarp();
            group_top2(k32, p, lane, top, second);
            __syncwarp();
        }
        // what the group is worth, and how far that may be off
        uint32_t worth = top;
        float off = 2 * err, common = 0.0f;
        if constexpr (KEYS != kKeysLogits) {
            if (by_logits && !p.group_max && uneven_groups(p, top, second)) common = __ldg(p.bias);
        }
        if (!p.group_max && top) {
            float v = value_of(top), w = second ? value_of(second) : 0.0f;
            if (KEYS >= kKeysSigmoid && by_logits) {
                const float lv = v, lw = w;
                v = KEYS == kKeysSigmoid ? sigmoid_approx(lv) : expf(lv - m) / sum;
                w = !second ? 0.0f : KEYS == kKeysSigmoid ? sigmoid_approx(lw) : expf(lw - m) / sum;
                off = score_error<KEYS, VPL>(v, KEYS == kKeysSigmoid ? lv : m - lv) +
                      score_error<KEYS, VPL>(w, KEYS == kKeysSigmoid ? lw : m - lw);
            }
            if (common != 0.0f) {
                v += common;
                w += common;
                off += kUlp * (fabsf(v) + fabsf(w));
            }
            if (second) v += w;
            off += kUlp * fabsf(v);
            worth = order_of(v);
        }
        uint32_t low, high;  // the least worth that stays, the best that goes
        bool stay;
        if (lanes) {
            // the best groups leave one by one, of equal ones the first (lanes past the last group hold nothing: 0)
            uint32_t left = worth;
            low = 0xffffffffu;
            for (int g = 0; g < p.top_groups; ++g) {
                const uint32_t most = __reduce_max_sync(kFull, left);
                if (most == 0u) break;
                low = most;
                const int src = __ffs(__ballot_sync(kFull, left == most)) - 1;
                if (((lane ^ src) & -lanes) == 0) left = 0u;  // of the same group
            }
            high = __reduce_max_sync(kFull, left);
            stay = left == 0u;
            if (!stay) {
#pragma unroll
                for (int i = 0; i < VPL; ++i) ord[i] = 0u;
            }
        } else {
            const uint32_t mask = best_groups(worth, p, lane);
            stay = mask >> lane & 1u;
            low = __reduce_min_sync(kFull, stay ? worth : 0xffffffffu);
            high = __reduce_max_sync(kFull, stay ? 0u : worth);
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                if (!(mask >> (min(lane * VPL + i, p.E - 1) / size) & 1u)) ord[i] = 0u;
        }
        if (high && !(by_logits && p.group_max)) {
            // groups on both sides of the cut that are no further apart than their bounds are told apart in 64 bits, but
            // where all of them have the same two logits: they tie, and lie in order
            const float a = value_of(low), c = value_of(high), v = value_of(worth);
            off = 2 * __uint_as_float(__reduce_max_sync(kFull, worth ? __float_as_uint(off) : 0u));
            if (!(a - c > off)) {
                const bool near = worth && !(stay ? v - c > off : a - v > off);
                const bool ties = by_logits &&
                                  __reduce_max_sync(kFull, near ? top : 0u) == __reduce_min_sync(kFull, near ? top : ~0u) &&
                                  __reduce_max_sync(kFull, near ? second : 0u) == __reduce_min_sync(kFull, near ? second : ~0u);
                doubt = !ties;
            }
        }
    }

    int mine = -1, candidate = -1, total = 0;
    uint32_t my_ord = 0;
    uint32_t best = ord[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) best = max(best, ord[i]);
    const int wanted = p.top_k + (err > 0.0f ? 1 : 0);
    bool one_by_one = true;
    if constexpr (kCandidates) {
        uint32_t left = best, least = 1u;
        for (int j = 0; j < wanted; ++j) {  // equal ones leave together: there are then more candidates
            least = __reduce_max_sync(kFull, left);
            if (least == 0u) break;
            if (left == least) left = 0u;
        }
        if (least == 0u || err == INFINITY) least = 1u;  // few are left, or nothing is known: all
        else if (KEYS != kKeysLogits && err > 0.0f) least = order_of(value_of(least) - 4 * err);
        int n = 0;
#pragma unroll
        for (int i = 0; i < VPL; ++i) n += ord[i] >= least;
        total = __reduce_add_sync(kFull, n);
        if (total <= 32) {
            one_by_one = false;
            // in any order: they are told apart by their experts
            __syncwarp();
            int at = n ? atomicAdd(&filled[warp], n) : 0;
            if (n) {
#pragma unroll
                for (int i = 0; i < VPL; ++i)
                    if (ord[i] >= least) candidates[warp][at++] = make_uint2(~(uint32_t)(lane * VPL + i), ord[i]);
            }
            __syncwarp();
            uint2 c = make_uint2(0u, 0u);
            if (lane < total) {
                c = candidates[warp][lane];
                candidate = (int)~c.x;
            }
            const unsigned long long own = (unsigned long long)c.y << 32 | c.x;
            int rank = 0;
#pragma unroll 4
            for (int j = 0; j < total; ++j) rank += reinterpret_cast<const unsigned long long*>(candidates[warp])[j] > own;
            __syncwarp();
            if (lane < total) candidates[warp][rank] = c;
            __syncwarp();
            if (lane < min(total, wanted)) {
                c = candidates[warp][lane];
                my_ord = c.y;
                mine = (int)~c.x;
            }
        }
    }
    if (one_by_one) {
        for (int j = 0; j < wanted; ++j) {
            const uint32_t top = __reduce_max_sync(kFull, best);
            if (top == 0u) break;
            const int src = __ffs(__ballot_sync(kFull, best == top)) - 1;
            int e = 0;
            if (lane == src) {
                bool found = false;
                best = 0u;
#pragma unroll
                for (int i = 0; i < VPL; ++i) {
                    if (!found && ord[i] == top) {
                        found = true;
                        e = lane * VPL + i;
                        ord[i] = 0u;
                    }
                    best = max(best, ord[i]);
                }
            }
            e = __shfl_sync(kFull, e, src);
            if (lane == j) {
                mine = e;
                my_ord = top;
            }
        }
    }
    if constexpr (KEYS != kKeysLogits) {
        if (err > 0.0f) {
            const uint32_t next = __shfl_down_sync(kFull, my_ord, 1);
            // NaN and infinities compare as not further apart
            const bool close = lane < p.top_k && my_ord && next && !(value_of(my_ord) - value_of(next) > 2 * err);
            const bool order = __any_sync(kFull, close);
            if (kCandidates && order && !doubt && !one_by_one) {
                __syncwarp();
                mine = select_64_among(p, t, candidate, total, candidates[warp], lane);
            } else {
                doubt = doubt || order;
            }
        }
    }
    if (doubt) mine = select_64(p, t, by_logits, keys, lane);

    const bool in = lane < p.top_k && mine >= 0;
    const float w = weight_of(p, in, in ? logit_at(p, t, mine) : 0.0f, m, sum);
    if (p.experts != nullptr && lane < p.top_k) {
        p.experts[t * p.top_k + lane] = in ? mine : -1;
        p.weights[t * p.top_k + lane] = in ? w * p.scale : 0.0f;
    }
    if (p.dense != nullptr) {
        for (int e = lane; e < p.E; e += 32) p.dense[t * p.E + e] = -INFINITY;
        __syncwarp();  // orders the row before the values that take their places
        if (in) p.dense[t * p.E + mine] = w * p.scale;
    }
}

// The gradient: with p the unscaled weights and d = scale * dweights,
//   softmax over the selected (or renormalised):  dl_j = p_j (d_j - <p, d>)
//   softmax over all:                             dl_e = p_e ([e selected] d_e - <p, d>)
//   sigmoid:                                      dl_j = d_j s_j (1 - s_j)
//   sigmoid, renormalised:                        dl_j = p_j (d_j - <p, d>) (1 - s_j)
// and 0 for every other expert.  A warp a token: the row of zeros (or of the others' softmax), then the selected.
// 32768 tokens, 8 of 256, fp32: the selected alone 9.5 us for 5.5 of bytes (its 4-byte stores: DRAM 65%, issue slots 63% of
// their rate); softmax over all 18.4 for 10.3 (issue slots 80%: the row is read three times, with two exponentials a logit).
template <typename L>
__global__ void __launch_bounds__(kRouteWarps * 32) route_bwd_kernel(const RouteParams p) {
    const int lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * kRouteWarps + (threadIdx.x >> 5);
    if (t >= p.T) return;
    const L* row = static_cast<const L*>(p.logits) + t * p.E;
    L* out = static_cast<L*>(p.dlogits) + t * p.E;
    int e = -1;
    float d = 0.0f;
    if (lane < p.top_k) {
        e = p.experts[t * p.top_k + lane];
        d = p.dweights[t * p.top_k + lane] * p.scale;
    }
    const bool in = e >= 0 && e < p.E;
    const float l = in ? logit(row + e) : 0.0f;
    const bool dense = p.score == MX_SCORE_SOFTMAX_ALL && !p.renormalize;
    float m = 0.0f, sum = 1.0f;
    if (dense) {
        m = -INFINITY;
        for (int i = lane; i < p.E; i += 32) m = fmaxf(m, logit(row + i));
        m = warp_max(m);
        sum = 0.0f;
        for (int i = lane; i < p.E; i += 32) sum += expf(logit(row + i) - m);
        sum = warp_sum(sum);
    }
    const float w = weight_of(p, in, l, m, sum);
    float g;
    if (p.score == MX_SCORE_SIGMOID && !p.renormalize) {
        g = d * w * (1.0f / (1.0f + expf(l)));
    } else {
        const float mean = warp_sum(in ? w * d : 0.0f);
        g = w * (d - mean);
        if (p.score == MX_SCORE_SIGMOID) g *= 1.0f / (1.0f + expf(l));
        if (dense && __any_sync(kFull, in)) {
            for (int i = lane; i < p.E; i += 32) put(out + i, -(expf(logit(row + i) - m) / sum) * mean);
            __syncwarp();
            if (in) put(out + e, g);
            return;
        }
    }
    for (int i = lane; i < p.E; i += 32) put(out + i, 0.0f);
    __syncwarp();  // orders the row's zeros before the values that take their places
    if (in) put(out + e, g);
}

// ---------------------------------------------------------------- the plan
// A stable counting sort by expert.  A CTA takes a run of choices, a warp a part of it, 32 choices a step,
// in turn: a choice's rank among its warp's is the count so far plus the lanes before it with the same expert (a
// warp-wide match), so no atomics and no order that could vary.  With several CTAs a first kernel counts each run.
// Bound by latency: 262144 choices of 256 experts take 12.3 us, of which the counts of 128 runs, which every CTA sums, 4.7,
// and the scattered slots 2 (CTAs of 1024 threads 13.4, longer runs 18, the second kernel launched while the first runs 13.1).
constexpr int kPlanThreads = 512;
constexpr int kPlanWarps = kPlanThreads / 32;
// Steps of a run: few, so that many CTAs share the work; more where there are enough of them (1.6 million choices of 64 experts
// 27.6 us, 35.5 with 16 steps; 4 million of 256, 59, 65 with 4 steps).
constexpr int kPlanShort = 4, kPlanLong = 8;
constexpr int64_t kPlanLongFrom = 1 << 20;
static int plan_steps(int64_t choices) { return choices < kPlanLongFrom ? kPlanShort : kPlanLong; }
static int64_t plan_runs(int64_t choices) {
    const int64_t run = (int64_t)kPlanThreads * plan_steps(choices);
    return max64(1, (choices + run - 1) / run);
}
// More counts, or more runs, than these are summed up by a kernel of their own, as what every CTA reads grows with them.
// Choices, experts, us with every CTA for itself / with the kernel: 262144, 256 12.1 / 12.9;  524288, 256 20.4 / 17.2;  800000, 64
// 18.0 / 21.7;  800000, 128 23.6 / 22.1;  2 million, 64 35.8 / 32.4;  2 million, 16 22.3 / 24.0;  8 million, 16 90 / 73;
// 34 million, 256 2630 / 427.
constexpr int64_t kPlanScanCounts = 32768, kPlanScanRuns = 500;
static bool plan_scanned(int64_t runs, int32_t E) { return runs * E > kPlanScanCounts ? runs > 1 : runs > kPlanScanRuns; }
static int64_t plan_hist_rows(int64_t runs, int32_t E) { return runs == 1 ? 0 : runs + plan_scanned(runs, E); }

struct PlanParams {
    const void* experts;
    int64_t n;  // choices
    int32_t E, multiple, runs;
    int64_t rows;
    int32_t *offs, *counts, *slot, *place;
    int32_t* hist;  // [runs][E]: a run's counts; scanned: those of the runs before it, and [E] behind, of all
    bool scanned;
};

template <typename I>
__device__ __forceinline__ int expert_of(const PlanParams& p, int64_t i) {  // -1: none
    if (i >= p.n) return -1;
    const I e = static_cast<const I*>(p.experts)[i];
    return e >= 0 && e < (I)p.E ? (int)e : -1;
}

template <typename I, int STEPS>
__global__ void __launch_bounds__(kPlanThreads) plan_count_kernel(const PlanParams p) {
    __shared__ int32_t count[kMaxGroups];
    for (int e = threadIdx.x; e < p.E; e += kPlanThreads) count[e] = 0;
    __syncthreads();
    const int64_t base = (int64_t)blockIdx.x * (kPlanThreads * STEPS);
    int ex[STEPS];
#pragma unroll
    for (int s = 0; s < STEPS; ++s) ex[s] = expert_of<I>(p, base + s * kPlanThreads + threadIdx.x);
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
        if (ex[s] >= 0) atomicAdd(&count[ex[s]], 1);
    __syncthreads();
    for (int e = threadIdx.x; e < p.E; e += kPlanThreads) p.hist[(int64_t)blockIdx.x * p.E + e] = count[e];
}

// hist: the runs' counts -> those of the runs before each, and of all.  A CTA takes 32 experts, a warp a 32nd of the runs.
constexpr int kScanWarps = 32;
__global__ void __launch_bounds__(kScanWarps * 32) plan_scan_kernel(const PlanParams p) {
    __shared__ int32_t part[kScanWarps][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, e = blockIdx.x * 32 + lane;
    const int per = (p.runs + kScanWarps - 1) / kScanWarps, from = min(p.runs, warp * per), to = min(p.runs, from + per);
    int32_t sum = 0;
    if (e < p.E) {
#pragma unroll 16
        for (int r = from; r < to; ++r) sum += __ldcg(p.hist + (int64_t)r * p.E + e);
    }
    part[warp][lane] = sum;
    __syncthreads();
    if (e >= p.E) return;
    int32_t before = 0;
    for (int w = 0; w < warp; ++w) before += part[w][lane];
    if (warp == kScanWarps - 1) p.hist[(int64_t)p.runs * p.E + e] = before + sum;
    for (int r0 = from; r0 < to; r0 += 16) {
        int32_t c[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) c[i] = r0 + i < to ? __ldcg(p.hist + (int64_t)(r0 + i) * p.E + e) : 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            if (r0 + i < to) p.hist[(int64_t)(r0 + i) * p.E + e] = before;
            before += c[i];
        }
    }
}

template <typename I, int STEPS>
__global__ void __launch_bounds__(kPlanThreads) plan_place_kernel(const PlanParams p) {
    extern __shared__ int32_t plan_smem[];
    int32_t* table = plan_smem;                  // [kPlanWarps][E]: counts, then first rows
    int32_t* before = table + kPlanWarps * p.E;  // [E]: choices of earlier runs
    int32_t* total = before + p.E;               // [E]: choices of all runs
    int32_t* start = total + p.E;                // [E]: first row of the group
    __shared__ int32_t warp_part[kPlanWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t base = (int64_t)blockIdx.x * (kPlanThreads * STEPS) + warp * 32 * STEPS + lane;
    int ex[STEPS], rank[STEPS];
#pragma unroll
    for (int s = 0; s < STEPS; ++s) ex[s] = expert_of<I>(p, base + s * 32);
    for (int i = threadIdx.x; i < kPlanWarps * p.E; i += kPlanThreads) table[i] = 0;
    for (int e = threadIdx.x; e < p.E; e += kPlanThreads) before[e] = total[e] = 0;
    __syncthreads();
    int32_t* mine = table + warp * p.E;
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
        const uint32_t same = __match_any_sync(kFull, ex[s]);
        const int ahead = __popc(same & ((1u << lane) - 1u));
        if (ex[s] >= 0) rank[s] = mine[ex[s]] + ahead;
        __syncwarp();
        if (ex[s] >= 0 && ahead == 0) mine[ex[s]] += __popc(same);
        __syncwarp();
    }
    __syncthreads();
    if (p.runs == 1) {
        for (int e = threadIdx.x; e < p.E; e += kPlanThreads) {
            int32_t c = 0;
#pragma unroll
            for (int w = 0; w < kPlanWarps; ++w) c += table[w * p.E + e];
            total[e] = c;
        }
    } else if (p.scanned) {
        for (int e = threadIdx.x; e < p.E; e += kPlanThreads) {
            before[e] = __ldcg(p.hist + (int64_t)blockIdx.x * p.E + e);
            total[e] = __ldcg(p.hist + (int64_t)p.runs * p.E + e);
        }
    } else {
        // the counts of all runs, and of those before this one: several threads an expert where there are enough
        const int parts = max(1, kPlanThreads / p.E), part = threadIdx.x / p.E;
        for (int e = parts > 1 ? threadIdx.x - part * p.E : threadIdx.x; e < p.E && part < parts; e += kPlanThreads) {
            int32_t lo = 0, all = 0;
#pragma unroll 16
            for (int r = parts > 1 ? part : 0; r < p.runs; r += parts) {
                const int32_t c = __ldcg(p.hist + (int64_t)r * p.E + e);
                all += c;
                if (r < (int)blockIdx.x) lo += c;
            }
            atomicAdd(before + e, lo);  // integers: any order
            atomicAdd(total + e, all);
        }
    }
    __syncthreads();
    // the groups' first rows: a scan of the padded sizes, kMaxGroups / kPlanThreads neighbours a thread
    constexpr int kPer = kMaxGroups / kPlanThreads;
    int32_t size[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = threadIdx.x * kPer + i;
        size[i] = e < p.E ? (total[e] + p.multiple - 1) / p.multiple * p.multiple : 0;
        // one group is all rows: that is how the quantizations lay its scales out, whatever its end
        if (p.E == 1 && e == 0) size[i] = (int32_t)p.rows;
        sum += size[i];
    }
    int32_t incl = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int32_t o = __shfl_up_sync(kFull, incl, d);
        if (lane >= d) incl += o;
    }
    if (lane == 31) warp_part[warp] = incl;
    __syncthreads();
    int32_t at = incl - sum, end = 0;
#pragma unroll
    for (int w = 0; w < kPlanWarps; ++w) {
        const int32_t c = warp_part[w];
        if (w < warp) at += c;
        end += c;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = threadIdx.x * kPer + i;
        if (e < p.E) {
            start[e] = at;
            if (blockIdx.x == 0) {
                p.offs[e] = at + size[i];
                p.counts[e] = total[e];
            }
        }
        at += size[i];
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.E; e += kPlanThreads) {
        int32_t row = start[e] + before[e];
#pragma unroll
        for (int w = 0; w < kPlanWarps; ++w) {
            const int32_t c = table[w * p.E + e];
            table[w * p.E + e] = row;
            row += c;
        }
    }
    __syncthreads();
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
        const int64_t i = base + s * 32;
        if (i >= p.n) continue;
        int32_t row = -1;
        if (ex[s] >= 0) {
            row = mine[ex[s]] + rank[s];
            p.slot[row] = (int32_t)i;
        }
        p.place[i] = row;
    }
    // rows without a token: each group's padding, by the CTAs in turn, a warp a group; and what follows the last group
    for (int e = blockIdx.x * kPlanWarps + warp; e < p.E; e += gridDim.x * kPlanWarps) {
        const int32_t from = start[e] + total[e], to = e + 1 < p.E ? start[e + 1] : end;
        for (int64_t r = (int64_t)from + lane; r < to; r += 32) p.slot[r] = -1;  // (rows may come near 2^31)
    }
    for (int64_t r = end + (int64_t)blockIdx.x * kPlanThreads + threadIdx.x; r < p.rows; r += (int64_t)gridDim.x * kPlanThreads)
        p.slot[r] = -1;
}

// ---------------------------------------------------------------- host side
static mxfp8_status_t route_check(const RouteParams& p, int32_t type) {
    if (p.T < 0 || p.E < 1 || p.E > MXFP8_MAX_GROUPS || p.top_k < 1 || p.top_k > MX_MAX_TOP_K || p.top_k > p.E)
        return MXFP8_ERR_SHAPE;
    if (p.T * (int64_t)p.top_k > INT32_MAX) return MXFP8_ERR_SHAPE;
    if (p.score < MX_SCORE_SOFTMAX || p.score > MX_SCORE_SIGMOID || type < MX_LOGITS_FP32 || type > MX_LOGITS_FP16)
        return MXFP8_ERR_LAYOUT;
    return MXFP8_OK;
}
static bool aligned_to(const void* p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(bytes - 1)) == 0; }

template <int VPL>
static mxfp8_status_t route_launch(RouteParams& p, cudaStream_t st) {
    p.group_size = p.E / p.groups;
    const int lanes = p.group_size / VPL;
    p.group_lanes = p.group_size % VPL == 0 && (lanes & (lanes - 1)) == 0 ? lanes : 0;
    // 32 KB at most; none where logits are ranked as they are
    const int smem = p.groups > 1 || p.bias ? kRouteWarps * p.E * (int)sizeof(unsigned long long) : 0;
    const unsigned grid = (unsigned)((p.T + kRouteWarps - 1) / kRouteWarps);
    const bool scored = p.bias != nullptr || (p.groups > 1 && !p.group_max);
    if (scored && p.score == MX_SCORE_SIGMOID) route_kernel<VPL, kKeysSigmoid><<<grid, kRouteWarps * 32, smem, st>>>(p);
    else if (scored && p.score == MX_SCORE_SOFTMAX_ALL) route_kernel<VPL, kKeysSoftmax><<<grid, kRouteWarps * 32, smem, st>>>(p);
    else if (p.bias) route_kernel<VPL, kKeysBias><<<grid, kRouteWarps * 32, smem, st>>>(p);
    else route_kernel<VPL, kKeysLogits><<<grid, kRouteWarps * 32, smem, st>>>(p);
    return host::last_launch_status();
}
static mxfp8_status_t route_run(RouteParams& p, cudaStream_t st) {
    if (p.E <= 32) return route_launch<1>(p, st);
    if (p.E <= 64) return route_launch<2>(p, st);
    if (p.E <= 128) return route_launch<4>(p, st);
    if (p.E <= 256) return route_launch<8>(p, st);
    if (p.E <= 512) return route_launch<16>(p, st);
    return route_launch<32>(p, st);
}

template <typename I, int STEPS>
static mxfp8_status_t plan_run(const PlanParams& p, cudaStream_t st) {
    if (p.runs > 1) {
        plan_count_kernel<I, STEPS><<<p.runs, kPlanThreads, 0, st>>>(p);
        if (mxfp8_status_t s = host::last_launch_status(); s != MXFP8_OK) return s;
    }
    if (p.scanned) {
        plan_scan_kernel<<<(p.E + 31) / 32, kScanWarps * 32, 0, st>>>(p);
        if (mxfp8_status_t s = host::last_launch_status(); s != MXFP8_OK) return s;
    }
    static std::atomic<int> attr_set[host::kMaxDevices];
    constexpr int most = (kPlanWarps + 3) * MXFP8_MAX_GROUPS * 4;
    if (!host::ensure_smem(reinterpret_cast<const void*>(plan_place_kernel<I, STEPS>), most, attr_set)) return MXFP8_ERR_LAUNCH;
    plan_place_kernel<I, STEPS><<<p.runs, kPlanThreads, (kPlanWarps + 3) * p.E * 4, st>>>(p);
    return host::last_launch_status();
}

}  // namespace mx

using namespace mx;

extern "C" mxfp8_status_t mx_moe_route(const void* logits, int32_t logits_type, int64_t T, int32_t E, int32_t top_k,
                                       int32_t score, const float* bias, int32_t groups, int32_t top_groups,
                                       int32_t group_score, int32_t renormalize, float scale, int32_t* experts,
                                       float* weights, float* dense, mxfp8_stream_t stream) {
    RouteParams p{};
    p.logits = logits;
    p.type = logits_type;
    p.bias = bias;
    p.experts = experts;
    p.weights = weights;
    p.dense = dense;
    p.T = T;
    p.E = E;
    p.top_k = top_k;
    p.score = score;
    p.groups = groups;
    p.top_groups = top_groups;
    p.group_max = group_score == MX_GROUP_MAX;
    p.renormalize = renormalize != 0;
    p.scale = scale;
    if (mxfp8_status_t s = route_check(p, logits_type); s != MXFP8_OK) return s;
    if (groups < 1 || groups > 32 || E % groups || top_groups < 1 || top_groups > groups || top_k > top_groups * (E / groups))
        return MXFP8_ERR_SHAPE;
    if (group_score != MX_GROUP_TOP2 && group_score != MX_GROUP_MAX) return MXFP8_ERR_LAYOUT;
    if (T == 0) return MXFP8_OK;  // an empty tensor may have no address
    if (!logits || !experts != !weights || (!experts && !dense)) return MXFP8_ERR_NULL;
    if (!aligned_to(logits, logits_type == MX_LOGITS_FP32 ? 4 : 2) || !aligned_to(bias, 4) || !aligned_to(experts, 4) ||
        !aligned_to(weights, 4) || !aligned_to(dense, 4))
        return MXFP8_ERR_ALIGN;
    if (mxfp8_status_t a = host::check_arch(); a != MXFP8_OK) return a;
    return route_run(p, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" mxfp8_status_t mx_moe_route_bwd(const void* logits, int32_t logits_type, int64_t T, int32_t E, int32_t top_k,
                                           int32_t score, int32_t renormalize, float scale, const int32_t* experts,
                                           const float* dweights, void* dlogits, mxfp8_stream_t stream) {
    RouteParams p{};
    p.logits = logits;
    p.experts = const_cast<int32_t*>(experts);
    p.dweights = dweights;
    p.dlogits = dlogits;
    p.T = T;
    p.E = E;
    p.top_k = top_k;
    p.score = score;
    p.renormalize = renormalize != 0;
    p.scale = scale;
    if (mxfp8_status_t s = route_check(p, logits_type); s != MXFP8_OK) return s;
    if (T == 0) return MXFP8_OK;
    if (!logits || !experts || !dweights || !dlogits) return MXFP8_ERR_NULL;
    const int size = logits_type == MX_LOGITS_FP32 ? 4 : 2;
    if (!aligned_to(logits, size) || !aligned_to(dlogits, size) || !aligned_to(experts, 4) || !aligned_to(dweights, 4))
        return MXFP8_ERR_ALIGN;
    if (mxfp8_status_t a = host::check_arch(); a != MXFP8_OK) return a;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const unsigned grid = (unsigned)((T + kRouteWarps - 1) / kRouteWarps);
    if (logits_type == MX_LOGITS_FP32) route_bwd_kernel<float><<<grid, kRouteWarps * 32, 0, st>>>(p);
    else if (logits_type == MX_LOGITS_BF16) route_bwd_kernel<__nv_bfloat16><<<grid, kRouteWarps * 32, 0, st>>>(p);
    else route_bwd_kernel<__half><<<grid, kRouteWarps * 32, 0, st>>>(p);
    return host::last_launch_status();
}

static bool plan_sizes(int64_t T, int32_t top_k, int32_t E, int32_t multiple) {
    if (T < 0 || T > INT32_MAX || top_k < 1 || top_k > MX_MAX_TOP_K || E < 1 || E > MXFP8_MAX_GROUPS || multiple < 1 ||
        multiple > 1024)
        return false;
    return T * top_k + (int64_t)E * multiple <= INT32_MAX;
}

extern "C" int64_t mx_moe_plan_rows(int64_t T, int32_t top_k, int32_t E, int32_t multiple) {
    if (!plan_sizes(T, top_k, E, multiple)) return -1;
    const int64_t n = T * top_k;
    return (n + min64(E, n) * (multiple - 1)) / multiple * multiple;
}

extern "C" size_t mx_moe_plan_workspace(int64_t T, int32_t top_k, int32_t E) {
    if (!plan_sizes(T, top_k, E, 1)) return 0;
    return (size_t)(plan_hist_rows(plan_runs(T * top_k), E) * E * 4);
}

extern "C" mxfp8_status_t mx_moe_plan(const void* experts, int32_t index_bytes, int64_t T, int32_t top_k, int32_t E,
                                      int32_t multiple, int64_t rows, int32_t* offs, int32_t* counts, int32_t* slot,
                                      int32_t* place, void* workspace, size_t workspace_bytes, mxfp8_stream_t stream) {
    if (!plan_sizes(T, top_k, E, multiple) || rows < mx_moe_plan_rows(T, top_k, E, multiple) || rows > INT32_MAX)
        return MXFP8_ERR_SHAPE;
    if (index_bytes != 4 && index_bytes != 8) return MXFP8_ERR_LAYOUT;
    const size_t need = mx_moe_plan_workspace(T, top_k, E);
    if (!offs || !counts || (rows && !slot) || (T && (!experts || !place)) || (need && !workspace)) return MXFP8_ERR_NULL;
    if (workspace_bytes < need) return MXFP8_ERR_SHAPE;
    if (!aligned_to(experts, index_bytes) || !aligned_to(offs, 4) || !aligned_to(counts, 4) || !aligned_to(slot, 4) ||
        !aligned_to(place, 4) || !aligned_to(workspace, 16))
        return MXFP8_ERR_ALIGN;
    if (mxfp8_status_t a = host::check_arch(); a != MXFP8_OK) return a;
    PlanParams p{};
    p.experts = experts;
    p.n = T * top_k;
    p.E = E;
    p.multiple = multiple;
    p.runs = (int32_t)plan_runs(p.n);
    p.scanned = plan_scanned(p.runs, E);
    p.rows = rows;
    p.offs = offs;
    p.counts = counts;
    p.slot = slot;
    p.place = place;
    p.hist = static_cast<int32_t*>(workspace);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (plan_steps(p.n) == kPlanShort)
        return index_bytes == 4 ? plan_run<int32_t, kPlanShort>(p, st) : plan_run<int64_t, kPlanShort>(p, st);
    return index_bytes == 4 ? plan_run<int32_t, kPlanLong>(p, st) : plan_run<int64_t, kPlanLong>(p, st);
}
