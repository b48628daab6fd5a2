// moe_tokens.cuh -- what the two kernels of the routed layer for a few tokens share: sizes, parameters and the routing.
#pragma once

#include "host_common.h"
#include "mx4.cuh"

namespace mx {

constexpr int kMtMaxTokens = 64;
constexpr int kMtMaxExperts = 256;
constexpr int kMtMaxTopK = 16;
constexpr int kMtRouteThreads = 128;
constexpr int kMtHeader = 256;  // workspace bytes before the tile counters

// Words of the workspace's header: CTAs that have arrived at each grid-wide point.  One word each: a CTA does not
// wait at a point that it has no use for, so arrivals at different points mix.
enum MtPoint : int { kMtXDone = 0, kMtHDone = 1, kMtSumsDone = 2, kMtExits = 3 };

struct MtParams {
    const uint8_t* x;        // bf16 [T][D]
    const float* logits;     // [T][E]
    const uint8_t* q_gate;   // codes [E][H][D], [E][H][D], [E][D][H]
    const uint8_t* q_up;
    const uint8_t* q_down;
    const uint8_t* s_gate;   // blocked scales, per expert
    const uint8_t* s_up;
    const uint8_t* s_down;
    uint8_t* xq;             // workspace: codes [T][D], scales [ct(D)][512]
    uint8_t* xs;
    uint8_t* hq;             // codes [active][T][H], scales [active][ct(H)][512]
    uint8_t* hs;
    float* part;             // [CTA][2][2][T][128] partial sums
    uint32_t* header;        // arrivals at the grid-wide points (MtPoint)
    uint32_t* counters;      // arrivals per tile: first half, then second half
    __nv_bfloat16* y;        // [T][D]
    int32_t* dev_status;
    uint64_t timeout_ns;
    int64_t D, H;
    int T, E, top_k, score;
    int ncounters;
};

__device__ __forceinline__ void fence_proxy_async() { asm volatile("fence.proxy.async;" ::: "memory"); }

__device__ __forceinline__ uint32_t ld_acquire(const uint32_t* p) {
    uint32_t v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

// The routing tables, in shared memory.
struct MtRoute {
    uint32_t mask[kMtMaxExperts][2];            // tokens of each active expert, a bit each
    uint32_t active[kMtMaxExperts / 32];        // experts that some token selected
    float sel_w[kMtMaxTokens * kMtMaxTopK];     // the selected experts' logits, then their weights
    uint16_t sel_e[kMtMaxTokens * kMtMaxTopK];  // a token's experts [T][top_k], best first (0xFFFF: none)
    uint16_t list[kMtMaxExperts];               // active experts, ascending
    int active_n;
};

__device__ __forceinline__ void route_sync() { asm volatile("bar.sync 2, 128;" ::: "memory"); }

// Top-k of every token and the list of active experts, by threads 0 .. 127 of a CTA (barrier 2); the caller
// orders what they wrote before anyone reads it.  keys: [T][E] words of scratch memory.  setup() runs while the
// logits are on their way.
template <class Setup>
__device__ __forceinline__ void mt_route(const MtParams& p, uint32_t* keys, MtRoute& r, int tid, Setup setup) {
            const int T = p.T, E = p.E;
            for (int i0 = tid; i0 < T * E; i0 += 8 * kMtRouteThreads) {
                uint32_t b[8];
    #pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int i = i0 + j * kMtRouteThreads;
                    b[j] = i < T * E ? __float_as_uint(p.logits[i]) : 0u;
                }
    #pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int i = i0 + j * kMtRouteThreads;
                    // unsigned keys that order as the logits do: NaN above everything, -0 equal to +0
                    uint32_t k = (b[j] & 0x80000000u) ? ~b[j] : b[j] | 0x80000000u;
                    if ((b[j] & 0x7FFFFFFFu) > 0x7F800000u) k = 0xFFFFFFFFu;
                    if (b[j] == 0x80000000u) k = 0x80000000u;
                    if (i < T * E) keys[i] = k;
                }
            }
            for (int i = tid; i < T * p.top_k; i += kMtRouteThreads) r.sel_e[i] = 0xFFFFu;
            if (tid < kMtMaxExperts / 32) r.active[tid] = 0;
            for (int i = tid; i < 2 * kMtMaxExperts; i += kMtRouteThreads) r.mask[i >> 1][i & 1] = 0;
    setup();
            route_sync();
            for (int i = tid; i < T * E; i += kMtRouteThreads) {
                const int t = i / E, e = i - t * E;
                const uint32_t k = keys[i];
                const uint32_t* row = keys + t * E;
                int rank = 0;  // logits before this one: larger, or equal at a lower index
    #pragma unroll 8
                for (int o = 0; o < E; ++o) rank += (row[o] > k) || (row[o] == k && o < e);
                if (rank < p.top_k && k != 0x007FFFFFu) {  // -inf is never selected
                    r.sel_e[t * p.top_k + rank] = (uint16_t)e;
                    r.sel_w[t * p.top_k + rank] = __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k);  // the logit again
                    atomicOr(&r.active[e >> 5], 1u << (e & 31));
                }
            }
            route_sync();
            if (tid < T) {
                const uint16_t* se = r.sel_e + tid * p.top_k;
                float* sw = r.sel_w + tid * p.top_k;
                if (p.score == MX_SCORE_SIGMOID) {
                    for (int j = 0; j < p.top_k && se[j] != 0xFFFFu; ++j) sw[j] = 1.0f / (1.0f + expf(-sw[j]));
                } else {
                    const float m = se[0] != 0xFFFFu ? sw[0] : 0.0f;  // the largest logit
                    float sum = 0.0f;
                    if (p.score == MX_SCORE_SOFTMAX) {
                        for (int j = 0; j < p.top_k && se[j] != 0xFFFFu; ++j) sum += expf(sw[j] - m);
                    } else {
                        for (int e = 0; e < E; ++e) sum += expf(p.logits[tid * E + e] - m);
                    }
                    for (int j = 0; j < p.top_k && se[j] != 0xFFFFu; ++j) sw[j] = expf(sw[j] - m) / sum;
                }
            }
            for (int i = tid; i < T * p.top_k; i += kMtRouteThreads) {
                const int e = r.sel_e[i];
                if (e == 0xFFFF) continue;
                int a = __popc(r.active[e >> 5] & ((1u << (e & 31)) - 1u));  // the expert's place among the active
                for (int w = 0; w < (e >> 5); ++w) a += __popc(r.active[w]);
                const int t = i / p.top_k;
                r.list[a] = (uint16_t)e;
                atomicOr(&r.mask[a][t >> 5], 1u << (t & 31));
            }
            if (tid == 0) {
                int n = 0;
                for (int w = 0; w < kMtMaxExperts / 32; ++w) n += __popc(r.active[w]);
                r.active_n = n;
            }
}

// Whether every CTA has arrived at a grid-wide point; for one thread.
__device__ __forceinline__ bool mt_grid_wait(const MtParams& p, int point, volatile int* abort_flag) {
    const uint64_t t0 = globaltimer_ns();
    while (ld_acquire(p.header + point) < gridDim.x) {
        if (*abort_flag) return false;
        if (globaltimer_ns() - t0 > p.timeout_ns) {
            *abort_flag = 1;
            report(p.dev_status, MXFP8_ERR_TIMEOUT);
            return false;
        }
    }
    fence_proxy_async();  // what the other CTAs wrote, before TMA reads it
    return true;
}

// The last CTA to leave puts the arrivals back to zero for the next launch; for one thread of a CTA.
__device__ __forceinline__ void mt_leave(const MtParams& p) {
    __threadfence();
    if (atomicAdd(p.header + kMtExits, 1u) + 1u == gridDim.x) {
        for (int i = 0; i <= kMtExits; ++i) p.header[i] = 0u;
        __threadfence();
    }
}

// The kernel for 8 tokens at most (moe_token_rows.cu): whether it takes these sizes, and its launch.
bool mt_rows_takes(const MtParams& p, int bits);
mxfp8_status_t mt_rows_launch(const MtParams& p, int bits, cudaStream_t st);

}  // namespace mx
