// moe_tokens.cu -- a whole routed SwiGLU layer for 1 .. 64 tokens in one kernel, expert weights in MXFP8 or
// MXFP4 (activations quantized to the same format), for sm_103a.
//
//   S_t = the k largest of token t's router logits;  w_te = softmax over S_t (or over all, or sigmoid)
//   h_te = silu(xq_t Wg_e^T) * (xq_t Wu_e^T),   y_t = bf16( sum_{e in S_t} w_te MX(h_te) Wd_e^T )
//
// With few tokens the layer is one pass over the weights of the experts that any token selected, so every
// choice serves that stream.  One cooperative launch, one CTA per SM, weights through TMA into a ring of
// stages that never drains: the same ring runs through both halves of the layer, and the down weights are
// on their way while the last gate/up tiles finish.  Weights are the tensor cores' 128-row operand,
// tokens the narrow one (N = 16, 32 or 64 columns): every token is multiplied with every selected expert,
// which costs no bandwidth and no gather, and a routing mask decides which columns are used -- so a NaN in an
// expert's weights reaches only the tokens routed to it.
//
// A unit of work is a stage of two weight tiles of 128 or 64 rows and 128 bytes of the contraction (32 or 16 KB):
//   first half   tile = 128 or 64 rows of one expert's gate and up matrices; units of one step along D
//   second half  tile = 128 or 64 rows of D; units of two steps, along every selected expert's H in turn
// Each half is cut into runs, one a CTA, in the way that should take least time (mt_split): whole tiles of 128
// or 64 rows, or equal runs of units that end anywhere.  A run that ends inside a tile leaves fp32 partial sums
// in the workspace.  In the first half the CTA that arrives last at a tile adds them, in the second all CTAs do
// after a grid-wide point; both in the order of the runs, so that the result does not depend on arrival.
//
//   warp 0      weight producer (TMA tiles and their scale tiles); waits for nothing but free stages
//   warp 1      token producer (quantized x or h and their scales); waits at the two grid-wide points:
//               x is quantized, h is complete
//   warp 2      tensor-core issuer: scale copies into tensor memory, then the block-scaled MMAs
//   warps 4-11  plan the CTA's work for every number of experts that may turn out selected, quantize its share of x
//               (and, for many logits, select experts with the rest); then the epilogues
//   warps 0-3   route first, every CTA the same
// Every wait is bounded by time (MXFP8_ERR_TIMEOUT and an orderly exit).

#include "host_common.h"
#include "mx4.cuh"

namespace mx {

constexpr int kMtMaxTokens = 64;
constexpr int kMtMaxExperts = 256;
constexpr int kMtMaxTopK = 16;
constexpr int kMtRouteThreads = 128;
constexpr int kMtThreads = 384;
constexpr int kMtHeader = 256;  // workspace bytes before the tile counters

// Words of the workspace's header: CTAs that have arrived at each grid-wide point.  One word each: a CTA does not
// wait at a point that it has no use for, so arrivals at different points mix.
enum MtPoint : int { kMtXDone = 0, kMtHDone = 1, kMtSumsDone = 2, kMtExits = 3 };

struct MtParams {
    const uint8_t* x;        // bf16 [T][D]
    const float* logits;     // [T][E]
    const uint8_t* s_gate;   // blocked scales, per expert
    const uint8_t* s_up;
    const uint8_t* s_down;
    uint8_t* xq;             // workspace: codes [T][D], scales [ct(D)][512]
    uint8_t* xs;
    uint8_t* hq;             // codes [active][T][H], scales [active][ct(H)][512]
    uint8_t* hs;
    float* part;             // [CTA][2][2][T][128] partial sums
    uint32_t* header;        // arrivals at the grid-wide points (MtPoint)
    uint32_t* counters;      // arrivals per shared tile of the first half
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
    float sel_w[kMtMaxTokens * kMtMaxTopK];     // the selected experts' logits, then their weights
    uint16_t sel_e[kMtMaxTokens * kMtMaxTopK];  // a token's experts [T][top_k], best first (0xFFFF: none)
    uint16_t list[kMtMaxExperts];               // active experts, ascending
    int active_n;
};

__device__ __forceinline__ void route_sync() { asm volatile("bar.sync 2, 128;" ::: "memory"); }

// The scratch memory of the routing: the [T][E] keys, a mask of tokens for every expert, and a plan for every number of
// active experts that there can be.  (A plan takes a dozen divisions, most of a microsecond: the epilogue warps make
// them while the routing warps find out the number.)
template <class Plan>
struct MtScratch {
    uint32_t *keys, *masks;
    Plan* plans;
    int most;  // active experts at most
    __device__ __forceinline__ MtScratch(void* at, const MtParams& p)
        : keys(static_cast<uint32_t*>(at)), masks(keys + p.T * p.E), plans(reinterpret_cast<Plan*>(masks + 2 * p.E)),
          most(min(p.E, p.T * p.top_k)) {}
};

// Barrier 4: the routing warps go on once the epilogue warps have made the plans.
__device__ __forceinline__ void plans_arrive() { asm volatile("bar.arrive 4, 384;" ::: "memory"); }
// Barrier 5: the keys, where the epilogue warps take a share of the selection.
__device__ __forceinline__ void keys_sync() { asm volatile("bar.sync 5, 384;" ::: "memory"); }
__device__ __forceinline__ void plans_wait() { asm volatile("bar.sync 4, 384;" ::: "memory"); }

constexpr int kMtFewLogits = 8 * kMtRouteThreads;  // as many as the routing warps load at once
// Whether the epilogue warps take a share of the selection: for more logits than that, it is worth waiting for them.
__device__ __forceinline__ bool mt_shared_selection(const MtParams& p) { return p.T * p.E > kMtFewLogits; }

__device__ __forceinline__ float mt_logit(uint32_t key) {  // the logit that a key was made of
    return __uint_as_float((key & 0x80000000u) ? key ^ 0x80000000u : ~key);
}

// Every token's top_k experts out of the keys, by `threads` threads: sel_e, sel_w (the logits) and the experts' masks.
// Up to 32 experts, every logit's rank among its token's: T E^2 comparisons, of which a thread makes four at a time.  More
// experts: a warp holds a token's keys, KEYS in a lane, and takes its best top_k times, 100 to 400 clocks a round.
// 64 tokens over small experts, the layer with ranks and with rounds: top 4 of 16 21.3 and 22.5 us, top 8 of 64 41 and 27, top 8
// of 256 272 and 48.
__device__ __forceinline__ void mt_rank(const uint32_t* keys, uint32_t* masks, MtRoute& r, int T, int E, int top_k, int tid,
                                        int threads) {
    // i / E for i < 2^14, E <= 2^8: the error of the reciprocal times i stays under 1
    const uint32_t inv_e = 0xFFFFFFFFu / (uint32_t)E + 1;
    for (int i = tid; i < T * E; i += threads) {
        const int t = E == 1 ? i : (int)__umulhi((uint32_t)i, inv_e), e = i - t * E;
        const uint32_t k = keys[i];
        const uint32_t* row = keys + t * E;
        // logits before this one: larger, or equal at a lower index (no key is 0: -inf has the least, 0x007FFFFF)
        int rank = 0;
        auto count = [&](uint32_t key, int o) { rank += key > (o < e ? k - 1 : k); };
        if (E % 4 == 0) {
            for (int o = 0; o < E; o += 4) {
                const uint4 q = *reinterpret_cast<const uint4*>(row + o);
                count(q.x, o);
                count(q.y, o + 1);
                count(q.z, o + 2);
                count(q.w, o + 3);
            }
        } else {
            for (int o = 0; o < E; ++o) count(row[o], o);
        }
        if (rank < top_k && k != 0x007FFFFFu) {  // -inf is never selected
            r.sel_e[t * top_k + rank] = (uint16_t)e;
            r.sel_w[t * top_k + rank] = mt_logit(k);
            atomicOr(&masks[2 * e + (t >> 5)], 1u << (t & 31));
        }
    }
}
template <int KEYS>
__device__ __forceinline__ void mt_rounds(const uint32_t* keys, uint32_t* masks, MtRoute& r, int T, int E, int top_k, int tid,
                                          int threads) {
    const int lane = tid & 31;
    for (int t = tid >> 5; t < T; t += threads / 32) {
        uint32_t k[KEYS];
#pragma unroll
        for (int j = 0; j < KEYS; ++j) k[j] = lane + 32 * j < E ? keys[t * E + lane + 32 * j] : 0u;
        uint32_t my_e = 0, my_key = 0;  // lane `place` keeps what round `place` took
        for (int place = 0; place < top_k; ++place) {
            uint32_t best = k[0];
#pragma unroll
            for (int j = 1; j < KEYS; ++j) best = max(best, k[j]);
            best = __reduce_max_sync(0xffffffffu, best);
            if (best <= 0x007FFFFFu) break;  // only -inf is left (padding has 0)
            uint32_t e = 0;  // of equal ones the first
#pragma unroll
            for (int j = KEYS - 1; j >= 0; --j) {
                const uint32_t have = __ballot_sync(0xffffffffu, k[j] == best);
                if (have) e = 32 * j + __ffs(have) - 1;
            }
#pragma unroll
            for (int j = 0; j < KEYS; ++j)
                if (e == (uint32_t)(lane + 32 * j)) k[j] = 0u;
            if (lane == place) {
                my_e = e;
                my_key = best;
            }
        }
        if (my_key) {
            r.sel_e[t * top_k + lane] = (uint16_t)my_e;
            r.sel_w[t * top_k + lane] = mt_logit(my_key);
            atomicOr(&masks[2 * my_e + (t >> 5)], 1u << (t & 31));
        }
        __syncwarp();
    }
}
__device__ __forceinline__ void mt_select(const uint32_t* keys, uint32_t* masks, MtRoute& r, int T, int E, int k, int tid,
                                          int threads) {
    if (E <= 32) mt_rank(keys, masks, r, T, E, k, tid, threads);
    else if (E <= 64) mt_rounds<2>(keys, masks, r, T, E, k, tid, threads);
    else if (E <= 128) mt_rounds<4>(keys, masks, r, T, E, k, tid, threads);
    else mt_rounds<8>(keys, masks, r, T, E, k, tid, threads);
}
// (Not inlined: it would stand in the way of the code around it, in both kinds of warps.)
__device__ __noinline__ void mt_select_shared(const uint32_t* keys, uint32_t* masks, MtRoute& r, int T, int E, int k,
                                              int tid) {
    mt_select(keys, masks, r, T, E, k, tid, kMtThreads);
}

// Top-k of every token, the list of active experts and the plan for their number, by threads 0 .. 127 of a CTA
// (barrier 2); the caller orders what they wrote before anyone reads it, and adds the weights (mt_weights).
// setup() runs while the logits are on their way.
template <class Plan, class Setup>
__device__ __forceinline__ void mt_route(const MtParams& p, const MtScratch<Plan>& scratch, MtRoute& r, Plan& plan, int tid,
                                         Setup setup) {
    const int E = p.E, n = p.T * E;
    uint32_t *keys = scratch.keys, *masks = scratch.masks;
    uint32_t b[8];  // the first kMtFewLogits; the rest straight to shared memory
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int i = tid + j * kMtRouteThreads;
        b[j] = 0;
        if (i < n) asm volatile("ld.global.u32 %0, [%1];" : "=r"(b[j]) : "l"(p.logits + i));
    }
    for (int i = tid + kMtFewLogits; i < n; i += kMtRouteThreads)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(keys + i)), "l"(p.logits + i) : "memory");
    for (int i = tid; i < p.T * p.top_k; i += kMtRouteThreads) r.sel_e[i] = 0xFFFFu;
    for (int i = tid; i < 2 * E; i += kMtRouteThreads) masks[i] = 0;
    setup();
    // unsigned keys that order as the logits do: NaN above everything, -0 equal to +0
    auto key_of = [](uint32_t v) -> uint32_t {
        uint32_t k = (v & 0x80000000u) ? ~v : v | 0x80000000u;
        if ((v & 0x7FFFFFFFu) > 0x7F800000u) k = 0xFFFFFFFFu;
        if (v == 0x80000000u) k = 0x80000000u;
        return k;
    };
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int i = tid + j * kMtRouteThreads;
        if (i < n) keys[i] = key_of(b[j]);
    }
    if (mt_shared_selection(p)) {
        asm volatile("cp.async.wait_all;" ::: "memory");
        for (int i = tid + kMtFewLogits; i < n; i += kMtRouteThreads) keys[i] = key_of(keys[i]);
        keys_sync();
        mt_select_shared(keys, masks, r, p.T, E, p.top_k, tid);
    } else {
        route_sync();
        mt_select(keys, masks, r, p.T, E, p.top_k, tid, kMtRouteThreads);
    }
    plans_wait();  // and the masks, of all that made them
    const int lane = tid & 31;
    int active = 0;
    for (int e0 = 0; e0 < E; e0 += 32) {  // every warp counts them all, and lists its share
        const int e = e0 + lane;
        const uint32_t m0 = e < E ? masks[2 * e] : 0u, m1 = e < E ? masks[2 * e + 1] : 0u;
        const uint32_t any = __ballot_sync(0xffffffffu, (m0 | m1) != 0);
        if ((m0 | m1) != 0 && (tid >> 5) == ((e0 >> 5) & (kMtRouteThreads / 32 - 1))) {
            const int a = active + __popc(any & ((1u << lane) - 1u));  // the expert's place
            r.list[a] = (uint16_t)e;
            r.mask[a][0] = m0;
            r.mask[a][1] = m1;
        }
        active += __popc(any);
    }
    if (tid == 0) r.active_n = active;
    constexpr int kWords = sizeof(Plan) / 4;
    static_assert(kWords <= kMtRouteThreads, "a thread copies a word");
    if (active && tid < kWords)
        reinterpret_cast<uint32_t*>(&plan)[tid] = reinterpret_cast<const uint32_t*>(scratch.plans + active - 1)[tid];
}

// The selected experts' logits -> their weights, by one warp.
__device__ __forceinline__ void mt_weights(const MtParams& p, MtRoute& r, int lane) {
    for (int t0 = 0; t0 < p.T; t0 += 32) {
        const int t = t0 + lane;
        const bool in = t < p.T;
        const uint16_t* se = r.sel_e + (in ? t : 0) * p.top_k;
        float* sw = r.sel_w + (in ? t : 0) * p.top_k;
        int n = 0;
        while (in && n < p.top_k && se[n] != 0xFFFFu) ++n;
        if (p.score == MX_SCORE_SIGMOID) {
            for (int j = 0; j < n; ++j) sw[j] = 1.0f / (1.0f + expf(-sw[j]));
            continue;
        }
        const float m = n ? sw[0] : 0.0f;  // the largest logit
        float sum = 0.0f;
        if (p.score == MX_SCORE_SOFTMAX) {
            for (int j = 0; j < n; ++j) sum += expf(sw[j] - m);
        } else {  // over all experts: a token at a time, its logits spread over the lanes
            for (int u = 0; u < 32 && t0 + u < p.T; ++u) {
                const float mu = __shfl_sync(0xffffffffu, m, u);
                float part = 0.0f;
                for (int e = lane; e < p.E; e += 32) part += expf(p.logits[(t0 + u) * p.E + e] - mu);
#pragma unroll
                for (int d = 16; d; d >>= 1) part += __shfl_xor_sync(0xffffffffu, part, d);
                if (u == lane) sum = part;
            }
        }
        for (int j = 0; j < n; ++j) sw[j] = expf(sw[j] - m) / sum;
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

constexpr int kMtEpiWarp0 = 4;
constexpr int kMtEpiThreads = 256;
constexpr int kMtStatic = 10 * 1024;  // static shared memory at most

constexpr int kMtStages = 10;  // at most
// For what is certain to finish, whatever the limit of the other waits: copies and products that have been issued.
constexpr uint64_t kMtDrainNs = 2000000000ull;

template <int BITS, int N>
struct MtCfg {
    static constexpr int kKE = BITS == 8 ? 128 : 256;   // contraction elements of a step (128 bytes)
    static constexpr int kSfTiles = kKE / 128;          // 512-byte scale tiles of a step
    static constexpr int kSfCols = 16 * kSfTiles;       // tensor-memory columns of a stage's scales
    static constexpr int kSfCol0 = 4 * N;               // after two buffers of two accumulators
    static constexpr int kSmem = 227 * 1024 - kMtStatic;
    static_assert(kSfCol0 + 4 * kSfCols <= 512, "tensor memory overflow");
};

// The tensor maps, by rows of a box: 128 and 64.
struct MtMaps {
    CUtensorMap gate[2], up[2], down[2], x, h;
};

__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
// One column: a value per lane.
__device__ __forceinline__ uint32_t tmem_ld_col(uint32_t taddr) {
    uint32_t r;
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(taddr));
    return r;
}
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&r)[16]) { tmem_ld_32x32b_x16(taddr, r); }
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&r)[32]) { tmem_ld_32x32b_x32(taddr, r); }

__device__ __forceinline__ void epi_sync() {
    __syncwarp();
    asm volatile("bar.sync 1, 256;" ::: "memory");
}
// Whether every epilogue thread says yes (and a barrier for them).
__device__ __forceinline__ bool epi_all(bool yes) {
    uint32_t r;
    __syncwarp();
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.and.pred q, 1, 256, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)yes)
        : "memory");
    return r != 0;
}

// The epilogue warps wait here for the routing tables; the other four warps only arrive.
__device__ __forceinline__ void routed_arrive() { asm volatile("bar.arrive 3, 384;" ::: "memory"); }
__device__ __forceinline__ void routed_wait() { asm volatile("bar.sync 3, 384;" ::: "memory"); }
// v = *p where `yes`, past L1; a predicate and not a branch, so that many are in flight.
__device__ __forceinline__ void ld_if(float& v, const float* p, bool yes) {
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %2, 0;\n\t@q ld.global.cg.f32 %0, [%1];\n\t}"
                 : "+f"(v)
                 : "l"(p), "r"((uint32_t)yes));
}

__device__ __forceinline__ void ld_if(float4& v, const float* p, bool yes) {
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %5, 0;\n\t@q ld.global.cg.v4.f32 {%0, %1, %2, %3}, [%4];\n\t}"
                 : "+f"(v.x), "+f"(v.y), "+f"(v.z), "+f"(v.w)
                 : "l"(p), "r"((uint32_t)yes));
}

// How one half of the layer is cut into runs, one a CTA.  Work is counted in units (a stage of weights each), `per` of
// them a tile; a run begins and ends at multiples of `grain` units: at tiles (grain == per), so that no CTA shares one,
// or anywhere (grain == 1).
struct MtSplit {
    uint32_t grains, n, grain, per;
    int rows;  // weight rows of a tile: 128, or 64 (half of the 128-row band its scales lie in)
    __device__ __forceinline__ static uint32_t div(uint64_t a, uint32_t b) {
        return a >> 32 ? (uint32_t)(a / b) : (uint32_t)a / b;  // 64-bit division is several times as long
    }
    __device__ __forceinline__ uint32_t start(uint32_t c) const {  // the first grain of run c
        return div((uint64_t)c * grains, n);
    }
    __device__ __forceinline__ uint32_t owner(uint32_t u) const {  // the run that holds unit u
        return div(((uint64_t)u / grain + 1) * n - 1, grains);
    }
    // whether run `c`, which holds some of the tile that begins at unit `begin`, also holds an earlier tile
    __device__ __forceinline__ bool earlier(uint32_t c, uint32_t begin) const { return start(c) * grain < begin; }
    __device__ __forceinline__ bool shared() const { return grain != per; }
};

// The cut that should take least, by clocks.  A half's bytes take their time at HBM's rate; a run takes its own on its
// SM, 900 clocks a unit of 128-row tiles and `half_unit` one of 64-row tiles (600 with 16 token columns, 800 with more: the
// products of a unit are issued in 250 to 500, the rest is the wait for the next stage).  Sharing tiles evens the runs out but
// costs an exchange of partial sums, 7000 clocks under load (two trips through L2 and the gathering).  bands: 128-row
// bands; per: units of one of them; g: CTAs.  Measured, best cut against shared tiles throughout and whole tiles throughout: one token
// over MXFP4 experts of 8192 x 5120 23.2 us / 27.4 / 23.4; four tokens, top 4 of 16 MXFP8 experts of 2048 x 7168 89.6 / 88.5 / 89.9;
// 64 tokens over the same in MXFP4 77 / 89 / 83; five tokens, six experts of 160 x 352 14.0 / 20.1 / 14.7.  With 800 for 16 columns
// too: eight tokens over eight experts of 1024 x 4096 28.2 in place of 26.2, two tokens over 16 of 1536 x 4096 24.8, not 25.9.
constexpr float kMtHbm = 3300.0f;  // bytes a clock
constexpr float kMtExchange = 7000.0f;
__host__ __device__ constexpr float mt_half_unit(int columns) { return columns == 16 ? 600.0f : 800.0f; }

__host__ __device__ __forceinline__ MtSplit mt_split(uint32_t bands, uint32_t per, float half_unit, uint32_t g) {
    const float hbm = (float)per * (32768.0f * (1.0f / kMtHbm));  // a band's bytes at HBM's rate
    // m rounds of a tile for every CTA, then one for the other r tiles
    auto rounds = [&](uint32_t m, uint32_t r, float bytes, float own) -> float {
        return (float)m * fmaxf(own, (float)g * bytes) + (r ? fmaxf(own, (float)r * bytes) : 0.0f);
    };
    const uint32_t m = bands / g, r = bands - m * g, over = 2 * r >= g ? 1 : 0;
    const float whole = rounds(m, r, hbm, (float)per * 900.0f),
                half = rounds(2 * m + over, 2 * r - over * g, 0.5f * hbm, (float)per * half_unit);
    const uint32_t units = bands * per, runs = min(g, (units + 1) / 2);
    const float longest = units < 2 * g ? 2.0f : (float)units / (float)g;
    const float cut = fmaxf((float)bands * hbm, ceilf(longest) * 900.0f) + kMtExchange;
    if (whole <= half && whole <= cut) return MtSplit{bands, min(g, bands), per, per, 128};
    if (half <= cut) return MtSplit{2 * bands, min(g, 2 * bands), per, per, 64};
    return MtSplit{units, runs, 1u, per, 128};
}

// What a CTA does in one half, for one number of active experts.
struct MtHalf {
    MtSplit cut;
    uint32_t u0, u1;      // its units
    uint32_t tile, part;  // the tile they begin in, and which part of its band that is
    uint32_t a, j;        // first half: the tile's active expert and the band of its rows; second: the active expert, and
                          // how many units of it come before
};
struct MtPlan {
    MtHalf half[2];
};

__device__ __forceinline__ MtHalf mt_half(int which, uint32_t bands, uint32_t per, uint32_t inner, uint32_t cta,
                                          float half_unit) {
    MtHalf h;
    h.cut = mt_split(bands, per, half_unit, gridDim.x);
    const uint32_t g0 = h.cut.start(cta);
    h.u0 = h.u1 = h.tile = h.part = h.a = h.j = 0;
    if (cta >= h.cut.n) return h;
    h.u0 = g0 * h.cut.grain;
    h.u1 = h.cut.start(cta + 1) * h.cut.grain;
    h.tile = h.cut.shared() ? h.u0 / per : g0;
    const uint32_t sh = h.cut.rows == 64 ? 1 : 0, band = h.tile >> sh;
    h.part = h.tile & sh;
    const uint32_t from = which ? h.u0 - h.tile * per : band;
    h.a = from / inner;
    h.j = from - h.a * inner;
    return h;
}

template <int BITS, int N>
__global__ void __launch_bounds__(kMtThreads, 1)
    moe_tokens_kernel(const __grid_constant__ MtMaps maps, const MtParams p) {
    using C = MtCfg<BITS, N>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t full[kMtStages], empty[kMtStages], tfull[2], tempty[2], drain;
    __shared__ MtRoute route;
    __shared__ MtPlan plan_s;
    __shared__ float w_s[2][kMtMaxTokens];
    __shared__ uint32_t tmem_base_s, last_s;
    __shared__ uint32_t issued_s[2];  // stages that the weight and the token producer have asked for
    __shared__ int abort_s;
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int T = p.T;
    volatile int* abort_flag = &abort_s;

    const int64_t D = p.D, H = p.H;
    const uint32_t cta = blockIdx.x;
    const int et = tid - kMtEpiWarp0 * 32;
    const uint32_t ct_d = (uint32_t)((D + 127) / 128), ct_h = (uint32_t)((H + 127) / 128);
    const uint32_t K1 = (uint32_t)((D + C::kKE - 1) / C::kKE), K2 = (uint32_t)((H + C::kKE - 1) / C::kKE);
    // first half: tiles (active expert, band of H, part), units of one step; second: tiles (band of D, part), units of two
    // steps of one active expert's H
    const uint32_t K2u = (K2 + 1) / 2;
    // A stage: two weight tiles, their scale tiles, two token tiles (the first half uses one), theirs.  A 64-row tile is
    // multiplied as its half of a 128-row one: the other half is whatever lies beside it in shared memory (half a
    // tile of room is left at both ends) and its results are not looked at.
    struct Layout {
        uint32_t sfa, b, sfb, bytes, edge, stages;
        __device__ constexpr Layout(uint32_t R1, uint32_t R2)
            : sfa(2 * (R1 > R2 ? R1 : R2) * 128), b(sfa + 2 * C::kSfTiles * 512), sfb(b + 2 * N * 128),
              bytes(sfb + 2 * C::kSfTiles * 512), edge(R1 < 128 || R2 < 128 ? 64 * 128 : 0),
              stages((C::kSmem - 1024 - 2 * edge) / bytes) {
            if (stages > (uint32_t)kMtStages) stages = kMtStages;
            if (stages > (uint32_t)(512 - C::kSfCol0) / C::kSfCols) stages = (512 - C::kSfCol0) / C::kSfCols;
        }
    };
    const MtScratch<MtPlan> scratch(smem, p);  // in the ring's memory, before it is filled

    if (warp >= kMtEpiWarp0) {
        // ------------------------------------------------ plans, by the last warps
        for (int i = kMtEpiThreads - 1 - et; i < 2 * scratch.most; i += kMtEpiThreads) {
            const uint32_t A = (uint32_t)(i >> 1) + 1;
            scratch.plans[i >> 1].half[i & 1] =
                mt_half(i & 1, i & 1 ? ct_d : A * ct_h, i & 1 ? A * K2u : K1, i & 1 ? K2u : ct_h, cta,
                        mt_half_unit(N));
        }
        const bool shared = mt_shared_selection(p);
        __syncwarp();
        if (!shared) plans_arrive();
        // ------------------------------------------------ quantize a share of x, zero the tile counters
        // (before any weight is asked for: x's loads would wait behind megabytes of them)
        const int64_t per_row = D / 8, items = T * per_row;  // 8 elements each; 4 neighbours make a block
        for (int64_t i0 = (int64_t)cta * kMtEpiThreads + et - lane; i0 < items;
             i0 += (int64_t)gridDim.x * kMtEpiThreads) {
            const int64_t i = i0 + lane;
            const bool in = i < items;
            const int64_t t = in ? i / per_row : 0, c = in ? (i - t * per_row) * 8 : 0;
            uint4 u = make_uint4(0, 0, 0, 0);
            if (in) u = *reinterpret_cast<const uint4*>(p.x + i * 16);
            float v[8] = {bf16lo(u.x), bf16hi(u.x), bf16lo(u.y), bf16hi(u.y),
                          bf16lo(u.z), bf16hi(u.z), bf16lo(u.w), bf16hi(u.w)};
            uint32_t m = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7FFFFFFFu);
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
            if (!in) continue;
            const uint32_t s = e8m0_of<BITS == 8 ? 8 : 2>(m);
            const float f = s == 0xFFu ? __uint_as_float(0x7FC00000u) : __uint_as_float((254u - s) << 23);
            if constexpr (BITS == 8) {
                uint2 q;
                q.x = cvt_e4m3x2(v[0] * f, v[1] * f) | (cvt_e4m3x2(v[2] * f, v[3] * f) << 16);
                q.y = cvt_e4m3x2(v[4] * f, v[5] * f) | (cvt_e4m3x2(v[6] * f, v[7] * f) << 16);
                *reinterpret_cast<uint2*>(p.xq + i * 8) = q;
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] *= f;  // a NaN scale makes the block NaN whatever its codes
                *reinterpret_cast<uint32_t*>(p.xq + i * 4) = cvt_e2m1x8(v);
            }
            if ((lane & 3) == 0) {
                const int64_t kb = c / 32;
                uint8_t* w = p.xs + (kb >> 2) * 512 + (t & 31) * 16 + (t >> 5) * 4;
                w[kb & 3] = (uint8_t)s;
                if (c + 32 >= D)  // the rest of the last tile's word is padding
                    for (int64_t z = (kb & 3) + 1; z < 4; ++z) w[z] = 0;
            }
        }
        for (int i = cta * kMtEpiThreads + et; i < p.ncounters; i += gridDim.x * kMtEpiThreads) p.counters[i] = 0;
        epi_sync();
        if (et == 0) {
            __threadfence();  // (the proxy fence is the reader's)
            atomicAdd(p.header + kMtXDone, 1u);
        }
        if (shared) {
            keys_sync();
            mt_select_shared(scratch.keys, scratch.masks, route, T, p.E, p.top_k, tid);
            __syncwarp();
            plans_arrive();
        }
        routed_wait();
    } else {
        // ------------------------------------------------ routing (every CTA, the same), barriers
        mt_route(p, scratch, route, plan_s, tid, [&] {
            if (warp == 2) {
                if (lane == 0) {
                    for (int s = 0; s < kMtStages; ++s) {
                        mbar_init(&full[s], 2);  // the weight and the token producer
                        mbar_init(&empty[s], 1);
                    }
                    for (int b = 0; b < 2; ++b) {
                        mbar_init(&tfull[b], 1);
                        mbar_init(&tempty[b], kMtEpiThreads / 32);
                    }
                    mbar_init(&drain, 1);
                    abort_s = 0;
                    fence_barrier_init();
                    prefetch_tmap(&maps.x);
                    prefetch_tmap(&maps.h);
                    for (int i = 0; i < 2; ++i) {
                        prefetch_tmap(&maps.gate[i]);
                        prefetch_tmap(&maps.up[i]);
                        prefetch_tmap(&maps.down[i]);
                    }
                }
                __syncwarp();
                tmem_alloc(&tmem_base_s, 512);
                tmem_relinquish();
            }
        });
        fence_proxy_async();  // the scratch memory is TMA's from here on
        tc_fence_before();
        route_sync();
        if (warp == 3) mt_weights(p, route, lane);
        __syncwarp();
        routed_arrive();
    }
    tc_fence_after();
    const uint32_t tmem = tmem_base_s;
    const int A = __shfl_sync(0xffffffffu, route.active_n, 0);
    auto mask_of = [&](uint32_t a) -> uint64_t { return route.mask[a][0] | ((uint64_t)route.mask[a][1] << 32); };

    const MtHalf h1 = plan_s.half[0], h2 = plan_s.half[1];
    const MtSplit &sp1 = h1.cut, &sp2 = h2.cut;
    const uint32_t AK2 = (uint32_t)A * K2u, u1_0 = h1.u0, u1_1 = h1.u1, u2_0 = h2.u0, u2_1 = h2.u1;
    const uint32_t R1 = sp1.rows, R2 = sp2.rows, parts1 = R1 == 64 ? 2 : 1, parts2 = R2 == 64 ? 2 : 1;
    constexpr Layout both128(128, 128), both64(64, 64), mixed(128, 64);
    const Layout lay = R1 != R2 ? mixed : R1 == 64 ? both64 : both128;
    const uint32_t off_sfa = lay.sfa, off_b = lay.b, off_sfb = lay.sfb, stage_bytes = lay.bytes, stages = lay.stages;
    uint8_t* ring = smem + lay.edge;

    const uint32_t ring_at = __shfl_sync(0xffffffffu, smem_u32(ring), 0);

    auto grid_wait = [&](int point) -> bool { return mt_grid_wait(p, point, abort_flag); };
    // a wait by a whole warp that goes on, or gives up, together
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, mbar_wait_bounded<true>(bar, parity, p.timeout_ns, abort_flag, p.dev_status));
    };
    // A place in the ring.  Whether the next stage can be had is asked one stage ahead, while this one's instructions are
    // issued: a wait costs 130 clocks even at a barrier that is complete, a third of what a stage's products take.
    struct Place {
        uint32_t stage = 0, phase = 0, ready = 0;
    };
    auto take = [&](Place& at, uint64_t* bars, uint32_t flip) -> bool {  // waits for stage at.stage, then looks at the next
        if (!at.ready && !wait(&bars[at.stage], at.phase ^ flip)) return false;
        const bool wraps = at.stage + 1 == stages;
        at.ready = peek(&bars[wraps ? 0 : at.stage + 1], at.phase ^ flip ^ (wraps ? 1u : 0u));
        return true;
    };
    auto pass = [&](Place& at) {
        if (++at.stage == stages) {
            at.stage = 0;
            at.phase ^= 1u;
        }
    };
    auto next1 = [&](MtHalf& t) {
        ++t.tile;
        if (++t.part < parts1) return;
        t.part = 0;
        if (++t.j < ct_h) return;
        t.j = 0;
        ++t.a;
    };
    auto next2 = [&](MtHalf& t) {
        if (++t.a < (uint32_t)A) return;
        t.a = 0;
        ++t.tile;
        t.part ^= parts2 - 1;
    };

    if (A == 0) {
        for (int64_t i = (int64_t)cta * kMtThreads + tid; i < T * D; i += (int64_t)gridDim.x * kMtThreads)
            p.y[i] = __float2bfloat16(0.0f);
    } else if (warp == 0) {
        // ------------------------------------------------ weight producer
        // (Warps 0-2 walk their loops whole and an elected lane issues, so that addresses and descriptors stay in uniform
        // registers, where these instructions take them from; divisions are paid once a tile.)
        const uint32_t one = elect_one();
        Place at;
        uint32_t issued = 0;
        bool ok = true;
        auto claim = [&](uint32_t bytes) -> bool {
            if (!take(at, empty, 1u)) return false;
            expect_tx(one, &full[at.stage], bytes);
            ++issued;
            return true;
        };
        const CUtensorMap *mg = &maps.gate[parts1 - 1], *mu = &maps.up[parts1 - 1], *md = &maps.down[parts2 - 1];
        MtHalf t1 = h1;
        for (uint32_t u = u1_0; u < u1_1 && ok; next1(t1)) {
            const uint32_t end = min(u1_1, (t1.tile + 1) * K1);
            const uint32_t e = __shfl_sync(0xffffffffu, (uint32_t)route.list[t1.a], 0);
            const int32_t row = (int32_t)((int64_t)e * H + t1.j * 128 + t1.part * R1);
            uint32_t k = u - t1.tile * K1;
            const int64_t so = (((int64_t)e * ct_h + t1.j) * ct_d + k * C::kSfTiles) * 512;
            const uint8_t *sg = p.s_gate + so, *su = p.s_up + so;
            for (; u < end; ++u, ++k, sg += C::kSfTiles * 512, su += C::kSfTiles * 512) {
                const uint32_t n = min((uint32_t)C::kSfTiles, ct_d - k * C::kSfTiles) * 512;
                if (!(ok = claim(2 * (R1 * 128 + n)))) break;
                const uint32_t st = ring_at + at.stage * stage_bytes;
                load_2d(one, st, mg, (int32_t)(k * 128), row, &full[at.stage]);
                load_2d(one, st + R1 * 128, mu, (int32_t)(k * 128), row, &full[at.stage]);
                load_bulk(one, st + off_sfa, sg, n, &full[at.stage]);
                load_bulk(one, st + off_sfa + C::kSfTiles * 512, su, n, &full[at.stage]);
                pass(at);
            }
        }
        MtHalf t2 = h2;
        for (uint32_t u = u2_0; u < u2_1 && ok; next2(t2)) {
            const uint32_t base = t2.tile * AK2 + t2.a * K2u, end = min(u2_1, base + K2u);
            const uint32_t band = t2.tile >> (parts2 - 1);
            const uint32_t e = __shfl_sync(0xffffffffu, (uint32_t)route.list[t2.a], 0);
            const int32_t row = (int32_t)((int64_t)e * D + band * 128 + t2.part * R2);
            uint32_t k = 2 * (u - base);
            const uint8_t* sd = p.s_down + (((int64_t)e * ct_d + band) * ct_h + k * C::kSfTiles) * 512;
            for (; u < end; ++u, k += 2, sd += 2 * C::kSfTiles * 512) {
                const uint32_t n = min(2u * C::kSfTiles, ct_h - k * C::kSfTiles) * 512;
                const bool two = k + 1 < K2;
                if (!(ok = claim((two ? 2 : 1) * R2 * 128 + n))) break;
                const uint32_t st = ring_at + at.stage * stage_bytes;
                load_2d(one, st, md, (int32_t)(k * 128), row, &full[at.stage]);
                if (two) load_2d(one, st + R2 * 128, md, (int32_t)(k * 128 + 128), row, &full[at.stage]);
                load_bulk(one, st + off_sfa, sd, n, &full[at.stage]);
                pass(at);
            }
        }
        if (lane == 0) issued_s[0] = issued;
    } else if (warp == 1) {
        // ------------------------------------------------ token producer
        const uint32_t one = elect_one();
        Place at;
        uint32_t issued = 0;
        // steps k .. k + n - 1 of the contraction: tiles of plane z of the map, scale tiles at s
        auto load = [&](const CUtensorMap* m, int32_t z, const uint8_t* s, uint32_t k, uint32_t n, uint32_t ct) -> bool {
            if (!take(at, empty, 1u)) return false;
            const uint32_t st = ring_at + at.stage * stage_bytes;
            const uint32_t sfb = min(n * C::kSfTiles, ct - k * C::kSfTiles) * 512;
            expect_tx(one, &full[at.stage], n * N * 128u + sfb);
            load_3d(one, st + off_b, m, (int32_t)(k * 128), 0, z, &full[at.stage]);
            if (n == 2) load_3d(one, st + off_b + N * 128, m, (int32_t)(k * 128 + 128), 0, z, &full[at.stage]);
            load_bulk(one, st + off_sfb, s, sfb, &full[at.stage]);
            ++issued;
            pass(at);
            return true;
        };
        bool ok = __all_sync(0xffffffffu, grid_wait(kMtXDone));
        uint32_t k = u1_0 - h1.tile * K1;
        const uint8_t* s = p.xs + k * C::kSfTiles * 512;
        for (uint32_t u = u1_0; u < u1_1 && ok; ++u) {
            ok = load(&maps.x, 0, s, k, 1, ct_d);
            s += C::kSfTiles * 512;
            if (++k == K1) {
                k = 0;
                s = p.xs;
            }
        }
        if (ok && u2_0 < u2_1) ok = __all_sync(0xffffffffu, grid_wait(kMtHDone));
        uint32_t a = h2.a;
        k = 2 * h2.j;
        s = p.hs + ((int64_t)a * ct_h + k * C::kSfTiles) * 512;
        for (uint32_t u = u2_0; u < u2_1 && ok; ++u) {
            ok = load(&maps.h, (int32_t)a, s, k, k + 1 < K2 ? 2 : 1, ct_h);
            s += 2 * C::kSfTiles * 512;
            if ((k += 2) >= K2) {
                k = 0;
                if (++a == (uint32_t)A) a = 0;
                s = p.hs + (int64_t)a * ct_h * 512;
            }
        }
        if (lane == 0) issued_s[1] = issued;
    } else if (warp == 2) {
        {
            // -------------------------------------------- tensor-core issuer
            const uint32_t one = elect_one();
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
            Place at;
            int buf = 0;
            uint32_t buf_phase = 0;
            // one product of K = 32 (E4M3) or 64 (E2M1): quarter s of the steps at a (weights) and b (tokens)
            auto mma = [&](uint32_t d, uint32_t a, uint32_t b, uint32_t sfa, uint32_t sfb, int s, uint32_t acc) {
                const uint64_t ad = desc_of((a + 2 * s) | kDescLbo, kDescTile), bd = desc_of((b + 2 * s) | kDescLbo, kDescTile);
                if constexpr (BITS == 8) {
                    mma_mxf8(one, d, ad, bd, idesc_mxf8(128, N, s, s), sfa, sfb, acc);
                } else {
                    constexpr uint32_t id0 = (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | (1u << 23) |
                                             (1u << 27);  // E2M1 x E2M1, E8M0, M = 128
                    const uint32_t id = (uint32_t)(s & 1) * 2;
                    mma_mxf4(one, d, ad, bd, id0 | (id << 4) | (id << 29), sfa + 4 * (s >> 1), sfb + 4 * (s >> 1), acc);
                }
            };
            // quarters of step k that hold any of K elements
            auto quarters = [&](uint32_t k, uint32_t K) -> uint32_t {
                return min(4u, (K - k * C::kKE + C::kKE / 4 - 1) / (C::kKE / 4));
            };
            const uint32_t q_d = quarters(K1 - 1, (uint32_t)D), q_h = quarters(K2 - 1, (uint32_t)H);
            auto open = [&]() -> bool {
                if (!peek(&tempty[buf], buf_phase ^ 1u) && !wait(&tempty[buf], buf_phase ^ 1u)) return false;
                tc_fence_after();
                return true;
            };
            // the quarters of a step, of which the first q hold anything
            auto each = [](uint32_t q, auto&& quarter) {
                quarter(0);
                if (q == 4) {
                    quarter(1);
                    quarter(2);
                    quarter(3);
                } else {
                    if (q > 1) quarter(1);
                    if (q > 2) quarter(2);
                }
            };
            auto close = [&] {
                commit(one, &tfull[buf]);
                if (++buf == 2) { buf = 0; buf_phase ^= 1u; }
            };
            auto release = [&] {
                commit(one, &empty[at.stage]);
                pass(at);
            };
            bool ok = true;
            MtHalf t1 = h1;
            for (uint32_t u = u1_0; u < u1_1 && ok; next1(t1)) {
                const uint32_t end = min(u1_1, (t1.tile + 1) * K1), back = t1.part * R1 * 8;
                if (!(ok = open())) break;
                const uint32_t d0 = tm + buf * 2 * N;
                for (uint32_t k = u - t1.tile * K1, acc = 0; u < end; ++u, ++k) {
                    if (!(ok = take(at, full, 0u))) break;
                    tc_fence_after();
                    // descriptors of a stage differ from its first only in their address field (in units of 16 bytes)
                    const uint32_t st = (ring_at + at.stage * stage_bytes) >> 4, sf = tm + C::kSfCol0 + at.stage * C::kSfCols;
                    const uint32_t a = st - back, b = st + (off_b >> 4);
#pragma unroll
                    for (int i = 0; i < 2 * C::kSfTiles; ++i)
                        cp_scales(one, sf + 4 * i, desc_of(st + (off_sfa >> 4) + 32 * i, kDescScale));
#pragma unroll
                    for (int i = 0; i < C::kSfTiles; ++i)
                        cp_scales(one, sf + 8 * C::kSfTiles + 4 * i, desc_of(st + (off_sfb >> 4) + 32 * i, kDescScale));
                    auto quarter = [&](int s) {
                        mma(d0, a, b, sf, sf + 8 * C::kSfTiles, s, acc);
                        mma(d0 + N, a + R1 * 8, b, sf + 4 * C::kSfTiles, sf + 8 * C::kSfTiles, s, acc);
                        acc = 1;
                    };
                    each(k + 1 == K1 ? q_d : 4u, quarter);
                    release();
                }
                if (ok) close();
            }
            MtHalf t2 = h2;
            for (uint32_t u = u2_0; u < u2_1 && ok; next2(t2)) {
                const uint32_t base = t2.tile * AK2 + t2.a * K2u, end = min(u2_1, base + K2u);
                const uint32_t back = t2.part * R2 * 8;
                if (!(ok = open())) break;
                const uint32_t d0 = tm + buf * 2 * N;
                for (uint32_t k = 2 * (u - base), acc = 0; u < end; ++u, k += 2) {
                    if (!(ok = take(at, full, 0u))) break;
                    tc_fence_after();
                    const uint32_t st = (ring_at + at.stage * stage_bytes) >> 4, sf = tm + C::kSfCol0 + at.stage * C::kSfCols;
                    const uint32_t a = st - back, b = st + (off_b >> 4);
#pragma unroll
                    for (int i = 0; i < 2 * C::kSfTiles; ++i) {
                        cp_scales(one, sf + 4 * i, desc_of(st + (off_sfa >> 4) + 32 * i, kDescScale));
                        cp_scales(one, sf + 8 * C::kSfTiles + 4 * i, desc_of(st + (off_sfb >> 4) + 32 * i, kDescScale));
                    }
                    auto half = [&](int w, uint32_t q) {
                        each(q, [&](int s) {
                            mma(d0, a + w * R2 * 8, b + w * N * 8, sf + 4 * C::kSfTiles * w, sf + (8 + 4 * w) * C::kSfTiles, s,
                                acc);
                            acc = 1;
                        });
                    };
                    half(0, k + 1 == K2 ? q_h : 4u);
                    if (k + 1 < K2) half(1, k + 2 == K2 ? q_h : 4u);
                    release();
                }
                if (ok) close();
            }
            commit(one, &drain);
            volatile int no_abort = 0;
            mbar_wait_bounded<true>(&drain, 0, kMtDrainNs, &no_abort, p.dev_status);
        }
    } else if (warp >= kMtEpiWarp0) {
        const int quarter = warp & 3, cg = (warp - kMtEpiWarp0) >> 2;
        const int r = quarter * 32 + lane;  // row of a weight tile = tensor-memory lane
        const uint32_t lane_base = tmem + ((uint32_t)(quarter * 32) << 16);
        int buf = 0;
        uint32_t buf_phase = 0;
        bool ok = true;
        const uint32_t slot_words = 2u * (uint32_t)T * 128u;  // one partial tile pair
        // A run leaves partial sums of at most two tiles: the one it begins in and the one it ends in.
        auto slot = [&](uint32_t c, bool second) -> float* {
            return p.part + (int64_t)(2 * c + (second ? 1 : 0)) * slot_words;
        };
        // every epilogue thread has written its partial sums: true for the CTA that completes the tile
        auto arrive_last = [&](uint32_t* counter, uint32_t of) -> bool {
            epi_sync();
            if (et == 0) {
                __threadfence();  // the CTA's writes, ordered before this by the barrier
                last_s = atomicAdd(counter, 1u) + 1u == of;
                __threadfence();
            }
            epi_sync();
            return last_s != 0;
        };

        // ------------------------------------------------ first half: gate, up, SwiGLU, quantize h
        // Token columns are those that the expert's mask names, one at a time and the odd ones by warps 8-11: tensor
        // memory and the partial sums are both addressed by column, so nothing is done for the others, and the code
        // stays short (four columns at a time, it took 1 us longer to get through once: instruction fetches).
        auto columns = [&](uint64_t left, auto&& f) {
            for (int turn = 0; left; left &= left - 1, ++turn)
                if ((turn & 1) == cg) f(__ffsll(left) - 1);
        };
        MtHalf t1 = h1;
        for (uint32_t u = u1_0; u < u1_1 && ok;) {
            const uint32_t tile = t1.tile, a = t1.a, j = t1.j;
            const uint32_t end = min(u1_1, (tile + 1) * K1), r0 = t1.part * R1;
            next1(t1);
            const bool whole = u == tile * K1 && end == (tile + 1) * K1;
            u = end;
            ok = epi_all(mbar_wait_bounded<true>(&tfull[buf], buf_phase, p.timeout_ns, abort_flag, p.dev_status));
            if (!ok) break;
            tc_fence_after();
            const uint64_t mask = mask_of(a);
            const uint32_t acc = lane_base + buf * 2 * N;
            // SwiGLU and quantization of a column; the warp's 32 rows are one block of the token's h
            const int64_t row = (int64_t)j * 128 + r;
            const bool mine = quarter * 32 >= r0 && quarter * 32 < r0 + R1;  // this warp's rows are in the tile
            const bool in = row < H;
            auto finish = [&](int col, float g, float h) {
                const float v = in ? g / (1.0f + expf(-g)) * h : 0.0f;
                const uint32_t s = e8m0_of<BITS == 8 ? 8 : 2>(__reduce_max_sync(0xffffffffu, __float_as_uint(v) & 0x7FFFFFFFu));
                const float f = s == 0xFFu ? __uint_as_float(0x7FC00000u) : __uint_as_float((254u - s) << 23);
                const int64_t at = (int64_t)a * T + col;
                if constexpr (BITS == 8) {
                    if (in) p.hq[at * H + row] = (uint8_t)cvt_e4m3x2(v * f, 0.0f);
                } else {
                    const float next = __shfl_down_sync(0xffffffffu, v * f, 1);
                    if (in && (lane & 1) == 0) p.hq[at * (H / 2) + row / 2] = cvt_e2m1x2(v * f, next);
                }
                if (lane == 0)
                    p.hs[((int64_t)a * ct_h + j) * 512 + (col & 31) * 16 + (col >> 5) * 4 + quarter] = (uint8_t)(in ? s : 0u);
            };
            float* own = slot(cta, u1_0 < tile * K1);
            columns(mine ? mask : 0, [&](int col) {
                uint32_t x = tmem_ld_col(acc + col), y = tmem_ld_col(acc + N + col);
                tmem_ld_wait();
                asm volatile("" : "+r"(x), "+r"(y));  // not before the wait
                const float g = __uint_as_float(x), h = __uint_as_float(y);
                if (whole) {
                    finish(col, g, h);
                } else {
                    __stcg(own + col * 128 + r, g);
                    __stcg(own + (T + col) * 128 + r, h);
                }
            });
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&tempty[buf]);
            if (++buf == 2) { buf = 0; buf_phase ^= 1u; }
            if (whole) continue;
            const uint32_t lo = sp1.owner(tile * K1), hi = sp1.owner((tile + 1) * K1 - 1);
            const bool lo_second = sp1.earlier(lo, tile * K1);  // the others begin in this tile
            if (!arrive_last(p.counters + tile, hi - lo + 1)) continue;
            columns(mask, [&](int col) {
                float g = 0.0f, h = 0.0f;
                constexpr int kRuns = 8;  // runs whose sums are in flight together
                for (uint32_t o = lo; o <= hi; o += kRuns) {
                    float v[kRuns], w[kRuns];
#pragma unroll
                    for (int x = 0; x < kRuns; ++x) {
                        const bool have = o + x <= hi;
                        const float* q = slot(o + x, o + x == lo && lo_second);
                        v[x] = w[x] = 0.0f;
                        ld_if(v[x], q + col * 128 + r, have);
                        ld_if(w[x], q + (T + col) * 128 + r, have);
                    }
#pragma unroll
                    for (int x = 0; x < kRuns; ++x) {
                        g += v[x];
                        h += w[x];
                    }
                }
                finish(col, g, h);
            });
        }
        epi_sync();
        if (et == 0) {
            __threadfence();
            atomicAdd(p.header + kMtHDone, 1u);
        }

        // ------------------------------------------------ second half: down, weighted sum over experts
        // (an accumulator for each expert: a token's column is added in, with its weight, if it was routed there)
        constexpr int NC = N / 2;  // token columns of this warp
        const int c0 = cg * NC;
        float total[NC];
        MtHalf t2 = h2;
        for (uint32_t u = u2_0; u < u2_1 && ok;) {
            const uint32_t tile = t2.tile, t_end = min(u2_1, (tile + 1) * AK2);
            const bool whole = u == tile * AK2 && t_end == (tile + 1) * AK2;
            const uint32_t band = tile >> (parts2 - 1), r0 = t2.part * R2;
            const bool mine = quarter * 32 >= r0 && quarter * 32 < r0 + R2;
#pragma unroll
            for (int c = 0; c < NC; ++c) total[c] = 0.0f;
            for (; u < t_end; next2(t2)) {
                const uint32_t a = t2.a;
                u = min(t_end, tile * AK2 + (a + 1) * K2u);
                if (et < T) {  // token et's weight for this expert
                    const int e = route.list[a];
                    float w = 0.0f;
                    for (int j = 0; j < p.top_k; ++j)
                        if (route.sel_e[et * p.top_k + j] == e) w = route.sel_w[et * p.top_k + j];
                    w_s[buf][et] = w;
                }
                ok = epi_all(mbar_wait_bounded<true>(&tfull[buf], buf_phase, p.timeout_ns, abort_flag, p.dev_status));
                if (!ok) break;
                tc_fence_after();
                const uint32_t mask = (uint32_t)(mask_of(a) >> c0);
                if (mine && (mask & (uint32_t)((1ull << NC) - 1ull)) != 0) {
                    uint32_t v[NC];
                    tmem_ld_cols(lane_base + buf * 2 * N + c0, v);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < NC; ++i)
                        if ((mask >> i) & 1u) total[i] += w_s[buf][c0 + i] * __uint_as_float(v[i]);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&tempty[buf]);
                if (++buf == 2) { buf = 0; buf_phase ^= 1u; }
            }
            if (!ok) break;
            if (!whole) {  // (a shared tile has all 128 rows)
                float* w = slot(cta, u2_0 < tile * AK2);
#pragma unroll
                for (int c = 0; c < NC; ++c)
                    if (c0 + c < T) __stcg(w + (c0 + c) * 128 + r, total[c]);
                continue;
            }
            const int64_t d = (int64_t)band * 128 + r;
            if (mine && d < D)
#pragma unroll
                for (int c = 0; c < NC; ++c)
                    if (c0 + c < T) p.y[(c0 + c) * D + d] = __float2bfloat16(total[c]);
        }
        // ------------------------------------------------ add up the tiles that several runs share
        // All CTAs take part, four columns of one token a thread; a tile's sums are added in its runs' order.
        if (sp2.shared()) {
            epi_sync();
            if (et == 0) {
                __threadfence();
                atomicAdd(p.header + kMtSumsDone, 1u);
                ok = ok && grid_wait(kMtSumsDone);
            }
            ok = epi_all(ok);
            // A warp takes a tile's 128 columns of kTok tokens at a time: the runs of its tile are found once and
            // its loads are whole lines, kTok * kRuns of them in flight.
            constexpr int kTok = N == 16 ? 1 : N == 32 ? 2 : 4, kRuns = 12 / kTok;
            const uint32_t groups = (T + kTok - 1) / kTok;
            for (uint32_t i = (et >> 5) * gridDim.x + cta; ok && i < ct_d * groups;
                 i += gridDim.x * (kMtEpiThreads / 32)) {
                const uint32_t gr = i / ct_d, tile = i - gr * ct_d;
                const uint32_t lo = sp2.owner(tile * AK2), hi = sp2.owner((tile + 1) * AK2 - 1);
                if (lo == hi) continue;  // one run had the whole tile
                const bool lo_second = sp2.earlier(lo, tile * AK2);
                const uint32_t d = tile * 128 + lane * 4, t0 = gr * kTok;
                float4 sum[kTok];
#pragma unroll
                for (int t = 0; t < kTok; ++t) sum[t] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                for (uint32_t o = lo; o <= hi; o += kRuns) {
                    float4 v[kRuns][kTok];
#pragma unroll
                    for (int x = 0; x < kRuns; ++x) {
                        const float* q = slot(o + x, o + x == lo && lo_second) + (int64_t)t0 * 128 + lane * 4;
#pragma unroll
                        for (int t = 0; t < kTok; ++t) {
                            v[x][t] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                            ld_if(v[x][t], q + t * 128, o + x <= hi && t0 + t < (uint32_t)T);
                        }
                    }
#pragma unroll
                    for (int x = 0; x < kRuns; ++x)
#pragma unroll
                        for (int t = 0; t < kTok; ++t) {
                            sum[t].x += v[x][t].x;
                            sum[t].y += v[x][t].y;
                            sum[t].z += v[x][t].z;
                            sum[t].w += v[x][t].w;
                        }
                }
#pragma unroll
                for (int t = 0; t < kTok; ++t)
                    if (d < D && t0 + t < (uint32_t)T)  // D is a multiple of 32
                        *reinterpret_cast<uint2*>(p.y + (int64_t)(t0 + t) * D + d) =
                            make_uint2(pack_bf16x2(sum[t].x, sum[t].y), pack_bf16x2(sum[t].z, sum[t].w));
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (abort_s && tid == 0) {
        // Given up: the copies in flight land before the CTA's memory goes.  A stage's barrier wants both producers; where
        // only one got to it, this thread arrives for the other.  (They are never further apart than the ring is long: a
        // stage is given out again after its products, which want both.)  Of the stages before the last ring's length of
        // them, all copies have landed.
        const uint32_t lo = min(issued_s[0], issued_s[1]), hi = max(issued_s[0], issued_s[1]);
        for (uint32_t i = lo; i < hi; ++i) mbar_arrive(&full[i % stages]);
        volatile int no_abort = 0;
        for (uint32_t i = hi > stages ? hi - stages : 0; i < hi; ++i)
            mbar_wait_bounded<true>(&full[i % stages], (i / stages) & 1u, kMtDrainNs, &no_abort, p.dev_status);
    }
    __syncthreads();
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    if (tid == 0) mt_leave(p);
}

// ---------------------------------------------------------------- host side
static int64_t up256(int64_t v) { return (v + 255) / 256 * 256; }

static int mt_columns(int T) { return T <= 16 ? 16 : T <= 32 ? 32 : 64; }  // token columns of the products

struct MtLayout {
    int64_t counters, ncounters, xq, xs, hq, hs, part, total;
};

static MtLayout mt_layout(int64_t T, int64_t E, int64_t D, int64_t H, int64_t k, int bits) {
    const int64_t A = std::min(E, T * k), ct_d = (D + 127) / 128, ct_h = (H + 127) / 128;
    MtLayout l;
    l.counters = kMtHeader;
    l.ncounters = A * ct_h;
    l.xq = l.counters + up256(l.ncounters * 4);
    l.xs = l.xq + up256(T * D * bits / 8);
    l.hq = l.xs + up256(ct_d * 512);
    l.hs = l.hq + up256(A * T * H * bits / 8);
    l.part = l.hs + up256(A * ct_h * 512);
    l.total = l.part + (int64_t)host::num_sms() * 2 * 2 * T * 128 * 4;
    return l;
}

static bool mt_map(CUtensorMap* m, const void* base, int64_t cols, int64_t rows, int64_t planes, int box_rows) {
    host::EncodeTiledFn fn = host::encode_fn();
    if (!fn) return false;
    const int rank = planes > 0 ? 3 : 2;
    cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)planes};
    cuuint64_t strides[2] = {(cuuint64_t)cols, (cuuint64_t)(cols * rows)};
    cuuint32_t box[3] = {128, (cuuint32_t)box_rows, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, rank, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int BITS, int N>
static mxfp8_status_t mt_launch(const MtMaps& m, const MtParams& p, cudaStream_t st) {
    using C = MtCfg<BITS, N>;
    static std::atomic<int> attr_set[host::kMaxDevices];
    if (!host::ensure_smem(reinterpret_cast<const void*>(moe_tokens_kernel<BITS, N>), C::kSmem, attr_set))
        return MXFP8_ERR_LAUNCH;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;  // every CTA is resident: they wait for one another
    attr[0].val.cooperative = 1;
    cfg.gridDim = dim3((unsigned)host::num_sms());
    cfg.blockDim = dim3(kMtThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, moe_tokens_kernel<BITS, N>, m, p) != cudaSuccess) {
        cudaGetLastError();
        return MXFP8_ERR_LAUNCH;
    }
    return host::last_launch_status();
}

static mxfp8_status_t mt_shape(int64_t T, int64_t E, int64_t D, int64_t H, int32_t k, int32_t bits) {
    if (T < 0 || T > kMtMaxTokens || E < 1 || E > kMtMaxExperts || D <= 0 || H <= 0 || k < 1 || k > kMtMaxTopK || k > E ||
        E * D > INT32_MAX || E * H > INT32_MAX)
        return MXFP8_ERR_SHAPE;
    if (bits != 4 && bits != 8) return MXFP8_ERR_LAYOUT;
    // units of work are counted in 32 bits
    if (E * ((H + 127) / 128) * ((D + 127) / 128) > INT32_MAX) return MXFP8_ERR_SHAPE;
    return (D % 32 || H % 32) ? MXFP8_ERR_ALIGN : MXFP8_OK;
}

}  // namespace mx

using namespace mx;

extern "C" size_t mx_moe_tokens_workspace(int32_t max_tokens, int32_t E, int64_t D, int64_t H, int32_t top_k,
                                          int32_t bits) {
    if (max_tokens < 1 || mt_shape(max_tokens, E, D, H, top_k, bits) != MXFP8_OK) return 0;
    return (size_t)mt_layout(max_tokens, E, D, H, top_k, bits).total;
}

static mxfp8_status_t mt_run(const void* x_bf16, const float* router_logits, int32_t T, int32_t E, int64_t D, int64_t H,
                             int32_t top_k, int32_t score, int32_t bits, const void* gate_q, const void* gate_s,
                             const void* up_q, const void* up_s, const void* down_q, const void* down_s, void* workspace,
                             size_t workspace_bytes, void* y_bf16, int32_t* dev_status, uint64_t limit_ns,
                             mxfp8_stream_t stream) {
    if (mxfp8_status_t s = mt_shape(T, E, D, H, top_k, bits); s != MXFP8_OK) return s;
    if (score < MX_SCORE_SOFTMAX || score > MX_SCORE_SIGMOID) return MXFP8_ERR_LAYOUT;
    if (T == 0) return MXFP8_OK;
    const void* ptrs[] = {x_bf16, gate_q, gate_s, up_q, up_s, down_q, down_s, workspace, y_bf16};
    if (!router_logits) return MXFP8_ERR_NULL;
    for (const void* q : ptrs)
        if (!q) return MXFP8_ERR_NULL;
    for (const void* q : ptrs)
        if (!host::aligned16(q)) return MXFP8_ERR_ALIGN;
    if (reinterpret_cast<uintptr_t>(router_logits) & 3u) return MXFP8_ERR_ALIGN;
    if (mxfp8_status_t a = host::check_arch(); a != MXFP8_OK) return a;
    const MtLayout l = mt_layout(T, E, D, H, top_k, bits);
    if (workspace_bytes < (size_t)l.total) return MXFP8_ERR_SHAPE;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    const int N = mt_columns(T);
    const int64_t Db = D * bits / 8, Hb = H * bits / 8;
    MtParams p{};
    p.x = static_cast<const uint8_t*>(x_bf16);
    p.logits = router_logits;
    p.s_gate = static_cast<const uint8_t*>(gate_s);
    p.s_up = static_cast<const uint8_t*>(up_s);
    p.s_down = static_cast<const uint8_t*>(down_s);
    p.xq = ws + l.xq;
    p.xs = ws + l.xs;
    p.hq = ws + l.hq;
    p.hs = ws + l.hs;
    p.part = reinterpret_cast<float*>(ws + l.part);
    p.header = reinterpret_cast<uint32_t*>(ws);
    p.counters = reinterpret_cast<uint32_t*>(ws + l.counters);
    p.y = static_cast<__nv_bfloat16*>(y_bf16);
    p.dev_status = dev_status;
    p.timeout_ns = limit_ns;
    p.D = D;
    p.H = H;
    p.T = T;
    p.E = E;
    p.top_k = top_k;
    p.score = score;
    p.ncounters = (int)l.ncounters;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    MtMaps m;
    for (int i = 0; i < 2; ++i)
        if (!mt_map(&m.gate[i], gate_q, Db, (int64_t)E * H, 0, 128 >> i) ||
            !mt_map(&m.up[i], up_q, Db, (int64_t)E * H, 0, 128 >> i) ||
            !mt_map(&m.down[i], down_q, Hb, (int64_t)E * D, 0, 128 >> i))
            return MXFP8_ERR_DRIVER;
    if (!mt_map(&m.x, ws + l.xq, Db, T, 1, N) ||
        !mt_map(&m.h, ws + l.hq, Hb, T, std::min<int64_t>(E, (int64_t)T * top_k), N))
        return MXFP8_ERR_DRIVER;
    if (bits == 8)
        return N == 16 ? mt_launch<8, 16>(m, p, st) : N == 32 ? mt_launch<8, 32>(m, p, st) : mt_launch<8, 64>(m, p, st);
    return N == 16 ? mt_launch<4, 16>(m, p, st) : N == 32 ? mt_launch<4, 32>(m, p, st) : mt_launch<4, 64>(m, p, st);
}

extern "C" mxfp8_status_t mx_moe_tokens(const void* x_bf16, const float* router_logits, int32_t T, int32_t E, int64_t D,
                                        int64_t H, int32_t top_k, int32_t score, int32_t bits, const void* gate_q,
                                        const void* gate_s, const void* up_q, const void* up_s, const void* down_q,
                                        const void* down_s, void* workspace, size_t workspace_bytes, void* y_bf16,
                                        int32_t* dev_status, mxfp8_stream_t stream) {
    return mt_run(x_bf16, router_logits, T, E, D, H, top_k, score, bits, gate_q, gate_s, up_q, up_s, down_q, down_s, workspace,
                  workspace_bytes, y_bf16, dev_status, 2000000000ull, stream);
}

extern "C" mxfp8_status_t mx_debug_moe_tokens(const void* x_bf16, const float* router_logits, int32_t T, int32_t E, int64_t D,
                                              int64_t H, int32_t top_k, int32_t score, int32_t bits, const void* gate_q,
                                              const void* gate_s, const void* up_q, const void* up_s, const void* down_q,
                                              const void* down_s, void* workspace, size_t workspace_bytes, void* y_bf16,
                                              int32_t* dev_status, uint64_t limit_ns, mxfp8_stream_t stream) {
    if (limit_ns > 10000000000ull) return MXFP8_ERR_SHAPE;
    return mt_run(x_bf16, router_logits, T, E, D, H, top_k, score, bits, gate_q, gate_s, up_q, up_s, down_q, down_s, workspace,
                  workspace_bytes, y_bf16, dev_status, limit_ns, stream);
}

extern "C" int32_t mx_debug_moe_tokens_cut(int32_t half, int32_t T, int32_t active, int64_t D, int64_t H, int32_t bits,
                                           int32_t ctas) {
    if (half < 0 || half > 1 || T < 1 || ctas < 1 || mt_shape(T, active, D, H, 1, bits) != MXFP8_OK) return 0;
    const uint32_t ct_d = (uint32_t)((D + 127) / 128), ct_h = (uint32_t)((H + 127) / 128);
    const uint32_t step = bits == 8 ? 128 : 256, K1 = (uint32_t)((D + step - 1) / step), K2 = (uint32_t)((H + step - 1) / step);
    const MtSplit c = half ? mt_split(ct_d, active * ((K2 + 1) / 2), mt_half_unit(mt_columns(T)), ctas)
                           : mt_split(active * ct_h, K1, mt_half_unit(mt_columns(T)), ctas);
    return c.grain != c.per ? 1 : c.rows;
}
