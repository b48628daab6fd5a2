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
// tokens the narrow one (N = 32 or 64 columns): every token is multiplied with every selected expert, which
// costs no bandwidth and no gather, and a routing mask decides which columns are used -- so a NaN in an
// expert's weights reaches only the tokens routed to it.
//
// A unit of work is one 128-byte step along the contraction of two 128-row weight tiles (32 KB):
//   first half   tile = 128 rows of one expert's gate and up matrices; steps along D
//   second half  tile = 256 rows of D; steps along every selected expert's H in turn
// Each half's units, in order, are cut into equal runs, one per CTA, so the load is even however few experts
// or tiles there are.  A run that ends inside a tile leaves fp32 partial sums in the workspace; the CTA
// that arrives last at a tile adds them in the order of their runs (the result does not depend on arrival).
//
//   warp 0      weight producer (TMA tiles and their scale tiles); waits for nothing but free stages
//   warp 1      token producer (quantized x or h and their scales); waits at the two grid-wide points:
//               x is quantized, h is complete
//   warp 2      tensor-core issuer: scale copies into tensor memory, then the block-scaled MMAs
//   warps 4-11  quantize this CTA's share of x; then the epilogues
// Every wait is bounded by time (MXFP8_ERR_TIMEOUT and an orderly exit).

#include "moe_tokens.cuh"

namespace mx {

constexpr int kMtThreads = 384;
constexpr int kMtEpiWarp0 = 4;
constexpr int kMtEpiThreads = 256;
constexpr int kMtStatic = 10 * 1024;  // static shared memory at most

template <int BITS, int N>
struct MtCfg {
    static constexpr int kKE = BITS == 8 ? 128 : 256;   // contraction elements of a step (128 bytes)
    static constexpr int kSfTiles = kKE / 128;          // 512-byte scale tiles of a step
    static constexpr int kOffSfA = 2 * 128 * 128;       // within a stage: two weight tiles, ...
    static constexpr int kOffB = kOffSfA + 2 * kSfTiles * 512;
    static constexpr int kOffSfB = kOffB + N * 128;
    static constexpr int kStage = (kOffSfB + kSfTiles * 512 + 1023) / 1024 * 1024;
    static constexpr int kSfCols = 3 * 4 * kSfTiles;    // tensor-memory columns of a stage's scales
    static constexpr int kSfCol0 = 4 * N;               // after two buffers of two accumulators
    static constexpr int kStages = (227 * 1024 - kMtStatic - 1024) / kStage;
    static constexpr int kSmem = kStages * kStage + 1024;
    static_assert(kStages >= 5, "too few stages to cover HBM's latency");
    static_assert(kOffB % 1024 == 0, "swizzled tiles start on 1024-byte boundaries");
    static_assert(kSfCol0 + kStages * kSfCols <= 512, "tensor memory overflow");
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

constexpr uint32_t kMtWholeSteps = 6;

// One half's units cut into n equal runs (n <= units, so none is empty).
struct MtSplit {
    uint32_t units, n;
    __device__ __forceinline__ static uint32_t div(uint64_t a, uint32_t b) {
        return a >> 32 ? (uint32_t)(a / b) : (uint32_t)a / b;  // 64-bit division is several times as long
    }
    __device__ __forceinline__ uint32_t start(uint32_t c) const { return div((uint64_t)c * units, n); }
    __device__ __forceinline__ uint32_t owner(uint32_t u) const {  // the run that holds unit u
        return div(((uint64_t)u + 1) * n - 1, units);
    }
    // whether run `c`, which holds some of the tile that begins at unit `begin`, also holds an earlier tile
    __device__ __forceinline__ bool earlier(uint32_t c, uint32_t begin) const { return start(c) < begin; }
};
// Tiles of few steps are not cut (an exchange of partial sums costs about 3 us, a step 0.3 us) where they fit
// one to a CTA; other runs hold at least two units.  On 5 tokens, 6 experts, D = 352, H = 160: 16.0 us; with a
// limit of 12 steps and four units 18.0 us.
__device__ __forceinline__ MtSplit mt_split(uint32_t units, uint32_t per_tile) {
    if (units == 0) return MtSplit{0u, 1u};
    const uint32_t tiles = units / per_tile;
    if (tiles <= gridDim.x && per_tile <= kMtWholeSteps) return MtSplit{units, tiles};
    return MtSplit{units, min(gridDim.x, (units + 1) / 2)};
}

template <int BITS, int N>
__global__ void __launch_bounds__(kMtThreads, 1)
    moe_tokens_kernel(const __grid_constant__ CUtensorMap map_gate, const __grid_constant__ CUtensorMap map_up,
                      const __grid_constant__ CUtensorMap map_down, const __grid_constant__ CUtensorMap map_x,
                      const __grid_constant__ CUtensorMap map_h, const MtParams p) {
    using C = MtCfg<BITS, N>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t full[C::kStages], empty[C::kStages], tfull[2], tempty[2], drain;
    __shared__ MtRoute route;
    __shared__ float w_s[2][kMtMaxTokens];
    __shared__ uint32_t tmem_base_s, last_s;
    __shared__ int abort_s;
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int T = p.T;
    volatile int* abort_flag = &abort_s;

    const int64_t D = p.D, H = p.H;
    const uint32_t cta = blockIdx.x;
    const int et = tid - kMtEpiWarp0 * 32;

    if (warp >= kMtEpiWarp0) {
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
        fence_proxy_async();
        epi_sync();
        if (et == 0) {
            __threadfence();
            atomicAdd(p.header + kMtXDone, 1u);
        }
        routed_wait();
    } else {
        // ------------------------------------------------ routing (every CTA, the same), barriers
        mt_route(p, reinterpret_cast<uint32_t*>(smem), route, tid, [&] {  // the keys, before the first stage is filled
            if (warp == 2) {
                if (lane == 0) {
                    for (int s = 0; s < C::kStages; ++s) {
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
                    prefetch_tmap(&map_gate);
                    prefetch_tmap(&map_up);
                    prefetch_tmap(&map_down);
                    prefetch_tmap(&map_x);
                    prefetch_tmap(&map_h);
                }
                __syncwarp();
                tmem_alloc(&tmem_base_s, 512);
                tmem_relinquish();
            }
        });
        fence_proxy_async();  // the keys' shared memory is TMA's from here on
        tc_fence_before();
        route_sync();
        routed_arrive();
    }
    tc_fence_after();
    const uint32_t tmem = tmem_base_s;
    const int A = __shfl_sync(0xffffffffu, route.active_n, 0);
    auto mask_of = [&](uint32_t a) -> uint64_t { return route.mask[a][0] | ((uint64_t)route.mask[a][1] << 32); };

    const uint32_t ct_d = (uint32_t)((D + 127) / 128), ct_h = (uint32_t)((H + 127) / 128);
    const uint32_t K1 = (uint32_t)((D + C::kKE - 1) / C::kKE), K2 = (uint32_t)((H + C::kKE - 1) / C::kKE);
    const uint32_t TH = ct_h, TD = (uint32_t)((D + 255) / 256);
    const uint32_t AK2 = (uint32_t)A * K2;
    const MtSplit sp1 = mt_split((uint32_t)A * TH * K1, K1), sp2 = mt_split(TD * AK2, AK2);
    const uint32_t u1_0 = cta < sp1.n ? sp1.start(cta) : 0, u1_1 = cta < sp1.n ? sp1.start(cta + 1) : 0;
    const uint32_t u2_0 = cta < sp2.n ? sp2.start(cta) : 0, u2_1 = cta < sp2.n ? sp2.start(cta + 1) : 0;

    auto grid_wait = [&](int point) -> bool { return mt_grid_wait(p, point, abort_flag); };

    if (A == 0) {
        for (int64_t i = (int64_t)cta * kMtThreads + tid; i < T * D; i += (int64_t)gridDim.x * kMtThreads)
            p.y[i] = __float2bfloat16(0.0f);
    } else if (warp == 0) {
        if (lane == 0) {
            // -------------------------------------------- weight producer
            // A place in this CTA's two runs, one after the other.  Stepping costs a few additions: the
            // divisions (hundreds of cycles each on one thread) are paid once a run.
            struct Place {
                const CUtensorMap *m0, *m1;
                const uint8_t *s0, *s1;
                int32_t row0, row1;       // row1 < 0: no second tile
                uint32_t k, K, left;      // step, steps of this tile and expert, units left in this half
                uint32_t a, j;            // active expert, tile
                uint32_t ct;
                bool first;
            };
            auto settle = [&](Place& q) {  // rows, scales of (a, j) from step k on
                const uint32_t e = route.list[q.a];
                if (q.first) {
                    const int64_t so = (((int64_t)e * ct_h + q.j) * ct_d + q.k * C::kSfTiles) * 512;
                    q.row0 = q.row1 = (int32_t)((int64_t)e * H + q.j * 128);
                    q.s0 = p.s_gate + so;
                    q.s1 = p.s_up + so;
                } else {
                    q.row0 = (int32_t)((int64_t)e * D + q.j * 256);
                    q.row1 = 2 * q.j + 1 < ct_d ? q.row0 + 128 : -1;
                    q.s0 = p.s_down + (((int64_t)e * ct_d + 2 * q.j) * ct_h + q.k * C::kSfTiles) * 512;
                    q.s1 = q.s0 + (int64_t)ct_h * 512;
                }
            };
            auto second = [&](Place& q) {
                const uint32_t r = u2_0 % AK2;
                q.first = false;
                q.m0 = q.m1 = &map_down;
                q.j = u2_0 / AK2;
                q.a = r / K2;
                q.k = r - q.a * K2;
                q.K = K2;
                q.ct = ct_h;
                q.left = u2_1 - u2_0;
            };
            auto begin = [&]() -> Place {
                Place q;
                if (u1_0 < u1_1) {
                    const uint32_t tile = u1_0 / K1;
                    q.first = true;
                    q.m0 = &map_gate;
                    q.m1 = &map_up;
                    q.a = tile / TH;
                    q.j = tile - q.a * TH;
                    q.k = u1_0 - tile * K1;
                    q.K = K1;
                    q.ct = ct_d;
                    q.left = u1_1 - u1_0;
                } else {
                    second(q);
                }
                settle(q);
                return q;
            };
            auto step = [&](Place& q) {
                --q.left;
                if (++q.k < q.K && q.left != 0) {
                    q.s0 += C::kSfTiles * 512;
                    q.s1 += C::kSfTiles * 512;
                    return;
                }
                if (q.left == 0) {
                    if (!q.first || u2_0 == u2_1) return;  // the end
                    second(q);
                } else {
                    q.k = 0;
                    if (q.first) {
                        if (++q.j == TH) { q.j = 0; ++q.a; }
                    } else {
                        if (++q.a == (uint32_t)A) { q.a = 0; ++q.j; }
                    }
                }
                settle(q);
            };
            auto sf_bytes = [&](const Place& q) { return min((uint32_t)C::kSfTiles, q.ct - q.k * C::kSfTiles) * 512u; };
            const uint32_t total = (u1_1 - u1_0) + (u2_1 - u2_0);
            if (total != 0) {
                int stage = 0;
                uint32_t phase = 0;
                Place q = begin();
                for (uint32_t i = 0; i < total; ++i) {
                    if (!mbar_wait_bounded<true>(&empty[stage], phase ^ 1u, p.timeout_ns, abort_flag, p.dev_status)) break;
                    uint8_t* st = smem + stage * C::kStage;
                    const uint32_t n = sf_bytes(q);
                    const int32_t x = (int32_t)(q.k * 128);
                    mbar_arrive_expect_tx(&full[stage], (q.row1 >= 0 ? 2u : 1u) * (16384u + n));
                    tma_load_2d(st, q.m0, x, q.row0, &full[stage]);
                    bulk_load(st + C::kOffSfA, q.s0, n, &full[stage]);
                    if (q.row1 >= 0) {
                        tma_load_2d(st + 16384, q.m1, x, q.row1, &full[stage]);
                        bulk_load(st + C::kOffSfA + C::kSfTiles * 512, q.s1, n, &full[stage]);
                    }
                    step(q);
                    if (++stage == C::kStages) { stage = 0; phase ^= 1u; }
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            // -------------------------------------------- token producer
            int stage = 0;
            uint32_t phase = 0;
            // step k of the contraction: tile (k, plane z) of the map, scale tiles at s
            auto load = [&](const CUtensorMap* m, int32_t z, const uint8_t* s, uint32_t k, uint32_t ct) -> bool {
                if (!mbar_wait_bounded<true>(&empty[stage], phase ^ 1u, p.timeout_ns, abort_flag, p.dev_status))
                    return false;
                uint8_t* st = smem + stage * C::kStage;
                const uint32_t sfb = min((uint32_t)C::kSfTiles, ct - k * C::kSfTiles) * 512;
                mbar_arrive_expect_tx(&full[stage], N * 128u + sfb);
                tma_load_3d(st + C::kOffB, m, (int32_t)(k * 128), 0, z, &full[stage]);
                bulk_load(st + C::kOffSfB, s, sfb, &full[stage]);
                if (++stage == C::kStages) { stage = 0; phase ^= 1u; }
                return true;
            };
            bool ok = grid_wait(kMtXDone);
            uint32_t k = u1_0 % K1;
            const uint8_t* s = p.xs + k * C::kSfTiles * 512;
            for (uint32_t u = u1_0; u < u1_1 && ok; ++u) {
                ok = load(&map_x, 0, s, k, ct_d);
                s += C::kSfTiles * 512;
                if (++k == K1) {
                    k = 0;
                    s = p.xs;
                }
            }
            if (ok && u2_0 < u2_1) ok = grid_wait(kMtHDone);
            uint32_t a = u2_0 % AK2 / K2;
            k = u2_0 % K2;  // AK2 is a multiple of K2
            s = p.hs + ((int64_t)a * ct_h + k * C::kSfTiles) * 512;
            for (uint32_t u = u2_0; u < u2_1 && ok; ++u) {
                ok = load(&map_h, (int32_t)a, s, k, ct_h);
                s += C::kSfTiles * 512;
                if (++k == K2) {
                    k = 0;
                    if (++a == (uint32_t)A) a = 0;
                    s = p.hs + (int64_t)a * ct_h * 512;
                }
            }
        }
    } else if (warp == 2) {
        {
            // -------------------------------------------- tensor-core issuer
            // The whole warp walks the loop and one elected lane issues, so that descriptors and addresses stay in
            // uniform registers, where these instructions take them from.
            const uint32_t one = elect_one();
            const uint32_t ring = __shfl_sync(0xffffffffu, smem_u32(smem), 0);
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
            auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
                return __all_sync(0xffffffffu,
                                  mbar_wait_bounded<true>(bar, parity, p.timeout_ns, abort_flag, p.dev_status));
            };
            int stage = 0, buf = 0;
            uint32_t phase = 0, buf_phase = 0;
            // steps k0 .. k1-1 of a contraction of K elements into the next accumulator pair
            auto contract = [&](uint32_t k0, uint32_t k1, int64_t K) -> bool {
                if (!wait(&tempty[buf], buf_phase ^ 1u))
                    return false;
                tc_fence_after();
                const uint32_t d0 = tm + buf * 2 * N;
                for (uint32_t k = k0; k < k1; ++k) {
                    if (!wait(&full[stage], phase))
                        return false;
                    tc_fence_after();
                    // descriptors of a stage differ from its first only in their address field
                    const uint32_t at = (ring + stage * C::kStage) >> 4;
                    const uint32_t sf = tm + C::kSfCol0 + stage * C::kSfCols;
#pragma unroll
                    for (int i = 0; i < 3 * C::kSfTiles; ++i) {
                        const int off = i < 2 * C::kSfTiles ? C::kOffSfA + 512 * i
                                                            : C::kOffSfB + 512 * (i - 2 * C::kSfTiles);
                        cp_scales(one, sf + 4 * i, desc_of(at + off / 16, kDescScale));
                    }
                    auto mma = [&](int s, uint32_t acc) {
                        const uint64_t bd = desc_of((at + (C::kOffB + 32 * s) / 16) | kDescLbo, kDescTile);
#pragma unroll
                        for (int w = 0; w < 2; ++w) {
                            const uint64_t ad = desc_of((at + (w * 16384 + 32 * s) / 16) | kDescLbo, kDescTile);
                            if constexpr (BITS == 8) {
                                mma_mxf8(one, d0 + w * N, ad, bd, idesc_mxf8(128, N, s, s), sf + 4 * w, sf + 8, acc);
                            } else {
                                constexpr uint32_t id0 = (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) |
                                                         (1u << 23) | (1u << 27);  // E2M1 x E2M1, E8M0, M = 128
                                const uint32_t id = (uint32_t)(s & 1) * 2;
                                mma_mxf4(one, d0 + w * N, ad, bd, id0 | (id << 4) | (id << 29),
                                            sf + 8 * w + 4 * (s >> 1), sf + 16 + 4 * (s >> 1), acc);
                            }
                        }
                    };
                    if ((int64_t)(k + 1) * C::kKE <= K) {
                        mma(0, k != k0);
                        mma(1, 1u);
                        mma(2, 1u);
                        mma(3, 1u);
                    } else {  // the contraction's last elements
                        const int steps = (int)((K - (int64_t)k * C::kKE + C::kKE / 4 - 1) / (C::kKE / 4));
                        mma(0, k != k0);
                        if (steps > 1) mma(1, 1u);
                        if (steps > 2) mma(2, 1u);
                        if (steps > 3) mma(3, 1u);
                    }
                    commit(one, &empty[stage]);
                    if (++stage == C::kStages) { stage = 0; phase ^= 1u; }
                }
                commit(one, &tfull[buf]);
                if (++buf == 2) { buf = 0; buf_phase ^= 1u; }
                return true;
            };
            bool ok = true;
            for (uint32_t u = u1_0; u < u1_1 && ok;) {
                const uint32_t tile = u / K1, end = min(u1_1, (tile + 1) * K1);
                ok = contract(u - tile * K1, end - tile * K1, D);
                u = end;
            }
            for (uint32_t u = u2_0; u < u2_1 && ok;) {
                const uint32_t base = u / K2 * K2, end = min(u2_1, base + K2);  // AK2 is a multiple of K2
                ok = contract(u - base, end - base, H);
                u = end;
            }
            commit(one, &drain);
            volatile int no_abort = 0;
            mbar_wait_bounded<true>(&drain, 0, p.timeout_ns, &no_abort, p.dev_status);
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
        // Token columns are taken kCols at a time from those the expert's mask names, the odd batches by warps
        // 8-11: tensor memory and the partial sums are both addressed by column, so nothing is done for the others
        // and the code stays a short loop (unrolled over all columns it did not fit the instruction cache).
        constexpr int kCols = 4;
        for (uint32_t u = u1_0; u < u1_1 && ok;) {
            const uint32_t tile = u / K1, a = tile / TH, j = tile - a * TH;
            const uint32_t end = min(u1_1, (tile + 1) * K1);
            const bool whole = u == tile * K1 && end == (tile + 1) * K1;
            u = end;
            ok = epi_all(mbar_wait_bounded<true>(&tfull[buf], buf_phase, p.timeout_ns, abort_flag, p.dev_status));
            if (!ok) break;
            tc_fence_after();
            const uint64_t mask = mask_of(a);
            const uint32_t acc = lane_base + buf * 2 * N;
            // the next batch of columns: their indexes (the last repeated), and how many
            auto batch = [&](uint64_t& left, int (&col)[kCols]) -> int {
                int n = 0;
#pragma unroll
                for (int i = 0; i < kCols; ++i) {
                    if (left) {
                        col[i] = __ffsll(left) - 1;
                        left &= left - 1;
                        n = i + 1;
                    } else {
                        col[i] = i ? col[i - 1] : 0;
                    }
                }
                return n;
            };
            auto from_tmem = [&](const int (&col)[kCols], float (&g)[kCols], float (&h)[kCols]) {
                uint32_t x[kCols], y[kCols];
#pragma unroll
                for (int i = 0; i < kCols; ++i) {
                    x[i] = tmem_ld_col(acc + col[i]);
                    y[i] = tmem_ld_col(acc + N + col[i]);
                }
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < kCols; ++i) {
                    asm volatile("" : "+r"(x[i]), "+r"(y[i]));  // not before the wait
                    g[i] = __uint_as_float(x[i]);
                    h[i] = __uint_as_float(y[i]);
                }
            };
            // SwiGLU and quantization of n columns; the warp's 32 rows are one block of a token's h
            const int64_t row = (int64_t)j * 128 + r;
            const bool in = row < H;
            auto finish = [&](const int (&col)[kCols], int n, const float (&g)[kCols], const float (&h)[kCols]) {
                float v[kCols];
                uint32_t m[kCols];
#pragma unroll
                for (int i = 0; i < kCols; ++i) {
                    v[i] = in ? g[i] / (1.0f + expf(-g[i])) * h[i] : 0.0f;
                    m[i] = __reduce_max_sync(0xffffffffu, __float_as_uint(v[i]) & 0x7FFFFFFFu);
                }
#pragma unroll
                for (int i = 0; i < kCols; ++i) {
                    const uint32_t s = e8m0_of<BITS == 8 ? 8 : 2>(m[i]);
                    const float f = s == 0xFFu ? __uint_as_float(0x7FC00000u) : __uint_as_float((254u - s) << 23);
                    const int64_t at = (int64_t)a * T + col[i];
                    if constexpr (BITS == 8) {
                        if (in && i < n) p.hq[at * H + row] = (uint8_t)cvt_e4m3x2(v[i] * f, 0.0f);
                    } else {
                        const float q8[8] = {v[i] * f, __shfl_down_sync(0xffffffffu, v[i] * f, 1), 0, 0, 0, 0, 0, 0};
                        if (in && i < n && (lane & 1) == 0) p.hq[at * (H / 2) + row / 2] = (uint8_t)cvt_e2m1x8(q8);
                    }
                    if (lane == 0 && i < n)
                        p.hs[((int64_t)a * ct_h + j) * 512 + (col[i] & 31) * 16 + (col[i] >> 5) * 4 + quarter] =
                            (uint8_t)(in ? s : 0u);
                }
            };
            float* own = slot(cta, u1_0 < tile * K1);
            uint64_t left = mask;
            for (int turn = 0; left; ++turn) {
                int col[kCols];
                const int n = batch(left, col);
                if ((turn & 1) != cg) continue;
                float g[kCols], h[kCols];
                from_tmem(col, g, h);
                if (whole) {
                    finish(col, n, g, h);
                } else {
#pragma unroll
                    for (int i = 0; i < kCols; ++i)
                        if (i < n) {
                            __stcg(own + col[i] * 128 + r, g[i]);
                            __stcg(own + (T + col[i]) * 128 + r, h[i]);
                        }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&tempty[buf]);
            if (++buf == 2) { buf = 0; buf_phase ^= 1u; }
            if (whole) continue;
            const uint32_t lo = sp1.owner(tile * K1), hi = sp1.owner((tile + 1) * K1 - 1);
            const bool lo_second = sp1.earlier(lo, tile * K1);  // the others begin in this tile
            if (!arrive_last(p.counters + tile, hi - lo + 1)) continue;
            left = mask;
            for (int turn = 0; left; ++turn) {
                int col[kCols];
                const int n = batch(left, col);
                if ((turn & 1) != cg) continue;
                float g[kCols], h[kCols];
#pragma unroll
                for (int i = 0; i < kCols; ++i) g[i] = h[i] = 0.0f;
                constexpr int kRuns = 4;  // runs whose sums are in flight together
                for (uint32_t o = lo; o <= hi; o += kRuns) {
                    float v[kRuns][kCols], w[kRuns][kCols];
#pragma unroll
                    for (int x = 0; x < kRuns; ++x) {
                        const bool have = o + x <= hi;
                        const float* q = slot(o + x, o + x == lo && lo_second);
#pragma unroll
                        for (int i = 0; i < kCols; ++i) {
                            v[x][i] = w[x][i] = 0.0f;
                            ld_if(v[x][i], q + col[i] * 128 + r, have && i < n);
                            ld_if(w[x][i], q + (T + col[i]) * 128 + r, have && i < n);
                        }
                    }
#pragma unroll
                    for (int x = 0; x < kRuns; ++x)
#pragma unroll
                        for (int i = 0; i < kCols; ++i) {
                            g[i] += v[x][i];
                            h[i] += w[x][i];
                        }
                }
                finish(col, n, g, h);
            }
        }
        fence_proxy_async();
        epi_sync();
        if (et == 0) {
            __threadfence();
            atomicAdd(p.header + kMtHDone, 1u);
        }

        // ------------------------------------------------ second half: down, weighted sum over experts
        constexpr int kLd = N < 32 ? N : 32;
        float total[N];  // warps 4-7: rows 0-127 of the tile, warps 8-11: rows 128-255
        for (uint32_t u = u2_0; u < u2_1 && ok;) {
            const uint32_t tile = u / AK2, t_end = min(u2_1, (tile + 1) * AK2);
            const bool whole = u == tile * AK2 && t_end == (tile + 1) * AK2;
#pragma unroll
            for (int c = 0; c < N; ++c) total[c] = 0.0f;
            uint32_t a = (u - tile * AK2) / K2;
            for (; u < t_end; ++a) {
                u = min(t_end, tile * AK2 + (a + 1) * K2);
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
                const uint64_t mask = mask_of(a);
#pragma unroll
                for (int c = 0; c < N; c += kLd) {
                    if (((mask >> c) & ((1ull << kLd) - 1ull)) == 0) continue;
                    uint32_t v[kLd];
                    tmem_ld_cols(lane_base + buf * 2 * N + cg * N + c, v);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < kLd; ++i)
                        if ((mask >> (c + i)) & 1u) total[c + i] += w_s[buf][c + i] * __uint_as_float(v[i]);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&tempty[buf]);
                if (++buf == 2) { buf = 0; buf_phase ^= 1u; }
            }
            if (!ok) break;
            if (!whole) {
                float* w = slot(cta, u2_0 < tile * AK2) + cg * T * 128;
#pragma unroll
                for (int c = 0; c < N; ++c)
                    if (c < T) __stcg(w + c * 128 + r, total[c]);
                continue;
            }
            const int64_t d = (int64_t)tile * 256 + cg * 128 + r;
            if (d < D)
#pragma unroll
                for (int c = 0; c < N; ++c)
                    if (c < T) p.y[c * D + d] = __float2bfloat16(total[c]);
        }
        // ------------------------------------------------ add up the tiles that several runs share
        // All CTAs take part, four columns of one token a thread; a tile's sums are added in its runs' order.
        if (sp2.units % sp2.n != 0 || sp2.units / sp2.n % AK2 != 0) {
            epi_sync();
            if (et == 0) {
                __threadfence();
                atomicAdd(p.header + kMtSumsDone, 1u);
                ok = ok && grid_wait(kMtSumsDone);
            }
            ok = epi_all(ok);
            // A warp takes 128 columns (half a tile) of kTok tokens at a time: the runs of its tile are found once and
            // its loads are whole lines, kTok * kRuns of them in flight.
            constexpr int kTok = N == 16 ? 1 : N == 32 ? 2 : 4, kRuns = 12 / kTok;
            const uint32_t halves = ct_d, groups = (T + kTok - 1) / kTok;
            for (uint32_t i = (et >> 5) * gridDim.x + cta; ok && i < halves * groups;
                 i += gridDim.x * (kMtEpiThreads / 32)) {
                const uint32_t gr = i / halves, hf = i - gr * halves, tile = hf >> 1;
                const uint32_t lo = sp2.owner(tile * AK2), hi = sp2.owner((tile + 1) * AK2 - 1);
                if (lo == hi) continue;  // one run had the whole tile
                const bool lo_second = sp2.earlier(lo, tile * AK2);
                const uint32_t d = hf * 128 + lane * 4, t0 = gr * kTok;
                float4 sum[kTok];
#pragma unroll
                for (int t = 0; t < kTok; ++t) sum[t] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                for (uint32_t o = lo; o <= hi; o += kRuns) {
                    float4 v[kRuns][kTok];
#pragma unroll
                    for (int x = 0; x < kRuns; ++x) {
                        const float* q = slot(o + x, o + x == lo && lo_second) + ((int64_t)(hf & 1) * T + t0) * 128 + lane * 4;
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
    if (abort_s && tid == 0) {  // given up: let the copies in flight land before the CTA's memory goes
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 1000000ull) __nanosleep(1000);
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

struct MtLayout {
    int64_t counters, ncounters, xq, xs, hq, hs, part, total;
};

static MtLayout mt_layout(int64_t T, int64_t E, int64_t D, int64_t H, int64_t k, int bits) {
    const int64_t A = std::min(E, T * k), ct_d = (D + 127) / 128, ct_h = (H + 127) / 128;
    MtLayout l;
    l.counters = kMtHeader;
    l.ncounters = A * ct_h + (D + 255) / 256;
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
static mxfp8_status_t mt_launch(const CUtensorMap (&m)[5], const MtParams& p, cudaStream_t st) {
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
    if (cudaLaunchKernelEx(&cfg, moe_tokens_kernel<BITS, N>, m[0], m[1], m[2], m[3], m[4], p) != cudaSuccess) {
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

extern "C" mxfp8_status_t mx_moe_tokens(const void* x_bf16, const float* router_logits, int32_t T, int32_t E, int64_t D,
                                        int64_t H, int32_t top_k, int32_t score, int32_t bits, const void* gate_q,
                                        const void* gate_s, const void* up_q, const void* up_s, const void* down_q,
                                        const void* down_s, void* workspace, size_t workspace_bytes, void* y_bf16,
                                        int32_t* dev_status, mxfp8_stream_t stream) {
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
    const int N = T <= 16 ? 16 : T <= 32 ? 32 : 64;
    const int64_t Db = D * bits / 8, Hb = H * bits / 8;
    MtParams p{};
    p.x = static_cast<const uint8_t*>(x_bf16);
    p.logits = router_logits;
    p.q_gate = static_cast<const uint8_t*>(gate_q);
    p.q_up = static_cast<const uint8_t*>(up_q);
    p.q_down = static_cast<const uint8_t*>(down_q);
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
    p.timeout_ns = 2000000000ull;
    p.D = D;
    p.H = H;
    p.T = T;
    p.E = E;
    p.top_k = top_k;
    p.score = score;
    p.ncounters = (int)l.ncounters;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (mt_rows_takes(p, bits)) return mt_rows_launch(p, bits, st);
    CUtensorMap m[5];
    if (!mt_map(&m[0], gate_q, Db, (int64_t)E * H, 0, 128) || !mt_map(&m[1], up_q, Db, (int64_t)E * H, 0, 128) ||
        !mt_map(&m[2], down_q, Hb, (int64_t)E * D, 0, 128) || !mt_map(&m[3], ws + l.xq, Db, T, 1, N) ||
        !mt_map(&m[4], ws + l.hq, Hb, T, std::min<int64_t>(E, (int64_t)T * top_k), N))
        return MXFP8_ERR_DRIVER;
    if (bits == 8)
        return N == 16 ? mt_launch<8, 16>(m, p, st) : N == 32 ? mt_launch<8, 32>(m, p, st) : mt_launch<8, 64>(m, p, st);
    return N == 16 ? mt_launch<4, 16>(m, p, st) : N == 32 ? mt_launch<4, 32>(m, p, st) : mt_launch<4, 64>(m, p, st);
}
