// mxfp4_mm.cu -- block-scaled MXFP4 grouped GEMM for sm_103a on the 5th-generation tensor cores.
//
//   out[m, n] = sum_k A[m,k] W[g][n,k]  for the rows m of group g, bf16,
// A [M, K] and W [G, N, K] as packed E2M1 codes with one E8M0 scale per 32 along K in the blocked layout.
//
// A cluster of two CTAs (cta_group::2) owns a 256 x 256 output tile.  A stage is 128 bytes = 256 elements of
// K: each CTA stages its own 128 rows of A and 128 rows of B, and both halves' scale tiles (two 128 x 4 tiles
// per 128 rows); the even CTA issues four M=256 x N=256 x K=64 tcgen05.mma.kind::mxf4 per stage, each with
// two scale bytes a row (scale_vec::2X: bytes 0-1 or 2-3 of the 32-bit scale word).
//   warp 0       TMA producer (both CTAs; every copy completes on the even CTA's stage barrier)
//   warp 1       MMA issuer (even CTA)
//   warps 2-9    epilogue: tensor memory -> bf16 -> shared memory -> 32-byte row pieces
//   warp 10      scale copies, shared -> tensor memory (even CTA, both CTAs' tiles)
// Rows past a group's end are read (they are the next group's) and masked at the store; a K that is not a
// multiple of 256 multiplies only the 64-wide steps that hold any of it (a row's tail past K is TMA's zero
// fill and the scale layout's zero padding).  Every wait is bounded.
//
// At 4 bits a stage's four MMAs take 0.28 us at the nominal rate of their K = 64 form (four times bf16's; the form with
// K = 96, which is not used, has six times), so what the issuing threads do per stage decides.  8 experts, 16384 tokens,
// N = 8192, K = 5120: 249 us (5.5 PFLOP/s) with one thread issuing from a lane == 0 branch, 210 us with whole warps and an
// elected lane (mx4.cuh) and one copy for both of B's scale tiles, 204 us (6.7 PFLOP/s) with six stages instead of five.
// Four times the measured bf16 rate would be 181 us.  What is left has no single cause: with a quarter of the MMAs the same
// kernel takes 166 us, with half the operand loads 186, without its stores 195.  A serial part of every tile is the drain of
// the only accumulator, which the next tile's MMAs wait for; a second one of 256 columns does not fit beside the scale
// columns as they are, a slot for each of the six stages.  Rastering bands of 8 or 32 tiles instead of 16: 218 and 223 us.

#include "host_common.h"
#include "mx4.cuh"

namespace mx {

constexpr int kF4EpiWarps = 8;
constexpr int kF4SfWarp = 2 + kF4EpiWarps;
constexpr int kF4Threads = 96 + 32 * kF4EpiWarps;
constexpr int kF4Band = 16;  // 256-row tiles per raster band (tiles of a band share B tiles in L2)

// The group tables (three words a group) share the block's memory with the ring: six stages up to kMostGroups
// groups, five beyond.
template <int STAGES>
struct CfgF4 {
    static constexpr int kStages = STAGES;
    static constexpr int kABytes = 128 * 128;
    static constexpr int kBBytes = 128 * 128;
    static constexpr int kSfaBytes = 2 * 512;      // two scale tiles: 256 elements of K
    static constexpr int kSfbBytes = 2 * 2 * 512;  // both 128-row halves of B
    static constexpr int kTx = 2 * (kABytes + kBBytes + kSfaBytes + kSfbBytes);
    static constexpr int kSfCols = 8 + 16;
    static constexpr int kSfCol0 = 256;
    static constexpr int kTmemCols = 512;
    static_assert(kSfCol0 + kStages * kSfCols <= kTmemCols, "tensor memory overflow");
    static constexpr int kOffB = kStages * kABytes;
    static constexpr int kOffSfa = kOffB + kStages * kBBytes;
    static constexpr int kOffSfb = kOffSfa + kStages * kSfaBytes;
    static constexpr int kOffStage = kOffSfb + kStages * kSfbBytes;
    static constexpr int kOffBar = kOffStage + kF4EpiWarps * 1024;
    static constexpr int kOffTable = kOffBar + (3 * kStages + 4) * 8 + 16;
    static constexpr int kMost = 226 * 1024;  // the static variables take the last KB
    static constexpr int smem(int G) { return kOffTable + 12 * G + 1024; }
    static constexpr int kMostGroups = (kMost - smem(0)) / 12;
};
static_assert(CfgF4<6>::kMostGroups >= 256 && CfgF4<5>::kMostGroups >= MXFP8_MAX_GROUPS, "shared memory");

struct F4Params {
    const int32_t* offs;
    int32_t G;
    int64_t M, N, K;
    __nv_bfloat16* out;
    int32_t* dev_status;
    uint64_t timeout_ns;
};

// Instruction descriptor of kind::mxf4: E2M1 x E2M1, K-major, E8M0 scales, dense, K = 64.
__host__ __device__ constexpr uint32_t idesc_mxf4(uint32_t M, uint32_t N, uint32_t a_sf, uint32_t b_sf) {
    return ((b_sf & 3u) << 4) | (1u << 7) | (1u << 10) | ((N >> 3) << 17) | (1u << 23) | ((M >> 7) << 27) |
           ((a_sf & 3u) << 29);
}

struct F4Tile {
    int64_t a_row, b_row;
    int64_t sfa_chunk, sfb_chunk;     // scale tile (512 bytes) of K element 0; 128-row chunk of B
    __nv_bfloat16* out;               // first element of this CTA's 128 rows
    int valid_rows, valid_cols;
    int rows;                         // of both CTAs together
};

// Tile t seen from CTA `half` of the pair.  pt_s: 128-row padded tiles before each group (scale bands);
// tt_s: 256-row tiles before it.
__device__ __forceinline__ F4Tile f4_tile(const F4Params& p, int64_t t, int half, const int32_t* ends_s,
                                          const int32_t* pt_s, const int32_t* tt_s) {
    const int64_t nt = (p.N + 255) / 256, ct = (p.K + 127) / 128, nchunk = (p.N + 127) / 128;
    int lo = 0, hi = p.G;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if ((int64_t)tt_s[mid] * nt <= t) lo = mid + 1;
        else hi = mid;
    }
    const int g = lo - 1;
    const int64_t start = g ? ends_s[g - 1] : 0, size = ends_s[g] - start, mt = (size + 255) / 256;
    const int64_t l = t - (int64_t)tt_s[g] * nt;
    const int64_t band = l / (kF4Band * nt), bm = min64(kF4Band, mt - band * kF4Band);
    const int64_t idx = l - band * kF4Band * nt, n = idx / bm, m = band * kF4Band + (idx - n * bm);
    const int64_t rows0 = m * 256 + half * 128;
    F4Tile ti;
    ti.a_row = start + rows0;
    ti.b_row = (int64_t)g * p.N + n * 256 + half * 128;
    // clamped: rows past the group are masked (so are columns past N, whose scales are the next expert's or 0)
    ti.sfa_chunk = (pt_s[g] + min64(2 * m + half, (size + 127) / 128 - 1)) * ct;
    ti.sfb_chunk = (int64_t)g * nchunk + 2 * n;
    ti.out = p.out + ti.a_row * p.N + n * 256;
    ti.rows = (int)min64(256, size - m * 256);
    ti.valid_rows = max(0, min(128, ti.rows - half * 128));
    ti.valid_cols = (int)min64(256, p.N - n * 256);
    return ti;
}

// SHORT: groups of few rows.  A is copied in boxes of 32 rows, those that the group reaches: what stays in the rest of
// a stage meets only rows that are masked at the store.
template <int STAGES, bool SHORT>
__global__ void __launch_bounds__(kF4Threads, 1)
    mxfp4_grouped_mm_kernel(const __grid_constant__ CUtensorMap tmap_a, const __grid_constant__ CUtensorMap tmap_b,
                            const __grid_constant__ CUtensorMap tmap_sfa,
                            const __grid_constant__ CUtensorMap tmap_sfb, const F4Params p) {
    using C = CfgF4<STAGES>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ int32_t ttotal_s;
    __shared__ uint32_t tmem_base_s;
    __shared__ int abort_s;

    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
    uint64_t* empty = full + C::kStages;
    uint64_t* sfull = empty + C::kStages;
    uint64_t* tfull = sfull + C::kStages;
    uint64_t* tempty = tfull + 1;
    uint64_t* drain = tempty + 1;
    uint64_t* sfdrain = drain + 1;
    int32_t* ends_s = reinterpret_cast<int32_t*>(smem + C::kOffTable);
    int32_t* pt_s = ends_s + p.G;
    int32_t* tt_s = pt_s + p.G;

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int half = (int)(cluster_ctarank() & 1u);
    const bool leader = half == 0;

    if (warp == 0) {
        // clamped monotone ends, and the exclusive sums of each group's 128-row and 256-row tiles
        const int G = p.G, per = (G + 31) / 32, g0 = lane * per, g1 = min(G, g0 + per);
        const int32_t Mc = (int32_t)p.M;
        int32_t mx = 0;
        for (int g = g0; g < g1; ++g) mx = max(mx, min(max(p.offs[g], 0), Mc));
        int32_t incl = mx;
        for (int d = 1; d < 32; d <<= 1) {
            const int32_t o = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl = max(incl, o);
        }
        int32_t run = __shfl_up_sync(0xffffffffu, incl, 1);
        if (lane == 0) run = 0;
        int32_t prev = run, psum = 0, tsum = 0;
        for (int g = g0; g < g1; ++g) {
            const int32_t e = max(prev, min(max(p.offs[g], 0), Mc));
            ends_s[g] = e;
            psum += (e - prev + 127) / 128;
            tsum += (e - prev + 255) / 256;
            prev = e;
        }
        int32_t pi = psum, tincl = tsum;
        for (int d = 1; d < 32; d <<= 1) {
            const int32_t o = __shfl_up_sync(0xffffffffu, pi, d), q = __shfl_up_sync(0xffffffffu, tincl, d);
            if (lane >= d) {
                pi += o;
                tincl += q;
            }
        }
        int32_t pe = pi - psum, te = tincl - tsum;
        prev = run;
        for (int g = g0; g < g1; ++g) {
            const int32_t e = ends_s[g];
            pt_s[g] = pe;
            tt_s[g] = te;
            pe += (e - prev + 127) / 128;
            te += (e - prev + 255) / 256;
            prev = e;
        }
        if (lane == 31) ttotal_s = tincl;
        if (lane == 0) {
            abort_s = 0;
            prefetch_tmap(&tmap_a);
            prefetch_tmap(&tmap_b);
            prefetch_tmap(&tmap_sfa);
            prefetch_tmap(&tmap_sfb);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            for (int s = 0; s < C::kStages; ++s) {
                mbar_init(&full[s], 1);
                mbar_init(&empty[s], 1);
                mbar_init(&sfull[s], 1);
            }
            mbar_init(tfull, 1);
            mbar_init(tempty, 2 * kF4EpiWarps);  // every epilogue warp of both CTAs
            mbar_init(drain, 1);
            mbar_init(sfdrain, 1);
            fence_barrier_init();
        }
        __syncwarp();
        tmem_alloc_pair(&tmem_base_s, C::kTmemCols);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // the peer may signal this CTA's barriers from here on
    tc_fence_after();

    const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_base_s, 0);
    const uint32_t ring = __shfl_sync(0xffffffffu, smem_u32(smem), 0);
    volatile int* abort_flag = &abort_s;
    const int64_t ntiles = (int64_t)__shfl_sync(0xffffffffu, ttotal_s, 0) * ((p.N + 255) / 256);
    const int64_t cid = blockIdx.x >> 1, ncl = gridDim.x >> 1;
    const int k_tiles = (int)((p.K + 255) / 256);
    // a wait by a whole warp that goes on, or gives up, together
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, mbar_wait_bounded<true>(bar, parity, p.timeout_ns, abort_flag, p.dev_status));
    };

    if (warp == 0) {
        // ------------------------------------------------ TMA producer (both CTAs)
        const uint32_t one = elect_one();
        int stage = 0;
        uint32_t phase = 0, issued = 0, last_phase = 0;
        bool ok = true;
        for (int64_t t = cid; t < ntiles && ok; t += ncl) {
            const F4Tile ti = f4_tile(p, t, half, ends_s, pt_s, tt_s);
            const int32_t a_row = __shfl_sync(0xffffffffu, (int32_t)ti.a_row, 0);
            const int32_t b_row = __shfl_sync(0xffffffffu, (int32_t)ti.b_row, 0);
            const int32_t sfa = __shfl_sync(0xffffffffu, (int32_t)(2 * ti.sfa_chunk), 0);
            const int32_t sfb = __shfl_sync(0xffffffffu, (int32_t)ti.sfb_chunk, 0);
            int boxes = 0;  // 32-row boxes of this CTA's A
            uint32_t tx = C::kTx;
            if constexpr (SHORT) {
                const int rows = __shfl_sync(0xffffffffu, ti.rows, 0), even = (min(rows, 128) + 31) / 32,
                          odd = (max(rows - 128, 0) + 31) / 32;
                boxes = leader ? even : odd;
                tx -= (8 - even - odd) * (32 * 128);
            }
            for (int kt = 0; kt < k_tiles; ++kt) {
                if (!wait(&empty[stage], phase ^ 1u)) {
                    ok = false;
                    break;
                }
                const uint32_t fb = cluster_addr(&full[stage], 0);
                if (leader) expect_tx(one, &full[stage], tx);
                if constexpr (SHORT) {
                    for (int i = 0; i < boxes; ++i)
                        load_2d_pair(one, ring + stage * C::kABytes + i * (32 * 128), &tmap_a, kt * 128, a_row + 32 * i, fb);
                } else {
                    load_2d_pair(one, ring + stage * C::kABytes, &tmap_a, kt * 128, a_row, fb);
                }
                load_2d_pair(one, ring + C::kOffB + stage * C::kBBytes, &tmap_b, kt * 128, b_row, fb);
                // two scale tiles a copy (an odd count's last copy reads one tile further, which nothing uses)
                load_2d_pair(one, ring + C::kOffSfa + stage * C::kSfaBytes, &tmap_sfa, 0, sfa + 4 * kt, fb);
                load_3d_pair(one, ring + C::kOffSfb + stage * C::kSfbBytes, &tmap_sfb, 0, 4 * kt, sfb, fb);
                issued |= 1u << stage;
                last_phase = (last_phase & ~(1u << stage)) | (phase << stage);
                if (++stage == C::kStages) { stage = 0; phase ^= 1u; }
            }
        }
        if (!ok && leader) {  // given up: let the copies in flight land before the pair exits
            volatile int no_abort = 0;
            for (int s = 0; s < C::kStages; ++s)
                if (issued & (1u << s))
                    mbar_wait_bounded<true>(&full[s], (last_phase >> s) & 1u, p.timeout_ns, &no_abort, nullptr);
        }
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer (even CTA)
        if (leader) {
            const uint32_t one = elect_one();
            int stage = 0;
            uint32_t phase = 0, acc_phase = 0;
            bool ok = true;
            constexpr uint32_t idesc0 = idesc_mxf4(256, 256, 0, 0);
            for (int64_t t = cid; t < ntiles && ok; t += ncl) {
                if (!wait(tempty, acc_phase ^ 1u)) break;
                tc_fence_after();
                for (int kt = 0; kt < k_tiles; ++kt) {
                    if (!wait(&full[stage], phase) || !wait(&sfull[stage], phase)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sf = tmem + C::kSfCol0 + stage * C::kSfCols;
                    const uint32_t a_s = ((ring + stage * C::kABytes) >> 4) | kDescLbo;
                    const uint32_t b_s = ((ring + C::kOffB + stage * C::kBBytes) >> 4) | kDescLbo;
                    auto mma = [&](int k, uint32_t acc) {
                        const uint32_t id = (uint32_t)(k & 1) * 2;  // scale bytes 0-1 or 2-3 of the word
                        mma_pair_mxf4(one, tmem, desc_of(a_s + 2 * k, kDescTile), desc_of(b_s + 2 * k, kDescTile),
                                      idesc0 | (id << 4) | (id << 29), sf + 4 * (k >> 1), sf + 8 + 8 * (k >> 1), acc);
                    };
                    if ((int64_t)(kt + 1) * 256 <= p.K) {
                        mma(0, kt != 0);
                        mma(1, 1u);
                        mma(2, 1u);
                        mma(3, 1u);
                    } else {  // the contraction's last elements
                        const int steps = (int)((p.K - (int64_t)kt * 256 + 63) / 64);
                        mma(0, kt != 0);
                        if (steps > 1) mma(1, 1u);
                        if (steps > 2) mma(2, 1u);
                        if (steps > 3) mma(3, 1u);
                    }
                    commit_pair(one, &empty[stage], 0x3);
                    if (++stage == C::kStages) { stage = 0; phase ^= 1u; }
                }
                if (!ok) break;
                commit_pair(one, tfull, 0x3);
                acc_phase ^= 1u;
            }
            // all tensor-core work of the pair is done before the columns are freed
            commit_pair(one, drain, 0x1);
            volatile int no_abort = 0;
            mbar_wait_bounded<true>(drain, 0, p.timeout_ns, &no_abort, p.dev_status);
        }
    } else if (warp == kF4SfWarp) {
        // ------------------------------------------------ scale copies (even CTA)
        if (leader) {
            const uint32_t one = elect_one();
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int64_t t = cid; t < ntiles && ok; t += ncl) {
                for (int kt = 0; kt < k_tiles; ++kt) {
                    if (!wait(&full[stage], phase)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sf = tmem + C::kSfCol0 + stage * C::kSfCols;
                    const uint32_t sa = (ring + C::kOffSfa + stage * C::kSfaBytes) >> 4;
                    const uint32_t sb = (ring + C::kOffSfb + stage * C::kSfbBytes) >> 4;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        cp_scales_pair(one, sf + 4 * h, desc_of(sa + 32 * h, kDescScale));
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            cp_scales_pair(one, sf + 8 + 8 * h + 4 * j, desc_of(sb + 64 * j + 32 * h, kDescScale));
                    }
                    commit_pair(one, &sfull[stage], 0x1);
                    if (++stage == C::kStages) { stage = 0; phase ^= 1u; }
                }
            }
            commit_pair(one, sfdrain, 0x1);
            volatile int no_abort = 0;
            mbar_wait_bounded<true>(sfdrain, 0, p.timeout_ns, &no_abort, p.dev_status);
        }
    } else if (warp >= 2) {
        // ------------------------------------------------ epilogue (both CTAs: own 128 rows)
        // Warp w drains lane quarter w % 4 and column half (w - 2) / 4.
        const int quarter = warp & 3;
        const int c_base = ((warp - 2) >> 2) * 128;
        uint8_t* stg = smem + C::kOffStage + (warp - 2) * 1024;  // 32 rows x 32 bytes
        const uint32_t tempty_leader = cluster_addr(tempty, 0);
        uint32_t acc_phase = 0;
        for (int64_t t = cid; t < ntiles; t += ncl) {
            const F4Tile ti = f4_tile(p, t, half, ends_s, pt_s, tt_s);
            __nv_bfloat16* wout = ti.out + (int64_t)(quarter * 32) * p.N + c_base;
            const int vrows = ti.valid_rows - quarter * 32;
            const int vcols = ti.valid_cols - c_base;
            if (!mbar_wait_bounded<true>(tfull, acc_phase, p.timeout_ns, abort_flag, p.dev_status)) break;
            acc_phase ^= 1u;
            tc_fence_after();
            uint32_t packed[64];
            const uint32_t taddr = tmem + ((uint32_t)(quarter * 32) << 16) + c_base;
#pragma unroll
            for (int c = 0; c < 128; c += 64) {
                uint32_t v0[32], v1[32];
                tmem_ld_32x32b_x32(taddr + c, v0);
                tmem_ld_32x32b_x32(taddr + c + 32, v1);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    packed[c / 2 + i] = pack_bf16x2(__uint_as_float(v0[2 * i]), __uint_as_float(v0[2 * i + 1]));
                    packed[c / 2 + 16 + i] = pack_bf16x2(__uint_as_float(v1[2 * i]), __uint_as_float(v1[2 * i + 1]));
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster_relaxed(tempty_leader);
            // 16 columns a pass: lane = row parks two 16-byte pieces (order flipped every 4 rows: no bank
            // conflicts), then two lanes a row store whole 32-byte pieces of 16 rows per instruction
#pragma unroll
            for (int ch = 0; ch < 8; ++ch) {
                if (ch * 16 >= vcols) break;
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    st_shared_v4(stg + lane * 32 + ((j ^ ((lane >> 2) & 1)) * 16),
                                 make_uint4(packed[ch * 8 + 4 * j], packed[ch * 8 + 4 * j + 1],
                                            packed[ch * 8 + 4 * j + 2], packed[ch * 8 + 4 * j + 3]));
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int rl = (lane >> 1) + 16 * i, piece = lane & 1;
                    const uint4 val = ld_shared_v4(stg + rl * 32 + ((piece ^ ((rl >> 2) & 1)) * 16));
                    if (rl < vrows && ch * 16 + piece * 8 < vcols)
                        *reinterpret_cast<uint4*>(wout + (int64_t)rl * p.N + ch * 16 + piece * 8) = val;
                }
                __syncwarp();
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // neither CTA frees tensor memory or exits while the pair still works
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, C::kTmemCols);
    }
}

// ---------------------------------------------------------------- host side
// uint8 [planes][rows][cols], boxes of box_planes x box_rows x box_cols bytes.
static bool f4_map(CUtensorMap* m, const void* base, int64_t rows, int64_t cols, int box_rows, int box_cols,
                   bool swizzle, int64_t planes = 1, int box_planes = 1) {
    host::EncodeTiledFn fn = host::encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)planes};
    cuuint64_t strides[2] = {(cuuint64_t)cols, (cuuint64_t)(cols * rows)};
    cuuint32_t box[3] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows, (cuuint32_t)box_planes};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, box_planes > 1 ? 3 : 2, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int STAGES, bool SHORT>
static mxfp8_status_t f4_launch(const CUtensorMap& ma, const CUtensorMap& mb, const CUtensorMap& msa,
                                const CUtensorMap& msb, const F4Params& p, int clusters, cudaStream_t st) {
    using C = CfgF4<STAGES>;
    static std::atomic<int> attr_set[host::kMaxDevices];
    if (!host::ensure_smem(reinterpret_cast<const void*>(mxfp4_grouped_mm_kernel<STAGES, SHORT>), C::kMost, attr_set))
        return MXFP8_ERR_LAUNCH;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(2 * (unsigned)clusters);
    cfg.blockDim = dim3(kF4Threads);
    cfg.dynamicSmemBytes = C::smem(p.G);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, mxfp4_grouped_mm_kernel<STAGES, SHORT>, ma, mb, msa, msb, p) != cudaSuccess) {
        cudaGetLastError();
        return MXFP8_ERR_LAUNCH;
    }
    return host::last_launch_status();
}

}  // namespace mx

using namespace mx;

extern "C" mxfp8_status_t mxfp4_grouped_mm_fwd(const void* a_q, const void* a_s, const void* w_q, const void* w_s,
                                               const int32_t* offs, int32_t G, int64_t M, int64_t N, int64_t K,
                                               void* out_bf16, int32_t* dev_status, mxfp8_stream_t stream) {
    if (!offs || !w_q || !w_s) return MXFP8_ERR_NULL;
    if (G < 1 || G > MXFP8_MAX_GROUPS || M < 0 || N <= 0 || K <= 0 || M > INT32_MAX || K > INT32_MAX ||
        (int64_t)G * N > INT32_MAX)
        return MXFP8_ERR_SHAPE;
    if (K % 32 || N % 32) return MXFP8_ERR_ALIGN;
    if (M == 0) return MXFP8_OK;  // empty tensors may have no address
    if (!a_q || !a_s || !out_bf16) return MXFP8_ERR_NULL;
    const void* ptrs[] = {a_q, a_s, w_q, w_s, out_bf16};
    for (const void* q : ptrs)
        if (!host::aligned16(q)) return MXFP8_ERR_ALIGN;
    const int64_t ct = (K + 127) / 128;
    const int64_t sfa_rows = ((M + 127) / 128 + G) * ct * 2, sfb_rows = (int64_t)G * ((N + 127) / 128) * ct * 2;
    if (sfa_rows > INT32_MAX - 4 || sfb_rows > INT32_MAX - 4) return MXFP8_ERR_SHAPE;  // TMA coordinates
    if (mxfp8_status_t a = host::check_arch(); a != MXFP8_OK) return a;
    // Groups of 64 rows and less on average: 16 groups of one row, N = 2048, K = 7168 take 30 us in place of 36, others the
    // same time; for longer ones the count of boxes costs the issuing warp 2%.
    const bool few = M <= 64 * (int64_t)G;
    CUtensorMap ma, mb, msa, msb;
    if (!f4_map(&ma, a_q, M, K / 2, few ? 32 : 128, 128, true) || !f4_map(&mb, w_q, (int64_t)G * N, K / 2, 128, 128, true) ||
        !f4_map(&msa, a_s, sfa_rows, 256, 4, 256, false) || !f4_map(&msb, w_s, ct * 2, 256, 4, 256, false, (int64_t)G * ((N + 127) / 128), 2))
        return MXFP8_ERR_DRIVER;
    F4Params p{};
    p.offs = offs;
    p.G = G;
    p.M = M;
    p.N = N;
    p.K = K;
    p.out = static_cast<__nv_bfloat16*>(out_bf16);
    p.dev_status = dev_status;
    p.timeout_ns = 2000000000ull;
    const int64_t bound = ((M + 255) / 256 + G) * ((N + 255) / 256);
    const int clusters = (int)max64(1, min64(bound, host::num_sms() / 2));
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (G > CfgF4<6>::kMostGroups)
        return few ? f4_launch<5, true>(ma, mb, msa, msb, p, clusters, st)
                   : f4_launch<5, false>(ma, mb, msa, msb, p, clusters, st);
    return few ? f4_launch<6, true>(ma, mb, msa, msb, p, clusters, st)
               : f4_launch<6, false>(ma, mb, msa, msb, p, clusters, st);
}
