// moe_token_rows.cu -- the routed SwiGLU layer for 1 .. 8 tokens (see moe_tokens.cu for the formulas): every CTA computes
// whole rows, so that no partial sums are exchanged between CTAs.
//
// For a token or two the layer is a stream of weights and a few waits, and the waits decide: adding up tiles that two
// CTAs share costs two trips through L2 under full load, twice a layer.  Here each CTA owns an equal run of rows over
// their whole contraction -- first rows h of the active experts' gate and up matrices, then rows d of the down matrices,
// over all active experts -- and its 16 warps split the contraction.  One grid-wide point is left (h is complete), and
// the down weights are already in flight while the grid gathers there.
//
//   warp 16     weight producer: a stage is 16 rows (8 of gate and the same 8 of up; or 16 of down) times up to 2 KB of
//               each, contiguous in memory: 16 bulk copies into padded rows
//   warps 0-15  a 128-byte slice of the stage's rows each (the slices move on from stage to stage): ldmatrix, two codes
//               to an f16 pair (exact), m16n8k16 tensor-core products of a 32-block with the 8 token columns, the
//               block's scales applied to its fp32 sum
// The row-wise layout of the f16 fragments puts gate row g and up row g into one lane, so SwiGLU needs no exchange.
// x (first) and the routed h (after the grid-wide point) are quantized by every CTA for itself into shared memory, as
// f16 element values and fp32 block scales.  The legacy tensor instruction is the right one here: it takes the
// weights from registers, where a 16-row tile of any rows can be put together, and its rate is not what bounds.

#include "moe_tokens.cuh"

namespace mx {

constexpr int kRwTokens = 8;
constexpr int kRwWarps = 16;
constexpr int kRwConsumers = kRwWarps * 32;
constexpr int kRwThreads = kRwConsumers + 32;
constexpr int kRwSeg = 2048;           // bytes of a row in a stage, at most
constexpr int kRwPitch = kRwSeg + 16;  // ldmatrix reads 8 rows from different banks
constexpr int kRwStage = 16 * kRwPitch;
constexpr int kRwPairs = kRwTokens * kMtMaxTopK;
constexpr int kRwMost = 32768;         // values of x, and of the routed h, that shared memory holds
constexpr int kRwAhead = 4;            // stages ahead whose scale words are loaded

struct RwLayout {  // dynamic shared memory, in bytes from its (128-byte aligned) start
    int pitch_x, pitch_h;  // f16 values of one token's x / one pair's h, in bytes
    int vals, fx, red, ring, stages, total;
};

__host__ __device__ inline int rw_pitch(int n) { return n * 2 % 128 == 0 ? n * 2 + 64 : n * 2; }

__host__ __device__ inline RwLayout rw_layout(int T, int pairs, int D, int H) {
    RwLayout l;
    l.pitch_x = rw_pitch(D);
    l.pitch_h = rw_pitch(H);
    const int v = T * l.pitch_x > pairs * l.pitch_h ? T * l.pitch_x : pairs * l.pitch_h;
    const int f = 4 * (T * (D / 32) > pairs * (H / 32) ? T * (D / 32) : pairs * (H / 32));
    l.vals = 0;
    l.fx = (v + 127) / 128 * 128;
    l.red = l.fx + (f + 127) / 128 * 128;
    l.ring = l.red + 2 * kRwWarps * 16 * T * 4;
    const int room = 226 * 1024 - 14 * 1024 - 128 - l.ring;
    l.stages = room / kRwStage;
    if (l.stages > 6) l.stages = 6;
    l.total = l.ring + l.stages * kRwStage + 128;
    return l;
}

__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Two E4M3 codes (half h of w) as an f16 pair, exactly.
template <int h>
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t w) {
    uint32_t r;
    if constexpr (h == 0)
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}" : "=r"(r) : "r"(w));
    else
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, b;\n\t}" : "=r"(r) : "r"(w));
    return r;
}
// Eight E2M1 codes as four f16 pairs, exactly.
__device__ __forceinline__ void e2m1x8_f16(uint32_t w, uint32_t (&r)[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
        : "r"(w));
}
// Block b's scale out of a word of four: 2^(byte - 127); byte 0xFF gives Inf (the caller sees to it that NaN comes out).
template <int b>
__device__ __forceinline__ float word_scale(uint32_t w) {
    const uint32_t v = (b < 3 ? w << (23 - 8 * b) : w >> 1) & 0x7F800000u;
    return __uint_as_float(max(v, 0x00400000u));
}
__device__ __forceinline__ bool has_ff(uint32_t w) { return (((w & 0x7F7F7F7Fu) + 0x01010101u) & w & 0x80808080u) != 0; }

__device__ __forceinline__ void rows_sync() {
    __syncwarp();
    asm volatile("bar.sync 1, 512;" ::: "memory");
}

// A thread's eight values of a block shared by four lanes -> f16 element values (packed pairs) and the block's scale.
template <int BITS>
__device__ __forceinline__ float quant8_f16(const float (&v)[8], uint32_t (&q)[4]) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7FFFFFFFu);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const uint32_t s = e8m0_of<BITS == 8 ? 8 : 2>(m);
    if (s == 0xFFu) {  // the scale is NaN; the elements must not be 0
#pragma unroll
        for (int j = 0; j < 4; ++j) q[j] = 0x3C003C00u;
        return e8m0_value(s);
    }
    const float f = __uint_as_float((254u - s) << 23);
    float z[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) z[j] = v[j] * f;
    if constexpr (BITS == 8) {
#pragma unroll
        for (int j = 0; j < 4; ++j) q[j] = e4m3x2_f16x2<0>(cvt_e4m3x2(z[2 * j], z[2 * j + 1]));
    } else {
        e2m1x8_f16(cvt_e2m1x8(z), q);
    }
    return e8m0_value(s);
}

template <int BITS>
__global__ void __launch_bounds__(kRwThreads, 1) moe_token_rows_kernel(const MtParams p) {
    constexpr int kBlkBytes = 32 * BITS / 8;       // bytes of a 32-block
    constexpr int kSliceBlk = 128 / kBlkBytes;     // blocks of a warp's slice
    constexpr int kWords = kSliceBlk / 4;          // scale words of a slice, per row
    extern __shared__ __align__(128) uint8_t smem_raw[];
    __shared__ MtRoute route;
    __shared__ __align__(8) uint64_t full[6], empty[6];
    __shared__ int8_t pair_s[kRwPairs][kRwTokens];  // (active expert, token) -> routed pair t * top_k + j, or -1
    __shared__ int abort_s;
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int T = p.T, D = (int)p.D, H = (int)p.H, top_k = p.top_k;
    const RwLayout l = rw_layout(T, T * top_k, D, H);
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
    float* fx = reinterpret_cast<float*>(smem + l.fx);
    float* red = reinterpret_cast<float*>(smem + l.red);
    uint8_t* ring = smem + l.ring;
    volatile int* abort_flag = &abort_s;
    const int n_h = H / 32, n_d = D / 32;  // 32-blocks of a contraction

    if (warp < 4) {
        for (int i = tid; i < kRwPairs * kRwTokens; i += kMtRouteThreads) (&pair_s[0][0])[i] = -1;
        mt_route(p, reinterpret_cast<uint32_t*>(ring), route, tid, [] {});
        route_sync();
        for (int i = tid; i < T * top_k; i += kMtRouteThreads) {
            const int e = route.sel_e[i];
            if (e == 0xFFFF) continue;
            int a = 0;  // the expert's place among the active (few)
            while (route.list[a] != e) ++a;
            pair_s[a][i / top_k] = (int8_t)i;
        }
    } else if (warp < kRwWarps) {
        const int items = T * (D / 8);
        for (int i0 = tid - lane - 128; i0 < items; i0 += kRwConsumers - 128) {
            const int i = i0 + lane, t = i < items ? i / (D / 8) : 0, c = i < items ? (i - t * (D / 8)) * 8 : 0;
            uint4 u = make_uint4(0, 0, 0, 0);
            if (i < items) u = *reinterpret_cast<const uint4*>(p.x + (int64_t)i * 16);
            const float v[8] = {bf16lo(u.x), bf16hi(u.x), bf16lo(u.y), bf16hi(u.y),
                                bf16lo(u.z), bf16hi(u.z), bf16lo(u.w), bf16hi(u.w)};
            uint32_t q[4];
            const float s = quant8_f16<BITS>(v, q);
            if (i < items) {
                *reinterpret_cast<uint4*>(smem + t * l.pitch_x + c * 2) = make_uint4(q[0], q[1], q[2], q[3]);
                if ((lane & 3) == 0) fx[t * n_d + c / 32] = s;
            }
        }
    } else if (lane == 0) {
        for (int s = 0; s < l.stages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], kRwWarps);
        }
        abort_s = 0;
        fence_barrier_init();
    }
    fence_proxy_async();  // the routing's scratch memory is the ring's from here on
    __syncthreads();

    const int A = __shfl_sync(0xffffffffu, route.active_n, 0);
    const uint32_t cta = blockIdx.x, n = gridDim.x;
    const uint32_t rows1 = (uint32_t)A * H;
    const uint32_t r1_0 = (uint32_t)((uint64_t)cta * rows1 / n), r1_1 = (uint32_t)((uint64_t)(cta + 1) * rows1 / n);
    const uint32_t r2_0 = (uint32_t)((uint64_t)cta * D / n), r2_1 = (uint32_t)((uint64_t)(cta + 1) * D / n);
    const uint32_t Db = D * BITS / 8, Hb = H * BITS / 8;  // bytes of a row
    // segments of a row: equal, whole slices, at most kRwSeg bytes
    const uint32_t ns1 = (Db + kRwSeg - 1) / kRwSeg, ns2 = (Hb + kRwSeg - 1) / kRwSeg;
    const uint32_t seg1 = ((Db + ns1 - 1) / ns1 + 127) / 128 * 128, seg2 = ((Hb + ns2 - 1) / ns2 + 127) / 128 * 128;
    const uint32_t g1 = (r1_1 - r1_0 + 7) / 8, g2 = (r2_1 - r2_0 + 15) / 16;  // groups of rows
    const uint32_t st1 = g1 * ns1, st2 = g2 * A * ns2;                        // stages
    const uint32_t ct_d = (D + 127) / 128, ct_h = (H + 127) / 128;

    if (A == 0) {
        for (int64_t i = (int64_t)cta * kRwThreads + tid; i < (int64_t)T * D; i += (int64_t)n * kRwThreads)
            p.y[i] = __float2bfloat16(0.0f);
    } else if (warp == kRwWarps) {
        // ------------------------------------------------ weight producer: lanes 0-15 a row each
        uint32_t stage = 0, phase = 0;
        auto issue = [&](const uint8_t* src, bool valid, uint32_t rows, uint32_t bytes) -> bool {
            if (!__all_sync(0xffffffffu,
                            mbar_wait_bounded<true>(&empty[stage], phase ^ 1u, p.timeout_ns, abort_flag, p.dev_status)))
                return false;
            if (lane == 0) mbar_arrive_expect_tx(&full[stage], rows * bytes);
            __syncwarp();
            if (valid) bulk_load(ring + stage * kRwStage + lane * kRwPitch, src, bytes, &full[stage]);
            if (++stage == (uint32_t)l.stages) {
                stage = 0;
                phase ^= 1u;
            }
            return true;
        };
        bool ok = true;
        for (uint32_t g = 0; g < g1 && ok; ++g) {
            const uint32_t left = min(8u, r1_1 - r1_0 - 8 * g), r = r1_0 + 8 * g + (lane & 7);
            const bool valid = lane < 16 && (lane & 7) < left;
            const uint32_t a = valid ? r / H : 0, h = valid ? r - a * H : 0, e = route.list[a];
            const uint8_t* src = (lane < 8 ? p.q_gate : p.q_up) + ((int64_t)e * H + h) * Db;
            for (uint32_t s = 0; s < ns1 && ok; ++s)
                ok = issue(src + s * seg1, valid, 2 * left, min(seg1, Db - s * seg1));
        }
        for (uint32_t g = 0; g < g2 && ok; ++g) {
            const uint32_t left = min(16u, r2_1 - r2_0 - 16 * g), d = r2_0 + 16 * g + lane;
            const bool valid = lane < left;
            for (int a = 0; a < A && ok; ++a) {
                const uint8_t* src = p.q_down + ((int64_t)route.list[a] * D + (valid ? d : 0)) * Hb;
                for (uint32_t s = 0; s < ns2 && ok; ++s)
                    ok = issue(src + s * seg2, valid, left, min(seg2, Hb - s * seg2));
            }
        }
    } else {
        const int g = lane >> 2, q = lane & 3;  // fragment row (and token column of B), fragment quarter
        uint32_t stage = 0, phase = 0;
        // which slice of a stage is this warp's: slices are dealt on from stage to stage
        uint32_t dealt = 0;
        auto my_slice = [&](uint32_t bytes, uint32_t& at) -> uint32_t {
            const uint32_t s = (warp + kRwWarps - at) & (kRwWarps - 1);
            at = (at + (bytes + 127) / 128) & (kRwWarps - 1);
            return s;
        };
        // The scale words of a slice for fragment rows g and g + 8.
        struct Scales {
            uint32_t lo[kWords], hi[kWords];
        };
        auto load_scales = [&](Scales& sc, const uint8_t* lo, const uint8_t* hi, uint32_t at_byte, uint32_t ct, bool mine) {
#pragma unroll
            for (int w = 0; w < kWords; ++w) {
                const uint32_t kt = at_byte / (4 * kBlkBytes) + w;
                sc.lo[w] = sc.hi[w] = 0;
                if (mine && kt < ct) {
                    sc.lo[w] = __ldg(reinterpret_cast<const uint32_t*>(lo + (int64_t)kt * 512));
                    sc.hi[w] = __ldg(reinterpret_cast<const uint32_t*>(hi + (int64_t)kt * 512));
                }
            }
        };
        // c += the slice's products: blocks k0 .. of `blocks`, values of token column g at vb, block scales of token
        // columns 2q and 2q + 1 at f0, f1
        auto slice = [&](float (&c)[4], const Scales& sc, uint32_t at, uint32_t k0, uint32_t blocks, const uint8_t* vb,
                         const float* f0, const float* f1) {
            const uint32_t base = smem_u32(ring) + stage * kRwStage + at;
            const uint32_t row = ((lane >> 3) & 1) * 8 + (lane & 7);
            bool bad_lo = false, bad_hi = false;
#pragma unroll
            for (int w = 0; w < kWords; ++w) {
                bad_lo |= has_ff(sc.lo[w]);
                bad_hi |= has_ff(sc.hi[w]);
            }
            auto block = [&](auto bc, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t a4, uint32_t a5,
                             uint32_t a6, uint32_t a7, uint4 b) {
                constexpr int i = decltype(bc)::value;
                float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                mma_f16(d, a0, a1, a2, a3, b.x, b.y);
                mma_f16(d, a4, a5, a6, a7, b.z, b.w);
                const float wl = word_scale<i & 3>(sc.lo[i >> 2]), wh = word_scale<i & 3>(sc.hi[i >> 2]);
                const float x0 = f0[k0 + i], x1 = f1[k0 + i];
                c[0] += d[0] * x0 * wl;
                c[1] += d[1] * x1 * wl;
                c[2] += d[2] * x0 * wh;
                c[3] += d[3] * x1 * wh;
            };
            auto one = [&](auto bc) {
                constexpr int i = decltype(bc)::value;
                if constexpr (BITS == 8) {
                    if (k0 + i >= blocks) return;
                    uint32_t r[4];  // rows 0-7 and 8-15 of bytes 0-15, then of bytes 16-31
                    ldmatrix_x4(r, base + row * kRwPitch + 32 * i + (lane >> 4) * 16);
                    const uint8_t* v = vb + (k0 + i) * 64 + q * 8;
                    const uint2 lo = *reinterpret_cast<const uint2*>(v), hi = *reinterpret_cast<const uint2*>(v + 32);
                    block(bc, e4m3x2_f16x2<0>(r[0]), e4m3x2_f16x2<0>(r[1]), e4m3x2_f16x2<1>(r[0]), e4m3x2_f16x2<1>(r[1]),
                          e4m3x2_f16x2<0>(r[2]), e4m3x2_f16x2<0>(r[3]), e4m3x2_f16x2<1>(r[2]), e4m3x2_f16x2<1>(r[3]),
                          make_uint4(lo.x, lo.y, hi.x, hi.y));
                } else {
                    if constexpr ((i & 1) == 0) {
                        if (k0 + i >= blocks) return;
                        uint32_t r[4], lo[4], hi[4];  // rows 0-7 and 8-15 of this block, then of the next
                        ldmatrix_x4(r, base + row * kRwPitch + 16 * i + (lane >> 4) * 16);
                        e2m1x8_f16(r[0], lo);
                        e2m1x8_f16(r[1], hi);
                        block(bc, lo[0], hi[0], lo[1], hi[1], lo[2], hi[2], lo[3], hi[3],
                              *reinterpret_cast<const uint4*>(vb + (k0 + i) * 64 + q * 16));
                        if (k0 + i + 1 >= blocks) return;
                        e2m1x8_f16(r[2], lo);
                        e2m1x8_f16(r[3], hi);
                        block(std::integral_constant<int, i + 1>{}, lo[0], hi[0], lo[1], hi[1], lo[2], hi[2], lo[3], hi[3],
                              *reinterpret_cast<const uint4*>(vb + (k0 + i + 1) * 64 + q * 16));
                    }
                }
            };
            one(std::integral_constant<int, 0>{});
            if constexpr (BITS == 8) one(std::integral_constant<int, 1>{});
            one(std::integral_constant<int, 2>{});
            if constexpr (BITS == 8) one(std::integral_constant<int, 3>{});
            if constexpr (kSliceBlk > 4) {
                one(std::integral_constant<int, 4>{});
                one(std::integral_constant<int, 6>{});
            }
            if (bad_lo) c[0] = c[1] = __uint_as_float(0x7FC00000u);
            if (bad_hi) c[2] = c[3] = __uint_as_float(0x7FC00000u);
        };
        auto land = [&] { mbar_wait_bounded<true>(&full[stage], phase, p.timeout_ns, abort_flag, p.dev_status); };
        auto next_stage = [&] {
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[stage]);
            if (++stage == (uint32_t)l.stages) {
                stage = 0;
                phase ^= 1u;
            }
        };
        // the 16 warps' sums of a fragment, by row and token
        auto park = [&](float* to, const float (&c)[4]) {
            float* w = to + warp * 16 * T;
            if (2 * q < T) {
                w[2 * q * 16 + g] = c[0];
                w[2 * q * 16 + g + 8] = c[2];
            }
            if (2 * q + 1 < T) {
                w[(2 * q + 1) * 16 + g] = c[1];
                w[(2 * q + 1) * 16 + g + 8] = c[3];
            }
        };
        auto added = [&](const float* from, int t, int row) -> float {
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < kRwWarps; ++w) s += from[(w * T + t) * 16 + row];
            return s;
        };
        const int tg = min(g, T - 1), t0 = min(2 * q, T - 1), t1 = min(2 * q + 1, T - 1);
        float* hbuf = p.part;  // fp32 h of the routed pairs [T * top_k][H]
        int parity = 0;

        // ------------------------------------------------ first half: rows of gate and up
        {
            // a place in the sequence of stages, for the scale words that are loaded ahead of the weights
            uint32_t fg = 0, fs = 0, fdealt = 0;
            const uint8_t *flo = nullptr, *fhi = nullptr;
            auto fetch = [&](Scales& sc) {
                if (fg >= g1) return;
                if (fs == 0) {
                    const uint32_t r = min(r1_0 + 8 * fg + g, r1_1 - 1), a = r / H, h = r - a * H;
                    const int64_t so = ((int64_t)route.list[a] * ct_h + (h >> 7)) * ct_d * 512 + (h & 31) * 16 + ((h >> 5) & 3) * 4;
                    flo = p.s_gate + so;
                    fhi = p.s_up + so;
                }
                const uint32_t bytes = min(seg1, Db - fs * seg1), s = my_slice(bytes, fdealt);
                load_scales(sc, flo, fhi, fs * seg1 + s * 128, ct_d, s * 128 < bytes);
                if (++fs == ns1) {
                    fs = 0;
                    ++fg;
                }
            };
            Scales sc[kRwAhead];
#pragma unroll
            for (int i = 0; i < kRwAhead; ++i) fetch(sc[i]);
            const uint8_t* vb = smem + tg * l.pitch_x;
            const float *f0 = fx + t0 * n_d, *f1 = fx + t1 * n_d;
            float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            uint32_t gr = 0, s = 0;
            for (uint32_t i = 0; i < st1; i += kRwAhead) {
#pragma unroll
                for (int j = 0; j < kRwAhead; ++j) {
                    if (i + j >= st1) break;
                    const uint32_t bytes = min(seg1, Db - s * seg1), sl = my_slice(bytes, dealt);
                    land();
                    if (sl * 128 < bytes)
                        slice(c, sc[j], sl * 128, (s * seg1 + sl * 128) / kBlkBytes, n_d, vb, f0, f1);
                    next_stage();
                    fetch(sc[j]);
                    if (++s < ns1) continue;
                    s = 0;
                    // the group's rows are complete
                    float* to = red + parity * kRwWarps * 16 * T;
                    parity ^= 1;
                    park(to, c);
                    c[0] = c[1] = c[2] = c[3] = 0.0f;
                    rows_sync();
                    if (tid < 8 * T) {
                        const int t = tid >> 3, row = tid & 7;
                        const uint32_t r = r1_0 + 8 * gr + row;
                        if (r < r1_1) {
                            const uint32_t a = r / H, pr = (uint32_t)(int)pair_s[a][t];
                            if ((int)pr >= 0) {
                                const float x1 = added(to, t, row), x3 = added(to, t, row + 8);
                                hbuf[(int64_t)pr * H + (r - a * H)] = x1 / (1.0f + expf(-x1)) * x3;
                            }
                        }
                    }
                    ++gr;
                }
            }
        }
        // ------------------------------------------------ h is complete: every CTA quantizes it for itself
        rows_sync();  // this CTA's h is written, and nobody reads x any more
        if (tid == 0) {
            __threadfence();
            atomicAdd(p.header + kMtHDone, 1u);
            if (r2_0 < r2_1) mt_grid_wait(p, kMtHDone, abort_flag);
        }
        rows_sync();
        if (r2_0 < r2_1) {
            const int items = T * top_k * (H / 8);
            for (int i0 = tid - lane; i0 < items; i0 += kRwConsumers) {
                const int i = i0 + lane, pr = i < items ? i / (H / 8) : 0, k = i < items ? (i - pr * (H / 8)) * 8 : 0;
                float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
                if (i < items) {  // an unused pair's values are never multiplied into a result
                    const float4* h = reinterpret_cast<const float4*>(hbuf + (int64_t)pr * H + k);
                    const float4 a = __ldcg(h), b = __ldcg(h + 1);
                    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
                    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
                }
                uint32_t z[4];
                const float s = quant8_f16<BITS>(v, z);
                if (i < items) {
                    *reinterpret_cast<uint4*>(smem + pr * l.pitch_h + k * 2) = make_uint4(z[0], z[1], z[2], z[3]);
                    if ((lane & 3) == 0) fx[pr * n_h + k / 32] = s;
                }
            }
        }
        rows_sync();

        // ------------------------------------------------ second half: rows of down, weighted sum over experts
        {
            uint32_t fg = 0, fa = 0, fs = 0, fdealt = dealt;
            const uint8_t *flo = nullptr, *fhi = nullptr;
            auto fetch = [&](Scales& sc) {
                if (fg >= g2) return;
                if (fs == 0) {
                    const uint32_t d0 = min(r2_0 + 16 * fg + g, r2_1 - 1), d1 = min(r2_0 + 16 * fg + g + 8, r2_1 - 1);
                    const int64_t e = (int64_t)route.list[fa] * ct_d;
                    flo = p.s_down + (e + (d0 >> 7)) * ct_h * 512 + (d0 & 31) * 16 + ((d0 >> 5) & 3) * 4;
                    fhi = p.s_down + (e + (d1 >> 7)) * ct_h * 512 + (d1 & 31) * 16 + ((d1 >> 5) & 3) * 4;
                }
                const uint32_t bytes = min(seg2, Hb - fs * seg2), s = my_slice(bytes, fdealt);
                load_scales(sc, flo, fhi, fs * seg2 + s * 128, ct_h, s * 128 < bytes);
                if (++fs == ns2) {
                    fs = 0;
                    if (++fa == (uint32_t)A) {
                        fa = 0;
                        ++fg;
                    }
                }
            };
            Scales sc[kRwAhead];
#pragma unroll
            for (int i = 0; i < kRwAhead; ++i) fetch(sc[i]);
            float c[4] = {0.0f, 0.0f, 0.0f, 0.0f}, total[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            uint32_t gr = 0, a = 0, s = 0;
            for (uint32_t i = 0; i < st2; i += kRwAhead) {
#pragma unroll
                for (int j = 0; j < kRwAhead; ++j) {
                    if (i + j >= st2) break;
                    const uint32_t bytes = min(seg2, Hb - s * seg2), sl = my_slice(bytes, dealt);
                    const int p0 = pair_s[a][t0], p1 = pair_s[a][t1];
                    land();
                    if (sl * 128 < bytes) {
                        const uint8_t* vb = smem + max((int)pair_s[a][tg], 0) * l.pitch_h;
                        slice(c, sc[j], sl * 128, (s * seg2 + sl * 128) / kBlkBytes, n_h, vb, fx + max(p0, 0) * n_h,
                              fx + max(p1, 0) * n_h);
                    }
                    next_stage();
                    fetch(sc[j]);
                    if (++s < ns2) continue;
                    s = 0;
                    // this expert's share, for the tokens routed to it
                    if (p0 >= 0) {
                        total[0] += route.sel_w[p0] * c[0];
                        total[2] += route.sel_w[p0] * c[2];
                    }
                    if (p1 >= 0) {
                        total[1] += route.sel_w[p1] * c[1];
                        total[3] += route.sel_w[p1] * c[3];
                    }
                    c[0] = c[1] = c[2] = c[3] = 0.0f;
                    if (++a < (uint32_t)A) continue;
                    a = 0;
                    float* to = red + parity * kRwWarps * 16 * T;
                    parity ^= 1;
                    park(to, total);
                    total[0] = total[1] = total[2] = total[3] = 0.0f;
                    rows_sync();
                    if (tid < 16 * T) {
                        const int t = tid >> 4, row = tid & 15;
                        const uint32_t d = r2_0 + 16 * gr + row;
                        if (d < r2_1) p.y[(int64_t)t * D + d] = __float2bfloat16(added(to, t, row));
                    }
                    ++gr;
                }
            }
        }
    }
    __syncthreads();
    if (tid == 0) {
        if (abort_s) {  // given up: let the copies in flight land before the CTA's memory goes
            const uint64_t w0 = globaltimer_ns();
            while (globaltimer_ns() - w0 < 1000000ull) __nanosleep(1000);
        }
        mt_leave(p);
    }
    __syncthreads();
}

// ---------------------------------------------------------------- host side
bool mt_rows_takes(const MtParams& p, int bits) {
    (void)bits;
    if (p.T > kRwTokens || p.T * p.D > kRwMost || (int64_t)p.T * p.top_k * p.H > kRwMost) return false;
    return rw_layout(p.T, p.T * p.top_k, (int)p.D, (int)p.H).stages >= 3;
}

template <int BITS>
static mxfp8_status_t rw_launch(const MtParams& p, cudaStream_t st) {
    static std::atomic<int> attr_set[host::kMaxDevices];
    if (!host::ensure_smem(reinterpret_cast<const void*>(moe_token_rows_kernel<BITS>), 212 * 1024, attr_set))
        return MXFP8_ERR_LAUNCH;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;  // every CTA is resident: they wait for one another
    attr[0].val.cooperative = 1;
    cfg.gridDim = dim3((unsigned)host::num_sms());
    cfg.blockDim = dim3(kRwThreads);
    cfg.dynamicSmemBytes = rw_layout(p.T, p.T * p.top_k, (int)p.D, (int)p.H).total;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, moe_token_rows_kernel<BITS>, p) != cudaSuccess) {
        cudaGetLastError();
        return MXFP8_ERR_LAUNCH;
    }
    return host::last_launch_status();
}

mxfp8_status_t mt_rows_launch(const MtParams& p, int bits, cudaStream_t st) {
    return bits == 8 ? rw_launch<8>(p, st) : rw_launch<4>(p, st);
}

}  // namespace mx
