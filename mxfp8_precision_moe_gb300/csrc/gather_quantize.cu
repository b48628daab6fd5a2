// gather_quantize.cu -- token rows quantized along the row into a plan's order: MXFP4, and MXFP8 where neither a
// column-wise copy nor weights are asked for.
//
// By token: a token's row is read and quantized once, and its codes and scales go to each of its top_k rows.  Going by the
// plan's rows, x is read and quantized top_k times: 8 rows a token of 8192 x 7168, MXFP4 153 us, MXFP8 206 us; by token
// 79 and 127, against 55 and 94 us for the bytes at the copy rate.  Codes go out by whole rows; the scales, whose layout
// keeps a row's 512 bytes apart, by 4-byte words of 128 columns, which L2 joins (14 and 17 us of the time).  Five CTAs an SM;
// four are up to 10% slower where a token has one row, six 3% where it has eight.

#include "groups.cuh"
#include "host_common.h"
#include "mx4.cuh"
#include "../../include/mxrouting.h"

namespace mx {

struct GatherParams {
    const uint8_t* x;      // bf16 [T][C]
    const int32_t* slot;   // [R]
    const int32_t* place;  // [T][k]
    const int32_t* offs;
    uint8_t* q;            // codes [R][C] or [R][C / 2]
    uint8_t* s;            // blocked scales
    int64_t R, T, C;
    int32_t G, k;
    int32_t parts;         // warps that share a token
    int64_t token_items, row_items, items;
};

constexpr int kGatherWarps = 8;

// EPT elements of a block (the other 32 / EPT - 1 shares are the neighbouring lanes') -> its scale byte, the codes in c.
__device__ __forceinline__ uint32_t q8_share_bf16(const uint32_t (&w)[8], uint32_t (&c)[4]) {
    uint32_t m = w[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) m = amax_pair(m, w[i]);
    m = max(m & 0x7FFFu, (m >> 16) & 0x7FFFu);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    const uint32_t s = e8m0_of<8>(m << 16);
    const uint32_t f = (254u - s) << 7;  // 2^(127 - s) as a bf16: s <= 246 for a finite amax
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 a = scale_pair(w[2 * i], f), b = scale_pair(w[2 * i + 1], f);
        c[i] = cvt_e4m3x2(a.x, a.y) | (cvt_e4m3x2(b.x, b.y) << 16);
    }
    if (s == 0xFFu) {  // NaN with each element's sign
#pragma unroll
        for (int i = 0; i < 4; ++i)
            c[i] = 0x7F7F7F7Fu | ((w[2 * i] >> 8) & 0x80u) | ((w[2 * i] >> 16) & 0x8000u) |
                   ((((w[2 * i + 1] >> 8) & 0x80u) | ((w[2 * i + 1] >> 16) & 0x8000u)) << 16);
    }
    return s;
}

template <int BITS>
__global__ void __launch_bounds__(kGatherWarps * 32, 5) gather_quantize_kernel(const GatherParams p) {
    __shared__ int32_t ends_s[kMaxGroups];
    __shared__ int32_t pstart_s[kMaxGroups];
    __shared__ int32_t ptotal_s;
    constexpr int EPT = BITS == 4 ? 32 : 16;    // elements of a lane: 16 bytes of codes, whole sectors by neighbours
    constexpr int kLanes = 128 / EPT;           // lanes of a scale word
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t R = p.R, C = p.C, ct = (C + 127) / 128;
    const int G = p.G;
    if (BITS == 8 && G == 1) {  // one group: the whole matrix, as for mxfp8_quantize_2d
        if (threadIdx.x == 0) {
            ends_s[0] = (int32_t)R;
            pstart_s[0] = 0;
        }
    } else if (threadIdx.x < 32) {
        build_group_table(p.offs, G, R, ends_s, pstart_s, &ptotal_s);
    }
    __syncthreads();
    // row r's place in the scales, -1: in no group
    auto padded = [&](int64_t r) -> int64_t {
        const int g = find_group(ends_s, G, r);
        return g < G ? pstart_s[g] + (r - (g ? ends_s[g - 1] : 0)) : -1;
    };
    auto word_at = [&](int64_t pr, int64_t k128) -> uint32_t* {
        return reinterpret_cast<uint32_t*>(p.s + ((pr >> 7) * ct + k128) * 512 + (pr & 31) * 16 + ((pr >> 5) & 3) * 4);
    };
    for (int64_t i = (int64_t)blockIdx.x * kGatherWarps + warp; i < p.items; i += (int64_t)gridDim.x * kGatherWarps) {
        if (i < p.token_items) {
            const int64_t t = i / p.parts;
            int64_t row = -1, pr = -1;  // lane j: the token's j-th
            if (lane < p.k) {
                const int32_t at = __ldg(p.place + t * p.k + lane);
                if (at >= 0 && at < R) {
                    row = at;
                    pr = padded(at);
                }
            }
            for (int64_t c0 = (i - t * p.parts) * (32 * EPT); c0 < C; c0 += (int64_t)p.parts * (32 * EPT)) {
                const int64_t c = c0 + lane * EPT;
                const bool in = c < C;
                uint32_t w[EPT / 2], codes[4];
#pragma unroll
                for (int j = 0; j < EPT / 8; ++j) {
                    uint4 u = make_uint4(0, 0, 0, 0);
                    if (in) u = __ldg(reinterpret_cast<const uint4*>(p.x + (t * C + c) * 2) + j);
                    w[4 * j] = u.x; w[4 * j + 1] = u.y; w[4 * j + 2] = u.z; w[4 * j + 3] = u.w;
                }
                uint32_t word;
                if constexpr (BITS == 4) word = q4_block_bf16(w, codes);
                else word = q8_share_bf16(w, codes);
                word <<= 8 * ((lane % kLanes) / (32 / EPT));
#pragma unroll
                for (int d = 32 / EPT; d < kLanes; d <<= 1) word |= __shfl_xor_sync(0xffffffffu, word, d);
                for (int j = 0; j < p.k; ++j) {
                    const int64_t to = __shfl_sync(0xffffffffu, row, j), pj = __shfl_sync(0xffffffffu, pr, j);
                    if (to < 0 || !in) continue;
                    *reinterpret_cast<uint4*>(p.q + (to * C + c) * BITS / 8) = make_uint4(codes[0], codes[1], codes[2], codes[3]);
                    if (lane % kLanes == 0 && pj >= 0) *word_at(pj, c >> 7) = word;
                }
            }
        } else if (i < p.token_items + p.row_items) {
            // 32 rows: those without a token are zeros
            const int64_t r0 = (i - p.token_items) * 32, mine = r0 + lane;
            const int32_t slot = mine < R ? __ldg(p.slot + mine) : 0;
            const bool none = slot < 0 || slot >= p.T * p.k;
            const int64_t pr = none ? padded(mine) : -1;
            uint32_t empty = __ballot_sync(0xffffffffu, none && (BITS == 8 || pr >= 0));
            while (empty) {
                const int j = __ffs(empty) - 1;
                empty &= empty - 1;
                const int64_t pj = __shfl_sync(0xffffffffu, pr, j);
                uint4* out = reinterpret_cast<uint4*>(p.q + (r0 + j) * C * BITS / 8);
                for (int64_t u = lane; u < C * BITS / 128; u += 32) out[u] = make_uint4(0, 0, 0, 0);
                if (pj >= 0)
                    for (int64_t u = lane; u < ct; u += 32) *word_at(pj, u) = 0u;
            }
        } else {
            // what is left of a group's last 128 rows in the scales, of 128 columns
            const int64_t n = i - p.token_items - p.row_items;
            const int g = (int)(n / ct);
            const int32_t size = ends_s[g] - (g ? ends_s[g - 1] : 0), over = size & 127;
            if (over == 0) continue;
            uint32_t* tile = word_at(pstart_s[g] + (size - over), n - g * ct);
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (32 * u + lane >= over) tile[lane * 4 + u] = 0u;
        }
    }
}

template <int BITS>
static mxfp8_status_t run_gather_quantize(GatherParams& p, cudaStream_t st) {
    constexpr int EPT = BITS == 4 ? 32 : 16;
    // Where a token has several rows, more CTAs than the five that fit on an SM, and more warps on a token, even the ends out.
    // Once (twice, 3, 4, 8 times) as many, us: 16384 tokens of 5120, MXFP8, one row 48.1 (49.0 50.1 50.9 58.4), two 61.1 (61.2
    // 63.4 62.0 68.3), three 79.2 (75.7 77.2 75.7 79.9), four 97.0 (91.4 93.7 89.9 92.9); MXFP4, one 37.1 (37.5 40.9 40.8 45.5),
    // two 44.4 (44.0 49.4 47.3 51.5), three 56.4 (52.1 56.2 54.0 57.7), four 67.4 (61.4 65.8 62.0 64.2); 8192 of 7168, eight rows
    // MXFP8 136.6 (134.8 134.4 127.3 123.1), MXFP4 87.9 (86.9 85.9 83.6 83.8).
    const int64_t chunks = (p.C + 32 * EPT - 1) / (32 * EPT), ctas = (int64_t)host::num_sms() * 5 * (p.k < 4 ? p.k : 4);
    // a warp takes a whole token, for which it looks its rows up once; of few tokens, several share one
    p.parts = (int32_t)max64(1, min64(chunks, (ctas * kGatherWarps + p.T - 1) / max64(p.T, 1)));
    p.token_items = p.T * p.parts;
    p.row_items = (p.R + 31) / 32;
    p.items = p.token_items + p.row_items + p.G * ((p.C + 127) / 128);
    const unsigned grid = (unsigned)min64(ctas, (p.items + kGatherWarps - 1) / kGatherWarps);
    gather_quantize_kernel<BITS><<<grid, kGatherWarps * 32, 0, st>>>(p);
    return host::last_launch_status();
}

mxfp8_status_t gather_quantize_rows(int bits, const void* x, const int32_t* slot, const int32_t* place, int64_t rows,
                                    int64_t T, int32_t top_k, int64_t D, const int32_t* offs, int32_t G, void* q, void* s,
                                    cudaStream_t st) {
    GatherParams p{};
    p.x = static_cast<const uint8_t*>(x);
    p.slot = slot;
    p.place = place;
    p.offs = offs;
    p.q = static_cast<uint8_t*>(q);
    p.s = static_cast<uint8_t*>(s);
    p.R = rows;
    p.T = T;
    p.C = D;
    p.G = G;
    p.k = top_k;
    return bits == 4 ? run_gather_quantize<4>(p, st) : run_gather_quantize<8>(p, st);
}

}  // namespace mx

using namespace mx;

extern "C" mxfp8_status_t mxfp4_gather_quantize(const void* x_bf16, const int32_t* slot, const int32_t* place, int64_t rows,
                                                int64_t T, int32_t top_k, int64_t D, const int32_t* offs, int32_t G, void* q,
                                                void* s, mxfp8_stream_t stream) {
    if (rows < 0 || rows > INT32_MAX || D <= 0 || D > INT32_MAX || T < 0 || top_k < 1 || top_k > MX_MAX_TOP_K ||
        T * top_k > INT32_MAX || G < 1 || G > MXFP8_MAX_GROUPS || !padded_rows_fit(rows, G))
        return MXFP8_ERR_SHAPE;
    if (D % 32) return MXFP8_ERR_ALIGN;
    if (rows == 0) return MXFP8_OK;  // an empty tensor may have no address
    if ((T && (!x_bf16 || !place)) || !slot || !offs || !q || !s) return MXFP8_ERR_NULL;
    if (!host::aligned16(x_bf16) || !host::aligned16(q) || !host::aligned16(s)) return MXFP8_ERR_ALIGN;
    for (const int32_t* v : {slot, place, offs})
        if (reinterpret_cast<uintptr_t>(v) & 3u) return MXFP8_ERR_ALIGN;
    if (mxfp8_status_t a = host::check_arch(); a != MXFP8_OK) return a;
    return gather_quantize_rows(4, x_bf16, slot, place, rows, T, top_k, D, offs, G, q, s, reinterpret_cast<cudaStream_t>(stream));
}
