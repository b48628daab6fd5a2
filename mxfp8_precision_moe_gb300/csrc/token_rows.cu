// token_rows.cu -- token rows into the order of a plan and back: gather, the weighted
// sum of a token's rows, and its backward.  Bound by HBM: every kernel goes by token,
// so that a token's row is read (or written) once for all of its top_k rows, and by
// 16-byte pieces, neighbouring threads along the row.

#include "common.cuh"
#include "host_common.h"
#include "../../include/mxrouting.h"

namespace mx {

struct RowsParams {
    const uint4* x;        // [T][C] token rows (the gather's input, the backward's dout), C pieces of 8 columns
    const uint4* y;        // [rows][C]
    const int32_t* slot;   // [rows]
    const int32_t* place;  // [T][k]
    const float* w;        // [T][k], or null: ones
    uint4* out;            // [T][C] or [rows][C]
    float* dw;             // [T][k]
    int64_t rows, T;
    int32_t k;
    uint32_t C;
    uint32_t token_ctas;   // of the gather: CTAs that take tokens; the others take padding rows
    uint32_t parts;        // warps that share a token
};

constexpr int kRowsThreads = 256;

__device__ __forceinline__ void unpack8(uint4 u, float (&v)[8]) {
    v[0] = bf16lo(u.x); v[1] = bf16hi(u.x); v[2] = bf16lo(u.y); v[3] = bf16hi(u.y);
    v[4] = bf16lo(u.z); v[5] = bf16hi(u.z); v[6] = bf16lo(u.w); v[7] = bf16hi(u.w);
}
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
    return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}
__device__ __forceinline__ int64_t row_or_none(const RowsParams& p, int64_t i) {
    const int32_t r = __ldg(p.place + i);
    return r >= 0 && r < p.rows ? r : -1;
}

// Rows without a token are zeros: a warp takes 32 rows' slots at a time.
__device__ __forceinline__ void zero_padding_rows(const RowsParams& p, int64_t cta) {
    const int lane = threadIdx.x & 31;
    const int64_t r0 = cta * kRowsThreads + (threadIdx.x & ~31);
    if (r0 >= p.rows) return;
    const int64_t mine = r0 + lane;
    const int32_t s = mine < p.rows ? __ldg(p.slot + mine) : 0;
    uint32_t empty = __ballot_sync(0xffffffffu, s < 0 || s >= p.T * p.k);
    while (empty) {
        const int64_t r = r0 + __ffs(empty) - 1;
        empty &= empty - 1;
        for (uint32_t c = lane; c < p.C; c += 32) p.out[r * p.C + c] = make_uint4(0, 0, 0, 0);
    }
}

// A warp a token, or a share of one where tokens are few: two pieces a lane at a time, read once, written to the token's
// rows (times their weights), which are looked up once, a lane each.
constexpr int kGatherPieces = 2;
template <bool kWeighted>
__global__ void __launch_bounds__(kRowsThreads) gather_rows_kernel(const RowsParams p) {
    if (blockIdx.x >= p.token_ctas) {
        zero_padding_rows(p, blockIdx.x - p.token_ctas);
        return;
    }
    constexpr int U = kGatherPieces;
    const int lane = threadIdx.x & 31;
    const int64_t item = (int64_t)blockIdx.x * (kRowsThreads / 32) + (threadIdx.x >> 5), t = item / p.parts;
    if (t >= p.T) return;
    int32_t mine = -1;
    float mine_w = 1.0f;
    if (lane < p.k) {
        mine = (int32_t)row_or_none(p, t * p.k + lane);
        if constexpr (kWeighted) mine_w = __ldg(p.w + t * p.k + lane);
    }
    for (uint32_t first = (uint32_t)(item - t * p.parts) * (32 * U); first < p.C; first += p.parts * (32 * U)) {
        const uint32_t c0 = first + lane;
        uint4 u[U];
#pragma unroll
        for (int q = 0; q < U; ++q)
            if (c0 + 32 * q < p.C) u[q] = __ldg(p.x + t * p.C + c0 + 32 * q);
        for (int j = 0; j < p.k; ++j) {
            const int32_t row = __shfl_sync(0xffffffffu, mine, j);
            const float w = kWeighted ? __shfl_sync(0xffffffffu, mine_w, j) : 1.0f;
            if (row < 0) continue;  // the same for the whole warp
#pragma unroll
            for (int q = 0; q < U; ++q) {
                uint4 o = u[q];
                if constexpr (kWeighted) {
                    float v[8];
                    unpack8(u[q], v);
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] *= w;
                    o = pack8(v);
                }
                if (c0 + 32 * q < p.C) p.out[(int64_t)row * p.C + c0 + 32 * q] = o;
            }
        }
    }
}

// A warp a token, or a share of one where tokens are few: it looks the token's rows up once, a lane each, and then takes U
// pieces a lane of up to KB rows at a time, U * KB loads in flight.
template <int KB, int U>
__global__ void __launch_bounds__(kRowsThreads) combine_kernel(const RowsParams p) {
    const int lane = threadIdx.x & 31;
    const int64_t item = (int64_t)blockIdx.x * (kRowsThreads / 32) + (threadIdx.x >> 5), t = item / p.parts;
    if (t >= p.T) return;
    int32_t mine = -1;
    float mine_w = 1.0f;
    if (lane < p.k) {
        mine = (int32_t)row_or_none(p, t * p.k + lane);
        if (p.w) mine_w = __ldg(p.w + t * p.k + lane);
    }
    for (uint32_t first = (uint32_t)(item - t * p.parts) * (32 * U); first < p.C; first += p.parts * (32 * U)) {
        const uint32_t c0 = first + lane;
        float acc[U][8];
#pragma unroll
        for (int q = 0; q < U; ++q)
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[q][e] = 0.0f;
        for (int j0 = 0; j0 < p.k; j0 += KB) {
            uint4 u[KB][U];
            int32_t row[KB];
#pragma unroll
            for (int b = 0; b < KB; ++b) {
                row[b] = __shfl_sync(0xffffffffu, mine, (j0 + b) & 31);
                if (j0 + b >= p.k) row[b] = -1;
                if (row[b] < 0) continue;  // the same for the whole warp
#pragma unroll
                for (int q = 0; q < U; ++q)
                    if (c0 + 32 * q < p.C) u[b][q] = __ldg(p.y + (int64_t)row[b] * p.C + c0 + 32 * q);
            }
#pragma unroll
            for (int b = 0; b < KB; ++b) {
                const float w = __shfl_sync(0xffffffffu, mine_w, (j0 + b) & 31);
                if (row[b] < 0) continue;
#pragma unroll
                for (int q = 0; q < U; ++q) {
                    float v[8];
                    unpack8(u[b][q], v);
#pragma unroll
                    for (int e = 0; e < 8; ++e) acc[q][e] = fmaf(w, v[e], acc[q][e]);
                }
            }
        }
#pragma unroll
        for (int q = 0; q < U; ++q)
            if (c0 + 32 * q < p.C) p.out[t * p.C + c0 + 32 * q] = pack8(acc[q]);
    }
}

// A CTA a token: each piece of dout is read once, with the pieces of the token's rows of y; dy's are written, and the
// threads' partial products <dout, y> are added up in a fixed order.  At the copy rate where a row fills the CTA: 16384 tokens,
// 4 rows of 5120 each, 224 us for 226 of bytes.  Shorter rows leave threads without a piece, and the adding up costs as much
// as ever: 65536 tokens, 4 rows of 1024, 301 us for 181; of 512 266 for 90; of 352 257 for 62.
template <int KB, bool kDy>
__global__ void __launch_bounds__(kRowsThreads) combine_bwd_kernel(const RowsParams p) {
    __shared__ float part[kRowsThreads / 32][MX_MAX_TOP_K];
    if (blockIdx.x >= p.T) {
        if constexpr (kDy) zero_padding_rows(p, blockIdx.x - p.T);
        return;
    }
    const int64_t t = blockIdx.x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int64_t at[KB];
    float w[KB], dot[KB];
#pragma unroll
    for (int j = 0; j < KB; ++j) {
        at[j] = j < p.k ? row_or_none(p, t * p.k + j) : -1;
        w[j] = at[j] >= 0 && p.w ? __ldg(p.w + t * p.k + j) : 1.0f;
        dot[j] = 0.0f;
    }
    for (uint32_t c = threadIdx.x; c < p.C; c += kRowsThreads) {
        const uint4 u = __ldg(p.x + t * p.C + c);
        uint4 s[KB];
#pragma unroll
        for (int j = 0; j < KB; ++j)
            if (at[j] >= 0) s[j] = __ldg(p.y + at[j] * p.C + c);
        float d[8];
        unpack8(u, d);
#pragma unroll
        for (int j = 0; j < KB; ++j) {
            if (at[j] < 0) continue;
            float v[8];
            unpack8(s[j], v);
#pragma unroll
            for (int q = 0; q < 8; ++q) dot[j] = fmaf(d[q], v[q], dot[j]);
            if constexpr (kDy) {
#pragma unroll
                for (int q = 0; q < 8; ++q) v[q] = d[q] * w[j];
                p.out[at[j] * p.C + c] = pack8(v);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < KB; ++j) {
#pragma unroll
        for (int m = 16; m; m >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], m);
        if (lane == 0) part[warp][j] = dot[j];
    }
    __syncthreads();
    if (threadIdx.x < p.k) {
        float sum = 0.0f;
#pragma unroll
        for (int v = 0; v < kRowsThreads / 32; ++v) sum += part[v][threadIdx.x];
        p.dw[t * p.k + threadIdx.x] = sum;
    }
}

// ---------------------------------------------------------------- host side
static mxfp8_status_t rows_check(RowsParams& p, int64_t rows, int64_t T, int32_t top_k, int64_t D) {
    if (rows < 0 || rows > INT32_MAX || T < 0 || top_k < 1 || top_k > MX_MAX_TOP_K || T * top_k > INT32_MAX || D < 1 ||
        D > INT32_MAX)
        return MXFP8_ERR_SHAPE;
    if (D % 8) return MXFP8_ERR_ALIGN;
    p.rows = rows;
    p.T = T;
    p.k = top_k;
    p.C = (uint32_t)(D / 8);
    return MXFP8_OK;
}
static bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
static int64_t padding_ctas(const RowsParams& p) { return (p.rows + kRowsThreads - 1) / kRowsThreads; }

// Warps for each token, of which one takes `width` pieces at a time: as many as fill the GPU twice (`times` over), or one
// for each width.
static uint32_t parts_of(const RowsParams& p, int width, int times) {
    const int64_t widths = (p.C + width - 1) / width, want = (int64_t)host::num_sms() * 128 * times;
    return (uint32_t)max64(1, min64(widths, (want + p.T - 1) / max64(p.T, 1)));
}
static int64_t token_ctas(const RowsParams& p) {
    constexpr int kWarps = kRowsThreads / 32;
    return (p.T * p.parts + kWarps - 1) / kWarps;
}

static mxfp8_status_t run_gather(RowsParams& p, cudaStream_t st) {
    if (p.rows == 0) return MXFP8_OK;
    // the more writes a token is, the more warps share it: once (twice, 4, 8, 16 times) over, 16384 tokens of 5120, us, one row
    // 52.8 (52.1 51.3 52.8 53.1), two 78.5 (78.6 77.8 78.0 77.4), three 106.1 (104.6 103.6 103.9 103.9), four 133.2 (131.0 129.7
    // 128.6 127.8); 8192 tokens of 7168, eight 179.5 (177.5 176.0 173.1 173.6)
    p.parts = parts_of(p, 32 * kGatherPieces, p.k < 4 ? p.k * p.k : 16);
    p.token_ctas = (uint32_t)token_ctas(p);
    const unsigned grid = (unsigned)(p.token_ctas + padding_ctas(p));
    if (p.w) gather_rows_kernel<true><<<grid, kRowsThreads, 0, st>>>(p);
    else gather_rows_kernel<false><<<grid, kRowsThreads, 0, st>>>(p);
    return host::last_launch_status();
}

template <int KB, int U>
static void run_combine(RowsParams& p, cudaStream_t st) {
    p.parts = parts_of(p, 32 * U, 1);
    combine_kernel<KB, U><<<(unsigned)token_ctas(p), kRowsThreads, 0, st>>>(p);
}

template <bool kDy>
static void run_combine_bwd(const RowsParams& p, unsigned grid, cudaStream_t st) {
    if (p.k == 1) combine_bwd_kernel<1, kDy><<<grid, kRowsThreads, 0, st>>>(p);
    else if (p.k == 2) combine_bwd_kernel<2, kDy><<<grid, kRowsThreads, 0, st>>>(p);
    else if (p.k <= 4) combine_bwd_kernel<4, kDy><<<grid, kRowsThreads, 0, st>>>(p);
    else if (p.k <= 8) combine_bwd_kernel<8, kDy><<<grid, kRowsThreads, 0, st>>>(p);
    else combine_bwd_kernel<16, kDy><<<grid, kRowsThreads, 0, st>>>(p);
}

}  // namespace mx

using namespace mx;

extern "C" mxfp8_status_t mx_moe_gather(const void* x_bf16, const int32_t* slot, const int32_t* place, int64_t rows,
                                        int64_t T, int32_t top_k, int64_t D, void* out_bf16, mxfp8_stream_t stream) {
    RowsParams p{};
    if (mxfp8_status_t s = rows_check(p, rows, T, top_k, D); s != MXFP8_OK) return s;
    if (rows == 0) return MXFP8_OK;  // an empty tensor may have no address
    if (!slot || !out_bf16 || (T && (!x_bf16 || !place))) return MXFP8_ERR_NULL;
    if (!host::aligned16(x_bf16) || !host::aligned16(out_bf16) || !aligned4(slot) || !aligned4(place)) return MXFP8_ERR_ALIGN;
    if (mxfp8_status_t a = host::check_arch(); a != MXFP8_OK) return a;
    p.x = static_cast<const uint4*>(x_bf16);
    p.slot = slot;
    p.place = place;
    p.out = static_cast<uint4*>(out_bf16);
    return run_gather(p, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" mxfp8_status_t mx_moe_combine(const void* y_bf16, const int32_t* place, const float* w, int64_t rows, int64_t T,
                                         int32_t top_k, int64_t D, void* out_bf16, mxfp8_stream_t stream) {
    RowsParams p{};
    if (mxfp8_status_t s = rows_check(p, rows, T, top_k, D); s != MXFP8_OK) return s;
    if (T == 0) return MXFP8_OK;
    if (!place || !out_bf16 || (rows && !y_bf16)) return MXFP8_ERR_NULL;
    if (!host::aligned16(y_bf16) || !host::aligned16(out_bf16) || !aligned4(place) || !aligned4(w)) return MXFP8_ERR_ALIGN;
    if (mxfp8_status_t a = host::check_arch(); a != MXFP8_OK) return a;
    p.y = static_cast<const uint4*>(y_bf16);
    p.place = place;
    p.w = w;
    p.out = static_cast<uint4*>(out_bf16);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    // rows at a time x pieces: 8 rows a token of 7168, four by two 154 us (one by eight 202, two by four 184, eight by two
    // 162); 4 of 5120, four by two 121 (four by one 160, two by four 139); 2, two by two 76 (two by four 86); 1, 55 and 56
    if (p.k > 2) run_combine<4, 2>(p, st);
    else if (p.k == 2) run_combine<2, 2>(p, st);
    else run_combine<1, 2>(p, st);
    return host::last_launch_status();
}

extern "C" mxfp8_status_t mx_moe_combine_bwd(const void* dout_bf16, const void* y_bf16, const int32_t* slot,
                                             const int32_t* place, const float* w, int64_t rows, int64_t T, int32_t top_k,
                                             int64_t D, void* dy_bf16, float* dw, mxfp8_stream_t stream) {
    RowsParams p{};
    if (mxfp8_status_t s = rows_check(p, rows, T, top_k, D); s != MXFP8_OK) return s;
    if ((T == 0 && rows == 0) || (!dy_bf16 && !dw)) return MXFP8_OK;
    if (T && (!dout_bf16 || !place)) return MXFP8_ERR_NULL;
    if (rows && ((dy_bf16 && !slot) || (dw && !y_bf16))) return MXFP8_ERR_NULL;
    if (!host::aligned16(dout_bf16) || !host::aligned16(y_bf16) || !host::aligned16(dy_bf16) || !aligned4(slot) ||
        !aligned4(place) || !aligned4(w) || !aligned4(dw))
        return MXFP8_ERR_ALIGN;
    if (mxfp8_status_t a = host::check_arch(); a != MXFP8_OK) return a;
    p.x = static_cast<const uint4*>(dout_bf16);
    p.y = static_cast<const uint4*>(y_bf16);
    p.slot = slot;
    p.place = place;
    p.w = w;
    p.out = static_cast<uint4*>(dy_bf16);
    p.dw = dw;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (!dw) return run_gather(p, st);
    const int64_t ctas = T + (dy_bf16 ? padding_ctas(p) : 0);
    if (ctas > INT32_MAX) return MXFP8_ERR_SHAPE;
    if (ctas == 0) return MXFP8_OK;
    if (dy_bf16) run_combine_bwd<true>(p, (unsigned)ctas, st);
    else run_combine_bwd<false>(p, (unsigned)ctas, st);
    return host::last_launch_status();
}
