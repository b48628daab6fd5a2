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

// This thread's piece of a [T][C] matrix: one long division a CTA, a short one a thread.
struct Piece {
    int64_t i, t;  // its index, its row
    uint32_t c;    // its place in the row
};
__device__ __forceinline__ Piece piece_of(uint32_t C) {
    const int64_t first = (int64_t)blockIdx.x * kRowsThreads, t0 = first / C;
    const uint32_t c0 = (uint32_t)(first - t0 * C) + threadIdx.x, more = c0 / C;
    return Piece{first + threadIdx.x, t0 + more, c0 - more * C};
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

// A thread a piece of a token's row: read once, written to the token's rows (times their weights).
template <bool kWeighted>
__global__ void __launch_bounds__(kRowsThreads) gather_rows_kernel(const RowsParams p) {
    if (blockIdx.x >= p.token_ctas) {
        zero_padding_rows(p, blockIdx.x - p.token_ctas);
        return;
    }
    const auto [i, t, c] = piece_of(p.C);
    if (t >= p.T) return;
    const uint4 u = __ldg(p.x + i);
    for (int j = 0; j < p.k; ++j) {
        const int64_t r = row_or_none(p, t * p.k + j);
        if (r < 0) continue;
        uint4 o = u;
        if constexpr (kWeighted) {
            const float w = __ldg(p.w + t * p.k + j);
            float v[8];
            unpack8(u, v);
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] *= w;
            o = pack8(v);
        }
        p.out[r * p.C + c] = o;
    }
}

// A thread a piece of a token's output; KB rows' loads in flight at a time.
template <int KB>
__global__ void __launch_bounds__(kRowsThreads) combine_kernel(const RowsParams p) {
    const auto [i, t, c] = piece_of(p.C);
    if (t >= p.T) return;
    float acc[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) acc[q] = 0.0f;
    for (int j0 = 0; j0 < p.k; j0 += KB) {
        uint4 u[KB];
        float w[KB];
        bool has[KB];
#pragma unroll
        for (int b = 0; b < KB; ++b) {
            const int64_t r = j0 + b < p.k ? row_or_none(p, t * p.k + j0 + b) : -1;
            has[b] = r >= 0;
            w[b] = 1.0f;
            if (has[b]) {
                u[b] = __ldg(p.y + r * p.C + c);
                if (p.w) w[b] = __ldg(p.w + t * p.k + j0 + b);
            }
        }
#pragma unroll
        for (int b = 0; b < KB; ++b)
            if (has[b]) {
                float v[8];
                unpack8(u[b], v);
#pragma unroll
                for (int q = 0; q < 8; ++q) acc[q] = fmaf(w[b], v[q], acc[q]);
            }
    }
    p.out[i] = pack8(acc);
}

// A CTA a token: each piece of dout is read once, with the pieces of the token's rows of y; dy's are written, and the
// threads' partial products <dout, y> are added up in a fixed order.
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
    if (T * p.C > (int64_t)INT32_MAX * kRowsThreads / 2) return MXFP8_ERR_SHAPE;
    return MXFP8_OK;
}
static bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
static int64_t padding_ctas(const RowsParams& p) { return (p.rows + kRowsThreads - 1) / kRowsThreads; }

static mxfp8_status_t run_gather(RowsParams& p, cudaStream_t st) {
    if (p.rows == 0) return MXFP8_OK;
    const int64_t tokens = (p.T * p.C + kRowsThreads - 1) / kRowsThreads;
    p.token_ctas = (uint32_t)tokens;
    const unsigned grid = (unsigned)(tokens + padding_ctas(p));
    if (p.w) gather_rows_kernel<true><<<grid, kRowsThreads, 0, st>>>(p);
    else gather_rows_kernel<false><<<grid, kRowsThreads, 0, st>>>(p);
    return host::last_launch_status();
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
    const unsigned grid = (unsigned)((T * p.C + kRowsThreads - 1) / kRowsThreads);
    if (p.k == 1) combine_kernel<1><<<grid, kRowsThreads, 0, st>>>(p);
    else if (p.k == 2) combine_kernel<2><<<grid, kRowsThreads, 0, st>>>(p);
    else if (p.k <= 4) combine_kernel<4><<<grid, kRowsThreads, 0, st>>>(p);
    else combine_kernel<8><<<grid, kRowsThreads, 0, st>>>(p);
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
