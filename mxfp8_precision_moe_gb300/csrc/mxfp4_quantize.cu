// mxfp4_quantize.cu -- MXFP4 quantization (plain, of expert weights, and of silu(h1) * h3) and its inverse.
//
// Per block of 32 elements along the row: e = floor(log2 amax) - 2, clamped at -127; codes
// RNE_E2M1(x 2^-e), saturated at 6; scale byte e + 127.  Bounded by HBM: 2 (4 for SwiGLU) bytes read and
// 17/32 written per element, about ten arithmetic instructions each (SwiGLU: thirty).
//
// A CTA of 8 warps owns 128 rows x 256 columns of a padded row tile (groups start on fresh 128-row tiles in
// the blocked scale layout, so a CTA's rows are one band of it and it also writes the band's padding); each
// warp 32 rows x 128 columns, two rows per load instruction, 16 lanes x 16 bytes a row.  A block of 32 spans
// 4 lanes (2 shuffles for its amax); the four scale bytes of a row's 128 columns meet in one 32-bit word
// (2 shuffles) and lane l stores the word of row l, so a warp writes its quarter of the 512-byte scale tile
// with one instruction.

#include "host_common.h"
#include "mx4.cuh"

namespace mx {

constexpr int kQ4Threads = 256;
constexpr int kQ4Cols = 256;   // columns of a CTA's tile
constexpr int kQ4Batch = 8;    // row pairs whose loads are in flight together

struct Q4Params {
    const uint8_t* x;      // bf16 [batch][R][C] (h1 for SwiGLU); dequantize: codes [batch][R][C/2]
    const uint8_t* x2;     // h3
    uint8_t* q;            // codes [batch][R][C/2]; dequantize: bf16 out
    uint8_t* s;            // scales
    int64_t R, C;
    int64_t tiles_r;       // padded row tiles per matrix (an upper bound with groups)
    int64_t s_bstride;     // scale bytes per matrix
    const int32_t* offs;   // row groups (batch == 1), nullptr: one group
    int32_t G;
    int blocked;
    int cols_per_cta;      // column tiles a CTA walks
};

enum Q4Kind : int { kQ4Plain = 0, kQ4Swiglu = 1, kQ4Dequant = 2 };

// The CTA's rows: matrix b, first row, rows inside, band of the scale layout.
struct Q4Rows {
    int64_t b, row0, band;
    int rows;
};

__device__ __forceinline__ Q4Rows q4_rows(const Q4Params& p) {
    __shared__ RowTile tile_s;
    Q4Rows r;
    if (p.offs != nullptr && p.blocked) {
        if (threadIdx.x < 32) {
            const RowTile t = locate_row_tile(p.offs, p.G, p.R, blockIdx.x);
            if (threadIdx.x == 0) tile_s = t;
        }
        __syncthreads();
        r.b = 0;
        r.band = blockIdx.x;
        r.row0 = tile_s.row0;
        r.rows = tile_s.g < 0 ? 0 : tile_s.rows;
    } else {
        r.b = blockIdx.x / p.tiles_r;
        r.band = blockIdx.x - r.b * p.tiles_r;
        r.row0 = r.band * 128;
        r.rows = (int)min64(128, p.R - r.row0);
    }
    return r;
}

__device__ __forceinline__ uint4 ld_stream(const uint8_t* p) {
    uint4 v;
    asm("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
        : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
        : "l"(p));
    return v;
}

__device__ __forceinline__ void unpack8(const uint4& u, float (&v)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16lo(w[i]);
        v[2 * i + 1] = bf16hi(w[i]);
    }
}

template <int KIND>
__global__ void __launch_bounds__(kQ4Threads) mxfp4_quantize_kernel(const Q4Params p) {
    const Q4Rows t = q4_rows(p);
    if (t.rows == 0) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int quarter = warp & 3, half = lane >> 4;
    const int64_t C = p.C, ct = (C + 127) / 128;
    const int64_t base = t.b * p.R + t.row0;  // first row among all matrices'
    const int rq = quarter * 32;              // the warp's first row in the tile
    uint8_t* sb = p.s + t.b * p.s_bstride;
    for (int cc = 0; cc < p.cols_per_cta; ++cc) {
        const int64_t k128 = (blockIdx.y * (int64_t)p.cols_per_cta + cc) * (kQ4Cols / 128) + (warp >> 2);
        if (k128 >= ct) break;
        const int64_t c = k128 * 128 + (lane & 15) * 8;  // C % 32 == 0: a lane's 8 columns are all in or all out
        const bool cin = c < C;
        uint32_t word = 0;  // scale bytes of row rq + lane
#pragma unroll
        for (int b0 = 0; b0 < 16; b0 += kQ4Batch) {
            uint4 u[kQ4Batch], u2[KIND == kQ4Swiglu ? kQ4Batch : 1];
#pragma unroll
            for (int i = 0; i < kQ4Batch; ++i) {
                const int r = rq + 2 * (b0 + i) + half;
                u[i] = make_uint4(0, 0, 0, 0);
                if (KIND == kQ4Swiglu) u2[i] = u[i];
                if (cin && r < t.rows) {
                    u[i] = ld_stream(p.x + ((base + r) * C + c) * 2);
                    if (KIND == kQ4Swiglu) u2[i] = ld_stream(p.x2 + ((base + r) * C + c) * 2);
                }
            }
#pragma unroll
            for (int i = 0; i < kQ4Batch; ++i) {
                const int r = rq + 2 * (b0 + i) + half;
                float v[8];
                unpack8(u[i], v);
                if constexpr (KIND == kQ4Swiglu) {
                    float g[8];
                    unpack8(u2[i], g);
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = v[j] / (1.0f + expf(-v[j])) * g[j];
                }
                uint32_t m = 0;  // magnitude bits order like the magnitudes, NaN above Inf above all else
#pragma unroll
                for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7FFFFFFFu);
                m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
                m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
                const uint32_t s = e8m0_of<2>(m);
                uint32_t codes;
                if (s == 0xFFu) {
                    codes = nonfinite_e2m1x8(v);
                } else {
                    const float f = __uint_as_float((254u - s) << 23);  // 2^(127 - s): s <= 252 here
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] *= f;
                    codes = cvt_e2m1x8(v);
                }
                if (cin && r < t.rows) *reinterpret_cast<uint32_t*>(p.q + ((base + r) * C + c) / 2) = codes;
                if (p.blocked) {
                    uint32_t w = s << (8 * ((lane >> 2) & 3));
                    w |= __shfl_xor_sync(0xffffffffu, w, 4);
                    w |= __shfl_xor_sync(0xffffffffu, w, 8);
                    w = __shfl_sync(0xffffffffu, w, (lane & 1) * 16);
                    if ((lane >> 1) == b0 + i) word = w;  // rows outside the group and columns past C: 0
                } else if (cin && r < t.rows && (lane & 3) == 0) {
                    sb[(t.row0 + r) * (C / 32) + c / 32] = (uint8_t)s;
                }
            }
        }
        if (p.blocked)
            *reinterpret_cast<uint32_t*>(sb + (t.band * ct + k128) * 512 + lane * 16 + quarter * 4) = word;
    }
}

__global__ void __launch_bounds__(kQ4Threads) mxfp4_dequantize_kernel(const Q4Params p) {
    const Q4Rows t = q4_rows(p);
    if (t.rows == 0) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int quarter = warp & 3, half = lane >> 4;
    const int64_t C = p.C, ct = (C + 127) / 128;
    const int64_t base = t.b * p.R + t.row0;
    const int rq = quarter * 32;
    const uint8_t* sb = p.s + t.b * p.s_bstride;
    for (int cc = 0; cc < p.cols_per_cta; ++cc) {
        const int64_t k128 = (blockIdx.y * (int64_t)p.cols_per_cta + cc) * (kQ4Cols / 128) + (warp >> 2);
        if (k128 >= ct) break;
        const int64_t c = k128 * 128 + (lane & 15) * 8;
        const bool cin = c < C;
        uint32_t word = 0;
        if (p.blocked)
            word = *reinterpret_cast<const uint32_t*>(sb + (t.band * ct + k128) * 512 + lane * 16 + quarter * 4);
        uint32_t codes[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int r = rq + 2 * i + half;
            codes[i] = 0;
            if (cin && r < t.rows) codes[i] = *reinterpret_cast<const uint32_t*>(p.x + ((base + r) * C + c) / 2);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int r = rq + 2 * i + half;
            const uint32_t w = __shfl_sync(0xffffffffu, word, 2 * i + half);
            uint32_t s = (w >> (8 * ((lane >> 2) & 3))) & 0xFFu;
            if (!cin || r >= t.rows) continue;
            if (!p.blocked) s = sb[(t.row0 + r) * (C / 32) + c / 32];
            const float f = e8m0_value(s);
            uint32_t o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 v = e2m1x2_value((codes[i] >> (8 * j)) & 0xFFu);
                o[j] = pack_bf16x2(v.x * f, v.y * f);
            }
            *reinterpret_cast<uint4*>(p.q + ((base + r) * C + c) * 2) = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
}

// ---------------------------------------------------------------- host side
static mxfp8_status_t q4_run(int kind, Q4Params& p, int32_t batch, int scale_layout, cudaStream_t st) {
    if (batch < 1 || batch > MXFP8_MAX_GROUPS || p.R < 0 || p.C <= 0 || p.R > INT32_MAX || p.C > INT32_MAX)
        return MXFP8_ERR_SHAPE;
    if (p.C % 32) return MXFP8_ERR_ALIGN;
    if (scale_layout != MXFP8_SCALES_COMPACT && scale_layout != MXFP8_SCALES_BLOCKED) return MXFP8_ERR_LAYOUT;
    if (p.offs != nullptr && (p.G < 1 || p.G > MXFP8_MAX_GROUPS)) return MXFP8_ERR_SHAPE;
    if (p.offs != nullptr && batch != 1) return MXFP8_ERR_LAYOUT;
    if (p.R == 0) return MXFP8_OK;  // an empty tensor may have no address
    if (!p.x || !p.q || !p.s || (kind == kQ4Swiglu && !p.x2)) return MXFP8_ERR_NULL;
    if (!host::aligned16(p.x) || !host::aligned16(p.x2) || !host::aligned16(p.q) || !host::aligned16(p.s))
        return MXFP8_ERR_ALIGN;
    if (mxfp8_status_t a = host::check_arch(); a != MXFP8_OK) return a;
    p.blocked = scale_layout == MXFP8_SCALES_BLOCKED;
    p.tiles_r = (p.R + 127) / 128;
    p.s_bstride = p.blocked ? p.tiles_r * ((p.C + 127) / 128) * 512 : p.R * (p.C / 32);
    const int64_t gx = (p.offs != nullptr && p.blocked) ? p.tiles_r + p.G : p.tiles_r * batch;
    const int64_t tc = (p.C + kQ4Cols - 1) / kQ4Cols;
    // a CTA walks several column tiles once there are enough CTAs to fill the GPU a few times over
    const int64_t want = 16 * (int64_t)host::num_sms();
    p.cols_per_cta = (int)max64(1, min64(tc, gx * tc / want));
    const int64_t gy = (tc + p.cols_per_cta - 1) / p.cols_per_cta;
    if (gx > INT32_MAX || gy > 65535) return MXFP8_ERR_SHAPE;
    const dim3 grid((unsigned)gx, (unsigned)gy);
    if (kind == kQ4Plain) mxfp4_quantize_kernel<kQ4Plain><<<grid, kQ4Threads, 0, st>>>(p);
    else if (kind == kQ4Swiglu) mxfp4_quantize_kernel<kQ4Swiglu><<<grid, kQ4Threads, 0, st>>>(p);
    else mxfp4_dequantize_kernel<<<grid, kQ4Threads, 0, st>>>(p);
    return host::last_launch_status();
}

}  // namespace mx

using namespace mx;

extern "C" mxfp8_status_t mxfp4_quantize_2d(const void* x_bf16, int64_t M, int64_t K, int scale_layout,
                                            const int32_t* offs, int32_t G, void* q, void* s, mxfp8_stream_t stream) {
    Q4Params p{};
    p.x = static_cast<const uint8_t*>(x_bf16);
    p.q = static_cast<uint8_t*>(q);
    p.s = static_cast<uint8_t*>(s);
    p.R = M;
    p.C = K;
    p.offs = offs;
    p.G = G;
    return q4_run(kQ4Plain, p, 1, scale_layout, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" mxfp8_status_t mxfp4_swiglu_quantize(const void* h1_bf16, const void* h3_bf16, int64_t M, int64_t K,
                                                int scale_layout, const int32_t* offs, int32_t G, void* q, void* s,
                                                mxfp8_stream_t stream) {
    Q4Params p{};
    p.x = static_cast<const uint8_t*>(h1_bf16);
    p.x2 = static_cast<const uint8_t*>(h3_bf16);
    p.q = static_cast<uint8_t*>(q);
    p.s = static_cast<uint8_t*>(s);
    p.R = M;
    p.C = K;
    p.offs = offs;
    p.G = G;
    return q4_run(kQ4Swiglu, p, 1, scale_layout, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" mxfp8_status_t mxfp4_quantize_3d_experts(const void* w_bf16, int32_t G, int64_t N, int64_t K,
                                                    int scale_layout, void* q, void* s, mxfp8_stream_t stream) {
    if (N <= 0) return MXFP8_ERR_SHAPE;
    Q4Params p{};
    p.x = static_cast<const uint8_t*>(w_bf16);
    p.q = static_cast<uint8_t*>(q);
    p.s = static_cast<uint8_t*>(s);
    p.R = N;
    p.C = K;
    return q4_run(kQ4Plain, p, G, scale_layout, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" mxfp8_status_t mxfp4_dequantize(const void* q, const void* s, int32_t batch, int64_t M, int64_t K,
                                           int scale_layout, const int32_t* offs, int32_t G, void* out_bf16,
                                           mxfp8_stream_t stream) {
    Q4Params p{};
    p.x = static_cast<const uint8_t*>(q);
    p.q = static_cast<uint8_t*>(out_bf16);
    p.s = static_cast<uint8_t*>(const_cast<void*>(s));
    p.R = M;
    p.C = K;
    p.offs = offs;
    p.G = G;
    return q4_run(kQ4Dequant, p, batch, scale_layout, reinterpret_cast<cudaStream_t>(stream));
}
