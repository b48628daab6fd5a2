// mxfp4_quantize.cu -- MXFP4 quantization (plain, of expert weights, and of silu(h1) * h3) and its inverse.
//
// Per block of 32 elements along the row: e = floor(log2 amax) - 2, clamped at -127; codes
// RNE_E2M1(x 2^-e), saturated at 6; scale byte e + 127.  2 (4 for SwiGLU) bytes read and 17/32 written per
// element, the inverse the other way round.
//
// A CTA of 8 warps owns 128 rows x 256 columns of a padded row tile (groups start on fresh 128-row tiles in
// the blocked scale layout, so a CTA's rows are one band of it and it also writes the band's padding), each
// warp 32 rows x 128 columns.
//   plain     a thread takes a whole block (four 16-byte loads, one 16-byte store of codes): no shuffles but
//             two that join a row's four scale bytes into one word.  Against four lanes a block this halves
//             the instructions per element: [16, 8192, 5120] takes 260 us instead of 303, 6.5 TB/s, which
//             is HBM's copy rate.  Five CTAs an SM; six spill, four leave loads too few.
//   SwiGLU    two threads a block, to fit six CTAs an SM.  126 us for 16384 x 8192, 4.8 TB/s, with neither the
//             issue slots nor DRAM full (68% each under ncu): a thread's next loads wait for its arithmetic, and only
//             the other warps fill the gap.  The quotient is a product with a reciprocal (silu2) in instructions of two
//             values; with the correctly rounded division 170 us (a block a thread 174-197 us then, four lanes
//             a block 169-190; five or seven CTAs 135 and 129 now).
//   inverse   four lanes a block: 16-byte stores of 8 values, whole 32-byte sectors by neighbouring lanes.
//             274 us for [16, 8192, 5120], 6.2 TB/s (write-heavy traffic).

#include "host_common.h"
#include "mx4.cuh"

namespace mx {

constexpr int kQ4Threads = 256;
constexpr int kQ4Cols = 256;   // columns of a CTA's tile

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
    int row_steps;         // of a tile's row steps, how many a CTA takes (blockIdx.z: which)
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

// Largest magnitude of each half of two bf16 pairs, NaN winning (the sign bits left are not used).
__device__ __forceinline__ uint32_t amax_pair(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// A bf16 pair times the bf16 power of two f, exact in fp32 (a -0 addend keeps the sign of a zero).
__device__ __forceinline__ float2 scale_pair(uint32_t w, uint32_t f) {
    float2 r;
    asm("{\n\t.reg .b16 a0, a1, b0, b1;\n\tmov.b32 {a0, a1}, %2;\n\tmov.b32 {b0, b1}, %3;\n\t"
        "fma.rn.f32.bf16 %0, a0, b0, 0f80000000;\n\tfma.rn.f32.bf16 %1, a1, b0, 0f80000000;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "r"(w), "r"(f));
    return r;
}

// A block of 32 bf16 (16 pairs) -> its scale byte, codes in c.
__device__ __forceinline__ uint32_t q4_block_bf16(const uint32_t (&w)[16], uint32_t (&c)[4]) {
    uint32_t m = w[0];
#pragma unroll
    for (int i = 1; i < 16; ++i) m = amax_pair(m, w[i]);
    const uint32_t s = e8m0_of<2>(max(m & 0x7FFFu, (m >> 16) & 0x7FFFu) << 16);
    const uint32_t f = (254u - s) << 7;  // 2^(127 - s) as a bf16: s <= 252 for a finite amax
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 r = scale_pair(w[4 * i + j], f);
            v[2 * j] = r.x;
            v[2 * j + 1] = r.y;
        }
        c[i] = cvt_e2m1x8(v);
    }
    if (s == 0xFFu) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float v[8] = {bf16lo(w[4 * i]), bf16hi(w[4 * i]), bf16lo(w[4 * i + 1]), bf16hi(w[4 * i + 1]),
                                bf16lo(w[4 * i + 2]), bf16hi(w[4 * i + 2]), bf16lo(w[4 * i + 3]), bf16hi(w[4 * i + 3])};
            c[i] = nonfinite_e2m1x8(v);
        }
    }
    return s;
}

// fp32 pairs, two lanes of one instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmul.rn.f32x2 z, x, y;\n\t"
        "mov.b64 {%0, %1}, z;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float rcp_approx(float x) {  // within 1 ulp
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// a / (1 + e^-a) of two values, as a/4 times the reciprocal of y = (1 + e^-a) / 4: that has no subnormal reciprocal
// below the largest finite e^-a.  One step of Newton's iteration, r + r (1 - y r), brings the reciprocal from 1 ulp to
// half of one, so that the whole is off by at most 2^-24 for the sum, the reciprocal and the product each, and
// expf's 2 ulp.  Where e^-a overflows, r is 0 and stays 0 (y is cut to a finite value in the step, 0 times it being 0):
// the result is -0, and NaN for a = -inf, as of the division.
__device__ __forceinline__ float2 silu2(float a, float b) {
    const float2 quarter = make_float2(0.25f, 0.25f);
    const float2 y = fma2(make_float2(expf(-a), expf(-b)), quarter, quarter);
    const float2 r = make_float2(rcp_approx(y.x), rcp_approx(y.y));
    const float2 e = fma2(make_float2(-fminf(y.x, 3.4e38f), -fminf(y.y, 3.4e38f)), r, make_float2(1.0f, 1.0f));
    return mul2(mul2(make_float2(a, b), quarter), fma2(r, e, r));
}

// EPT elements of a block (the other 32 / EPT - 1 shares are the neighbouring lanes') of silu(w) * g in fp32 -> the
// block's scale byte, this share's codes in c.
template <int EPT>
__device__ __forceinline__ uint32_t q4_share_swiglu(const uint32_t (&w)[EPT / 2], const uint32_t (&g)[EPT / 2],
                                                    uint32_t (&c)[EPT / 8]) {
    float v[EPT];
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < EPT / 2; ++i) {
        const float a = bf16lo(w[i]), b = bf16hi(w[i]);
        const float2 h = mul2(silu2(a, b), make_float2(bf16lo(g[i]), bf16hi(g[i])));
        v[2 * i] = h.x;
        v[2 * i + 1] = h.y;
        asm("max.NaN.abs.f32 %0, %0, %1, %2;" : "+f"(top) : "f"(h.x), "f"(h.y));  // NaN wins
    }
    uint32_t m = __float_as_uint(top);
#pragma unroll
    for (int d = 1; d < 32 / EPT; d <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
    const uint32_t s = e8m0_of<2>(m);
    const float f = __uint_as_float((254u - s) << 23);
#pragma unroll
    for (int i = 0; i < EPT / 8; ++i) {
        float z[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 h = mul2(make_float2(v[8 * i + 2 * j], v[8 * i + 2 * j + 1]), make_float2(f, f));
            z[2 * j] = h.x;
            z[2 * j + 1] = h.y;
        }
        c[i] = cvt_e2m1x8(z);
    }
    if (s == 0xFFu) {
#pragma unroll
        for (int i = 0; i < EPT / 8; ++i) {
            float z[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) z[j] = v[8 * i + j];
            c[i] = nonfinite_e2m1x8(z);
        }
    }
    return s;
}

// KIND's elements of a thread: a whole block of a plain quantization needs no shuffles, while SwiGLU's
// arithmetic wants more warps than its registers would leave with one.
template <int KIND>
__global__ void __launch_bounds__(kQ4Threads, KIND == kQ4Swiglu ? 6 : 5) mxfp4_quantize_kernel(const Q4Params p) {
    constexpr int EPT = KIND == kQ4Swiglu ? 16 : 32;
    constexpr int kLanes = 128 / EPT;        // lanes along a row's 128 columns
    constexpr int kRows = 32 / kLanes;       // rows a warp takes at a time
    const Q4Rows t = q4_rows(p);
    if (t.rows == 0) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int quarter = warp & 3;
    const int64_t C = p.C, ct = (C + 127) / 128;
    const int r0 = quarter * 32 + lane / kLanes;
    uint8_t* sb = p.s + t.b * p.s_bstride;
    for (int cc = 0; cc < p.cols_per_cta; ++cc) {
        const int64_t k128 = (blockIdx.y * (int64_t)p.cols_per_cta + cc) * (kQ4Cols / 128) + (warp >> 2);
        if (k128 >= ct) break;
        const int64_t c = k128 * 128 + (lane % kLanes) * EPT;
        const bool cin = c < C;
        int64_t at = (t.b * p.R + t.row0 + r0) * C + c;  // the thread's first element
        const int i0 = blockIdx.z * p.row_steps * kRows;
        at += i0 * C;
#pragma unroll 1
        for (int i = i0; i < i0 + p.row_steps * kRows; i += kRows, at += kRows * C) {
            const int r = r0 + i;
            const bool in = cin && r < t.rows;
            uint32_t w[EPT / 2], g[KIND == kQ4Swiglu ? EPT / 2 : 1], codes[EPT / 8], s;
#pragma unroll
            for (int j = 0; j < EPT / 8; ++j) {
                uint4 u = make_uint4(0, 0, 0, 0);
                if (in) u = *reinterpret_cast<const uint4*>(p.x + at * 2 + 16 * j);
                w[4 * j] = u.x; w[4 * j + 1] = u.y; w[4 * j + 2] = u.z; w[4 * j + 3] = u.w;
                if constexpr (KIND == kQ4Swiglu) {
                    if (in) u = *reinterpret_cast<const uint4*>(p.x2 + at * 2 + 16 * j);
                    g[4 * j] = u.x; g[4 * j + 1] = u.y; g[4 * j + 2] = u.z; g[4 * j + 3] = u.w;
                }
            }
            if constexpr (KIND == kQ4Swiglu) s = q4_share_swiglu<EPT>(w, g, codes);
            else s = q4_block_bf16(w, codes);
            if (in) {
                uint8_t* q = p.q + at / 2;
                if constexpr (EPT == 32) *reinterpret_cast<uint4*>(q) = make_uint4(codes[0], codes[1], codes[2], codes[3]);
                else if constexpr (EPT == 16) *reinterpret_cast<uint2*>(q) = make_uint2(codes[0], codes[1]);
                else *reinterpret_cast<uint32_t*>(q) = codes[0];
            }
            if (p.blocked) {
                // rows outside the group and columns past C were read as zeros: their scales are 0
                uint32_t word = s << (8 * ((lane % kLanes) / (32 / EPT)));
#pragma unroll
                for (int d = 32 / EPT; d < kLanes; d <<= 1) word |= __shfl_xor_sync(0xffffffffu, word, d);
                if (lane % kLanes == 0)
                    *reinterpret_cast<uint32_t*>(sb + (t.band * ct + k128) * 512 + (r & 31) * 16 + quarter * 4) = word;
            } else if (in && c % 32 == 0) {
                sb[(t.row0 + r) * (C / 32) + c / 32] = (uint8_t)s;
            }
        }
    }
}

__global__ void __launch_bounds__(kQ4Threads, 6) mxfp4_dequantize_kernel(const Q4Params p) {
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
#pragma unroll 1
        for (int b0 = blockIdx.z * p.row_steps * 8; b0 < (int)(blockIdx.z + 1) * p.row_steps * 8; b0 += 8) {
            uint32_t codes[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int r = rq + 2 * (b0 + i) + half;
                codes[i] = 0;
                if (cin && r < t.rows) codes[i] = *reinterpret_cast<const uint32_t*>(p.x + ((base + r) * C + c) / 2);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int r = rq + 2 * (b0 + i) + half;
                const uint32_t w = __shfl_sync(0xffffffffu, word, 2 * (b0 + i) + half);
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
    // few tiles: their row steps (a load's latency each) go to CTAs of their own
    const int steps = kind == kQ4Plain ? 4 : kind == kQ4Swiglu ? 8 : 2;
    int split = 1;
    while (split < steps && gx * gy * split * 2 <= 4 * (int64_t)host::num_sms()) split *= 2;
    p.row_steps = steps / split;
    const dim3 grid((unsigned)gx, (unsigned)gy, (unsigned)split);
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
