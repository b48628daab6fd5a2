// mx4.cuh -- device helpers of the MXFP4 kernels and of the routed layer for a few
// tokens: the E2M1 element rules and the lookup of a padded 128-row tile's group.
#pragma once

#include "common.cuh"
#include "../../include/mxfp4moe.h"

namespace mx {

// Shared scale byte of a block from the magnitude bits of its fp32 amax, for elements
// whose largest exponent is EMAX (2: E2M1, 8: E4M3): s = max(E - EMAX, 0), E the
// exponent field; Inf / NaN (E = 255) -> 0xFF.
template <int EMAX>
__device__ __forceinline__ uint32_t e8m0_of(uint32_t amax_bits) {
    const uint32_t E = amax_bits >> 23;
    if (E == 0xFFu) return 0xFFu;
    return E > (uint32_t)EMAX ? E - (uint32_t)EMAX : 0u;
}

// 2^(s - 127) as an fp32; 0xFF -> NaN, 0 -> the subnormal 2^-127.
__device__ __forceinline__ float e8m0_value(uint32_t s) {
    return __uint_as_float(s == 0xFFu ? 0x7FC00000u : s == 0u ? 0x00400000u : s << 23);
}

// Eight fp32 -> eight E2M1 codes (round to nearest even, saturated), v[0] in the lowest half byte.
__device__ __forceinline__ uint32_t cvt_e2m1x8(const float (&v)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

// The E2M1 codes of a non-finite block: 7 with each element's sign.
__device__ __forceinline__ uint32_t nonfinite_e2m1x8(const float (&v)[8]) {
    uint32_t r = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) r |= (7u | ((__float_as_uint(v[i]) >> 28) & 8u)) << (4 * i);
    return r;
}

// Two E2M1 codes (one byte) -> two fp32 values (exact).
__device__ __forceinline__ float2 e2m1x2_value(uint32_t byte) {
    uint32_t h;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b0;\n\t}"
        : "=r"(h)
        : "r"(byte));
    float lo, hi;
    asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(lo), "=f"(hi)
        : "r"(h));
    return make_float2(lo, hi);
}

// Where padded 128-row tile `t` of G row groups over M rows comes from.  Groups start on fresh
// 128-row tiles, so the tile's number is also its band in the blocked scale layout.
struct RowTile {
    int g;          // group, -1: past the last group
    int64_t row0;   // first source row
    int rows;       // its rows inside the group (1 .. 128)
};

// Called by one whole warp; the result is valid in every lane.  Offsets are clamped into [0, M] and made
// monotone, so that no row outside the matrix is ever named.
__device__ __forceinline__ RowTile locate_row_tile(const int32_t* offs, int G, int64_t M, int64_t t) {
    const int lane = threadIdx.x & 31;
    const int per = (G + 31) / 32;
    const int g0 = lane * per, g1 = min(G, g0 + per);
    const int32_t Mc = (int32_t)M;
    int32_t mx = 0;
    for (int g = g0; g < g1; ++g) mx = max(mx, min(max(offs[g], 0), Mc));
    int32_t incl = mx;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int32_t o = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl = max(incl, o);
    }
    int32_t run = __shfl_up_sync(0xffffffffu, incl, 1);
    if (lane == 0) run = 0;
    int32_t prev = run, tsum = 0;
    for (int g = g0; g < g1; ++g) {
        const int32_t e = max(prev, min(max(offs[g], 0), Mc));
        tsum += (e - prev + 127) / 128;
        prev = e;
    }
    int32_t tincl = tsum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int32_t o = __shfl_up_sync(0xffffffffu, tincl, d);
        if (lane >= d) tincl += o;
    }
    RowTile r{-1, 0, 0};
    int32_t first = tincl - tsum;
    prev = run;
    for (int g = g0; g < g1; ++g) {
        const int32_t e = max(prev, min(max(offs[g], 0), Mc));
        const int32_t n = (e - prev + 127) / 128;
        if (t >= first && t < first + n) {
            r.g = g;
            r.row0 = prev + (t - first) * 128;
            r.rows = (int)min64(128, e - r.row0);
        }
        first += n;
        prev = e;
    }
    const uint32_t who = __ballot_sync(0xffffffffu, r.g >= 0);
    const int src = who ? __ffs(who) - 1 : 0;
    r.g = __shfl_sync(0xffffffffu, r.g, src);
    r.row0 = __shfl_sync(0xffffffffu, r.row0, src);
    r.rows = __shfl_sync(0xffffffffu, r.rows, src);
    return r;
}

}  // namespace mx
