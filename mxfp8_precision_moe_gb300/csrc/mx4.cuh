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

// Two of them: one byte.
__device__ __forceinline__ uint8_t cvt_e2m1x2(float lo, float hi) {
    uint32_t r;
    asm("{\n\t.reg .b8 b;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %2, %1;\n\tmov.b32 %0, {b, b, b, b};\n\t}"
        : "=r"(r)
        : "f"(lo), "f"(hi));
    return (uint8_t)r;
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

// Shared-memory descriptors by halves: the low word is address / 16 (14 bits) with the leading offset above it
// (unused by 128-byte swizzled tiles; 1), the high word is constant for tiles (stride 1024 bytes between 8-row
// groups, version 1, 128-byte swizzle) and for 32 x 16-byte scale tiles (stride 128, no swizzle).
constexpr uint32_t kDescLbo = 1u << 16;
constexpr uint32_t kDescTile = (1024u >> 4) | (1u << 14) | (2u << 29);
constexpr uint32_t kDescScale = (128u >> 4) | (1u << 14);
__device__ __forceinline__ uint64_t desc_of(uint32_t lo, uint32_t hi) { return ((uint64_t)hi << 32) | lo; }

// One lane of a converged warp.
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r;
}
// Operations of the lane whose `one` is set, in a loop that the whole warp walks: their descriptors and addresses then
// stay in uniform registers, where these instructions take them from.  Issued from a lane == 0 branch, each
// tcgen05.mma took about 70 cycles and each tcgen05.cp 56, which is what bounds a kernel whose MMAs are short.
__device__ __forceinline__ void cp_scales(uint32_t one, uint32_t taddr, uint64_t sdesc) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %0, 0;\n\t"
        "@q tcgen05.cp.cta_group::1.32x128b.warpx4 [%1], %2;\n\t}" ::"r"(one),
        "r"(taddr), "l"(sdesc)
        : "memory");
}
__device__ __forceinline__ void commit(uint32_t one, uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %0, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%1];\n\t}" ::"r"(one),
        "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void mma_mxf8(uint32_t one, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                         uint32_t sfb, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.u32 q, %7, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(
            d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb), "r"(one)
        : "memory");
}
__device__ __forceinline__ void mma_mxf4(uint32_t one, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                         uint32_t sfb, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.u32 q, %7, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb), "r"(one)
        : "memory");
}

// Whether a phase of an mbarrier has completed, without waiting; the same answer for a whole warp.
__device__ __forceinline__ uint32_t peek(uint64_t* bar, uint32_t parity) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred q;\n\tmbarrier.test_wait.parity.shared::cta.b64 q, [%1], %2;\n\t"
        "vote.sync.all.pred q, q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return r;
}

__device__ __forceinline__ void expect_tx(uint32_t one, uint64_t* bar, uint32_t bytes) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %2, 0;\n\t"
        "@q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(smem_u32(bar)),
        "r"(bytes), "r"(one)
        : "memory");
}
__device__ __forceinline__ void load_2d(uint32_t one, uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y,
                                        uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %5, 0;\n\t"
        "@q cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n\t}" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_u32(bar)), "r"(one)
        : "memory");
}
__device__ __forceinline__ void load_3d(uint32_t one, uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y, int32_t z,
                                        uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %6, 0;\n\t"
        "@q cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];\n\t}" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar)), "r"(one)
        : "memory");
}
__device__ __forceinline__ void load_bulk(uint32_t one, uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %4, 0;\n\t"
        "@q cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n\t}" ::"r"(dst),
        "l"(src), "r"(bytes), "r"(smem_u32(bar)), "r"(one)
        : "memory");
}

// The same for a CTA pair.
__device__ __forceinline__ void cp_scales_pair(uint32_t one, uint32_t taddr, uint64_t sdesc) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %0, 0;\n\t"
        "@q tcgen05.cp.cta_group::2.32x128b.warpx4 [%1], %2;\n\t}" ::"r"(one),
        "r"(taddr), "l"(sdesc)
        : "memory");
}
__device__ __forceinline__ void commit_pair(uint32_t one, uint64_t* bar, uint16_t cta_mask) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %0, 0;\n\t"
        "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%1], %2;\n\t}" ::"r"(
            one),
        "r"(smem_u32(bar)), "h"(cta_mask)
        : "memory");
}
__device__ __forceinline__ void mma_pair_mxf4(uint32_t one, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                              uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.u32 q, %7, 0;\n\t"
        "@q tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb), "r"(one)
        : "memory");
}
__device__ __forceinline__ void load_2d_pair(uint32_t one, uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y,
                                             uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %5, 0;\n\t"
        "@q cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
        "%3}], [%4];\n\t}" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar), "r"(one)
        : "memory");
}
__device__ __forceinline__ void load_3d_pair(uint32_t one, uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y,
                                             int32_t z, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %6, 0;\n\t"
        "@q cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, "
        "%4}], [%5];\n\t}" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar), "r"(one)
        : "memory");
}

}  // namespace mx
