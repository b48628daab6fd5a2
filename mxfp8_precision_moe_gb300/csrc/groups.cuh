// groups.cuh -- row groups as the kernels look them up: end rows, and first rows in the layout whose groups start at
// multiples of 128.
#pragma once

#include "common.cuh"

namespace mx {

// Warp 0 builds, for G groups over R rows, the clamped monotone end rows and
// the padded start rows P[g] = sum_{h<g} ceil(size_h/128)*128 (also the scale
// column base of a column-grouped layout, in units of 32 rows: P[g]/32).
// Returns the padded total through *total.
static __device__ __forceinline__ void build_group_table(const int32_t* offs, int G, int64_t R, int32_t* ends_s, int32_t* pstart_s,
                                  int32_t* total) {
    const int lane = threadIdx.x & 31;
    const int per = (G + 31) / 32;
    const int g0 = lane * per, g1 = min(G, g0 + per);
    const int32_t Rc = (int32_t)R;
    // pass 1: running max of clamped offsets (makes them monotone)
    int32_t mx = 0;
    for (int g = g0; g < g1; ++g) mx = max(mx, min(max(offs[g], 0), Rc));
    int32_t incl = mx;
    for (int d = 1; d < 32; d <<= 1) {
        int32_t o = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl = max(incl, o);
    }
    int32_t run = __shfl_up_sync(0xffffffffu, incl, 1);
    if (lane == 0) run = 0;
    // pass 2: ends, padded sizes, exclusive scan of padded sizes
    int32_t prev = run, psum = 0;
    for (int g = g0; g < g1; ++g) {
        int32_t e = max(prev, min(max(offs[g], 0), Rc));
        ends_s[g] = e;
        psum += ((e - prev + 127) / 128) * 128;
        prev = e;
    }
    int32_t sincl = psum;
    for (int d = 1; d < 32; d <<= 1) {
        int32_t o = __shfl_up_sync(0xffffffffu, sincl, d);
        if (lane >= d) sincl += o;
    }
    int32_t sexcl = sincl - psum;
    prev = run;
    for (int g = g0; g < g1; ++g) {
        pstart_s[g] = sexcl;
        int32_t e = ends_s[g];
        sexcl += ((e - prev + 127) / 128) * 128;
        prev = e;
    }
    if (lane == 31) *total = sincl;
}

// The table's padded rows are 32-bit numbers.
static inline bool padded_rows_fit(int64_t R, int32_t G) { return R + (int64_t)127 * G <= INT32_MAX; }

// Group of row r (ends_s monotone): first g with r < ends_s[g]; G if none.
__device__ __forceinline__ int find_group(const int32_t* ends_s, int G, int64_t r) {
    int lo = 0, hi = G;
    while (lo < hi) {
        int mid = (lo + hi) >> 1;
        if (r < ends_s[mid]) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

}  // namespace mx
