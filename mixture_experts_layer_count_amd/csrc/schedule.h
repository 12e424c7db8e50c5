// The tile list of the grouped GEMMs (schedule.hip), for kernels that build it
// beside other work.
#pragma once

#include "common.h"

namespace moe {

// by one workgroup of 1024 threads; scan_lds: 16 ints
__device__ __forceinline__ void build_tiles(const int32_t *offsets, int G, int extra_rows, int bm, int32_t *tiles,
                                            int32_t *n_tiles, int32_t *group_tile_start, int32_t *zero, int n_zero,
                                            int *scan_lds) {
    for (int i = threadIdx.x; i < n_zero; i += 1024) zero[i] = 0;
    const int NG = G + (extra_rows > 0 ? 1 : 0);
    int carry = 0;
    // groups in rounds of 1024; each thread emits its group's tiles
    for (int g0 = 0; g0 < NG; g0 += 1024) {
        const int g = g0 + threadIdx.x;
        int lo = 0, hi = 0, n = 0;
        if (g < NG) {
            lo = offsets[g];
            hi = g < G ? offsets[g + 1] : lo + extra_rows;
            n = (hi - lo + bm - 1) / bm;
            if (n < 0) n = 0;
        }
        int total = 0;
        const int first = block_exclusive_scan(n, scan_lds, &total) + carry;
        if (g < NG && group_tile_start) group_tile_start[g] = first;
        for (int i = 0; i < n; ++i) {
            int *t = tiles + 4 * (first + i);
            t[0] = g;
            t[1] = lo + i * bm;
            t[2] = min(lo + (i + 1) * bm, hi);
            t[3] = 0;
        }
        carry += total;
    }
    if (threadIdx.x == 0) {
        *n_tiles = carry;
        if (group_tile_start) group_tile_start[NG] = carry;
    }
}

}  // namespace moe
