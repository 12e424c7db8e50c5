// Device-side tile list for the grouped GEMMs.
//
// Page "MOE推理流程解析" §二: one launch runs every expert's matrix even though
// their row counts differ. The row counts live on the device (they come out
// of the permutation), so the list of (expert, first row) tiles is built on
// the device too: no device-to-host copy, and the whole layer stays capturable
// in a HIP graph. The GEMM grids are sized for the worst case
// (ceil(M / bm) + G tiles) and surplus workgroups exit at once.
#include "schedule.h"

namespace moe {
namespace {

__global__ __launch_bounds__(1024) void build_tiles_kernel(const int32_t *offsets, int G, int extra_rows,
                                                           int bm, int32_t *tiles, int32_t *n_tiles,
                                                           int32_t *group_tile_start, int32_t *zero,
                                                           int n_zero) {
    __shared__ int scan_lds[16];
    build_tiles(offsets, G, extra_rows, bm, tiles, n_tiles, group_tile_start, zero, n_zero, scan_lds);
}

}  // namespace

hipError_t launch_build_tiles(const int32_t *offsets, int G, int extra_rows, int bm, int32_t *tiles,
                              int32_t *n_tiles, int32_t *group_tile_start, hipStream_t s, int32_t *zero,
                              int n_zero) {
    if (G < 1 || bm < 1 || extra_rows < 0 || n_zero < 0 || (n_zero > 0 && !zero)) return hipErrorInvalidValue;
    hipLaunchKernelGGL(build_tiles_kernel, dim3(1), dim3(1024), 0, s, offsets, G, extra_rows, bm, tiles,
                       n_tiles, group_tile_start, zero, n_zero);
    return hipGetLastError();
}

}  // namespace moe
