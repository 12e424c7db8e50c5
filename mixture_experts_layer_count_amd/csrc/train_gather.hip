// Token gradients of the FFN backward: the sum over a token's k expert rows,
//   dX[t] = sum_j rows[assign_row[t k + j]] (+ add[t]),
// in fp32 in ascending j, rounded once; and the routing weights' gradients,
//   dw[t, j] = sum over column tiles of dw_part[tile][assign_row[t k + j]].
// HBM-bound: fp32 rows read once, bf16 written. One block per token and 2048
// columns, 8 columns (two 16-byte loads a row) a thread. Rows outside [0, *n_rows)
// (picks that the permutation left out) contribute nothing.
#include "common.h"

namespace moe {

MOE_BOUNDS_FILE(train_gather)

namespace {

__global__ __launch_bounds__(256) void gather_grads_kernel(const float *rows, const int32_t *assign_row, int k,
                                                           const int32_t *n_rows, int M, int H, const uint16_t *add, uint16_t *dX) {
    const int t = blockIdx.x, c = (blockIdx.y * 256 + threadIdx.x) * 8;
    if (c >= H) return;
    M = min(M, *n_rows);
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.0f;
    for (int j = 0; j < k; ++j) {
        const int r = assign_row ? assign_row[(long long)t * k + j] : t;
        if (r < 0 || r >= M) continue;
        const f32x4 *p = reinterpret_cast<const f32x4 *>(rows + (long long)r * H + c);
        const f32x4 a = p[0], b = p[1];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] += a[i];
            v[4 + i] += b[i];
        }
    }
    const long long o = (long long)t * H + c;
    if (add) {
        const u32x4 s = *reinterpret_cast<const u32x4 *>(add + o);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] += bf16_lo(s[i]);
            v[2 * i + 1] += bf16_hi(s[i]);
        }
    }
    *reinterpret_cast<u32x4 *>(dX + o) = u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                               pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
}

__global__ __launch_bounds__(256) void gather_dw_kernel(const float *part, int n_part, const int32_t *assign_row,
                                                        long long A, const int32_t *n_rows, int M, float *dw) {
    const long long a = (long long)blockIdx.x * 256 + threadIdx.x;
    if (a >= A) return;
    const int r = assign_row ? assign_row[a] : (int)a;
    float v = 0.0f;
    if (r >= 0 && r < min(M, *n_rows))
        for (int q = 0; q < n_part; ++q) v += part[(long long)q * M + r];
    dw[a] = v;
}

}  // namespace

hipError_t launch_gather_grads(const float *rows, const float *dw_part, int n_part, const int32_t *assign_row, int T,
                               int k, const int32_t *n_rows, int M, int H, const void *add, void *dX, float *dw, hipStream_t s) {
    if (T < 1 || k < 1 || !n_rows || H % 8 || (!assign_row && k != 1)) return hipErrorInvalidValue;
    if (dX) {
        if (!rows) return hipErrorInvalidValue;
        hipLaunchKernelGGL(gather_grads_kernel, dim3((unsigned)T, (unsigned)((H + 2047) / 2048)), dim3(256), 0, s, rows,
                           assign_row, k, n_rows, M, H, static_cast<const uint16_t *>(add), static_cast<uint16_t *>(dX));
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (dw) {
        if (!dw_part) return hipErrorInvalidValue;
        const long long A = (long long)T * k;
        hipLaunchKernelGGL(gather_dw_kernel, dim3((unsigned)((A + 255) / 256)), dim3(256), 0, s, dw_part, n_part,
                           assign_row, A, n_rows, M, dw);
        return hipGetLastError();
    }
    return hipSuccess;
}

}  // namespace moe
