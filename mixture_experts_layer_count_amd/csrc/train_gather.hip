// What the FFN backward does token by token, between its products: the sum over
// a token's k expert rows,
//   dX[t] = sum_j rows[assign_row[t k + j]] (+ add[t]),
// in fp32 in ascending j, rounded once; the routing weights' gradients,
//   dw[t, j] = sum over column tiles of dw_part[tile][assign_row[t k + j]];
// and the token's row read back from its checkpoint for the weight gradients.
// HBM-bound: fp32 rows read once, bf16 written (65536 rows of 2048: 124 us,
// 5.0 TB/s). One block per token and 2048 columns, 8 columns (two 16-byte loads
// a row) a thread. As three launches: 12 us, so 5.4 (T 1536, k 2, H 640). Rows
// outside [0, *n_rows) (picks that the permutation left out) contribute nothing.
// A grid's dimension holds fewer than 2^32 threads (beyond, a launch takes their
// number mod 2^32 and reports nothing), and T may pass 2^24: the tokens go to
// the grid's z in runs of kRun.
#include "mx8.h"

namespace moe {

namespace {

constexpr int kRun = 1 << 16;  // tokens along x

__global__ __launch_bounds__(256) void gather_grads_kernel(GatherProblem p) {
    const int t = blockIdx.z * kRun + blockIdx.x, c = (blockIdx.y * 256 + threadIdx.x) * 8;
    if (t >= p.T) return;
    const int M = min(p.M, *p.n_rows);
    const long long o = (long long)t * p.H + c;
    u32x2 code;
    float scale;
    if (p.x && c < p.H) {  // on their way while the rows are summed
        code = *reinterpret_cast<const u32x2 *>(p.xq + o);
        scale = mx8::scale_of(p.xs[o / mx8::kGroup]);
    }
    if (p.dw && blockIdx.y == 0 && (int)threadIdx.x < p.k) {
        const long long a = (long long)t * p.k + threadIdx.x;
        const int r = p.assign_row ? p.assign_row[a] : t;
        float v = 0.0f;
        if (r >= 0 && r < M)
            for (int q = 0; q < p.n_part; ++q) v += p.dw_part[(long long)q * p.M + r];
        p.dw[a] = v;
    }
    if (c >= p.H) return;
    if (p.x) {
        const f32x4 a = mx8::values4(code[0], scale), b = mx8::values4(code[1], scale);
        *reinterpret_cast<u32x4 *>(p.x + o) = u32x4{pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]),
                                                    pack_bf16x2(b[0], b[1]), pack_bf16x2(b[2], b[3])};
    }
    if (!p.dX) return;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.0f;
    for (int j = 0; j < p.k; ++j) {
        const int r = p.assign_row ? p.assign_row[(long long)t * p.k + j] : t;
        if (r < 0 || r >= M) continue;
        const f32x4 *row = reinterpret_cast<const f32x4 *>(p.rows + (long long)r * p.H + c);
        const f32x4 a = row[0], b = row[1];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] += a[i];
            v[4 + i] += b[i];
        }
    }
    if (p.add) {
        const u32x4 s = *reinterpret_cast<const u32x4 *>(p.add + o);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] += bf16_lo(s[i]);
            v[2 * i + 1] += bf16_hi(s[i]);
        }
    }
    *reinterpret_cast<u32x4 *>(p.dX + o) = u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                 pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
}

}  // namespace

hipError_t launch_gather_grads(const GatherProblem &p, hipStream_t s) {
    if (p.T < 1 || p.k < 1 || p.k > 256 || !p.n_rows || p.H % 32 || (!p.assign_row && p.k != 1) || (p.dX && !p.rows) ||
        (p.dw && !p.dw_part) || (p.x && (!p.xq || !p.xs)))
        return hipErrorInvalidValue;
    if (!p.dX && !p.dw && !p.x) return hipSuccess;
    const unsigned columns = p.dX || p.x ? (unsigned)((p.H + 2047) / 2048) : 1;
    const unsigned runs = (unsigned)((p.T + (long long)kRun - 1) / kRun);
    hipLaunchKernelGGL(gather_grads_kernel, dim3((unsigned)(p.T < kRun ? p.T : kRun), columns, runs), dim3(256), 0, s,
                       p);
    return hipGetLastError();
}

}  // namespace moe
