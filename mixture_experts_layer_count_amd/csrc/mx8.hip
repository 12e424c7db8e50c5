// Activation checkpoints in 8 bits: packing rows to MXFP8 and reading them
// back (format: mx8.h).
//
// HBM-bound: bf16 in 2 B a value, 1 + 1/32 B out (and the reverse). A thread
// owns 16 consecutive values: two (fp32: four) 16-byte loads, one 16-byte
// code store; the two threads of a group exchange their maxima with one
// shuffle, and one of them stores the group's scale byte (32 contiguous bytes
// a wavefront). 32768 x 4096, medians: bf16 packed in 83 us (4.9 TB/s; at best
// 69), read back in 66 (6.2 TB/s; the 256 MB cache holds part of it); fp32
// packed in 119 (5.7 TB/s), read back in 174 (3.9 TB/s, 537 MB of it written).
#include "mx8.h"
#include "schedule.h"

namespace moe {
namespace {

using namespace mx8;

constexpr int kPer = 16;  // values per thread
constexpr long long kMaxThreads = 0xffffffffLL;  // of a launch (beyond, it takes their number mod 2^32)

// 16 values of X at element offset o
template <bool F32>
__device__ __forceinline__ void load16(const void *X, long long o, float (&v)[kPer]) {
    if constexpr (F32) {
        const f32x4 *p = reinterpret_cast<const f32x4 *>(reinterpret_cast<const float *>(X) + o);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const f32x4 x = p[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) v[4 * i + j] = x[j];
        }
    } else {
        const u32x4 *p = reinterpret_cast<const u32x4 *>(reinterpret_cast<const uint16_t *>(X) + o);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const u32x4 x = p[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[8 * i + 2 * j] = bf16_lo(x[j]);
                v[8 * i + 2 * j + 1] = bf16_hi(x[j]);
            }
        }
    }
}

template <bool F32>
__device__ __forceinline__ void pack16(const void *X, long long ldx, long long n, int C, uint8_t *Q, uint8_t *S,
                                       long long t) {
    const long long i = t * kPer;  // first value of this thread in the dense order
    // C is a multiple of 32: both threads of a group are in or out together
    if (i >= n) return;
    const long long row = i / C;
    float v[kPer];
    load16<F32>(X, ldx == C ? i : row * ldx + (i - row * C), v);
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) m = max(m, amax_bits(v[j]));
    m = max(m, (uint32_t)__shfl_xor((int)m, 1));
    const int e = scale_exp(m);
    const float inv = pow2(-e);
    u32x4 q;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        q[j] = codes4(scaled(v[4 * j], inv), scaled(v[4 * j + 1], inv), scaled(v[4 * j + 2], inv),
                      scaled(v[4 * j + 3], inv));
    *reinterpret_cast<u32x4 *>(Q + i) = q;
    if ((t & 1) == 0) S[i / kGroup] = (uint8_t)(e + 127);
}

template <bool F32>
__global__ __launch_bounds__(256) void mx8_pack_kernel(const void *X, long long ldx, long long n, int C, uint8_t *Q,
                                                       uint8_t *S) {
    pack16<F32>(X, ldx, n, C, Q, S, (long long)blockIdx.x * 256 + threadIdx.x);
}

// dense bf16 rows packed, and the tile list by the first workgroup (two
// launches took 2.4 us more of 53: 8 experts, T 1536, k 2, H 640, F 416)
__global__ __launch_bounds__(1024) void mx8_pack_tiles_kernel(const void *X, long long n, int C, uint8_t *Q, uint8_t *S,
                                                              TilesJob j) {
    __shared__ int scan_lds[16];
    if (blockIdx.x == 0)
        build_tiles(j.offsets, j.G, 0, j.bm, j.tiles, j.n_tiles, j.start, j.zero, j.n_zero, scan_lds);
    else
        pack16<false>(X, C, n, C, Q, S, (blockIdx.x - 1LL) * 1024 + threadIdx.x);
}

template <bool F32>
__global__ __launch_bounds__(256) void mx8_unpack_kernel(const uint8_t *Q, const uint8_t *S, long long n, void *Y) {
    const long long i = ((long long)blockIdx.x * 256 + threadIdx.x) * kPer;
    if (i >= n) return;
    const u32x4 q = *reinterpret_cast<const u32x4 *>(Q + i);
    const float s = scale_of(S[i / kGroup]);
    if constexpr (F32) {
        f32x4 *y = reinterpret_cast<f32x4 *>(reinterpret_cast<float *>(Y) + i);
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = values4(q[j], s);
    } else {
        u32x4 *y = reinterpret_cast<u32x4 *>(reinterpret_cast<uint16_t *>(Y) + i);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const f32x4 a = values4(q[2 * j], s), b = values4(q[2 * j + 1], s);
            y[j] = u32x4{pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]), pack_bf16x2(b[0], b[1]),
                         pack_bf16x2(b[2], b[3])};
        }
    }
}

}  // namespace

hipError_t launch_mx8_pack(const void *X, moe_dtype x_dt, long long ldx, long long R, int C, uint8_t *Q, uint8_t *S,
                           hipStream_t s) {
    if (R < 0 || C < mx8::kGroup || C % mx8::kGroup || ldx < C || (x_dt != MOE_F32 && x_dt != MOE_BF16))
        return hipErrorInvalidValue;
    if (R == 0) return hipSuccess;
    const long long n = R * C, blocks = (n / kPer + 255) / 256;
    if (blocks > kMaxThreads / 256) return hipErrorInvalidValue;
    if (x_dt == MOE_F32)
        hipLaunchKernelGGL(mx8_pack_kernel<true>, dim3((unsigned)blocks), dim3(256), 0, s, X, ldx, n, C, Q, S);
    else
        hipLaunchKernelGGL(mx8_pack_kernel<false>, dim3((unsigned)blocks), dim3(256), 0, s, X, ldx, n, C, Q, S);
    return hipGetLastError();
}

hipError_t launch_mx8_pack_tiles(const void *X, long long R, int C, uint8_t *Q, uint8_t *S, const TilesJob &tiles,
                                 hipStream_t s) {
    if (R < 0 || C < mx8::kGroup || C % mx8::kGroup || tiles.G < 1 || tiles.bm < 1 || tiles.n_zero < 0 ||
        (tiles.n_zero > 0 && !tiles.zero))
        return hipErrorInvalidValue;
    const long long n = R * C, blocks = (n / kPer + 1023) / 1024 + 1;
    if (blocks > kMaxThreads / 1024) return hipErrorInvalidValue;
    hipLaunchKernelGGL(mx8_pack_tiles_kernel, dim3((unsigned)blocks), dim3(1024), 0, s, X, n, C, Q, S, tiles);
    return hipGetLastError();
}

hipError_t launch_mx8_unpack(const uint8_t *Q, const uint8_t *S, long long R, int C, moe_dtype y_dt, void *Y,
                             hipStream_t s) {
    if (R < 0 || C < mx8::kGroup || C % mx8::kGroup || (y_dt != MOE_F32 && y_dt != MOE_BF16))
        return hipErrorInvalidValue;
    if (R == 0) return hipSuccess;
    const long long n = R * C, blocks = (n / kPer + 255) / 256;
    if (blocks > kMaxThreads / 256) return hipErrorInvalidValue;
    if (y_dt == MOE_F32)
        hipLaunchKernelGGL(mx8_unpack_kernel<true>, dim3((unsigned)blocks), dim3(256), 0, s, Q, S, n, Y);
    else
        hipLaunchKernelGGL(mx8_unpack_kernel<false>, dim3((unsigned)blocks), dim3(256), 0, s, Q, S, n, Y);
    return hipGetLastError();
}

}  // namespace moe
