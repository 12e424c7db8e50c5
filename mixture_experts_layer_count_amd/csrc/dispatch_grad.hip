// Gradients of the rows sorted by expert (moe_permute's Xp) and of the weighted
// sum back to tokens (moe_combine), for experts of any form.
//
// With r = assign_row[a], a = t k + j:
//   combine   dYp[r] = w[a] dY[t],  dw[a] = sum_h Yp[r, h] dY[t, h]
//   permute   dX[t] = sum_j dXp[r] (+ add[t])
// HBM-bound: combine reads T + M rows and writes M, permute reads M (+ T) and
// writes T: combine 118 us (4.8 TB/s) at M 65536, T 8192, H 2048, bf16; permute 113 us
// (5.2 TB/s) at M 32768, T 4096, H 7168 with add; a copy runs at 4.5 TB/s. Sums are
// fp32, in a fixed order, rounded once. Rows outside [0, min(M, *n_rows)) are picks that
// the permutation left out.
#include "train.h"

namespace moe {
namespace {

// V consecutive values as one access: 16 bytes, or 8 where H is no multiple of 8
template <typename E, int V>
struct Unit {
    static constexpr int words = V * (int)sizeof(E) / 4;
    uint32_t w[words];
    __device__ __forceinline__ float operator[](int i) const {
        if constexpr (sizeof(E) == 4) return __uint_as_float(w[i]);
        else return (i & 1) ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]);
    }
};
template <typename E, int V>
__device__ __forceinline__ Unit<E, V> load(const E *p) {
    Unit<E, V> u;
    if constexpr (Unit<E, V>::words == 4) {
        const u32x4 x = *reinterpret_cast<const u32x4 *>(p);
        u.w[0] = x[0], u.w[1] = x[1], u.w[2] = x[2], u.w[3] = x[3];
    } else {
        const u32x2 x = *reinterpret_cast<const u32x2 *>(p);
        u.w[0] = x[0], u.w[1] = x[1];
    }
    return u;
}
template <typename E, int V>
__device__ __forceinline__ void store(E *p, const float (&v)[V]) {
    if constexpr (sizeof(E) == 4)
        *reinterpret_cast<f32x4 *>(p) = f32x4{v[0], v[1], v[2], v[3]};
    else if constexpr (V == 8)
        *reinterpret_cast<u32x4 *>(p) = u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                              pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
    else
        *reinterpret_cast<u32x2 *>(p) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
}

// ---- combine: a workgroup a token. dY's row is kept in registers (U units a
// thread, more columns in further passes) while the token's k rows stream
// through; each wavefront's part of a dot product waits in LDS for the others ----
constexpr int kMaxPicks = 64;
template <typename E, int V, int BS, int U>
__global__ __launch_bounds__(BS) void combine_back_kernel(CombineBack p) {
    constexpr int NWV = BS / 64;
    __shared__ float part[NWV][kMaxPicks];
    const int t = blockIdx.x, lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    const int M = p.n_rows ? min(p.T * p.k, *p.n_rows) : p.T * p.k;
    const E *dY = reinterpret_cast<const E *>(p.dY) + (long long)t * p.H;
    const E *Yp = reinterpret_cast<const E *>(p.Yp);
    E *dYp = reinterpret_cast<E *>(p.dYp);
    for (int c0 = 0; c0 < p.H; c0 += BS * V * U) {
        Unit<E, V> d[U];
        int c[U];
        bool in[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            c[u] = c0 + (u * BS + threadIdx.x) * V;
            in[u] = c[u] < p.H;
            if (!in[u]) c[u] = 0;  // reads the row's first unit, which counts for nothing
            d[u] = load<E, V>(dY + c[u]);
        }
#pragma unroll 2
        for (int j = 0; j < p.k; ++j) {
            const long long a = (long long)t * p.k + j;
            const int r = p.assign_row[a];
            float dot = 0.0f;
            if (r >= 0 && r < M) {
                const float w = p.dYp ? p.w[a] : 0.0f;
                const long long o = (long long)r * p.H;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    Unit<E, V> y{};
                    if (p.dw) y = load<E, V>(Yp + o + c[u]);
                    float v[V], s = 0.0f;
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        s = fmaf(y[i], d[u][i], s);
                        v[i] = w * d[u][i];
                    }
                    if (in[u]) {
                        dot += s;
                        if (p.dYp) store<E, V>(dYp + o + c[u], v);
                    }
                }
            }
            if (p.dw) {
#pragma unroll
                for (int x = 32; x >= 1; x >>= 1) dot += __shfl_xor(dot, x);
                if (lane == 0) part[wv][j] = c0 == 0 ? dot : part[wv][j] + dot;
            }
        }
    }
    if (!p.dw) return;
    __syncthreads();
    for (int j = threadIdx.x; j < p.k; j += BS) {
        float s = part[0][j];
#pragma unroll
        for (int x = 1; x < NWV; ++x) s += part[x][j];
        p.dw[(long long)t * p.k + j] = s;
    }
}

// ---- combine of short rows: L lanes a token, a unit each, 256 / L tokens a workgroup;
// four of a token's rows in flight ----
template <typename E, int V, int L>
__global__ __launch_bounds__(256) void combine_back_short_kernel(CombineBack p) {
    const long long t = (long long)blockIdx.x * (256 / L) + threadIdx.x / L;
    if (t >= p.T) return;  // a token's lanes together
    const int lane = threadIdx.x % L, M = p.n_rows ? min(p.T * p.k, *p.n_rows) : p.T * p.k;
    const bool in = lane * V < p.H;
    const int c = in ? lane * V : 0;  // others read the row's first unit, which counts for nothing
    const E *Yp = reinterpret_cast<const E *>(p.Yp) + c;
    E *dYp = reinterpret_cast<E *>(p.dYp) + c;
    const Unit<E, V> d = load<E, V>(reinterpret_cast<const E *>(p.dY) + t * p.H + c);
    for (int j0 = 0; j0 < p.k; j0 += 4) {
        int r[4];
        float w[4], dot[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const long long a = t * p.k + j0 + u;
            r[u] = j0 + u < p.k ? p.assign_row[a] : -1;
            w[u] = j0 + u < p.k && p.dYp ? p.w[a] : 0.0f;
            if (r[u] >= M) r[u] = -1;
        }
        Unit<E, V> y[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            y[u] = Unit<E, V>{};
            if (p.dw && r[u] >= 0) y[u] = load<E, V>(Yp + (long long)r[u] * p.H);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            dot[u] = 0.0f;
            float v[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                dot[u] = fmaf(y[u][i], d[i], dot[u]);
                v[i] = w[u] * d[i];
            }
            if (!in || r[u] < 0) dot[u] = 0.0f;
            else if (p.dYp) store<E, V>(dYp + (long long)r[u] * p.H, v);
        }
        if (!p.dw) continue;
#pragma unroll
        for (int x = L / 2; x >= 1; x >>= 1)
#pragma unroll
            for (int u = 0; u < 4; ++u) dot[u] += __shfl_xor(dot[u], x);
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (lane == 0 && j0 + u < p.k) p.dw[t * p.k + j0 + u] = dot[u];
    }
}

// ---- permute: a thread a unit of a token's row; up to 8 rows in flight ----
template <typename E, int V>
__global__ __launch_bounds__(256) void permute_back_kernel(PermuteBack p, long long threads) {
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= threads) return;
    const int units = p.H / V;
    const int t = (int)(i / units), c = (int)(i - (long long)t * units) * V;
    const int M = p.n_rows ? min(p.T * p.k, *p.n_rows) : p.T * p.k;
    const E *rows = reinterpret_cast<const E *>(p.dXp);
    float v[V];
#pragma unroll
    for (int x = 0; x < V; ++x) v[x] = 0.0f;
    for (int j0 = 0; j0 < p.k; j0 += 8) {
        int r[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            r[u] = j0 + u < p.k ? p.assign_row[(long long)t * p.k + j0 + u] : -1;
            if (r[u] >= M) r[u] = -1;
        }
        Unit<E, V> y[8];
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (r[u] >= 0) y[u] = load<E, V>(rows + (long long)r[u] * p.H + c);
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (r[u] >= 0)
#pragma unroll
                for (int x = 0; x < V; ++x) v[x] += y[u][x];
    }
    const long long o = (long long)t * p.H + c;
    if (p.add) {
        const Unit<E, V> y = load<E, V>(reinterpret_cast<const E *>(p.add) + o);
#pragma unroll
        for (int x = 0; x < V; ++x) v[x] += y[x];
    }
    store<E, V>(reinterpret_cast<E *>(p.dX) + o, v);
}

template <typename E, int V, int BS, int U>
hipError_t combine_back(const CombineBack &p, hipStream_t s) {
    hipLaunchKernelGGL((combine_back_kernel<E, V, BS, U>), dim3((unsigned)p.T), dim3(BS), 0, s, p);
    return hipGetLastError();
}
template <typename E, int V, int L>
hipError_t combine_back_short(const CombineBack &p, hipStream_t s) {
    hipLaunchKernelGGL((combine_back_short_kernel<E, V, L>), dim3((unsigned)((p.T + 256 / L - 1) / (256 / L))), dim3(256),
                       0, s, p);
    return hipGetLastError();
}
template <typename E, int V>
hipError_t combine_back(const CombineBack &p, hipStream_t s) {
    // 32768 tokens, k 8, bf16, against a wavefront and workgroup a token: H 32 9.5 and 45 us,
    // H 128 24 and 47, H 512 113 and 118
    if (p.H <= 8 * V) return combine_back_short<E, V, 8>(p, s);
    if (p.H <= 16 * V) return combine_back_short<E, V, 16>(p, s);
    if (p.H <= 32 * V) return combine_back_short<E, V, 32>(p, s);
    if (p.H <= 64 * V) return combine_back_short<E, V, 64>(p, s);
    // bf16, 8192 tokens, k 8, us: H 1024 52 (two wavefronts 59, four 78), H 2048 118 (two
    // units a thread 126, one wavefront 137), H 4096 half the tokens 118 (one unit 120,
    // four 130); 64 tokens, k 8, H 7168 15 with four units, 18 with two, 25 with one
    if (p.H <= 128 * V) return combine_back<E, V, 64, 2>(p, s);
    if (p.H <= 256 * V) return combine_back<E, V, 256, 1>(p, s);
    if (p.H <= 512 * V) return combine_back<E, V, 256, 2>(p, s);
    return combine_back<E, V, 256, 4>(p, s);
}
template <typename E, int V>
hipError_t permute_back(const PermuteBack &p, hipStream_t s) {
    const long long threads = (long long)p.T * (p.H / V);
    hipLaunchKernelGGL((permute_back_kernel<E, V>), dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, s, p,
                       threads);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_combine_back(const CombineBack &p, moe_dtype dt, hipStream_t s) {
    if (p.T < 1 || p.T > kCombineBackTokens || p.k < 1 || p.k > kMaxPicks || p.H < 4 || p.H % 4)
        return hipErrorInvalidValue;
    if (dt == MOE_F32) return combine_back<float, 4>(p, s);
    return p.H % 8 ? combine_back<uint16_t, 4>(p, s) : combine_back<uint16_t, 8>(p, s);
}

hipError_t launch_permute_back(const PermuteBack &p, moe_dtype dt, hipStream_t s) {
    if (p.T < 1 || p.k < 1 || p.H < 4 || p.H % 4 || (long long)p.T * p.H > kPermuteBackValues)
        return hipErrorInvalidValue;
    if (dt == MOE_F32) return permute_back<float, 4>(p, s);
    return p.H % 8 ? permute_back<uint16_t, 4>(p, s) : permute_back<uint16_t, 8>(p, s);
}

}  // namespace moe
