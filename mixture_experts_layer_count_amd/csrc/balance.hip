// Balance loss, z loss and per-expert counts of a router, and the gradient at
// its logits.
//
// For tokens t with p = softmax(logits[t]) and lse = log sum exp(logits[t]),
// sequences b of n_b tokens (n_b > 0: B' of them, N tokens in all):
//   f_b[e]  = E / (k n_b) * #{(t in b, j): topk_idx[t, j] = e}
//   balance = alpha / B' sum_b sum_e f_b[e] 1/n_b sum_{t in b} p[t, e]
//   z       = beta / N sum_t lse[t]^2
//   dlogits[t, e] = d0 alpha / (B' n_b) p[t, e] (f_b[e] - sum_e' p[t, e'] f_b[e'])
//                 + d1 2 beta / N lse[t] p[t, e]
//                 + sum_{j: idx_j = e} w_j (dw_j - sum_j' w_j' dw_j')
// (counts have no gradient; the last line is the gradient of the
// renormalised top-k weights, a softmax over the k kept logits). A row whose
// logits are all -inf has p = 0 and lse = 0.
//
// Bound: instruction issue for many tokens (at 256 experts the VALU issues in
// 0.8 of the CUs' busy cycles, 104 instructions a token in the sums and 187 in
// the gradient, much of it lane reductions of six dependent steps that serve one
// token of a wavefront; the logits come at less than a copy's 4.9 TB/s), launch
// latency for few. A token's logits are held by LPT lanes, V = 4
// (16-byte loads) or 1 consecutive experts a lane, NI such pieces: LPT is the
// smallest power of two that covers E, so a layer of 8 experts puts 32 tokens
// on a wavefront and 256 experts one.
//
// Measured (sums, second kernel, gradient; medians): 64 tokens of 8 experts 3.0,
// 3.8 and 3.8 us; 8192 of 128 5.9, 7.2 and 8.2; 65536 of 256 19.6 (67 MB and the
// picks at 3.5 TB/s), 5.3 and 32.5 (140 MB at 4.3 TB/s).
//
// The sums over tokens are formed in a fixed order, so results are identical
// run to run: a block sums the tokens of one chunk, sequence by sequence, and
// writes one partial row per (chunk x, sequence b) it holds, at slot x + b
// (both only grow along the tokens, so slots are distinct and there are at
// most chunks + B). The second kernel adds a sequence's slots in ascending
// order; its last block to finish (a counter that the first kernel clears)
// adds the sequences. Counts are integers, so LDS atomics keep them exact.
#include <math.h>

#include <type_traits>

#include "train.h"

namespace moe {
namespace {

// x combined over the LPT lanes of a token (a power of two), in every lane of
// them: DPP permutations within 16 lanes, then row and half swaps. All VALU:
// with cross-lane LDS permutations these reductions were most of the kernels'
// time.
template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xf, 0xf, false));
}
template <int LPT, class Op>
__device__ __forceinline__ float combine_lanes(float x, Op op) {
    if constexpr (LPT >= 2) x = op(x, dpp<0xB1>(x));    // quad_perm [1,0,3,2]
    if constexpr (LPT >= 4) x = op(x, dpp<0x4E>(x));    // quad_perm [2,3,0,1]
    if constexpr (LPT >= 8) x = op(x, dpp<0x141>(x));   // row_half_mirror
    if constexpr (LPT >= 16) x = op(x, dpp<0x140>(x));  // row_mirror
    if constexpr (LPT >= 32) {
        const auto v = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
        x = op(__uint_as_float(v[0]), __uint_as_float(v[1]));
    }
    if constexpr (LPT >= 64) {
        const auto v = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
        x = op(__uint_as_float(v[0]), __uint_as_float(v[1]));
    }
    return x;
}
template <int LPT>
__device__ __forceinline__ float sum_lanes(float x) {
    return combine_lanes<LPT>(x, [](float p, float q) { return p + q; });
}
template <int LPT>
__device__ __forceinline__ float max_lanes(float x) {
    return combine_lanes<LPT>(x, [](float p, float q) { return fmaxf(p, q); });
}

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

struct BalanceArgs {
    const float *logits;
    const int32_t *idx;
    int T, E, k;
    const int32_t *seq;  // [B + 1] or null: one sequence of T tokens
    int B;
    int chunk;           // tokens per block
};

// tokens [lo, hi) of sequence b, kept inside [0, T)
__device__ __forceinline__ void seq_range(const BalanceArgs &a, int b, int &lo, int &hi) {
    lo = a.seq ? min(max(a.seq[b], 0), a.T) : 0;
    hi = a.seq ? min(max(a.seq[b + 1], lo), a.T) : a.T;
}
// the first sequence from b on that ends after token t (B if none). The offsets
// of a padded batch end in many empty sequences: one by one they took 0.17 us
// each (8192 tokens, the last 191 outside all of 1024 sequences: 207 us of loss
// and 149 of gradient in place of 43 and 13)
__device__ __forceinline__ int first_seq(const BalanceArgs &a, int b, int t) {
    if (!a.seq) return b;
    int lo = b, hi = a.B;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (a.seq[mid + 1] > t) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}
// the same where b itself is the likely one
__device__ __forceinline__ int next_seq(const BalanceArgs &a, int b, int t) {
    return b >= a.B || !a.seq || a.seq[b + 1] > t ? b : first_seq(a, b + 1, t);
}

template <int V, int NI, int LPT>
struct Row {
    static constexpr int per_wave = 64 / LPT;  // tokens per wavefront
    float x[NI][V];
    // expert of piece i, element 0, for lane li of the token's LPT
    static __device__ __forceinline__ int expert(int i, int li) { return (i * LPT + li) * V; }
    __device__ __forceinline__ void load(const float *row, int E, int li, bool ok) {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int e = expert(i, li);
            if constexpr (V == 4) {
                f32x4 v = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                if (ok && e < E) v = *reinterpret_cast<const f32x4 *>(row + e);
#pragma unroll
                for (int c = 0; c < 4; ++c) x[i][c] = v[c];
            } else {
                x[i][0] = (ok && e < E) ? row[e] : -INFINITY;
            }
        }
    }
    // x becomes p; returns lse (0 for a row of -inf only, with p = 0)
    __device__ __forceinline__ float softmax() {
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int c = 0; c < V; ++c) top = fmaxf(top, x[i][c]);
        top = max_lanes<LPT>(top);
        // a NaN logit is ignored by fmaxf and makes the sum, and so the row, NaN
        const float base = top == -INFINITY ? 0.0f : top;
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int c = 0; c < V; ++c) {
                // the hardware's exp2: p's relative error is about 2^-24 times
                // 2 + the logit's distance from the largest
                x[i][c] = __builtin_amdgcn_exp2f(1.4426950408889634f * (x[i][c] - base));
                sum += x[i][c];
            }
        sum = sum_lanes<LPT>(sum);
        const bool empty = sum == 0.0f;
        const float inv = empty ? 0.0f : 1.0f / sum;
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int c = 0; c < V; ++c) x[i][c] *= inv;
        return empty ? 0.0f : base + logf(sum);
    }
};

template <int V, int NI, int LPT>
__global__ __launch_bounds__(kThreads) void balance_sums_kernel(BalanceArgs a, float *partP, int32_t *partC,
                                                                float *partZ, int32_t *done, int32_t *counts) {
    typedef Row<V, NI, LPT> R;
    __shared__ float sP[kWaves][1024];
    __shared__ int32_t sC[1024];
    __shared__ float sZ[kWaves];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int li = lane % LPT, sub = lane / LPT;
    if (blockIdx.x == 0) {  // for the second kernel
        if (tid == 0) *done = 0;
        for (int e = tid; e < a.E; e += kThreads) counts[e] = 0;
    }
    const int t0 = blockIdx.x * a.chunk, t1 = min(t0 + a.chunk, a.T);
    for (int b = first_seq(a, 0, t0), pos = t0; b < a.B; b = next_seq(a, b + 1, pos)) {
        int lo, hi;
        seq_range(a, b, lo, hi);
        if (lo >= t1) break;
        lo = max(lo, t0);
        hi = min(hi, t1);
        pos = max(pos, hi);
        if (lo >= hi) continue;  // an empty sequence in front of all
        for (int e = tid; e < a.E; e += kThreads) sC[e] = 0;
        __syncthreads();
        for (long long i = (long long)lo * a.k + tid; i < (long long)hi * a.k; i += kThreads) {
            const int e = a.idx[i];
            if (e >= 0 && e < a.E) atomicAdd(&sC[e], 1);
        }
        float sum[NI][V], z = 0.0f;
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int c = 0; c < V; ++c) sum[i][c] = 0.0f;
        for (int tb = lo + w * R::per_wave; tb < hi; tb += kWaves * R::per_wave) {
            const int t = tb + sub;
            const bool ok = t < hi;
            R r;
            r.load(a.logits + (long long)(ok ? t : lo) * a.E, a.E, li, ok);
            const float lse = r.softmax();
            if (ok && li == 0) z += lse * lse;
#pragma unroll
            for (int i = 0; i < NI; ++i)
#pragma unroll
                for (int c = 0; c < V; ++c) sum[i][c] += r.x[i][c];
        }
        // the wavefront's tokens, then the block's wavefronts, in order
#pragma unroll
        for (int d = LPT; d < 64; d <<= 1)
#pragma unroll
            for (int i = 0; i < NI; ++i)
#pragma unroll
                for (int c = 0; c < V; ++c) sum[i][c] += __shfl_xor(sum[i][c], d);
#pragma unroll
        for (int d = 32; d >= 1; d >>= 1) z += __shfl_xor(z, d);
        if (sub == 0) {
#pragma unroll
            for (int i = 0; i < NI; ++i)
#pragma unroll
                for (int c = 0; c < V; ++c) {
                    const int e = R::expert(i, li) + c;
                    if (e < a.E) sP[w][e] = sum[i][c];
                }
        }
        if (lane == 0) sZ[w] = z;
        __syncthreads();
        const long long slot = (long long)blockIdx.x + b;
        for (int e = tid; e < a.E; e += kThreads) {
            float v = sP[0][e];
#pragma unroll
            for (int q = 1; q < kWaves; ++q) v += sP[q][e];
            partP[slot * a.E + e] = v;
            partC[slot * a.E + e] = sC[e];
        }
        if (tid == 0) partZ[slot] = (sZ[0] + sZ[1]) + (sZ[2] + sZ[3]);
        if (hi == t1) break;
        __syncthreads();
    }
}

// grid (slices of 64 experts, B): the sequence's counts and its share of the
// losses; the last block to finish adds the sequences
constexpr int kFinalThreads = 1024;
__global__ __launch_bounds__(kFinalThreads) void balance_final_kernel(BalanceArgs a, const float *partP,
                                                                      const int32_t *partC, const float *partZ,
                                                                      float alpha, float beta, int32_t *seq_counts,
                                                                      float *part_loss, int32_t *done, float *loss,
                                                                      int32_t *counts) {
    constexpr int NW = kFinalThreads / 64;
    __shared__ float sP[NW][64];
    __shared__ int32_t sC[NW][64];
    __shared__ int last;
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int b = blockIdx.y, e = blockIdx.x * 64 + lane, nsl = gridDim.x;
    int lo, hi;
    seq_range(a, b, lo, hi);
    const int x0 = lo / a.chunk, x1 = hi > lo ? (hi - 1) / a.chunk : x0 - 1;
    // wavefront w adds chunks x0 + w, x0 + w + NW, ..; then the wavefronts in order
    float p = 0.0f;
    int c = 0;
    if (e < a.E)
        for (int x = x0 + w; x <= x1; x += 4 * NW) {
            float pv[4];
            int cv[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const bool in = x + q * NW <= x1;
                const long long at = ((long long)(in ? x + q * NW : x) + b) * a.E + e;
                pv[q] = partP[at];
                cv[q] = partC[at];
                if (!in) {
                    pv[q] = 0.0f;
                    cv[q] = 0;
                }
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                p += pv[q];
                c += cv[q];
            }
        }
    sP[w][lane] = p;
    sC[w][lane] = c;
    __syncthreads();
    if (w == 0) {
#pragma unroll
        for (int q = 1; q < NW; ++q) {
            p += sP[q][lane];
            c += sC[q][lane];
        }
        if (e < a.E) {
            seq_counts[(long long)b * a.E + e] = c;
            if (c) atomicAdd(counts + e, c);
        }
        const float n = (float)(hi - lo);
        // f_b[e] P_b[e], the E experts of this slice
        float v = (e < a.E && hi > lo) ? ((float)c * (float)a.E / ((float)a.k * n)) * (p / n) : 0.0f;
        v = sum_lanes<64>(v);
        // the z sums of the sequence's chunks (slice 0)
        float z = 0.0f;
        if (blockIdx.x == 0) {
            for (int x = x0 + lane; x <= x1; x += 64) z += partZ[(long long)x + b];
            z = sum_lanes<64>(z);
        }
        // the partial losses and the count of finished blocks go past the L2 of
        // this XCD (device-scope accesses), the former complete before the
        // latter: no cache needs to be written back or dropped
        if (lane == 0) {
            float *mine = part_loss + 2 * ((long long)b * nsl + blockIdx.x);
            __hip_atomic_store(mine, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            __hip_atomic_store(mine + 1, z, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            last = __hip_atomic_fetch_add(done, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
                   (int)(gridDim.x * gridDim.y) - 1;
        }
    }
    __syncthreads();
    if (!last) return;
    if (w == 0) {
        // over sequences in 64 bits: they may be many
        double v = 0.0, z = 0.0;
        long long n = 0;
        int live = 0;
        for (int q = lane; q < a.B; q += 64) {
            int ql, qh;
            seq_range(a, q, ql, qh);
            n += qh - ql;
            live += qh > ql;
        }
        for (long long q = lane; q < (long long)a.B * nsl; q += 64) {
            v += __hip_atomic_load(part_loss + 2 * q, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            z += __hip_atomic_load(part_loss + 2 * q + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
#pragma unroll
        for (int d = 32; d >= 1; d >>= 1) {
            v += __shfl_xor(v, d);
            z += __shfl_xor(z, d);
            n += __shfl_xor(n, d);
            live += __shfl_xor(live, d);
        }
        if (lane == 0) {
            loss[0] = live ? (float)((double)alpha * v / live) : 0.0f;
            loss[1] = n ? (float)((double)beta * z / (double)n) : 0.0f;
        }
    }
}

struct RouteBackArgs {
    const float *w, *dw;        // [T, k] routing weights and their gradients (null: no routing term)
    const int32_t *seq_counts;  // [B, E] (null: no balance and z terms)
    const float *dloss;         // [2] (null: 1, 1)
    float alpha, beta;
    float *dlogits;
};

template <int V, int NI, int LPT>
__global__ __launch_bounds__(kThreads) void route_backward_kernel(BalanceArgs a, RouteBackArgs g) {
    typedef Row<V, NI, LPT> R;
    constexpr int KQ = V * NI < 4 ? V * NI : 4;  // picks per lane: k <= min(E, 64) <= KQ LPT
    __shared__ __attribute__((aligned(16))) float rows[kWaves][64 * NI * V];
    __shared__ int s_live, s_n;
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int li = lane % LPT, sub = lane / LPT;
    const int t0 = blockIdx.x * a.chunk, t1 = min(t0 + a.chunk, a.T);
    const bool aux = g.seq_counts != nullptr;
    // sequences that hold tokens, and their tokens
    if (aux) {
        if (w == 0) {
            int live = 0, n = 0;
            for (int q = lane; q < a.B; q += 64) {
                int ql, qh;
                seq_range(a, q, ql, qh);
                n += qh - ql;
                live += qh > ql;
            }
#pragma unroll
            for (int d = 32; d >= 1; d >>= 1) {
                n += __shfl_xor(n, d);
                live += __shfl_xor(live, d);
            }
            if (lane == 0) {
                s_live = live;
                s_n = n;
            }
        }
        __syncthreads();
    }
    const float d0 = g.dloss ? g.dloss[0] : 1.0f, d1 = g.dloss ? g.dloss[1] : 1.0f;
    // [pos, end): a run of tokens of one sequence, or of none
    int b = aux ? first_seq(a, 0, t0) : a.B;
    int pos = t0;
    while (pos < t1) {
        int end = t1;
        bool in_seq = false;
        int lo = 0, hi = 0;
        for (; b < a.B; b = next_seq(a, b + 1, pos)) {
            seq_range(a, b, lo, hi);
            if (hi <= pos) continue;  // behind
            in_seq = lo <= pos;
            end = min(t1, in_seq ? hi : lo);
            break;
        }
        // f_b[e] alpha d0 / (B' n_b) of this lane's experts
        float f[NI][V], zc = 0.0f;
        if (in_seq) {
            const float n = (float)(hi - lo);
            const float s = d0 * g.alpha * (float)a.E / ((float)a.k * n) / (n * (float)s_live);
            zc = d1 * 2.0f * g.beta / (float)s_n;
#pragma unroll
            for (int i = 0; i < NI; ++i)
#pragma unroll
                for (int c = 0; c < V; ++c) {
                    const int e = R::expert(i, li) + c;
                    f[i][c] = e < a.E ? s * (float)g.seq_counts[(long long)b * a.E + e] : 0.0f;
                }
        }
        for (int tb = pos + w * R::per_wave; tb < end; tb += kWaves * R::per_wave) {
            const int t = tb + sub;
            const bool ok = t < end;
            const long long row = ok ? t : pos;
            R r;
            int pick[KQ];
            float wv[KQ], dv[KQ];
            if (in_seq) r.load(a.logits + row * a.E, a.E, li, ok);
            if (g.dw) {
                // lane li holds picks li, li + LPT, ..
#pragma unroll
                for (int q = 0; q < KQ; ++q) {
                    const int j = li + q * LPT;
                    const bool in = ok && j < a.k;
                    const long long at = row * a.k + (in ? j : 0);
                    pick[q] = in ? a.idx[at] : -1;
                    wv[q] = in ? g.w[at] : 0.0f;
                    dv[q] = in ? g.dw[at] : 0.0f;
                }
            }
            if (in_seq) {
                const float lse = r.softmax();
                float dot = 0.0f;
#pragma unroll
                for (int i = 0; i < NI; ++i)
#pragma unroll
                    for (int c = 0; c < V; ++c) dot = fmaf(r.x[i][c], f[i][c], dot);
                dot = sum_lanes<LPT>(dot);
                const float base = zc * lse - dot;
#pragma unroll
                for (int i = 0; i < NI; ++i)
#pragma unroll
                    for (int c = 0; c < V; ++c) r.x[i][c] *= f[i][c] + base;
            } else {
#pragma unroll
                for (int i = 0; i < NI; ++i)
#pragma unroll
                    for (int c = 0; c < V; ++c) r.x[i][c] = 0.0f;
            }
            if (g.dw) {
                // w_j (dw_j - sum w dw) is added at its expert in an LDS copy of
                // the row (comparing every pick with every lane's experts in
                // registers took 8 us more of 54, 256 experts). Picks of one
                // expert are added in the order of their lanes
                float dot = 0.0f;
#pragma unroll
                for (int q = 0; q < KQ; ++q) dot = fmaf(wv[q], dv[q], dot);
                dot = sum_lanes<LPT>(dot);
                float *mine = rows[w] + sub * (LPT * NI * V);
#pragma unroll
                for (int i = 0; i < NI; ++i)
#pragma unroll
                    for (int c = 0; c < V; ++c) mine[R::expert(i, li) + c] = r.x[i][c];
                wave_lds_sync();
#pragma unroll
                for (int q = 0; q < KQ; ++q)
                    if (pick[q] >= 0 && pick[q] < a.E) atomicAdd(mine + pick[q], wv[q] * (dv[q] - dot));
                wave_lds_sync();
#pragma unroll
                for (int i = 0; i < NI; ++i)
#pragma unroll
                    for (int c = 0; c < V; ++c) r.x[i][c] = mine[R::expert(i, li) + c];
                wave_lds_sync();
            }
            if (!ok) continue;
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int e = R::expert(i, li);
                if (e >= a.E) continue;
                if constexpr (V == 4)
                    *reinterpret_cast<f32x4 *>(g.dlogits + row * a.E + e) =
                        f32x4{r.x[i][0], r.x[i][1], r.x[i][2], r.x[i][3]};
                else
                    g.dlogits[row * a.E + e] = r.x[i][0];
            }
        }
        pos = end;
    }
}

// tokens per block: enough blocks for every CU, at least 16 tokens each, and
// at most 64 (the partial rows stay below a sixteenth of the logits)
int chunk_tokens(int T) {
    int c = (int)((T + 1023LL) / 1024);
    c = (c + 15) / 16 * 16;
    return c < 16 ? 16 : c > 64 ? 64 : c;
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// calls fn with the row layout of E experts
template <class Fn>
void with_layout(int E, bool vec, Fn fn) {
    using std::integral_constant;
#define MOE_LAYOUT(V, NI, LPT) \
    fn(integral_constant<int, V>{}, integral_constant<int, NI>{}, integral_constant<int, LPT>{})
    if (vec) {
        if (E <= 8) MOE_LAYOUT(4, 1, 2);
        else if (E <= 16) MOE_LAYOUT(4, 1, 4);
        else if (E <= 32) MOE_LAYOUT(4, 1, 8);
        else if (E <= 64) MOE_LAYOUT(4, 1, 16);
        else if (E <= 128) MOE_LAYOUT(4, 1, 32);
        else if (E <= 256) MOE_LAYOUT(4, 1, 64);
        else if (E <= 512) MOE_LAYOUT(4, 2, 64);
        else MOE_LAYOUT(4, 4, 64);
    } else {
        if (E <= 16) MOE_LAYOUT(1, 1, 16);
        else if (E <= 64) MOE_LAYOUT(1, 1, 64);
        else if (E <= 256) MOE_LAYOUT(1, 4, 64);
        else MOE_LAYOUT(1, 16, 64);
    }
#undef MOE_LAYOUT
}

struct BalanceWs {
    float *partP, *partZ, *part_loss;
    int32_t *partC, *done;
};
size_t carve(void *ws, int T, int E, int B, BalanceWs &w) {
    const long long slots = ((long long)T + chunk_tokens(T) - 1) / chunk_tokens(T) + B;
    const long long nsl = (E + 63) / 64;
    size_t used = 0;
    auto take = [&](size_t bytes) {
        char *p = ws ? static_cast<char *>(ws) + used : nullptr;
        used += (bytes + 255) / 256 * 256;
        return p;
    };
    w.partP = reinterpret_cast<float *>(take(sizeof(float) * slots * E));
    w.partC = reinterpret_cast<int32_t *>(take(sizeof(int32_t) * slots * E));
    w.partZ = reinterpret_cast<float *>(take(sizeof(float) * slots));
    w.part_loss = reinterpret_cast<float *>(take(sizeof(float) * 2 * B * nsl));
    w.done = reinterpret_cast<int32_t *>(take(sizeof(int32_t)));
    return used;
}

}  // namespace

size_t balance_ws_bytes(int T, int E, int B) {
    BalanceWs w;
    return carve(nullptr, T, E, B, w);
}

hipError_t launch_balance_loss(const float *logits, const int32_t *idx, int T, int E, int k, const int32_t *seq, int B,
                               float alpha, float beta, float *loss, int32_t *counts, int32_t *seq_counts, void *ws,
                               hipStream_t s) {
    if (T < 0 || E < 1 || E > 1024 || k < 1 || k > 64 || B < 1 || B > 65535 || (!seq && B != 1))
        return hipErrorInvalidValue;
    BalanceWs w;
    carve(ws, T, E, B, w);
    const BalanceArgs a{logits, idx, T, E, k, seq, B, chunk_tokens(T)};
    // no tokens: one block, which only clears the counter
    const dim3 grid((unsigned)(T > 0 ? (T + a.chunk - 1) / a.chunk : 1));
    with_layout(E, E % 4 == 0 && aligned16(logits), [&](auto v, auto ni, auto lpt) {
        hipLaunchKernelGGL((balance_sums_kernel<decltype(v)::value, decltype(ni)::value, decltype(lpt)::value>), grid,
                           dim3(kThreads), 0, s, a, w.partP, w.partC, w.partZ, w.done, counts);
    });
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(balance_final_kernel, dim3((unsigned)((E + 63) / 64), (unsigned)B), dim3(kFinalThreads), 0, s, a,
                       w.partP, w.partC, w.partZ, alpha, beta, seq_counts, w.part_loss, w.done, loss, counts);
    return hipGetLastError();
}

hipError_t launch_route_backward(const float *logits, const int32_t *idx, const float *w, const float *dw, int T, int E,
                                 int k, const int32_t *seq, int B, const int32_t *seq_counts, float alpha, float beta,
                                 const float *dloss, float *dlogits, hipStream_t s) {
    if (T < 1 || E < 1 || E > 1024 || k < 1 || k > 64 || k > E || B < 1 || B > 65535 || (!seq && B != 1))
        return hipErrorInvalidValue;
    const BalanceArgs a{logits, idx, T, E, k, seq, B, chunk_tokens(T)};
    const RouteBackArgs g{w, dw, seq_counts, dloss, alpha, beta, dlogits};
    const dim3 grid((unsigned)((T + a.chunk - 1) / a.chunk));
    with_layout(E, E % 4 == 0 && aligned16(logits) && aligned16(dlogits), [&](auto v, auto ni, auto lpt) {
        hipLaunchKernelGGL((route_backward_kernel<decltype(v)::value, decltype(ni)::value, decltype(lpt)::value>), grid,
                           dim3(kThreads), 0, s, a, g);
    });
    return hipGetLastError();
}

}  // namespace moe
