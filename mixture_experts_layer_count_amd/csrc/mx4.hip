// MXFP4 quantisation of rows and of weight matrices, and reading them back
// (format: mx4.h).
//
// HBM-bound: 2 (fp32: 4) bytes a value in, 17/32 out, and the reverse. A value's
// arithmetic is about one instruction (a conversion takes two values and the packed
// maximum two), so bf16 stays in pairs as it lies in memory. About the copy's rate of 4.5 TB/s
// or above, fastest and median of 20 calls. bf16: rows 32768 x 4096 (339 MB) 64 and 78 us
// (5.3 and 4.3 TB/s), back 49 and 50; weights 8 x 4096 x 14336 (1.19 GB) 225 and 260 (5.3 and
// 4.6), back 194 and 195 (6.1). fp32: rows 16384 x 7168 (532 MB) 95 and 103 (5.6 and 5.2),
// back 89 and 94; the same weights (2.13 GB) 400 and 411 (5.3 and 5.2), back 384 and 391.
#include "mx4.h"
#include "schedule.h"
#include "train.h"

namespace moe {

MOE_BOUNDS_FILE(mx4)

namespace {

using namespace mx4;

constexpr long long kMaxThreads = 0xffffffffLL;  // of a launch (beyond, it takes their number mod 2^32)
// fewer threads of two words take one: 16384: 4.0 against 4.5 us, 32768: 6.6 against 5.2
constexpr long long kFewThreads = 1 << 15;
constexpr int kPer = 16;  // values per thread of the row kernels

// the largest of a lane and its neighbour, and of the four lanes of a quad
__device__ __forceinline__ uint32_t pair_max(uint32_t v) {
    return max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xb1, 0xf, 0xf, true));  // lanes 1 0 3 2
}
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
    v = pair_max(v);
    return max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4e, 0xf, 0xf, true));  // lanes 2 3 0 1
}

// 8 consecutive fp32 values
__device__ __forceinline__ void load8(const float *p, float (&v)[8]) {
    const f32x4 a = reinterpret_cast<const f32x4 *>(p)[0], b = reinterpret_cast<const f32x4 *>(p)[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = a[i];
        v[4 + i] = b[i];
    }
}

// ---- rows: a thread owns 16 consecutive values; the two threads of a group
// exchange their maxima, and one of them stores the scale byte ----
template <bool F32>
__global__ __launch_bounds__(256) void mx4_rows_kernel(const void *X, long long ldx, long long n, int C, uint8_t *Q,
                                                       uint8_t *S) {
    const long long t = (long long)blockIdx.x * 256 + threadIdx.x, i = t * kPer;
    // C is a multiple of 32: both threads of a group are in or out together
    if (i >= n) return;
    long long o = i;
    if (ldx != C) {
        const long long row = i / C;
        o = row * ldx + (i - row * C);
    }
    uint32_t m, b;
    u32x2 q;
    if constexpr (F32) {
        float v[2][8];
        load8(static_cast<const float *>(X) + o, v[0]);
        load8(static_cast<const float *>(X) + o + 8, v[1]);
        m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, max(mag_bits(v[0][j]), mag_bits(v[1][j])));
        b = scale_byte(pair_max(m));
        q = u32x2{codes8(v[0], b), codes8(v[1], b)};
    } else {
        const u32x4 *x = reinterpret_cast<const u32x4 *>(reinterpret_cast<const uint16_t *>(X) + o);
        const u32x4 x0 = x[0], x1 = x[1];
        b = scale_byte(pair_max(max(max_bits(x0), max_bits(x1))));
        q = u32x2{codes8(x0, b), codes8(x1, b)};
    }
    *reinterpret_cast<u32x2 *>(Q + i / 2) = q;
    if ((t & 1) == 0) S[i / kGroup] = (uint8_t)b;
}

typedef float f32x2 __attribute__((ext_vector_type(2)));

// the NaN scale of a group, applied by the caller (the conversions read
// exponent 255 as a power of two)
__device__ __forceinline__ float nan_if(uint32_t byte, float x) {
    return byte == 255u ? __uint_as_float(0x7fc00000u) : x;
}

// 16 bytes of values: 8 of bf16, 4 of fp32
template <bool F32>
__device__ __forceinline__ void store16(void *Y, long long o, const float *v) {
    if constexpr (F32)
        *reinterpret_cast<f32x4 *>(reinterpret_cast<float *>(Y) + o) = f32x4{v[0], v[1], v[2], v[3]};
    else
        *reinterpret_cast<u32x4 *>(reinterpret_cast<uint16_t *>(Y) + o) =
            u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
}
template <bool F32>
constexpr int kBack = F32 ? 4 : 8;  // values of a store

// A store of 16 bytes a lane, a wavefront's one after the other, and 16 / kBack of them a
// thread: 16384 x 7168 fp32 89 us, bf16 52 (16 consecutive values a thread: 148, 55)
template <bool F32>
__global__ __launch_bounds__(256) void mx4_rows_back_kernel(const uint8_t *Q, const uint8_t *S, long long n, void *Y) {
    constexpr int U = kBack<F32>;
    const long long base = (long long)blockIdx.x * 256 * kPer + threadIdx.x * U;
    uint32_t q[kPer / U], b[kPer / U];
#pragma unroll
    for (int u = 0; u < kPer / U; ++u) {
        const long long i = base + u * 256 * U;
        q[u] = b[u] = 0;
        if (i >= n) continue;
        if constexpr (F32) q[u] = *reinterpret_cast<const uint16_t *>(Q + i / 2);
        else q[u] = *reinterpret_cast<const uint32_t *>(Q + i / 2);
        b[u] = S[i / kGroup];
    }
#pragma unroll
    for (int u = 0; u < kPer / U; ++u) {
        const long long i = base + u * 256 * U;
        const f32x2 x[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[u], scale_of(b[u]), 0),
                            __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[u], scale_of(b[u]), 1),
                            __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[u], scale_of(b[u]), 2),
                            __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[u], scale_of(b[u]), 3)};
        float v[U];
#pragma unroll
        for (int j = 0; j < U; ++j) v[j] = nan_if(b[u], x[j / 2][j & 1]);
        if (i < n) store16<F32>(Y, i, v);
    }
}

// byte J of a code word, from the values of two rows: fp32 bits, or the bf16 of
// columns J & 1 in two words of two columns
template <int J>
__device__ __forceinline__ uint32_t codes_f32(uint32_t w, uint32_t lo, uint32_t hi, float s) {
    return (uint32_t)__builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, __uint_as_float(lo), __uint_as_float(hi), s, J);
}
template <int J>
__device__ __forceinline__ uint32_t codes_bf16(uint32_t w, uint32_t lo, uint32_t hi, float s) {
    const uint32_t pair = __builtin_amdgcn_perm(hi, lo, J & 1 ? 0x07060302u : 0x05040100u);
    return (uint32_t)__builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, pair_of(pair), s, J);
}

// ---- weights [G][K][N]: a thread owns 4 WORDS columns of one group of 32 K rows
// (bf16 with 2 WORDS: a wavefront's rows are 1 KB of values, 512 bytes of codes), its
// values kept in registers between the maximum and the codes. fp32 takes one word:
// two would be 256 registers of values ----
template <bool F32, int WORDS>
__global__ __launch_bounds__(256) void mx4_weights_kernel(const void *W, long long threads, int N, uint8_t *Q,
                                                          uint8_t *S) {
    typedef uint32_t Words __attribute__((ext_vector_type(WORDS)));
    constexpr int kCols = 4 * WORDS, kRegs = F32 ? kCols : kCols / 2;  // registers a row
    typedef uint32_t Row __attribute__((ext_vector_type(kRegs)));
    const long long t = (long long)blockIdx.x * 256 + threadIdx.x;
    if (t >= threads) return;
    const int per = N / kCols;
    const long long g = t / per;  // group of 32 rows, over all matrices (K is a multiple of 32)
    const int c = (int)(t - g * per) * kCols;
    Row v[32];
#pragma unroll
    for (int r = 0; r < 32; ++r) {
        const long long o = (32 * g + r) * N + c;
        v[r] = *reinterpret_cast<const Row *>(static_cast<const char *>(W) + (F32 ? 4 : 2) * o);
    }
    uint32_t m[kCols];  // bits of the largest magnitudes
    if constexpr (F32) {
#pragma unroll
        for (int j = 0; j < kCols; ++j) {
            m[j] = 0;
#pragma unroll
            for (int r = 0; r < 32; ++r) m[j] = max(m[j], v[r][j] & 0x7fffffffu);
        }
    } else {
#pragma unroll
        for (int j = 0; j < kRegs; ++j) {
            u16x2 most = mags(v[0][j]);
#pragma unroll
            for (int r = 1; r < 32; ++r) most = __builtin_elementwise_max(most, mags(v[r][j]));
            m[2 * j] = (uint32_t)most[0] << 16;
            m[2 * j + 1] = (uint32_t)most[1] << 16;
        }
    }
    Words b, keep;  // scale bytes; a mask of the columns without the NaN scale
    float s[kCols];
#pragma unroll
    for (int w = 0; w < WORDS; ++w) b[w] = keep[w] = 0;
#pragma unroll
    for (int j = 0; j < kCols; ++j) {
        const uint32_t byte = scale_byte(m[j]);
        s[j] = scale_of(byte == 255u ? 127u : byte);
        b[j / 4] |= byte << (8 * (j & 3));
        keep[j / 4] |= (byte == 255u ? 0u : 255u) << (8 * (j & 3));
    }
#pragma unroll
    for (int r = 0; r < 16; ++r) {
        const Row lo = v[2 * r], hi = v[2 * r + 1];
        Words q;
#pragma unroll
        for (int w = 0; w < WORDS; ++w) {
            uint32_t x = 0;
            // byte j: the codes of rows 2 r (low) and 2 r + 1 of column 4 w + j
            if constexpr (F32) {
                x = codes_f32<0>(x, lo[4 * w], hi[4 * w], s[4 * w]);
                x = codes_f32<1>(x, lo[4 * w + 1], hi[4 * w + 1], s[4 * w + 1]);
                x = codes_f32<2>(x, lo[4 * w + 2], hi[4 * w + 2], s[4 * w + 2]);
                x = codes_f32<3>(x, lo[4 * w + 3], hi[4 * w + 3], s[4 * w + 3]);
            } else {
                x = codes_bf16<0>(x, lo[2 * w], hi[2 * w], s[4 * w]);
                x = codes_bf16<1>(x, lo[2 * w], hi[2 * w], s[4 * w + 1]);
                x = codes_bf16<2>(x, lo[2 * w + 1], hi[2 * w + 1], s[4 * w + 2]);
                x = codes_bf16<3>(x, lo[2 * w + 1], hi[2 * w + 1], s[4 * w + 3]);
            }
            q[w] = x & keep[w];
        }
        *reinterpret_cast<Words *>(Q + (16 * g + r) * N + c) = q;
    }
    *reinterpret_cast<Words *>(S + g * N + c) = b;
}

template <bool F32>
__global__ __launch_bounds__(256) void mx4_weights_back_kernel(const uint8_t *Q, const uint8_t *S, long long threads,
                                                               int N, void *W) {
    constexpr int U = kBack<F32>, kWords = U / 4;  // columns a thread
    typedef uint32_t Words __attribute__((ext_vector_type(kWords)));
    const long long t = (long long)blockIdx.x * 256 + threadIdx.x;
    if (t >= threads) return;
    const int per = N / U;
    const long long g = t / per;
    const int c = (int)(t - g * per) * U;
    Words q[16];
#pragma unroll
    for (int r = 0; r < 16; ++r) q[r] = *reinterpret_cast<const Words *>(Q + (16 * g + r) * N + c);
    const Words sw = *reinterpret_cast<const Words *>(S + g * N + c);
    uint32_t b[U];
#pragma unroll
    for (int j = 0; j < U; ++j) b[j] = sw[j >> 2] >> (8 * (j & 3)) & 255u;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
        float lo[U], hi[U];
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const f32x2 x = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[r][j >> 2] >> (8 * (j & 3)), scale_of(b[j]), 0);
            lo[j] = nan_if(b[j], x[0]);
            hi[j] = nan_if(b[j], x[1]);
        }
        store16<F32>(W, (32 * g + 2 * r) * N + c, lo);
        store16<F32>(W, (32 * g + 2 * r + 1) * N + c, hi);
    }
}

// a / gk of 0 <= a < 2^31 as a product: (a mul) >> (31 + shift), mul = floor(2^(31 +
// shift) / gk) + 1, 2^shift >= gk. (mul gk exceeds 2^(31 + shift) by at most gk <=
// 2^shift, so the product is off by less than 1 / gk.) A division by an argument
// takes about 35 instructions, for every row of every thread
struct Divide {
    uint32_t mul, shift;
    explicit Divide(int gk) : shift(0) {
        while ((1LL << shift) < gk) ++shift;
        mul = (uint32_t)((1ULL << (31 + shift)) / gk + 1);
    }
    __device__ __forceinline__ int operator()(int a) const {
        return (int)(((unsigned long long)(uint32_t)a * mul) >> (31 + shift));
    }
};

// ---- rows in the product's layout: 16 lanes a row and panel (8 values each, four
// lanes a group), RPT rows of one panel each, 64 RPT rows of a panel a workgroup ----

// what the first launch of two, or the first workgroups of one, do beside the rows
__device__ __forceinline__ void first_jobs(const Mx4Panels &p, const TilesJob &j, int blk, int *scan_lds) {
    if (blk == 0 && j.tiles)
        build_tiles(j.offsets, j.G, 0, j.bm, j.tiles, j.n_tiles, j.start, j.zero, j.n_zero, scan_lds);
}
// the tile list, and which row holds an assignment
__global__ __launch_bounds__(1024) void mx4_row_of_kernel(Mx4Panels p, TilesJob j) {
    __shared__ int scan_lds[16];
    first_jobs(p, j, blockIdx.x, scan_lds);
    const int used = p.n_rows ? min(p.rows, *p.n_rows) : p.rows;
    for (int r = blockIdx.x * 1024 + threadIdx.x; r < used; r += gridDim.x * 1024) {
        const int a = p.row_src[r];
        if (a >= 0 && a < p.rows) p.scratch[a] = r;
    }
}

// the row of X that holds assignment a's token
__device__ __forceinline__ int source(int a, const Divide &token) {
    if (MOE_BOUNDS_FAIL(a >= 0, BOUNDS_A_ROW)) a = 0;
    return token(a);
}
__device__ __forceinline__ u32x4 load_panel(const Mx4Panels &p, long long row, int c) {
    if (MOE_BOUNDS_FAIL(row >= 0 && (p.a_rows <= 0 || row < p.a_rows), BOUNDS_A_ROW)) row = 0;
    const u32x4 x = *reinterpret_cast<const u32x4 *>(reinterpret_cast<const uint16_t *>(p.X) + row * p.C +
                                                     (c < p.C ? c : 0));
    return c < p.C ? x : u32x4{0, 0, 0, 0};
}
__device__ __forceinline__ void store_panel(const Mx4Panels &p, int kb, int row, int sub, uint32_t codes, uint32_t b) {
    if (MOE_BOUNDS_FAIL(row >= 0 && row < p.ld, BOUNDS_QUANT_ROW)) return;
    const long long o = kb * p.ld + row;
    *reinterpret_cast<uint32_t *>(p.A + o * 64 + 4 * sub) = codes;
    if ((sub & 3) == 0) reinterpret_cast<uint8_t *>(p.As + o)[sub >> 2] = (uint8_t)b;
}

// row by row
template <int RPT>
__global__ __launch_bounds__(1024) void mx4_panels_kernel(Mx4Panels p, TilesJob j, int chunks, Divide token) {
    __shared__ int scan_lds[16];
    int blk = blockIdx.x;
    if (j.tiles && blk-- == 0) {
        first_jobs(p, j, 0, scan_lds);
        return;
    }
    const int kb = blk / chunks, r0 = blk % chunks * (64 * RPT) + (threadIdx.x >> 4);
    const int sub = threadIdx.x & 15, c = 128 * kb + 8 * sub;
    const int used = p.n_rows ? min(p.rows, *p.n_rows) : p.rows;
    bool in[RPT];  // a row's 16 lanes together
    long long src[RPT];
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const int r = r0 + 64 * i;
        in[i] = r < used || (r >= p.rows && r < p.rows + p.extra);
        src[i] = !in[i] ? 0 : r >= p.rows ? r - p.rows : p.row_src ? source(p.row_src[r], token) : r;
    }
    u32x4 x[RPT];
#pragma unroll
    for (int i = 0; i < RPT; ++i) x[i] = in[i] ? load_panel(p, src[i], c) : u32x4{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const uint32_t b = scale_byte(quad_max(max_bits(x[i])));
        if (in[i]) store_panel(p, kb, r0 + 64 * i, sub, codes8(x[i], b), b);
    }
}

// token by token: its row is read and coded once and stored at the rows of its gk
// assignments. Lane i of a token's 16 looks up assignments i, i + 16, ..
template <int RPT>
__global__ __launch_bounds__(1024) void mx4_panels_token_kernel(Mx4Panels p, int chunks, int tokens, Divide token) {
    const int kb = blockIdx.x / chunks, chunk = blockIdx.x % chunks, t0 = chunk * (64 * RPT) + (threadIdx.x >> 4);
    const int sub = threadIdx.x & 15, c = 128 * kb + 8 * sub;
    const int used = p.n_rows ? min(p.rows, *p.n_rows) : p.rows;
    for (int j0 = 0; j0 < p.gk; j0 += 16) {
        int row[RPT];
        u32x4 x[RPT];
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            const int t = t0 + 64 * i;
            const long long a = (long long)t * p.gk + j0 + sub;
            row[i] = t < tokens && j0 + sub < p.gk && a < p.rows ? p.row_of[a] : -1;
            if (row[i] < 0 || row[i] >= used || p.row_src[row[i]] != (int)a) row[i] = -1;
        }
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            // a token that no row names is not read (X may end before it)
            const int t = t0 + 64 * i;
            const bool some = (__ballot(row[i] >= 0) >> (threadIdx.x & 48) & 0xffffu) != 0 || t < p.extra;
            x[i] = some ? load_panel(p, t, c) : u32x4{0, 0, 0, 0};
        }
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            const uint32_t b = scale_byte(quad_max(max_bits(x[i]))), codes = codes8(x[i], b);
            for (int j = 0; j < 16 && j0 + j < p.gk; ++j) {
                const int r = __shfl(row[i], j, 16);
                if (r >= 0) store_panel(p, kb, r, sub, codes, b);
            }
            if (j0 == 0 && t0 + 64 * i < p.extra) store_panel(p, kb, p.rows + t0 + 64 * i, sub, codes, b);
        }
    }
    // rows that no entry of row_of names (an assignment that two rows hold, or one past
    // the rows' number): a lane looks at one, and its 16 lanes code what they find
    for (int base = chunk * 1024; base < used; base += chunks * 1024) {
        const int r = base + threadIdx.x;
        const int a = r < used ? p.row_src[r] : 0;
        const bool own = r < used && ((uint32_t)a >= (uint32_t)p.rows || p.row_of[a] != r);
        uint32_t left = (uint32_t)(__ballot(own) >> (threadIdx.x & 48)) & 0xffffu;
        while (__any(left != 0)) {
            const int i = left ? __ffs((int)left) - 1 : 0, t = source(__shfl(a, i, 16), token);
            const u32x4 x = left ? load_panel(p, t, c) : u32x4{0, 0, 0, 0};
            const uint32_t b = scale_byte(quad_max(max_bits(x)));
            if (left) store_panel(p, kb, r - sub + i, sub, codes8(x, b), b);
            left &= left - 1;
        }
    }
}

}  // namespace

// workgroups of 1024 threads for 256 rows and a panel, and one for the tile list
bool mx4_panels_fit(long long rows, int C) {
    return (rows + 255) / 256 * mx4::panels(C) + 1 <= kMaxThreads / 1024;
}

hipError_t launch_mx4_panels(const Mx4Panels &p, const TilesJob *tiles, hipStream_t s) {
    if (p.rows < 0 || p.extra < 0 || p.C < kGroup || p.C % kGroup || p.gk < 1 || !p.A || !p.As ||
        p.ld < (long long)p.rows + p.extra)
        return hipErrorInvalidValue;
    const long long rows = (long long)p.rows + p.extra;
    if (rows == 0 && !tiles) return hipSuccess;
    if (!mx4_panels_fit(rows, p.C)) return hipErrorInvalidValue;
    const int np = panels(p.C);
    // few blocks of 64 rows and a panel: a row a thread, for more workgroups (H 2048, 256
    // blocks: 3.4 against 5.1 us with four, 1024: 7.6 and 8.1, 4096: 17.5 and 16.5)
    const long long work = (rows + 63) / 64 * np;
    const bool few = work <= 1024;
    const TilesJob job = tiles ? *tiles : TilesJob{};
    const Divide token(p.gk);
    const dim3 block(1024);
    // 65536 rows of 8192 tokens, C 2048: 53 us by row (268 MB of tokens read from beyond
    // the L2s, at 5 TB/s), 37 + 6 for row_of by token. 8192 rows of 4096 tokens, C 4096: 21
    // by row, 20 + 5 by token. The launch for row_of takes 5 us or more. (More than a layer's
    // 64 picks a token: by row, whose time does not grow with them)
    if (p.row_src && p.gk >= 4 && p.gk <= 64 && (p.row_of ? !few : p.scratch && work >= 8192)) {
        Mx4Panels q = p;
        if (!q.row_of) {
            const long long n = (rows + 1023) / 1024;
            hipLaunchKernelGGL(mx4_row_of_kernel, dim3((unsigned)(n < 512 ? n : 512)), block, 0, s, p, job);
            q.row_of = p.scratch;
        } else if (tiles) {
            return hipErrorInvalidValue;
        }
        long long tokens = (p.rows + (long long)p.gk - 1) / p.gk;
        if (tokens < p.extra) tokens = p.extra;
        const long long chunks = (tokens + 255) / 256;
        hipLaunchKernelGGL(mx4_panels_token_kernel<4>, dim3((unsigned)(chunks * np)), block, 0, s, q, (int)chunks,
                           (int)tokens, token);
        return hipGetLastError();
    }
    const long long chunks = (rows + (few ? 64 : 256) - 1) / (few ? 64 : 256);
    const long long blocks = chunks * np + (tiles ? 1 : 0);
    if (few)
        hipLaunchKernelGGL(mx4_panels_kernel<1>, dim3((unsigned)blocks), block, 0, s, p, job, (int)chunks, token);
    else
        hipLaunchKernelGGL(mx4_panels_kernel<4>, dim3((unsigned)blocks), block, 0, s, p, job, (int)chunks, token);
    return hipGetLastError();
}

}  // namespace moe

// ---------------------------------------------------------------------------
// public entry points
// ---------------------------------------------------------------------------
#include "abi_util.h"

using namespace moe;

namespace {

// values of one call: a launch of 256 threads per 4096 values of rows (of weights 32768 or
// 65536, by the columns a thread takes), and a grid's dimension holds fewer than 2^32 threads
constexpr long long kMaxValues = (1LL << 36) - 4096;

bool off16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) != 0; }
bool off8(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 7) != 0; }

moe_status check_rows(long long R, int C, moe_dtype dt) {
    if (R < 0 || C < 1) return MOE_ERR_INVALID_ARG;
    if ((dt != MOE_F32 && dt != MOE_BF16) || C % 32 || C > kMaxDim || R > kMaxValues / C) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}
moe_status check_weights(int G, int K, int N, moe_dtype dt) {
    if (G < 0 || K < 1 || N < 1) return MOE_ERR_INVALID_ARG;
    if ((dt != MOE_F32 && dt != MOE_BF16) || K % 32 || N % 8 || K > kMaxDim || N > kMaxDim ||
        G > kMaxValues / ((long long)K * N))
        return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

}  // namespace

extern "C" {

moe_status moe_quantize_mxfp4_rows(const void *X, moe_dtype x_dt, long long ldx, long long R, int C, uint8_t *Q,
                                   uint8_t *S, hipStream_t stream) {
    const moe_status st = check_rows(R, C, x_dt);
    if (st != MOE_OK) return st;
    if (ldx < C) return MOE_ERR_INVALID_ARG;
    if (ldx % (x_dt == MOE_F32 ? 4 : 8)) return MOE_ERR_UNSUPPORTED;
    if (R == 0) return MOE_OK;
    if (!X || !Q || !S) return MOE_ERR_INVALID_ARG;
    if (off16(X) || off8(Q)) return MOE_ERR_UNSUPPORTED;
    const long long n = R * C;
    const dim3 grid((unsigned)((n / kPer + 255) / 256));
    if (x_dt == MOE_F32) hipLaunchKernelGGL(mx4_rows_kernel<true>, grid, dim3(256), 0, stream, X, ldx, n, C, Q, S);
    else hipLaunchKernelGGL(mx4_rows_kernel<false>, grid, dim3(256), 0, stream, X, ldx, n, C, Q, S);
    return hip_status(hipGetLastError());
}

moe_status moe_dequantize_mxfp4_rows(const uint8_t *Q, const uint8_t *S, long long R, int C, moe_dtype y_dt, void *Y,
                                     hipStream_t stream) {
    const moe_status st = check_rows(R, C, y_dt);
    if (st != MOE_OK) return st;
    if (R == 0) return MOE_OK;
    if (!Q || !S || !Y) return MOE_ERR_INVALID_ARG;
    if (off8(Q) || off16(Y)) return MOE_ERR_UNSUPPORTED;
    const long long n = R * C;
    const dim3 grid((unsigned)((n / kPer + 255) / 256));
    if (y_dt == MOE_F32) hipLaunchKernelGGL(mx4_rows_back_kernel<true>, grid, dim3(256), 0, stream, Q, S, n, Y);
    else hipLaunchKernelGGL(mx4_rows_back_kernel<false>, grid, dim3(256), 0, stream, Q, S, n, Y);
    return hip_status(hipGetLastError());
}

moe_status moe_quantize_mxfp4_weights(const void *W, moe_dtype w_dt, int G, int K, int N, uint8_t *Q, uint8_t *S,
                                      hipStream_t stream) {
    const moe_status st = check_weights(G, K, N, w_dt);
    if (st != MOE_OK) return st;
    if (G == 0) return MOE_OK;
    if (!W || !Q || !S) return MOE_ERR_INVALID_ARG;
    if (off16(W) || off8(Q) || off8(S)) return MOE_ERR_UNSUPPORTED;
    const long long words = (long long)G * (K / 32) * (N / 4);
    const bool one = w_dt == MOE_F32 || words / 2 < kFewThreads;
    const long long threads = one ? words : words / 2;
    const dim3 grid((unsigned)((threads + 255) / 256));
    if (w_dt == MOE_F32)
        hipLaunchKernelGGL((mx4_weights_kernel<true, 1>), grid, dim3(256), 0, stream, W, threads, N, Q, S);
    else if (one) hipLaunchKernelGGL((mx4_weights_kernel<false, 1>), grid, dim3(256), 0, stream, W, threads, N, Q, S);
    else hipLaunchKernelGGL((mx4_weights_kernel<false, 2>), grid, dim3(256), 0, stream, W, threads, N, Q, S);
    return hip_status(hipGetLastError());
}

moe_status moe_dequantize_mxfp4_weights(const uint8_t *Q, const uint8_t *S, int G, int K, int N, moe_dtype w_dt,
                                        void *W, hipStream_t stream) {
    const moe_status st = check_weights(G, K, N, w_dt);
    if (st != MOE_OK) return st;
    if (G == 0) return MOE_OK;
    if (!Q || !S || !W) return MOE_ERR_INVALID_ARG;
    if (off8(Q) || off8(S) || off16(W)) return MOE_ERR_UNSUPPORTED;
    const long long threads = (long long)G * (K / 32) * (N / (w_dt == MOE_F32 ? kBack<true> : kBack<false>));
    const dim3 grid((unsigned)((threads + 255) / 256));
    if (w_dt == MOE_F32)
        hipLaunchKernelGGL(mx4_weights_back_kernel<true>, grid, dim3(256), 0, stream, Q, S, threads, N, W);
    else hipLaunchKernelGGL(mx4_weights_back_kernel<false>, grid, dim3(256), 0, stream, Q, S, threads, N, W);
    return hip_status(hipGetLastError());
}

}  // extern "C"
