// Weight gradients of the grouped FFN: for every expert g,
//   dW_g[m][n] = sum over its rows r of A(r)[m] B(r)[n]
// in one launch: dW1 and dW3 (A = the token rows read back from their
// checkpoint, B = [dg | du]) or dW2 (A = w h, B = dY), the token operand
// gathered by row. The sum runs over rows, so both operands are contiguous
// across it: LDS tiles keep the matrices' [row][column] layout and both MFMA
// operands are read with ds_read_b64_tr_b16.
//
// A work item is one 256 x 256 tile of one expert's output; its K loop is that
// expert's rows, 32 a step (rows past the end read zeros, so NaN or infinite
// rows of another expert never enter). An expert without rows writes zeros.
// 8 wavefronts in 2 x 4 (128 x 64 each), a ring of 4 stages as in
// tiled_gemm_kernel.h. The gathered rows' token numbers are kept in LDS,
// kWindow rows at a time, so that the ring's vector-memory count holds
// only copies.
// Items are handed to the XCDs in runs of 32 (one per CU) of consecutive
// tiles of an expert, in turn: an XCD's L2 serves a run's panels, and an
// expert with many rows is spread over the XCDs.
// build-flags: -mllvm -amdgpu-mfma-vgpr-form
#include "tiled_gemm_kernel.h"

namespace moe {

MOE_BOUNDS_FILE(train_weights)

namespace tiled {
namespace {

// what rows past an expert's end are read from
__device__ __attribute__((aligned(16))) const uint32_t kZeroPiece[4] = {0, 0, 0, 0};

struct WRing {
    static constexpr int tile = 32 * 512;  // one operand: 32 rows of 256 bf16
    static constexpr int stage = 2 * tile;
    static constexpr int S = 4;
    static constexpr int nC = 4;           // copies per wavefront and step (2 of each operand)
    static constexpr int MI = 8, NB = 4;
    static constexpr int kWindow = 4096;   // rows per K loop
    static constexpr int idx = S * stage;
    static constexpr int lds = idx + kWindow * 4;
    static constexpr int old = 64 + 8;     // epilogue staging (bf16), 16 rows a wavefront
    static_assert(lds <= 160 * 1024 && 8 * 16 * old * 2 <= S * stage, "LDS");
};

template <bool F32>
__global__ __launch_bounds__(512, 1) void weights_gemm_kernel(WeightsProblem p, int nM, int nN) {
    typedef WRing R;
    constexpr int S = R::S, MI = R::MI, NB = R::NB, NC = R::nC, NR = 2 * (MI + NB);
    __shared__ __attribute__((aligned(1024))) uint8_t lds[R::lds];
    int *idx = reinterpret_cast<int *>(lds + R::idx);

    // ---- this workgroup's item ----
    const int mats = p.C1 ? 2 : 1;
    const long long per_group = (long long)nM * nN * mats;
    const int xcd = blockIdx.x % kXcds, slot = blockIdx.x / kXcds;
    const long long id = ((long long)(slot / kBlocksPerXcd) * kXcds + xcd) * kBlocksPerXcd + slot % kBlocksPerXcd;
    const int g = (int)(id / per_group);
    if (g >= p.G) return;
    const int t = (int)(id % per_group);
    const int m0 = 256 * (t / (nN * mats)), nt = t % (nN * mats);
    const int half = nt >= nN ? 1 : 0, n0 = 256 * (nt - half * nN);
    const int lo = min(max(p.offsets[g], 0), p.M), hi = min(max(p.offsets[g + 1], lo), p.M);
    if (lo == hi && p.accumulate) return;

    const int tid = threadIdx.x;
    const int lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), wr = w / 4, wc = w % 4;
    const int i16 = lane & 15, gq = lane >> 4;

    // ---- copies: q < 2 operand A, else B; copy q of wavefront w fills rows
    // 2 (2 w + q % 2) + lane / 32 of the step, the lane's 16-byte chunk being
    // the one the swizzle puts there ----
    const uint16_t *base[NC];
    int krow[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int k = 2 * (2 * w + q) + (lane >> 5);
        const int c = 8 * ((lane & 31) ^ bswz16(k));
        krow[q] = k;
        base[q] = p.A + min(m0 + c, p.MD - 8);
        base[2 + q] = p.B + (long long)half * p.ND + min(n0 + c, p.ND - 8);
    }
    const int32_t *src = p.a_src ? p.a_src : p.b_src;
    int w0 = lo;  // first row of the window
    auto copy = [&](int q, int kt, int stage) {
        const int k = kt * 32 + krow[q & 1];
        const bool gathered = q < 2 ? p.a_src != nullptr : p.b_src != nullptr;
        const int r = gathered ? idx[k] : (w0 + k < hi ? w0 + k : -1);
        const void *s = r < 0 ? (const void *)kZeroPiece
                              : (const void *)(base[q] + (long long)r * (q < 2 ? p.lda : p.ldb));
        copy16(s, lds + stage * R::stage + (q < 2 ? 0 : R::tile) + (2 * w + (q & 1)) * 1024);
    };

    // ---- fragment reads: r = 2 block + half; blocks 0..MI-1 of A, then B ----
    struct Frag {
        bf16x8 a[MI], b[NB];
        u32x2 raw[MI + NB][2];
    };
    auto read = [&](Frag &f, int r, int stage) {
        const int blk = r >> 1, kh = r & 1;
        const int k = 8 * gq + 4 * kh + (i16 >> 2);
        const int n = (blk < MI ? 128 * wr + 16 * blk : 64 * wc + 16 * (blk - MI)) + 4 * (i16 & 3);
        f.raw[blk][kh] = ds_tr16(lds_addr(lds + stage * R::stage + (blk < MI ? 0 : R::tile)) + k * 512 +
                                 16 * ((n >> 3) ^ bswz16(k)) + 2 * (n & 7));
    };
    auto land = [&](Frag &f) {
        wait_lds();
#pragma unroll
        for (int b = 0; b < MI + NB; ++b) {
            fence(f.raw[b][0]);
            fence(f.raw[b][1]);
            const u32x4 v = {f.raw[b][0][0], f.raw[b][0][1], f.raw[b][1][0], f.raw[b][1][1]};
            if (b < MI) f.a[b] = __builtin_bit_cast(bf16x8, v);
            else f.b[b - MI] = __builtin_bit_cast(bf16x8, v);
        }
    };

    f32x4 acc[MI][NB];
#pragma unroll
    for (int m = 0; m < MI; ++m)
#pragma unroll
        for (int j = 0; j < NB; ++j) acc[m][j] = f32x4{};
    auto mma_rows = [&](const Frag &f, int m) {
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < NB; ++j)
            acc[m][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f.b[j], f.a[m], acc[m][j], 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
    };

    for (; w0 < hi; w0 += R::kWindow) {
        const int rows = min(hi - w0, R::kWindow), nk = (rows + 31) / 32;
        if (src) {
            const long long lim = p.a_src ? p.a_rows : p.b_rows;
            for (int i = tid; i < 32 * nk; i += 512) {
                int v = i < rows ? src[w0 + i] / p.gk : -1;
                if (MOE_BOUNDS_FAIL(v >= -1 && (lim <= 0 || v < lim), BOUNDS_A_ROW)) v = -1;
                idx[i] = v;
            }
            __syncthreads();
        }
        Frag fa, fb;
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
            for (int q = 0; q < NC; ++q) copy(q, min(s, nk - 1), s);
        wait_vm<(S - 1) * NC>();
        __builtin_amdgcn_s_barrier();
#pragma unroll
        for (int r = 0; r < NR; ++r) read(fa, r, 0);
        land(fa);
        int stage = 0;
        auto step = [&](Frag &cur, Frag &nxt, int kt) {
            const int nstage = stage + 1 == S ? 0 : stage + 1;
            const int from = min(kt + S, nk - 1);
            mma_rows(cur, 0);
            mma_rows(cur, 1);
            wait_vm<(S - 2) * NC>();
            __builtin_amdgcn_s_barrier();
            constexpr int SLOTS = MI - 2;
#pragma unroll
            for (int c = 0; c < SLOTS; ++c) {
#pragma unroll
                for (int q = c * NC / SLOTS; q < (c + 1) * NC / SLOTS; ++q) copy(q, from, stage);
#pragma unroll
                for (int r = c * NR / SLOTS; r < (c + 1) * NR / SLOTS; ++r) read(nxt, r, nstage);
                mma_rows(cur, c + 2);
            }
            land(nxt);
            stage = nstage;
        };
        int kt = 0;
        for (; kt + 1 < nk; kt += 2) {
            step(fa, fb, kt);
            step(fb, fa, kt + 1);
        }
        if (kt < nk) step(fa, fb, kt);
        wait_vm<0>();     // the repeated copies of the last steps have landed,
        __syncthreads();  // and every wavefront is done with the ring and the rows' numbers
    }

    // ---- store ----
    void *C = half ? p.C1 : p.C0;
    const long long out0 = (long long)g * p.MD * p.ND;
    const int c0 = n0 + 64 * wc;
    if constexpr (F32) {
        float *Cf = reinterpret_cast<float *>(C) + out0;
#pragma unroll
        for (int m = 0; m < MI; ++m) {
            const int row = m0 + 128 * wr + 16 * m + i16;
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                const int col = c0 + 16 * j + 4 * gq;
                if (row >= p.MD || col >= p.ND) continue;
                f32x4 *o = reinterpret_cast<f32x4 *>(Cf + (long long)row * p.ND + col);
                f32x4 v = acc[m][j];
                if (p.accumulate) v += *o;
                *o = v;
            }
        }
    } else {
        uint16_t *Cb = reinterpret_cast<uint16_t *>(C) + out0;
        uint16_t *stg = reinterpret_cast<uint16_t *>(lds) + w * 16 * R::old;
#pragma unroll
        for (int m = 0; m < MI; ++m) {
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                const int row = m0 + 128 * wr + 16 * m + i16, col = c0 + 16 * j + 4 * gq;
                f32x4 v = acc[m][j];
                if (p.accumulate && row < p.MD && col < p.ND) {
                    const u32x2 old = *reinterpret_cast<const u32x2 *>(Cb + (long long)row * p.ND + col);
                    v += f32x4{bf16_lo(old[0]), bf16_hi(old[0]), bf16_lo(old[1]), bf16_hi(old[1])};
                }
                *reinterpret_cast<u32x2 *>(stg + i16 * R::old + 16 * j + 4 * gq) =
                    u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int piece = lane + 64 * c, r = piece >> 3, col = 8 * (piece & 7);
                const int row = m0 + 128 * wr + 16 * m + r;
                if (row < p.MD && c0 + col < p.ND)
                    *reinterpret_cast<u32x4 *>(Cb + (long long)row * p.ND + c0 + col) =
                        *reinterpret_cast<const u32x4 *>(stg + r * R::old + col);
            }
        }
    }
}

}  // namespace
}  // namespace tiled

hipError_t launch_weights_gemm(const WeightsProblem &p, hipStream_t s) {
    if (!p.A || !p.B || !p.offsets || !p.C0 || p.G < 1 || p.M < 0 || p.MD < 32 || p.MD % 32 || p.ND < 32 ||
        p.ND % 32 || p.gk < 1 || (p.a_src && p.b_src) || p.lda < p.MD || p.ldb < (p.C1 ? 2 : 1) * p.ND ||
        (p.c_dt != MOE_F32 && p.c_dt != MOE_BF16))
        return hipErrorInvalidValue;
    const int nM = (p.MD + 255) / 256, nN = (p.ND + 255) / 256;
    const long long items = (long long)p.G * nM * nN * (p.C1 ? 2 : 1);
    constexpr long long run = tiled::kXcds * tiled::kBlocksPerXcd;
    const long long blocks = (items + run - 1) / run * run;
    if (blocks > 0x7fffffffLL) return hipErrorInvalidValue;
    if (p.c_dt == MOE_F32)
        hipLaunchKernelGGL(tiled::weights_gemm_kernel<true>, dim3((unsigned)blocks), dim3(512), 0, s, p, nM, nN);
    else
        hipLaunchKernelGGL(tiled::weights_gemm_kernel<false>, dim3((unsigned)blocks), dim3(512), 0, s, p, nM, nN);
    return hipGetLastError();
}

}  // namespace moe
