// Row gradients of the grouped FFN: C[r][n] = sum_k A(r)[k] B_g[n][k] over
// every expert's rows in one launch, with both operands contiguous in k (the
// forward's weight matrices [K][N], read for the product with their
// transpose). Two uses:
//  * SwiGLU backward (BACK): A(r) = dY[token of r], B = W2 [F][H], so the
//    accumulator is p = dY W2^T, before the routing weight. The epilogue reads
//    the checkpointed g and u (MXFP8) and forms, with s = 1 / (1 + e^-g):
//      h = g s u            dw[r] = sum_f p h        (gradient of the weight)
//      dg = w p u s (1 + g (1 - s))    du = w p g s    w h for dW2
//    dY is gathered by the copies and never multiplied by w in memory: the
//    combine's backward pass costs no pass of its own.
//  * plain: A = [dg | du] [M][2F], B = W1 then W3 [H][F] along k; fp32 rows
//    out (they are summed over a token's k rows before the one rounding).
// dg, du and w h are rounded to bf16: the operands of the bf16 matrix cores.
//
// Tile BM (128 or 256) rows x 256 columns, 32 deep a step, 8 wavefronts in
// 2 x 4, each BM/2 rows x 64 columns; copy ring, swizzle, waits and barriers
// as in tiled_gemm_kernel.h, whose A-operand layout (64-byte rows, 16-byte
// reads) serves both operands here: no transposing reads.
// build-flags: -mllvm -amdgpu-mfma-vgpr-form
#include "tiled_gemm_kernel.h"

namespace moe {

MOE_BOUNDS_FILE(train_rows)

namespace tiled {
namespace {

constexpr int kRowsBN = rows_gemm_bn;

template <int BM>
struct RowsRing {
    static constexpr int a_bytes = BM * 64;
    static constexpr int stage = a_bytes + kRowsBN * 64;
    static constexpr int S = kRingBudget / stage < 6 ? kRingBudget / stage : 6;
    static constexpr int nA = BM / 128;  // 1 KB copies (16 rows) per wavefront and step
    static constexpr int nB = 2;
    static constexpr int per_tile = nA + nB;
    static constexpr int MI = BM / 32;   // 16-row blocks per wavefront
    // epilogue staging per wavefront: a 16 x 64 block of each output (bf16,
    // padded rows) and of each code matrix
    static constexpr int old = 64 + 8, cld = 64 + 16;
    static constexpr int stg = 3 * 16 * old * 2 + 2 * 16 * cld;
    static constexpr int dw = 8 * stg;   // [4][BM] floats behind it
    static constexpr int lds = S * stage > dw + 16 * BM ? S * stage : dw + 16 * BM;
    static_assert(lds <= 160 * 1024, "LDS");
};

template <int BM, bool BACK>
__global__ __launch_bounds__(512, 1) void rows_gemm_kernel(RowsProblem p, int nN) {
    typedef RowsRing<BM> R;
    constexpr int S = R::S, MI = R::MI, NB = 4, NC = R::per_tile, NR = NB + MI;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[R::lds];

    GemmProblem order{};
    order.tiles = p.tiles;
    order.n_tiles = p.n_tiles;
    order.group_tile_start = p.group_tile_start;
    order.M = p.M;
    int mt, nt;
    if (!pick_tile(order, nN, BM, mt, nt)) return;
    if (MOE_BOUNDS_FAIL(mt < p.max_tiles, BOUNDS_TILE)) return;
    const int g = p.tiles[4 * mt], row0 = p.tiles[4 * mt + 1], row_end = p.tiles[4 * mt + 2];
    if (MOE_BOUNDS_FAIL(g >= 0 && g < p.n_groups && row0 >= 0 && row0 < row_end && row_end <= p.M, BOUNDS_TILE))
        return;
    const int n0 = nt * kRowsBN;
    const int tid = threadIdx.x;
    const int lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), wr = w / 4, wc = w % 4;
    const int i16 = lane & 15, gq = lane >> 4;
    const int nblk = min(max((row_end - row0 - wr * (BM / 2) + 15) >> 4, 0), MI);

    // ---- copy sources: lane -> row lane / 4 of a 16-row copy, chunk lane % 4 ----
    const uint16_t *a_src[R::nA], *b_src[R::nB];
#pragma unroll
    for (int q = 0; q < R::nA; ++q) {
        int r = row0 + 16 * (w * R::nA + q) + (lane >> 2);
        if (r >= row_end) r = row0;  // rows past the tile's end copy a valid row (never stored)
        long long src = p.row_src ? (long long)(p.row_src[r] / p.gk) : (long long)r;
        if (MOE_BOUNDS_FAIL(src >= 0 && (p.a_rows <= 0 || src < p.a_rows), BOUNDS_A_ROW)) src = 0;
        a_src[q] = p.A + src * p.lda + 8 * aswz_chunk(lane);
    }
    const long long b_stride = (long long)p.N * p.K0;
#pragma unroll
    for (int q = 0; q < R::nB; ++q) {
        const int n = min(n0 + 16 * (w * R::nB + q) + (lane >> 2), p.N - 1);
        b_src[q] = p.B0 + g * b_stride + (long long)n * p.K0 + 8 * aswz_chunk(lane);
    }
    const int nk0 = p.K0 / kBK, nk = p.B1 ? 2 * nk0 : nk0;
    // the second matrix continues k: its elements lie this far behind the
    // first's (two allocations: integer arithmetic on their addresses)
    const long long b_next = p.B1 ? (long long)((uintptr_t)p.B1 - (uintptr_t)p.B0) - 2LL * p.K0 : 0;
    auto copy = [&](int q, int kt, int stage) {
        uint8_t *st = lds + stage * R::stage;
        if (q < R::nA) {
            copy16(a_src[q] + kt * kBK, st + (w * R::nA + q) * 1024);
        } else {
            const char *b = reinterpret_cast<const char *>(b_src[q - R::nA]) + 2LL * kt * kBK;
            if (kt >= nk0) b += b_next;
            copy16(b, st + R::a_bytes + (w * R::nB + q - R::nA) * 1024);
        }
    };

    // ---- fragment reads: 16-byte pieces of 64-byte rows, both operands ----
    struct Frag {
        bf16x8 a[MI], b[NB];
    };
    const int chunk = 16 * (gq ^ ((lane >> 2) & 3));
    const int a_off = (wr * (BM / 2) + i16) * 64 + chunk;
    const int b_off = R::a_bytes + (64 * wc + i16) * 64 + chunk;
    auto read = [&](Frag &f, int r, int stage) {
        const uint8_t *st = lds + stage * R::stage;
        if (r < NB) f.b[r] = *reinterpret_cast<const bf16x8 *>(st + b_off + r * 1024);
        else f.a[r - NB] = *reinterpret_cast<const bf16x8 *>(st + a_off + (r - NB) * 1024);
    };

    f32x4 acc[MI][NB];
#pragma unroll
    for (int m = 0; m < MI; ++m)
#pragma unroll
        for (int j = 0; j < NB; ++j) acc[m][j] = f32x4{};
    // B first: a lane's four results are one row and four adjacent columns
    auto mma_rows = [&](const Frag &f, int m, auto act) {
        __builtin_amdgcn_sched_barrier(0);
        if (m < decltype(act)::value) {
#pragma unroll
            for (int j = 0; j < NB; ++j)
                acc[m][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f.b[j], f.a[m], acc[m][j], 0, 0, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
    };

    Frag fa, fb;
#pragma unroll
    for (int t = 0; t < S; ++t)
#pragma unroll
        for (int q = 0; q < NC; ++q) copy(q, min(t, nk - 1), t);
    wait_vm<(S - 1) * NC>();
    __builtin_amdgcn_s_barrier();
#pragma unroll
    for (int r = 0; r < NR; ++r) read(fa, r, 0);
    wait_lds();
    auto kloop = [&](auto act) {
        constexpr int ACT = decltype(act)::value;
        int stage = 0;
        auto step = [&](Frag &cur, Frag &nxt, int kt) {
            const int nstage = stage + 1 == S ? 0 : stage + 1;
            const int src = min(kt + S, nk - 1);
            constexpr int PRE = MI >= 8 ? 2 : 1, SLOTS = MI - PRE;
#pragma unroll
            for (int m = 0; m < PRE; ++m) mma_rows(cur, m, act);
            wait_vm<(S - 2) * NC>();
            __builtin_amdgcn_s_barrier();
#pragma unroll
            for (int c = 0; c < SLOTS; ++c) {
#pragma unroll
                for (int q = c * NC / SLOTS; q < (c + 1) * NC / SLOTS; ++q) copy(q, src, stage);
#pragma unroll
                for (int r = c * NR / SLOTS; r < (c + 1) * NR / SLOTS; ++r)
                    if (ACT > 0 && (r < NB || r - NB < ACT)) read(nxt, r, nstage);
                mma_rows(cur, c + PRE, act);
            }
            wait_lds();  // every read of the stage is done before anyone refills it
            stage = nstage;
        };
        int kt = 0;
        for (; kt + 1 < nk; kt += 2) {
            step(fa, fb, kt);
            step(fb, fa, kt + 1);
        }
        if (kt < nk) step(fa, fb, kt);
    };
    if (nblk == 0) kloop(std::integral_constant<int, 0>{});
    else if (MI >= 8 && nblk <= MI / 2) kloop(std::integral_constant<int, MI / 2>{});
    else kloop(std::integral_constant<int, MI>{});

    wait_vm<0>();  // the repeated copies of the last steps land before the LDS is used again
    if constexpr (!BACK) {
#pragma unroll
        for (int m = 0; m < MI; ++m) {
            const int row = row0 + wr * (BM / 2) + 16 * m + i16;
            if (row >= row_end) continue;
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                const int col = n0 + 64 * wc + 16 * j + 4 * gq;
                if (col < p.N) *reinterpret_cast<f32x4 *>(p.C + (long long)row * p.N + col) = acc[m][j];
            }
        }
        return;
    } else {
        __syncthreads();  // every wavefront is done with the ring
        // ---- SwiGLU backward, 16 rows at a time, through the wavefront's
        // staging area (its LDS operations complete in order) ----
        uint8_t *stg = lds + w * R::stg;
        uint16_t *so = reinterpret_cast<uint16_t *>(stg);
        uint8_t *sc = stg + 3 * 16 * R::old * 2;
        float *sdw = reinterpret_cast<float *>(lds + R::dw);
        const int c0 = n0 + 64 * wc;
        // code loads: lane -> row lane / 4 of the block, 16 codes at 16 (lane % 4)
        const int lr = lane >> 2, lc = 16 * (lane & 3);
        const int ngr = p.N >> 5;
        struct Codes {
            u32x4 g, u;
            uint8_t gs[2], us[2];
            float w;
        };
        auto load = [&](Codes &c, int m) {
            const int base = row0 + wr * (BM / 2) + 16 * m;
            const int r = base + lr;
            c.g = c.u = u32x4{0, 0, 0, 0};
            if (r < row_end && c0 + lc < p.N) {
                const long long o = (long long)r * p.N + c0 + lc;
                c.g = *reinterpret_cast<const u32x4 *>(p.gq + o);
                c.u = *reinterpret_cast<const u32x4 *>(p.uq + o);
            }
            const int rs = base + i16;
            c.w = 0.0f;
#pragma unroll
            for (int q = 0; q < 2; ++q) c.gs[q] = c.us[q] = 0;
            if (rs < row_end) {
                c.w = p.topk_w ? p.topk_w[p.w_src ? p.w_src[rs] : rs] : 1.0f;
#pragma unroll
                for (int q = 0; q < 2; ++q)
                    if (c0 + 32 * q < p.N) {
                        const long long o = (long long)rs * ngr + (c0 >> 5) + q;
                        c.gs[q] = p.gs[o];
                        c.us[q] = p.us[o];
                    }
            }
        };
        Codes cur;
        load(cur, 0);
#pragma unroll
        for (int m = 0; m < MI; ++m) {
            if (m >= nblk) {  // no rows of the group
                if (gq == 0) sdw[wc * BM + wr * (BM / 2) + 16 * m + i16] = 0.0f;
                continue;
            }
            Codes nxt = cur;
            if (m + 1 < MI) load(nxt, m + 1);
            *reinterpret_cast<u32x4 *>(sc + lr * R::cld + lc) = cur.g;
            *reinterpret_cast<u32x4 *>(sc + 16 * R::cld + lr * R::cld + lc) = cur.u;
            float dw = 0.0f;
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                const uint32_t gw = *reinterpret_cast<const uint32_t *>(sc + i16 * R::cld + 16 * j + 4 * gq);
                const uint32_t uw = *reinterpret_cast<const uint32_t *>(sc + (16 + i16) * R::cld + 16 * j + 4 * gq);
                const f32x4 gv = mx8::values4(gw, mx8::scale_of(cur.gs[j / 2]));
                const f32x4 uv = mx8::values4(uw, mx8::scale_of(cur.us[j / 2]));
                float dg[4], du[4], hw[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.4426950408889634f * gv[i]));
                    const float gsv = gv[i] * s, h = gsv * uv[i], pv = acc[m][j][i];
                    dw = fmaf(pv, h, dw);
                    const float pw = cur.w * pv;
                    du[i] = pw * gsv;
                    dg[i] = pw * uv[i] * s * (1.0f + gv[i] * (1.0f - s));
                    hw[i] = cur.w * h;
                }
                uint16_t *o = so + i16 * R::old + 16 * j + 4 * gq;
                *reinterpret_cast<u32x2 *>(o) = u32x2{pack_bf16x2(dg[0], dg[1]), pack_bf16x2(dg[2], dg[3])};
                *reinterpret_cast<u32x2 *>(o + 16 * R::old) = u32x2{pack_bf16x2(du[0], du[1]), pack_bf16x2(du[2], du[3])};
                *reinterpret_cast<u32x2 *>(o + 32 * R::old) = u32x2{pack_bf16x2(hw[0], hw[1]), pack_bf16x2(hw[2], hw[3])};
            }
            dw += __shfl_xor(dw, 16);
            dw += __shfl_xor(dw, 32);
            if (gq == 0) sdw[wc * BM + wr * (BM / 2) + 16 * m + i16] = c0 < p.N ? dw : 0.0f;
            // 16-byte pieces of the staged rows: 8 a row, 2 a lane and output
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int piece = lane + 64 * c, r = piece >> 3, col = 8 * (piece & 7);
                const int row = row0 + wr * (BM / 2) + 16 * m + r;
                const uint16_t *o = so + r * R::old + col;
                if (row < row_end && c0 + col < p.N) {
                    uint16_t *dgu = p.dGU + (long long)row * 2 * p.N + c0 + col;
                    *reinterpret_cast<u32x4 *>(dgu) = *reinterpret_cast<const u32x4 *>(o);
                    *reinterpret_cast<u32x4 *>(dgu + p.N) = *reinterpret_cast<const u32x4 *>(o + 16 * R::old);
                    *reinterpret_cast<u32x4 *>(p.Hw + (long long)row * p.N + c0 + col) =
                        *reinterpret_cast<const u32x4 *>(o + 32 * R::old);
                }
            }
            cur = nxt;
        }
        if (!p.dw_part) return;
        __syncthreads();
        for (int r = tid; r < BM; r += 512)
            if (row0 + r < row_end)
                p.dw_part[(long long)nt * p.M + row0 + r] =
                    (sdw[r] + sdw[BM + r]) + (sdw[2 * BM + r] + sdw[3 * BM + r]);
    }
}

template <int BM>
hipError_t launch_rows(const RowsProblem &p, bool back, hipStream_t s) {
    const int nN = (p.N + kRowsBN - 1) / kRowsBN;
    const long long per = ((long long)p.max_tiles * nN + kXcds - 1) / kXcds, blocks = per * kXcds;
    if (blocks <= 0) return hipSuccess;
    if (blocks > 0x7fffffffLL) return hipErrorInvalidValue;
    if (back)
        hipLaunchKernelGGL((rows_gemm_kernel<BM, true>), dim3((unsigned)blocks), dim3(512), 0, s, p, nN);
    else
        hipLaunchKernelGGL((rows_gemm_kernel<BM, false>), dim3((unsigned)blocks), dim3(512), 0, s, p, nN);
    return hipGetLastError();
}

}  // namespace
}  // namespace tiled

// 256-row tiles once experts average 192 rows (as the forward's tiles), else 128
int rows_gemm_bm(long long rows, int groups) { return groups > 0 && rows >= 192LL * groups ? 256 : 128; }

hipError_t launch_rows_gemm(const RowsProblem &p, bool back, int bm, hipStream_t s) {
    if (!p.A || !p.B0 || !p.tiles || !p.n_tiles || !p.group_tile_start || p.N < 32 || p.N % 32 || p.K0 < 32 ||
        p.K0 % 32 || p.gk < 1 || p.lda < (p.B1 ? 2 * p.K0 : p.K0))
        return hipErrorInvalidValue;
    if (back ? (!p.gq || !p.gs || !p.uq || !p.us || !p.dGU || !p.Hw || p.B1) : !p.C) return hipErrorInvalidValue;
    if (bm == 256) return tiled::launch_rows<256>(p, back, s);
    if (bm == 128) return tiled::launch_rows<128>(p, back, s);
    return hipErrorInvalidValue;
}

}  // namespace moe
