// build-flags: -mllvm -amdgpu-mfma-vgpr-form
// The expert FFN's row products in training: C[r] = A(r) B_g over every
// expert's rows in one launch, A(r) contiguous in k. Four uses:
//  * GATE_UP: A(r) = X[token of r], B = W1 and W3 [H][F]. The epilogue forms
//    h = silu(g) u (bf16) and writes g and u as MXFP8 checkpoints (mx8.h):
//    they never leave the chip in 16 bits.
//  * DOWN: A = h, B = W2 [F][H], bf16 rows out.
//  * BACK, the SwiGLU backward: A(r) = dY[token of r], B = W2^T, so the
//    accumulator is p = dY W2^T, before the routing weight. The epilogue reads
//    the checkpointed g and u and forms, with s = 1 / (1 + e^-g):
//      h = g s u            dw[r] = sum_f p h        (gradient of the weight)
//      dg = w p u s (1 + g (1 - s))    du = w p g s    w h for dW2
//    dY is gathered by the copies and never multiplied by w in memory: the
//    combine's backward pass costs no pass of its own.
//  * DX: A = [dg | du] [M][2F], B = W1^T then W3^T along k; fp32 rows out (they
//    are summed over a token's k rows before the one rounding).
// h, dg, du and w h are rounded to bf16: the operands of the bf16 matrix cores.
//
// Tile BM (128 or 256) rows x 256 columns, 64 deep a step, 8 wavefronts in
// 2 x 4, each BM/2 rows x 64 columns (GATE_UP: 128 columns of W1 and of W3).
// Operands contiguous in k (A; B of the two backward uses, whose weight rows
// are k) are copied as whole 128-byte lines of a row (32 deep, the 64-byte
// halves were separate requests to L2) by buffer loads: a lane's offset stays
// the same over k, the step only moves the scalar descriptor. LDS rows are 128
// bytes, 16-byte chunk c of row
// r at c ^ ((r >> 1) & 7): a ds_read_b128 serves lanes 0-3, 12-15 and 20-27
// (then the others) together, whose eight even and eight odd rows then hit all
// 64 banks once. The forward's B keeps the weights' [K][N] layout, two 64 x 128
// panels with 256-byte rows, and is read with ds_read_b64_tr_b16 (chunks
// swizzled by bswz16 of the row).
// A step's two 32-deep halves alternate in two register sets: the second
// half's fragments are read while the first is multiplied and the next step's
// first while the second is, so one barrier a step (after the next step's
// copies have landed) both publishes the next stage and frees this one.
//
// Measured (medians): 8 experts, 8192 rows, H 4096, F 14336: BACK 1052 us (914
// TFLOP/s, 0.44 of the matrix cores' cycles at 2.0 GHz), DX 1895 (1015); 128
// experts, 65536 rows, H 2048, F 768: GATE_UP 587 (at best 473), BACK 343, DX 591
// (698 TFLOP/s, 0.35 of the cycles. A quarter of the tiles' rows are past an
// expert's end, but empty blocks are left out by 64 rows and 6 % of the
// multiplied ones are empty: the rest is a tile's start of about 6 us, BACK's
// epilogue of 15 and DX's stores, beside 24 to 32 steps); 32 experts, 4096 rows,
// H 7168, F 2048: GATE_UP 506, DOWN 244, BACK 328, DX 493 (2.4 GB at 4.9 TB/s,
// a copy's rate). Time stamps show 13 to 18 % of the CUs' time between items
// and after the last, yet a persistent form that removed it took as long: the
// card runs at its power limit, and idle CUs leave their share to the others.
//
// Tail: the last, partial round of an XCD's items is split over k into up to
// kRowsParts parts, as many as one round of its CUs takes, where an item is
// long (8 experts of 4096 x 14336, 8192 rows: DX 2150 -> 1890 us, BACK 1195 ->
// 1140; 32 experts of 7168 x 2048, 4096 rows: GATE_UP 560 -> 511). Parts in a
// second round lose: the weights' bytes bound such a launch, and the CUs left
// in a partial round get them faster (BACK of those 32 experts, 18 items left:
// 293 us, as 54 parts 310). A part leaves its fp32 sums and the last one to
// finish adds them in part order, so results do not depend on which that is.
#include "mx8.h"
#include "train_kernel.h"

namespace moe {

MOE_BOUNDS_FILE(train_rows)

namespace tiled {
namespace {

constexpr int kRowsBN = rows_gemm_bn;
constexpr int kRowsBK = 64;
constexpr int kRowsParts = 4;        // parts of a split item at most
constexpr int kRowsPartSteps = 32;   // and steps a part has at least (a part's sums cost about 10 steps)
// Workgroups along x, the others along y: one dimension of a grid holds fewer
// than 2^32 threads (beyond, a launch takes their number mod 2^32 and reports
// nothing). A multiple of the XCDs, so that the order over them goes on
constexpr uint32_t kRowsRun = 4096;

template <int BM>
struct RowsRing {
    static constexpr int a_bytes = BM * 128;
    static constexpr int b_bytes = kRowsBN * 128;
    static constexpr int stage = a_bytes + b_bytes;
    static constexpr int S = kRingBudget / stage < 3 ? kRingBudget / stage : 3;
    static constexpr int nA = BM / 64;  // 1 KB copies (8 rows) per wavefront and step
    static constexpr int nB = kRowsBN / 64;
    static constexpr int per_tile = nA + nB;
    static constexpr int MI = BM / 32;   // 16-row blocks per wavefront
    // BACK's staging per wavefront: a 16 x 64 block of each code matrix (padded
    // rows) and its scale bytes
    static constexpr int cld = 64 + 16;
    static constexpr int stg = 2 * 16 * cld + 64;
    static constexpr int dw = 8 * stg;   // [4][BM] floats behind it
    // GATE_UP's: rows of 128 bf16 h, then of both projections' 128 codes
    // (padded), then of 4 scale bytes each
    static constexpr int hld = 128 + 8, qld = 256 + 16;
    static constexpr int codes = BM * hld * 2, scales = codes + BM * qld;
    static constexpr int epi = scales + 8 * BM > dw + 16 * BM ? scales + 8 * BM : dw + 16 * BM;
    static constexpr int lds = S * stage > epi ? S * stage : epi;
    static_assert(S >= 2 && lds <= 160 * 1024, "LDS");
};

// This workgroup's item, or part of one. Items are in tile_of's order, a
// contiguous run of them per XCD; the run's last `tail` items, one partial
// round of the XCD's CUs, are split.
__device__ __forceinline__ bool pick_rows(const RowsProblem &p, int nN, int nk, Unit &u) {
    GemmProblem order{};
    order.tiles = p.tiles;
    order.n_tiles = p.n_tiles;
    order.group_tile_start = p.group_tile_start;
    const int n_tiles = *p.n_tiles, n_work = n_tiles * nN;
    const int per = (n_work + kXcds - 1) / kXcds;
    const uint32_t block = blockIdx.y * kRowsRun + blockIdx.x;
    const int xcd = block % kXcds, slot = block / kXcds;
    const int first = xcd * per, n = min(per, n_work - first);
    if (n <= 0) return false;
    const int tail = n % kBlocksPerXcd, full = n - tail;
    const int parts = p.part && tail > 0 ? max(min(min(kRowsParts, kBlocksPerXcd / tail), nk / kRowsPartSteps), 1) : 1;
    int item = slot;
    if (slot >= full) {
        const int v = slot - full;
        if (v >= tail * parts) return false;
        item = full + v / parts;
        u.part = v % parts;
        u.parts = parts;
        u.tail_slot = xcd * kBlocksPerXcd + v / parts;
        u.part_slot = xcd * kBlocksPerXcd + v;
    }
    tile_of(order, nN, n_tiles, first + item, u.mt, u.nt);
    return true;
}

template <int BM, RowsUse USE>
__global__ __launch_bounds__(512, 1) void rows_gemm_kernel(RowsProblem p, int nN) {
    typedef RowsRing<BM> R;
    constexpr bool KN = USE == ROWS_GATE_UP || USE == ROWS_DOWN;  // B is [K][N]
    constexpr int BR = KN ? 2 : 1;                                // reads of a B block
    constexpr int S = R::S, MI = R::MI, NB = 4, NC = R::per_tile, NR = BR * NB + MI;
    constexpr int W = USE == ROWS_GATE_UP ? kRowsBN / 2 : kRowsBN;  // output columns per tile
    __shared__ __attribute__((aligned(1024))) uint8_t lds[R::lds];

    // steps of one B matrix (the last may be half) and of all
    const int nk0 = (p.K0 + kRowsBK - 1) / kRowsBK, nk_all = USE == ROWS_DX ? 2 * nk0 : nk0;
    Unit u;
    if (!pick_rows(p, nN, nk_all, u)) return;
    const int mt = u.mt, nt = u.nt;
    const int k_first = nk_all * u.part / u.parts;
    const int nk = nk_all * (u.part + 1) / u.parts - k_first;
    if (MOE_BOUNDS_FAIL(mt < p.max_tiles, BOUNDS_TILE)) return;
    const int g = p.tiles[4 * mt], row0 = p.tiles[4 * mt + 1], row_end = p.tiles[4 * mt + 2];
    if (MOE_BOUNDS_FAIL(g >= 0 && g < p.n_groups && row0 >= 0 && row0 < row_end && row_end <= p.M, BOUNDS_TILE))
        return;
    const int n0 = nt * W;
    const int tid = threadIdx.x;
    const int lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), wr = w / 4, wc = w % 4;
    const int i16 = lane & 15, gq = lane >> 4;
    const int nblk = min(max((row_end - row0 - wr * (BM / 2) + 15) >> 4, 0), MI);

    // ---- copy sources: lane -> row lane / 8 of an 8-row copy, physical chunk
    // lane % 8; byte offsets from the descriptor's start, which is the tile's
    // first row (gathered A: row 0) at the step's first column ----
    uint32_t a_off[R::nA], b_off[R::nB];
#pragma unroll
    for (int q = 0; q < R::nA; ++q) {
        const int tr = 8 * (w * R::nA + q) + (lane >> 3);
        int r = row0 + tr;
        if (r >= row_end) r = row0;  // rows past the tile's end copy a valid row (never stored)
        int src = p.row_src ? p.row_src[r] : r - row0;
        if (p.row_src) {
            if (MOE_BOUNDS_FAIL(src >= 0 && src < p.a_rows * p.gk, BOUNDS_A_ROW)) src = 0;
            src /= p.gk;
        }
        a_off[q] = 2u * ((uint32_t)src * p.lda + 8 * ((lane & 7) ^ ((tr >> 1) & 7)));
    }
    const char *a0 = reinterpret_cast<const char *>(p.A + (p.row_src ? 0LL : (long long)row0 * p.lda));
    // B [N][K0]: rows as A's. B [K0][N]: panel q / 2 of 128 columns, copy q % 2
    // of it fills rows 4 (2 w + q % 2) + lane / 16 of the step; columns past N
    // read the last ones, a DOWN panel past N the first panel (never stored)
    const char *b0, *b1;
    static_assert(!KN || R::nB == 4, "two copies a panel");
    const int panel1 = USE == ROWS_DOWN && p.N - n0 > 128 ? 128 : 0;
#pragma unroll
    for (int q = 0; q < R::nB; ++q) {
        if constexpr (KN) {
            const int k = 4 * (2 * w + (q & 1)) + (lane >> 4), first = n0 + (q < 2 ? 0 : panel1);
            b_off[q] = 2u * ((uint32_t)k * p.N + min(8 * ((lane & 15) ^ bswz16(k)), p.N - 8 - first));
        } else {
            const int tr = 8 * (w * R::nB + q) + (lane >> 3);
            b_off[q] = 2u * ((uint32_t)min(tr, p.N - 1 - n0) * p.K0 + 8 * ((lane & 7) ^ ((tr >> 1) & 7)));
        }
    }
    if constexpr (KN) {
        const long long first = (long long)g * p.K0 * p.N + n0;
        b0 = reinterpret_cast<const char *>(p.B0 + first);
        b1 = USE == ROWS_GATE_UP ? reinterpret_cast<const char *>(p.B1 + first) : b0 + 2 * panel1;
    } else {
        const long long first = ((long long)g * p.N + n0) * p.K0;
        b0 = reinterpret_cast<const char *>(p.B0 + first);
        b1 = USE == ROWS_DX ? reinterpret_cast<const char *>(p.B1 + first) : b0;
    }
    // bytes from the descriptor's start to the last row's end
    const uint32_t a_len = 2u * p.lda * (uint32_t)(p.row_src ? p.a_rows : row_end - row0);
    const uint32_t b_len = 2u * p.K0 * (uint32_t)min(kRowsBN, p.N - n0);
    // where K0 ends in the middle of a step, the lanes of the step's second 64
    // bytes get offsets past any range and so read zeros
    // (a copy's rows are 8 q' .. + 7, q' even or odd with q: its chunk swizzle
    // is (4 q' + lane / 16) % 8)
    static_assert(R::nA % 2 == 0 && R::nB % 2 == 0, "parity of a copy's rows");
    uint32_t second[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) second[q] = ((lane & 7) ^ (4 * q + (lane >> 4))) >= 4 ? gather_max_bytes : 0;
    auto copy = [&](int q, int kt, int stage) {
        uint8_t *st = lds + stage * R::stage;
        const int seg = USE == ROWS_DX && kt >= nk0 ? 1 : 0, k = kRowsBK * (kt - seg * nk0);  // first column of the step in its matrix
        const uint32_t cut = k + kRowsBK > p.K0 ? ~0u : 0u;
        if (q < R::nA) {
            const int ka = 2 * (k + seg * p.K0);
            copy16_buffer(a0 + ka, a_len - ka, a_off[q] | (second[q & 1] & cut), st + (w * R::nA + q) * 1024);
        } else if constexpr (KN) {
            // the rows left of K0 (the others of a last half step read zeros)
            const int s = (q - R::nA) / 2, i = (q - R::nA) % 2;
            const uint32_t len = 2u * ((uint32_t)min(kRowsBK, p.K0 - k) * p.N - n0 - (s ? panel1 : 0));
            copy16_buffer((s ? b1 : b0) + 2LL * k * p.N, len, b_off[q - R::nA],
                          st + R::a_bytes + s * (R::b_bytes / 2) + (2 * w + i) * 1024);
        } else {
            copy16_buffer((seg ? b1 : b0) + 2 * k, b_len - 2 * k, b_off[q - R::nA] | (second[(q - R::nA) & 1] & cut),
                          st + R::a_bytes + (w * R::nB + q - R::nA) * 1024);
        }
    };

    // ---- fragment reads of half h: B blocks, then A row blocks ----
    struct Frag {
        bf16x8 a[MI], b[NB];
        u32x2 raw[KN ? NB : 1][2];
    };
    const int swz = (i16 >> 1) & 7;  // of row i16 of any 16-row block
    const int a_row = (wr * (BM / 2) + i16) * 128, b_row = R::a_bytes + (64 * wc + i16) * 128;
    // B [K0][N]: the lane's k rows are 32 h + 8 gq + 4 (half of the read pair) +
    // i16 / 4 of the block's panel; column block j moves the chunk index in
    // bits that only the swizzle's XOR touches
    const int k0 = 8 * gq + (i16 >> 2), c0 = ((i16 & 3) >> 1) + (USE == ROWS_GATE_UP ? 4 * wc : 8 * (wc & 1));
    const uint32_t b_tr = R::a_bytes + (USE == ROWS_GATE_UP ? 0 : (wc >> 1) * (R::b_bytes / 2)) + k0 * 256 +
                          16 * (c0 ^ bswz16(k0)) + 8 * (i16 & 1);
    auto read = [&](Frag &f, int r, int stage, auto half) {
        constexpr int h = decltype(half)::value;
        const uint8_t *st = lds + stage * R::stage;
        if constexpr (KN) {
            if (r < 2 * NB) {
                const int j = r >> 1;
                // GATE_UP: blocks 0, 1 of W1's panel and 2, 3 of W3's
                const uint32_t at = (lds_addr(st) + b_tr) ^ (32 * (USE == ROWS_GATE_UP ? j & 1 : j));
                constexpr int panel = USE == ROWS_GATE_UP ? R::b_bytes / 2 : 0, kh = 4 * 256;
                if (j < 2) f.raw[j][r & 1] = r & 1 ? ds_tr16_at<h * 8192 + kh>(at) : ds_tr16_at<h * 8192>(at);
                else f.raw[j][r & 1] = r & 1 ? ds_tr16_at<h * 8192 + kh + panel>(at) : ds_tr16_at<h * 8192 + panel>(at);
                return;
            }
            r -= 2 * NB;
        } else {
            if (r < NB) {
                f.b[r] = *reinterpret_cast<const bf16x8 *>(st + 16 * ((4 * h + gq) ^ swz) + b_row + r * 2048);
                return;
            }
            r -= NB;
        }
        f.a[r] = *reinterpret_cast<const bf16x8 *>(st + 16 * ((4 * h + gq) ^ swz) + a_row + r * 2048);
    };
    // the reads have completed: hand the transposed ones to the compiler
    auto land = [&](Frag &f) {
        wait_lds();
        if constexpr (KN) {
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                fence(f.raw[j][0]);
                fence(f.raw[j][1]);
                f.b[j] = __builtin_bit_cast(
                    bf16x8, u32x4{f.raw[j][0][0], f.raw[j][0][1], f.raw[j][1][0], f.raw[j][1][1]});
            }
        }
    };
    constexpr std::integral_constant<int, 0> first_half;
    constexpr std::integral_constant<int, 1> second_half;

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

    const int k_last = k_first + nk - 1;
    Frag fa, fb;
#pragma unroll
    for (int t = 0; t < S; ++t)
#pragma unroll
        for (int q = 0; q < NC; ++q) copy(q, min(k_first + t, k_last), t);
    wait_vm<(S - 1) * NC>();
    __builtin_amdgcn_s_barrier();
#pragma unroll
    for (int r = 0; r < NR; ++r) read(fa, r, 0, first_half);
    land(fa);
    auto kloop = [&](auto act) {
        constexpr int ACT = decltype(act)::value;
        auto wanted = [](int r) { return ACT > 0 && (r < BR * NB || r - BR * NB < ACT); };
        int stage = 0;
        for (int kt = k_first; kt <= k_last; ++kt) {
            const int nstage = stage + 1 == S ? 0 : stage + 1;
            const int src = min(kt + S, k_last);
            // first half; the second's fragments are read
            constexpr int SA = MI - 1;
#pragma unroll
            for (int c = 0; c < MI; ++c) {
#pragma unroll
                for (int r = c * NR / SA; r < (c + 1) * NR / SA && r < NR; ++r)
                    if (wanted(r)) read(fb, r, stage, second_half);
                mma_rows(fa, c, act);
            }
            if (ACT > 0) land(fb);
            // second half; the next step's first fragments are read
            constexpr int PRE = MI >= 8 ? 2 : 1, SLOTS = MI - PRE;
#pragma unroll
            for (int m = 0; m < PRE; ++m) mma_rows(fb, m, act);
            wait_vm<(S - 2) * NC>();
            __builtin_amdgcn_s_barrier();
#pragma unroll
            for (int c = 0; c < SLOTS; ++c) {
#pragma unroll
                for (int q = c * NC / SLOTS; q < (c + 1) * NC / SLOTS; ++q) copy(q, src, stage);
#pragma unroll
                for (int r = c * NR / SLOTS; r < (c + 1) * NR / SLOTS; ++r)
                    if (wanted(r)) read(fa, r, nstage, first_half);
                mma_rows(fb, c + PRE, act);
            }
            if (ACT > 0) land(fa);
            stage = nstage;
        }
    };
    if (nblk == 0) kloop(std::integral_constant<int, 0>{});
    else if (MI >= 8 && nblk <= MI / 2) kloop(std::integral_constant<int, MI / 2>{});
    else kloop(std::integral_constant<int, MI>{});

    wait_vm<0>();  // the repeated copies of the last steps land before the LDS is used again
    if (u.parts > 1) {
        // leave this part's sums ([accumulator][thread] vectors); the last part
        // to count itself adds all of them in part order
        if (MOE_BOUNDS_FAIL(u.part_slot < rows_gemm_counters && u.part_slot >= u.part, BOUNDS_TAIL_SLOT)) return;
        f32x4 *mine = reinterpret_cast<f32x4 *>(p.part) + (long long)u.part_slot * (MI * NB * 512);
#pragma unroll
        for (int i = 0; i < MI * NB; ++i) mine[i * 512 + tid] = acc[i / NB][i % NB];
        wait_vm<0>();
        __syncthreads();
        int *last = reinterpret_cast<int *>(lds);
        if (tid == 0) {
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "agent");
            *last = __hip_atomic_fetch_add(p.part_cnt + u.tail_slot, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
                    u.parts - 1;
            if (*last) __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
        }
        __syncthreads();
        if (!*last) return;
        const f32x4 *part0 = mine - (long long)u.part * (MI * NB * 512);
#pragma unroll
        for (int i = 0; i < MI * NB; ++i) acc[i / NB][i % NB] = part0[i * 512 + tid];
        for (int q = 1; q < u.parts; ++q) {
            part0 += MI * NB * 512;
#pragma unroll
            for (int i = 0; i < MI * NB; ++i) acc[i / NB][i % NB] += part0[i * 512 + tid];
        }
        __syncthreads();  // the flag has been read: the LDS is free
    }
    // a 16 x 64 block of bf16 results, whole lines (of 64-byte pieces each is two
    // requests to L2)
    auto store_lines = [&](uint16_t *C, int ld, int m, const f32x4 (&x)[NB]) {
        u32x4 v[2] = {pair_columns(x[0], x[1]), pair_columns(x[2], x[3])};
        whole_lines(v[0], v[1]);
        const int col = n0 + 64 * wc + 32 * (i16 >> 3) + pair_column(gq);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int row = row0 + wr * (BM / 2) + 16 * m + 8 * i + (i16 & 7);
            if (row < row_end && col < p.N) *reinterpret_cast<u32x4 *>(C + (long long)row * ld + col) = v[i];
        }
    };
    if constexpr (USE == ROWS_DX) {
#pragma unroll
        for (int m = 0; m < MI; ++m) {
            if (m >= nblk) continue;
#pragma unroll
            for (int j = 0; j < NB; j += 2) {
                u32x4 v[2] = {__builtin_bit_cast(u32x4, acc[m][j]), __builtin_bit_cast(u32x4, acc[m][j + 1])};
                whole_lines(v[0], v[1]);
                const int col = n0 + 64 * wc + 16 * (j + (i16 >> 3)) + 4 * gq;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int row = row0 + wr * (BM / 2) + 16 * m + 8 * i + (i16 & 7);
                    if (row < row_end && col < p.N)
                        *reinterpret_cast<u32x4 *>(reinterpret_cast<float *>(p.C) + (long long)row * p.N + col) = v[i];
                }
            }
        }
    } else if constexpr (USE == ROWS_DOWN) {
        uint16_t *C = reinterpret_cast<uint16_t *>(p.C);
#pragma unroll
        for (int m = 0; m < MI; ++m) {
            if (m >= nblk) continue;
            store_lines(C, p.N, m, acc[m]);
        }
    } else if constexpr (USE == ROWS_GATE_UP) {
        __syncthreads();
        // the tile's h, codes and scale bytes in LDS, then 16-byte pieces of
        // rows. A wavefront's 32 columns of a projection are one scale group:
        // 8 values in each of the four lanes that share lane % 16
        uint16_t *sh = reinterpret_cast<uint16_t *>(lds);
#pragma unroll
        for (int m = 0; m < MI; ++m) {
            if (m >= nblk) continue;
            const int r = wr * (BM / 2) + 16 * m + i16;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float h[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) h[i] = silu_f32(acc[m][j][i]) * acc[m][j + 2][i];
                *reinterpret_cast<u32x2 *>(sh + r * R::hld + 32 * wc + 16 * j + 4 * gq) =
                    u32x2{pack_bf16x2(h[0], h[1]), pack_bf16x2(h[2], h[3])};
            }
#pragma unroll
            for (int half = 0; half < 2; ++half) {  // g, u
                const f32x4 (&v)[NB] = acc[m];
                uint32_t top = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) top = max(top, mx8::amax_bits(v[2 * half + i / 4][i % 4]));
                top = max(top, (uint32_t)__shfl_xor((int)top, 16));
                top = max(top, (uint32_t)__shfl_xor((int)top, 32));
                const int e = mx8::scale_exp(top);
                const float inv = mx8::pow2(-e);
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const f32x4 &x = v[2 * half + q];
                    *reinterpret_cast<uint32_t *>(lds + R::codes + r * R::qld + 128 * half + 32 * wc + 16 * q + 4 * gq) =
                        mx8::codes4(mx8::scaled(x[0], inv), mx8::scaled(x[1], inv), mx8::scaled(x[2], inv),
                                    mx8::scaled(x[3], inv));
                }
                if (gq == 0) lds[R::scales + r * 8 + 4 * half + wc] = (uint8_t)(e + 127);
            }
        }
        __syncthreads();
        uint16_t *C = reinterpret_cast<uint16_t *>(p.C);
        for (int i = tid; i < BM * 16; i += 512) {
            const int r = i >> 4, c = i & 15, row = row0 + r;
            if (row >= row_end) break;  // rows only grow
            if (n0 + 8 * c < p.N)
                *reinterpret_cast<u32x4 *>(C + (long long)row * p.N + n0 + 8 * c) =
                    *reinterpret_cast<const u32x4 *>(sh + r * R::hld + 8 * c);
            // 8 pieces of 16 codes of each projection (N % 32 == 0)
            const int half = c >> 3, col = n0 + 16 * (c & 7);
            if (col < p.N)
                *reinterpret_cast<u32x4 *>((half ? p.uq_out : p.gq_out) + (long long)row * p.N + col) =
                    *reinterpret_cast<const u32x4 *>(lds + R::codes + r * R::qld + 16 * c);
        }
        for (int i = tid; i < BM * 8; i += 512) {
            const int r = i >> 3, half = (i >> 2) & 1, q = i & 3, row = row0 + r;
            if (row < row_end && n0 + 32 * q < p.N)
                (half ? p.us_out : p.gs_out)[(long long)row * (p.N >> 5) + (n0 >> 5) + q] =
                    lds[R::scales + r * 8 + 4 * half + q];
        }
    } else {
        // ---- SwiGLU backward, 16 rows at a time; the codes come kAhead blocks
        // ahead of their use (one ahead each block waited for memory: 20 us a
        // tile) and change from rows of 16 to the accumulators' layout through
        // the wavefront's staging area ----
        constexpr int kAhead = MI < 4 ? MI : 4;
        uint8_t *sc = lds + w * R::stg, *ss = sc + 2 * 16 * R::cld;
        float *sdw = reinterpret_cast<float *>(lds + R::dw);
        const int c0 = n0 + 64 * wc, base = row0 + wr * (BM / 2);
        // code loads: lane -> row lane / 4 of the block, 16 codes at 16 (lane % 4)
        // and one of its scale bytes: g's two, then u's
        const int lr = lane >> 2, lc = 16 * (lane & 3);
        struct Codes {
            u32x4 g, u;
            uint8_t s;
        };
        Codes codes[kAhead];
        auto load = [&](int m) {
            Codes &c = codes[m % kAhead];
            const int r = base + 16 * m + lr, group = (c0 >> 5) + (lane & 1);
            c.g = c.u = u32x4{0, 0, 0, 0};
            c.s = 0;
            if (r >= row_end) return;
            if (c0 + lc < p.N) {
                const long long o = (long long)r * p.N + c0 + lc;
                c.g = *reinterpret_cast<const u32x4 *>(p.gq + o);
                c.u = *reinterpret_cast<const u32x4 *>(p.uq + o);
            }
            if (group < p.N >> 5) c.s = (lane & 2 ? p.us : p.gs)[(long long)r * (p.N >> 5) + group];
        };
        // the wavefront's routing weights, one row a lane
        float row_w[(MI + 3) / 4];
#pragma unroll
        for (int i = 0; i < (MI + 3) / 4; ++i) {
            const int r = base + 64 * i + lane;
            row_w[i] = 0.0f;
            if (r >= row_end || 64 * i + lane >= BM / 2) continue;
            int a = p.w_src ? p.w_src[r] : r;
            if (MOE_BOUNDS_FAIL(a >= 0 && a < p.M, BOUNDS_A_ROW)) a = 0;
            row_w[i] = p.topk_w ? p.topk_w[a] : 1.0f;
        }
#pragma unroll
        for (int m = 0; m < kAhead; ++m) load(m);
        __syncthreads();  // every wavefront is done with the ring
#pragma unroll
        for (int m = 0; m < MI; ++m) {
            if (m >= nblk) {  // no rows of the group
                if (gq == 0) sdw[wc * BM + wr * (BM / 2) + 16 * m + i16] = 0.0f;
                continue;
            }
            const Codes &cur = codes[m % kAhead];
            *reinterpret_cast<u32x4 *>(sc + lr * R::cld + lc) = cur.g;
            *reinterpret_cast<u32x4 *>(sc + (16 + lr) * R::cld + lc) = cur.u;
            ss[lane] = cur.s;
            if (m + kAhead < MI) load(m + kAhead);
            wave_lds_sync();
            const uint32_t sb = *reinterpret_cast<const uint32_t *>(ss + 4 * i16);
            const float wt = __shfl(row_w[m / 4], 16 * (m % 4) + i16);
            float dw = 0.0f, dw_half = 0.0f;
            f32x4 dg[NB], du[NB], hw[NB];
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                if (j == NB / 2) dw_half = dw;
                const uint32_t gw = *reinterpret_cast<const uint32_t *>(sc + i16 * R::cld + 16 * j + 4 * gq);
                const uint32_t uw = *reinterpret_cast<const uint32_t *>(sc + (16 + i16) * R::cld + 16 * j + 4 * gq);
                const f32x4 gv = mx8::values4(gw, mx8::scale_of((uint8_t)(sb >> (8 * (j / 2)))));
                const f32x4 uv = mx8::values4(uw, mx8::scale_of((uint8_t)(sb >> (16 + 8 * (j / 2)))));
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.4426950408889634f * gv[i]));
                    const float gsv = gv[i] * s, h = gsv * uv[i], pv = acc[m][j][i];
                    dw = fmaf(pv, h, dw);
                    const float pw = wt * pv;
                    du[j][i] = pw * gsv;
                    // s (1 + g (1 - s)) = s + g s (1 - s)
                    dg[j][i] = pw * uv[i] * fmaf(gsv, 1.0f - s, s);
                    hw[j][i] = wt * h;
                }
            }
            wave_lds_sync();
            store_lines(p.dGU, 2 * p.N, m, dg);
            store_lines(p.dGU + p.N, 2 * p.N, m, du);
            store_lines(p.Hw, p.N, m, hw);
            // columns past N (N % 32 == 0) have h = 0, but their p may be infinite
            if (c0 + 32 >= p.N) dw = dw_half;
            dw += __shfl_xor(dw, 16);
            dw += __shfl_xor(dw, 32);
            if (gq == 0) sdw[wc * BM + wr * (BM / 2) + 16 * m + i16] = c0 < p.N ? dw : 0.0f;
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
hipError_t launch_rows(const RowsProblem &p, RowsUse use, hipStream_t s) {
    const int nN = rows_gemm_columns(p.N, use);
    // items per XCD, and the parts that the last of them may be split into
    const long long per = ((long long)p.max_tiles * nN + kXcds - 1) / kXcds + (p.part ? kBlocksPerXcd : 0);
    const long long blocks = per * kXcds, runs = (blocks + kRowsRun - 1) / kRowsRun;
    if (blocks <= 0) return hipSuccess;
    if (runs > 0xffff) return hipErrorInvalidValue;
    auto launch = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)(runs > 1 ? kRowsRun : blocks), (unsigned)runs), dim3(512), 0, s, p,
                           nN);
    };
    switch (use) {
    case ROWS_GATE_UP: launch(rows_gemm_kernel<BM, ROWS_GATE_UP>); break;
    case ROWS_DOWN: launch(rows_gemm_kernel<BM, ROWS_DOWN>); break;
    case ROWS_BACK: launch(rows_gemm_kernel<BM, ROWS_BACK>); break;
    case ROWS_DX: launch(rows_gemm_kernel<BM, ROWS_DX>); break;
    }
    return hipGetLastError();
}

}  // namespace
}  // namespace tiled

// 256-row tiles read B half as often and have half as many items to start and
// end; 128-row ones leave fewer rows of an expert's last tile empty. Taken: 256
// where both hold, else 128.
//  * Experts average kTallRows rows. Whole calls, 128 against 256 (us; experts
//    x H x F): forward at 192 rows an expert 271 to 320 (16 x 4096 x 2048), 425
//    to 438 (128 x 2048 x 768), 836 to 853 (8 x 4096 x 14336), at 224 335 to
//    320, 458 to 451, 965 to 875, at 384 426 to 365, 660 to 608, 1389 to 1166;
//    backward at 224 678 to 688, 997 to 1017, 2020 to 2060, at 288 771 to 740,
//    1152 to 1151, 2377 to 2324, at 384 856 to 819, 1386 to 1392, 2807 to 2597.
//    (64 experts of 2048 x 768, the shape that gains least: 4 % slower at 256
//    in the forward, 1 % at 288 in the backward.)
//  * 128-row tiles would need a second round of the CUs. Forward at 128 tiles
//    of 256 rows 45 to 58 (4 x 1024 x 512), 126 to 142 (4 x 1536 x 2048), at 144
//    70 to 59, 153 to 146; backward at 126 132 to 156 (8 x 768 x 768), 258 to
//    281, at 144 178 to 165, 302 to 310, at 200 210 to 203, 391 to 402.
int rows_gemm_bm(RowsPass pass, long long rows, int groups, int columns) {
    const long long kTallRows = pass == ROWS_FORWARD ? 224 : 288;
    const long long tiles = rows / 256 + groups / 2;  // about half a tile of each expert is a rest
    const long long cus = tiled::kXcds * tiled::kBlocksPerXcd;
    return groups > 0 && rows >= kTallRows * groups && 2 * tiles * columns > cus ? 256 : 128;
}
int rows_gemm_columns(int N, RowsUse use) {
    const int w = use == ROWS_GATE_UP ? rows_gemm_bn / 2 : rows_gemm_bn;
    return (N + w - 1) / w;
}
static_assert(rows_gemm_counters == tiled::kXcds * tiled::kBlocksPerXcd, "one slot per CU");
size_t rows_gemm_part_bytes(int bm, RowsUse use, int K0) {
    // none where the steps are too few to split
    if (K0 * (use == ROWS_DX ? 2LL : 1LL) < 2LL * tiled::kRowsPartSteps * tiled::kRowsBK) return 0;
    return sizeof(float) * (size_t)rows_gemm_counters * bm * rows_gemm_bn;
}

hipError_t launch_rows_gemm(const RowsProblem &p, RowsUse use, int bm, hipStream_t s) {
    const bool two = use == ROWS_GATE_UP || use == ROWS_DX;
    if (!p.A || !p.B0 || two != (p.B1 != nullptr) || !p.tiles || !p.n_tiles || !p.group_tile_start || p.N < 32 ||
        p.N % 32 || p.K0 < 32 || p.K0 % 32 || p.gk < 1 || p.lda < (use == ROWS_DX ? 2 * p.K0 : p.K0) ||
        (p.row_src && (p.a_rows < 1 || 2LL * p.a_rows * p.lda > gather_max_bytes)) ||
        (p.part && !p.part_cnt))
        return hipErrorInvalidValue;
    if (use == ROWS_BACK ? (!p.gq || !p.gs || !p.uq || !p.us || !p.dGU || !p.Hw) : !p.C) return hipErrorInvalidValue;
    if (use == ROWS_GATE_UP && (!p.gq_out || !p.gs_out || !p.uq_out || !p.us_out)) return hipErrorInvalidValue;
    if (bm == 256) return tiled::launch_rows<256>(p, use, s);
    if (bm == 128) return tiled::launch_rows<128>(p, use, s);
    return hipErrorInvalidValue;
}

}  // namespace moe
