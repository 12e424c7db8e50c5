// W4A4 grouped GEMM: MXFP4 weights times MXFP4 rows on the scaled 4-bit matrix
// instruction.
// build-flags: -mllvm -amdgpu-mfma-vgpr-form
//
// Math: C[r, n] = sum over groups b of 32 K of
//   2^(sa[r, b] - 127) 2^(sw[b, n] - 127) sum_{k in b} qa[r, k] qw[k, n]
// One v_mfma_scale_f32_32x32x64_f8f6f4 takes two groups of a 32 x 32 output
// block, scales included, and adds in fp32: no arithmetic is left to the
// vector unit inside the K loop. (The 16 x 16 x 128 form reaches 3.5 to 5.2
// PFLOP/s from registers with random codes, this one 6.1 to 6.4; its issue
// rate allows 9.0, reached with zeros: the clock falls under load.)
//
// Tile: BM = 64 MI rows x 256 B-columns x 128 deep; 2 x 4 wavefronts, each 32 MI
// rows x 64 B-columns (MI x 2 blocks).
//  * gate/up (SWIGLU): B-columns 0..127 are W1[:, n0:n0+128], the rest
//    W3[:, n0:n0+128]. Wavefront column wc holds both accumulators of output
//    columns n0 + 32 wc .. + 31: one MXFP4 group, so h = silu(g) u is
//    quantised from the fp32 accumulators in registers and leaves as codes.
//  * down (PLAIN): B-columns are W2[:, n0:n0+256].
// Rows come in panels (mx4.h), so a K step of a tile is one contiguous piece of
// codes and one of scale words; a panel's rows past the tile's end are read and
// multiplied (they are other rows, or uninitialised ones) and never stored.
// Persistent: a workgroup walks its share of its XCD's contiguous run of the
// work order, and the ring of S stages (global -> LDS copies, a fixed count in
// flight) runs on from item to item. A stage's first half (64 deep) is
// multiplied while its second half is read to registers, its second half while
// the next stage's first is.
//  * A tile: 64-byte rows, 16-byte chunk c of row r at c ^ ((r >> 2) & 3): a
//    16-lane pass of the 16-byte operand reads touches all banks.
//  * B tile: two halves of 128 columns, [64 byte rows][128], each byte two K
//    rows of its column; 16-byte chunk c of byte row k at c ^ 2 ((k >> 1) & 3).
//    An operand (16 bytes of one column) is two ds_read_b64_tr_b8, 8 byte rows
//    each; the 8 rows x 32 bytes of 32 lanes fall into distinct banks.
//  * K not a multiple of 128: the rows' panels are filled up with zero codes;
//    the weights' rows past the end are the last one again (times zero).
//
// What bounds it. Few rows an expert: the weights' bytes (32 experts of 7168 x 2048, 8
// rows each: gate/up 499 MB in 108 us, down 250 MB in 56; 120 rows: 135 and 83; 128 on
// average, 6 to 592, 2.5 rounds of tiles: 172 to 177 and 89 to 96). Many: the matrix
// cores, at the clock that the card holds under them. 8 experts, 8192 rows, H 4096,
// F 14336: gate/up 515 to 565 us, 3.7 to 3.4 PFLOP/s, down 265 to 292; tiles are 12 % larger than
// the rows, and the matrix cores are busy for 60 % of the cycles at 1.5 to 1.8 GHz. A
// loop of the same products, LDS reads and a barrier a step reaches 4.8 PFLOP/s cold
// and 6.0 in the long run, at 1.3 to 1.7 GHz, against 8.7 at 2.4 GHz with zeros. Fewer
// cycles hence gain little: reads spread over the whole step with a wait for each row
// block took 5 % of the cycles and nothing of the median time away. 4 wavefronts of
// 128 x 128, two workgroups a CU of 128 x 256, ranges of equal steps in place of whole
// items, staggered starts: as fast or slower. Passing over the products of row blocks
// without rows costs a branch a half step: 610 to 640 us.
#include "mx4.h"
#include "tiled_gemm_kernel.h"

namespace moe {

MOE_BOUNDS_FILE(a4)

namespace tiled {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kA4BK = 128;    // K per step
constexpr int kA4Items = 64;  // work items per workgroup at most (LDS table)
constexpr int WR = 2, WC = 4, NW = WR * WC, NJ = 8 / WC;  // wavefronts; 32-column blocks of one

template <int MI>
struct RingA4 {
    static constexpr int BM = 32 * MI * WR;
    static constexpr int a_bytes = BM * 64;
    static constexpr int b_bytes = 64 * 256;
    static constexpr int sa_bytes = BM * 4;
    static constexpr int sb_bytes = 4 * 256;
    static constexpr int sb_at = a_bytes + b_bytes + sa_bytes;
    static constexpr int stage = sb_at + sb_bytes;
    static constexpr int at = 16 * kA4Items;  // the table of items comes first
    static constexpr int S = (160 * 1024 - at) / stage < 6 ? (160 * 1024 - at) / stage : 6;
    static constexpr int a_chunks = a_bytes / 1024;  // 1 KB copies, 16 rows each
    static constexpr int nA = (a_chunks + NW - 1) / NW;
    static constexpr int nB = 16 / NW;               // 1 KB copies, 8 byte rows of a half each
    static constexpr int slots = BM / 64 + 4;        // 256-byte scale copies
    static constexpr int nS = (slots + NW - 1) / NW;
    static constexpr int per_step = nA + nB + nS;
    static constexpr int lds = at + S * stage;
    static_assert(S >= 3 && BM % 64 == 0 && (S - 2) * per_step < 64, "ring");
};

// What steers the K loop is kept in scalar registers: a count that went through a
// vector load or a division leaves a loop of exec masks, 15 % slower
__device__ __forceinline__ int scalar(int x) { return __builtin_amdgcn_readfirstlane(x); }

template <int OPB, int OPA>
__device__ __forceinline__ f32x16 mfma4(const i32x4 &b, const i32x4 &a, const f32x16 &c, int sb, int sa) {
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(i32x8{b[0], b[1], b[2], b[3], 0, 0, 0, 0},
                                                           i32x8{a[0], a[1], a[2], a[3], 0, 0, 0, 0}, c, 4, 4, OPB, sb,
                                                           OPA, sa);
}
struct ItemA4 {
    int g, row0, row_end, n0;
};
// A workgroup's items: first + slot + i slots < first + n for i = 0, 1, .., or piece
// `piece` (64 MI rows) of item `first` alone (n: 1, or 0 for none)
struct Share {
    int first, n, piece;
};

// The work order's item `id`: its rows and its column tile
__device__ __forceinline__ void item_rows(const GemmProblem &p, int nN, int n_tiles, int slots, int id, int &g, int &r0,
                                          int &r1, int &nt) {
    int mt;
    // one round of about a tile an expert: no rows share weights, and the work order's
    // two dependent loads (0.6 us of 8) are spared
    if (n_tiles <= p.n_groups && n_tiles * nN <= slots * kXcds) {
        mt = id / nN;
        nt = id - mt * nN;
    } else {
        tile_of(p, nN, n_tiles, id, mt, nt);
    }
    const bool ok = mt < p.max_tiles;
    g = ok ? p.tiles[4 * mt] : 0, r0 = ok ? p.tiles[4 * mt + 1] : 0, r1 = ok ? p.tiles[4 * mt + 2] : 0;
    if (MOE_BOUNDS_FAIL(ok && g >= 0 && g < p.n_groups && r0 >= 0 && r0 < r1 && r1 <= p.M, BOUNDS_TILE)) {
        g = 0;
        r0 = 0;
        r1 = 1;
    }
}

template <bool SWIGLU, int MI>
__device__ __forceinline__ void run_items(const GemmProblem &p, int nN, int n_tiles, const Share &share, uint8_t *lds) {
    typedef RingA4<MI> R;
    constexpr int S = R::S;
    constexpr int W = SWIGLU ? 128 : 256;
    int *table = reinterpret_cast<int *>(lds);
    uint8_t *ring = lds + R::at;

    const int tid = threadIdx.x;
    const int lane = tid & 63, w = scalar(tid >> 6), wr = w / WC, wc = w % WC;
    const int l32 = lane & 31, hb = lane >> 5;
    const int nk = (p.K + kA4BK - 1) / kA4BK;
    const int slot = blockIdx.x / kXcds, slots = gridDim.x / kXcds;

    // ---- this workgroup's items ----
    const bool alone = share.piece >= 0;
    int count = alone ? share.n : slot < share.n ? scalar((share.n - slot + slots - 1) / slots) : 0;
    if (MOE_BOUNDS_FAIL(count <= kA4Items, BOUNDS_TILE)) return;
    {
        int g = 0, r0 = 0, r1 = 0, nt = 0;
        if (lane < count) {
            item_rows(p, nN, n_tiles, slots, share.first + (alone ? 0 : slot + slots * lane), g, r0, r1, nt);
            if (alone) {
                r0 += R::BM * share.piece;
                r1 = min(r1, r0 + R::BM);
            }
        }
        const unsigned long long some = __ballot(r0 < r1);  // a piece without rows is dropped
        if (w == 0 && r0 < r1)
            *reinterpret_cast<i32x4 *>(table + 4 * __popcll(some & ((1ULL << lane) - 1))) = i32x4{g, r0, r1, nt * W};
        count = scalar(__popcll(some));
    }
    __syncthreads();
    if (count == 0) return;
    auto item_at = [&](int j) {
        const i32x4 t = *reinterpret_cast<const i32x4 *>(table + 4 * j);
        return ItemA4{scalar(t[0]), scalar(t[1]), scalar(t[2]), scalar(t[3])};
    };

    // ---- copies: a uniform base that moves on each step, and a lane's offset.
    // A chunk i: rows 16 i + lane / 4. B chunk i: half i / 8, byte rows
    // 8 (i % 8) + lane / 8. Scale slot i: 64 rows' words, or (from BM / 64 on)
    // half h, K groups 2 q and 2 q + 1 of 128 columns. Surplus copies repeat
    // the last one, so every wavefront issues the same number ----
    auto a_chunk = [&](int q) { return min(w + NW * q, R::a_chunks - 1); };
    auto s_slot = [&](int q) { return min(w + NW * q, R::slots - 1); };
    const uint8_t *a_base, *b_base[2], *s_base[R::nS];
    uint32_t b_off[R::nB], s_off[R::nS];
    uint32_t a_off;  // of chunk 0
    {
        const int row = lane >> 2;  // 16 rows: the swizzle depends on these alone
        a_off = row * 64 + 16 * ((lane & 3) ^ ((row >> 2) & 3));
    }
    // byte rows and K groups of the last step that the weights have
    const int k_rows = p.K / 2 - 64 * (nk - 1), k_groups = p.K / 32 - 4 * (nk - 1);
    const bool ragged = p.K % kA4BK != 0;
    auto bytes = [](const void *x) { return static_cast<const uint8_t *>(x); };
    const uint8_t *wb0 = bytes(p.B0), *wb1 = bytes(p.B1), *ws0 = bytes(p.S0), *ws1 = bytes(p.S1);
    const uint8_t *xb0 = bytes(p.Bx0), *xb1 = bytes(p.Bx1), *xs0 = bytes(p.Sx0), *xs1 = bytes(p.Sx1);
    auto set_sources = [&](const ItemA4 &it) {
        int ln = lane;  // re-read: its multiples need not live through the K loop
        asm volatile("" : "+v"(ln));
        const bool extra = it.g == p.extra_group;
        a_base = reinterpret_cast<const uint8_t *>(p.A) + (long long)it.row0 * 64;
        const long long go = (extra ? 0 : (long long)it.g * p.b_stride);
        const long long so = (extra ? 0 : (long long)it.g * p.s_stride);
        const uint8_t *S0 = (extra ? xs0 : ws0) + so, *S1 = SWIGLU ? (extra ? xs1 : ws1) + so : S0;
        b_base[0] = (extra ? xb0 : wb0) + go;
        b_base[1] = SWIGLU ? (extra ? xb1 : wb1) + go : b_base[0];
#pragma unroll
        for (int q = 0; q < R::nB; ++q) {
            const int i = w + NW * q, row = 8 * (i & 7) + (ln >> 3);
            const int c = (ln & 7) ^ (2 * ((row >> 1) & 3));
            const int col = min(it.n0 + (SWIGLU ? 0 : 128 * (i >> 3)) + 16 * c, p.N - 16);
            b_off[q] = (uint32_t)row * (uint32_t)p.N + (uint32_t)col;
        }
#pragma unroll
        for (int q = 0; q < R::nS; ++q) {
            const int i = s_slot(q);
            if (i < R::BM / 64) {
                s_base[q] = reinterpret_cast<const uint8_t *>(p.As) + (long long)it.row0 * 4;
                s_off[q] = (64 * i + ln) * 4;
            } else {
                const int h = (i - R::BM / 64) >> 1, kg = 2 * ((i - R::BM / 64) & 1) + (ln >> 5);
                const int col = min(it.n0 + (SWIGLU ? 0 : 128 * h) + 4 * (ln & 31), p.N - 4);
                s_base[q] = h ? S1 : S0;
                s_off[q] = (uint32_t)kg * (uint32_t)p.N + (uint32_t)col;
            }
        }
    };
    // what the next copies are of: step c_kt of item c_item, c_left steps before the next item
    int c_item = 0, c_kt, c_left, c_step = 1;
    long long a_step = p.as_ld * 64, b_step = 64LL * p.N, s_step[R::nS];
#pragma unroll
    for (int q = 0; q < R::nS; ++q) s_step[q] = s_slot(q) < R::BM / 64 ? p.as_ld * 4 : 4LL * p.N;
    auto begin_item = [&]() {
        const ItemA4 it = item_at(c_item);
        c_kt = 0;
        c_left = nk;
        set_sources(it);
    };
    auto move = [&](long long by) {
        a_base += by * a_step;
        b_base[0] += by * b_step;
        b_base[1] += by * b_step;
#pragma unroll
        for (int q = 0; q < R::nS; ++q) s_base[q] += by * s_step[q];
        c_kt += (int)by * c_step;
    };
    // after an item's last step: the next item; past the last one its last step's
    // copies are repeated (into stages that nobody reads)
    auto next_item = [&]() {
        if (c_item + 1 < count) {
            ++c_item;
            begin_item();
        } else {
            move(-1);
            a_step = b_step = c_step = 0;
#pragma unroll
            for (int q = 0; q < R::nS; ++q) s_step[q] = 0;
            c_left = 0x7fffffff;
        }
    };
    auto copy = [&](int q, int stage) {
        uint8_t *st = ring + stage * R::stage;
        if (MOE_BOUNDS_FAIL(c_kt >= 0 && c_kt < nk, BOUNDS_TILE)) c_kt = nk - 1;
        const bool last = ragged && c_kt == nk - 1;
        if (q < R::nA) {
            copy16(a_base + (a_off + 1024u * (uint32_t)a_chunk(q)), st + a_chunk(q) * 1024);
        } else if (q < R::nA + R::nB) {
            const int i = w + NW * (q - R::nA);
            uint32_t o = b_off[q - R::nA];
            o -= last ? (uint32_t)max(8 * (i & 7) + (lane >> 3) - (k_rows - 1), 0) * (uint32_t)p.N : 0u;
            copy16(b_base[(NW * (q - R::nA)) >> 3] + o, st + R::a_bytes + i * 1024);
        } else {
            const int i = s_slot(q - R::nA - R::nB);
            uint32_t o = s_off[q - R::nA - R::nB];
            o -= last && i >= R::BM / 64
                     ? (uint32_t)max(2 * ((i - R::BM / 64) & 1) + (lane >> 5) - (k_groups - 1), 0) * (uint32_t)p.N
                     : 0u;
            copy4(s_base[q - R::nA - R::nB] + o, st + R::a_bytes + R::b_bytes + i * 256);
        }
    };
    // ---- operand reads of half kh (64 deep) of a stage, and of a stage's scales ----
    struct Frag {
        i32x4 a[MI], b[NJ];
        u32x2 raw[NJ][2];
    };
    const int i16 = lane & 15;
    // column block j of this wavefront: half-tile and column within it
    auto b_half = [&](int j) { return SWIGLU ? j / (NJ / 2) : (32 * (NJ * wc + j)) >> 7; };
    auto b_col = [&](int j) { return SWIGLU ? 32 * (NJ / 2 * wc + j % (NJ / 2)) : (32 * (NJ * wc + j)) & 127; };
    uint32_t tr_at[NJ];  // byte row 16 hb + i16 / 2 of the first half
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        const int c = (b_col(j) >> 4) + ((lane >> 4) & 1), row = 16 * hb + (i16 >> 1);
        tr_at[j] = R::a_bytes + b_half(j) * 8192 + row * 128 + 16 * (c ^ (2 * ((row >> 1) & 3))) + 8 * (i16 & 1);
    }
    const int a_row = wr * 32 * MI + l32;
    const int a_at = a_row * 64 + 16 * (hb ^ ((a_row >> 2) & 3));  // first half; the second: ^ 32
    const int sa_at = R::a_bytes + R::b_bytes + a_row * 4;
    // scales of the column blocks by one transposing read: its rows are (half,
    // block) pairs, so that a lane gets its column's bytes of all of them
    uint32_t sb_at;
    {
        const int r = (i16 >> 1) & (2 * NJ - 1), j = r % NJ, kh = r / NJ;
        sb_at = R::sb_at + b_half(j) * 512 + (2 * kh + hb) * 128 + b_col(j) + 16 * ((lane >> 4) & 1) + 8 * (i16 & 1);
    }
    u32x2 sb_raw, sb;        // read, in use: byte NJ kh + j
    int sa_raw[MI], sa[MI];  // byte 2 kh of the word in use
    constexpr int NRF = 2 * NJ + MI, NRS = MI + 1;  // reads of a half, and of a stage's scales
    auto read = [&](Frag &f, int r, int stage, auto kh_) {
        constexpr int kh = decltype(kh_)::value;
        const uint8_t *st = ring + stage * R::stage;
        if (r < 2 * NJ) {
            const int j = r >> 1;
            const uint32_t at = lds_addr(st) + tr_at[j];
            if (r & 1) f.raw[j][1] = ds_tr8_at<4096 * kh + 1024>(at);
            else f.raw[j][0] = ds_tr8_at<4096 * kh>(at);
        } else if (r < NRF) {
            f.a[r - 2 * NJ] = *reinterpret_cast<const i32x4 *>(st + (a_at ^ (32 * kh)) + 2048 * (r - 2 * NJ));
        } else if (r == NRF) {
            sb_raw = ds_tr8(lds_addr(st) + sb_at);
        } else {
            sa_raw[r - NRF - 1] = *reinterpret_cast<const int *>(st + sa_at + 128 * (r - NRF - 1));
        }
    };
    auto land = [&](Frag &f, bool scales) {
        wait_lds();
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            fence(f.raw[j][0]);
            fence(f.raw[j][1]);
            f.b[j] = i32x4{(int)f.raw[j][0][0], (int)f.raw[j][0][1], (int)f.raw[j][1][0], (int)f.raw[j][1][1]};
        }
        if (scales) {
            fence(sb_raw);
            sb = sb_raw;
#pragma unroll
            for (int m = 0; m < MI; ++m) sa[m] = sa_raw[m] >> (8 * hb);
        }
    };

    f32x16 acc[MI][NJ];
    auto clear = [&]() {
#pragma unroll
        for (int m = 0; m < MI; ++m)
#pragma unroll
            for (int j = 0; j < NJ; ++j)
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[m][j][i] = 0.0f;
    };
    clear();
    // the weights are the first operand: a lane's sixteen results are one row
    // (lane % 32 of its block) and columns 8 q + 4 (lane / 32) + 0..3, q < 4
    auto mma = [&](const Frag &f, int i, auto kh_) {
        constexpr int kh = decltype(kh_)::value;
        const int m = i / NJ, j = i % NJ;
        __builtin_amdgcn_sched_barrier(0);
        switch (2 * kh + j) {
        case 0: acc[m][j] = mfma4<0, 2 * kh>(f.b[j], f.a[m], acc[m][j], (int)sb[0], sa[m]); break;
        case 1: acc[m][j] = mfma4<1, 2 * kh>(f.b[j], f.a[m], acc[m][j], (int)sb[0], sa[m]); break;
        case 2: acc[m][j] = mfma4<2, 2 * kh>(f.b[j], f.a[m], acc[m][j], (int)sb[0], sa[m]); break;
        default: acc[m][j] = mfma4<3, 2 * kh>(f.b[j], f.a[m], acc[m][j], (int)sb[0], sa[m]); break;
        }
        __builtin_amdgcn_sched_barrier(0);
    };

    // ---- a finished tile. Every store is issued, so that the waits below can
    // count them: lanes without an output give an offset past the buffer's end,
    // which the store drops ----
    constexpr int kNowhere = 0x7ffffff0;
    auto rsrc = [](void *base, int bytes) {
        return __builtin_amdgcn_make_buffer_rsrc(base, 0, bytes, 0x00020000);
    };
    auto swap32 = [](uint32_t &x, uint32_t &y) {  // x's upper 32 lanes and y's lower ones change places
        const auto r = __builtin_amdgcn_permlane32_swap(x, y, false, false);
        x = r[0];
        y = r[1];
    };
    // h in MXFP4: a lane holds half of a row's 32 columns, lane ^ 32 the rest.
    // Of two row blocks the lower lanes store the first's rows, the upper ones
    // the second's: 16 bytes of codes and a scale byte a lane
    auto gate_up_out = [&](const ItemA4 &it) {
        int ln = lane;
        asm volatile("" : "+v"(ln));
        const long long at = (long long)(it.n0 >> 7) * p.cqs_ld + it.row0;
        const int rows = it.row_end - it.row0;
        const auto codes = rsrc(p.Cq + at * 64, rows * 64);
        const auto scales = rsrc(reinterpret_cast<uint8_t *>(p.Cqs) + at * 4, rows * 4);
#pragma unroll
        for (int j = 0; j < NJ / 2; ++j) {
            const int grp = NJ / 2 * wc + j;              // group of 32 of the tile's columns
            const bool pad = it.n0 + 32 * grp >= p.N;  // columns past the end: zero codes, scale 1
#pragma unroll
            for (int m = 0; m < MI; m += 2) {
                uint32_t code[2][2], byte[2];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    if (m + u >= MI) {
                        code[u][0] = code[0][0];
                        code[u][1] = code[0][1];
                        byte[u] = byte[0];
                        continue;
                    }
                    const f32x16 &g = acc[m + u][j], &x = acc[m + u][j + NJ / 2];
                    float v[16];
                    uint32_t t = 0;
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        v[i] = silu_f32(g[i]) * x[i];
                        t = max(t, mx4::mag_bits(v[i]));
                    }
                    uint32_t s = t;
                    swap32(t, s);
                    byte[u] = mx4::scale_byte(max(t, s));
                    code[u][0] = mx4::codes8(v, byte[u]);
                    code[u][1] = mx4::codes8(v + 8, byte[u]);
                    if (pad) {
                        code[u][0] = code[u][1] = 0;
                        byte[u] = 127;
                    }
                }
                u32x4 out;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t x = code[0][h], y = code[1][h];
                    swap32(x, y);
                    out[2 * h] = (x & 0xffffu) | y << 16;
                    out[2 * h + 1] = x >> 16 | (y & 0xffff0000u);
                }
                const bool up = ln >= 32;
                const int row = wr * 32 * MI + 32 * (up ? m + 1 : m) + (ln & 31);  // of the tile
                const bool in = row < rows && (!up || m + 1 < MI);
                __builtin_amdgcn_raw_buffer_store_b128(out, codes, in ? row * 64 + 16 * grp : kNowhere, 0, 0);
                __builtin_amdgcn_raw_buffer_store_b8((uint8_t)(up ? byte[1] : byte[0]), scales,
                                                     in ? row * 4 + grp : kNowhere, 0, 0);
            }
        }
    };
    // bf16 rows: a lane holds 4-column pieces of its row, lane ^ 32 the ones between.
    // Exchanges between the wavefront's halves and quarters leave 8 columns a lane
    // and the four lanes l, l + 16, .. with a row's 32: 64 bytes of 16 rows a store
    auto down_out = [&](const ItemA4 &it) {
        int ln = lane;
        asm volatile("" : "+v"(ln));
        const int rows = it.row_end - it.row0, ld = p.ldc;
        const auto C = rsrc(reinterpret_cast<uint16_t *>(p.C) + (long long)it.row0 * ld + it.n0, (rows * ld - it.n0) * 2);
        const int piece = 8 * ((ln >> 5) | ((ln >> 3) & 2));  // column of the lane's piece
#pragma unroll
        for (int m = 0; m < MI; ++m) {
            const int row = wr * 32 * MI + 32 * m + (ln & 15);  // of the tile
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                const f32x16 &x = acc[m][j];
                uint32_t v[2][4];  // columns 0..7 or 8..15 (upper lanes), and 16 more
#pragma unroll
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[h][e] = pack_bf16x2(x[8 * h + 2 * e], x[8 * h + 2 * e + 1]);
                    swap32(v[h][0], v[h][2]);
                    swap32(v[h][1], v[h][3]);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {  // rows 16..31's first pieces against rows 0..15's second
                    const auto r = __builtin_amdgcn_permlane16_swap(v[0][e], v[1][e], false, false);
                    v[0][e] = r[0];
                    v[1][e] = r[1];
                }
                const int col = 32 * (NJ * wc + j) + piece;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const bool in = row + 16 * h < rows && it.n0 + col < p.N;
                    __builtin_amdgcn_raw_buffer_store_b128(u32x4{v[h][0], v[h][1], v[h][2], v[h][3]}, C,
                                                           in ? ((row + 16 * h) * ld + col) * 2 : kNowhere, 0, 0);
                }
            }
        }
    };

    constexpr int ST = SWIGLU ? NJ * ((MI + 1) / 2) : 2 * NJ * MI;  // stores of a tile
    auto tile_out = [&](const ItemA4 &it) {
        if constexpr (SWIGLU) gate_up_out(it);
        else down_out(it);
    };

    // ---- fill the ring, then the steps of every item ----
    typedef std::integral_constant<int, 0> H0;
    typedef std::integral_constant<int, 1> H1;
    constexpr int NC = R::per_step;
    // A half step's products in order, with what is issued before each. Reads come
    // early, so that they have landed when the last products are issued; the copies
    // into a stage follow the barrier that frees it. PRE products stand before it
    constexpr int P = MI * NJ, PRE = P > 4 ? 2 : 1, PB = P - PRE;
    constexpr int RA = P > 4 ? P - 4 : 1, RB = PB > 4 ? PB - 4 : 1;
    auto upto = [](int i, int n, int slots) { return i >= slots ? n : i * n / slots; };
    begin_item();
#pragma unroll
    for (int t = 0; t < S; ++t) {
#pragma unroll
        for (int q = 0; q < NC; ++q) copy(q, t);
        move(1);
        if (--c_left == 0) next_item();
    }
    wait_vm<(S - 1) * NC>();
    __builtin_amdgcn_s_barrier();
    Frag f0, f1;
#pragma unroll
    for (int r = 0; r < NRF + NRS; ++r) read(f0, r, 0, H0{});
    land(f0, true);
    int stage = 0;
    // One step, without a branch: its products would sink past one, away from the
    // reads and copies that they hide
    auto step = [&](auto stores) {
        const int nstage = stage + 1 == S ? 0 : stage + 1;
#pragma unroll
        for (int i = 0; i < P; ++i) {
#pragma unroll
            for (int r = upto(i, NRF, RA); r < upto(i + 1, NRF, RA); ++r) read(f1, r, stage, H1{});
            mma(f0, i, H0{});
        }
        land(f1, false);  // the stage is read: its reads are done before anyone refills it
#pragma unroll
        for (int i = 0; i < PRE; ++i) mma(f1, i, H1{});
        wait_vm<(S - 2) * NC + decltype(stores)::value>();
        __builtin_amdgcn_s_barrier();
#pragma unroll
        for (int i = 0; i < PB; ++i) {
#pragma unroll
            for (int r = upto(i, NRF + NRS, RB); r < upto(i + 1, NRF + NRS, RB); ++r) read(f0, r, nstage, H0{});
#pragma unroll
            for (int q = upto(i, NC, PB); q < upto(i + 1, NC, PB); ++q) copy(q, stage);
            mma(f1, PRE + i, H1{});
        }
        move(1);
        land(f0, true);
        stage = nstage;
    };
    // Runs of steps up to the next event: the end of an item's copies, of its
    // products, or of the first steps after a stored tile, whose waits let its
    // stores (newer than the copies waited for) be under way
    ItemA4 it = item_at(0);
    int j = 0, left = nk, after = 0;
    for (;;) {
        int n = min(left, c_left);
        left -= n, c_left -= n;
        if (after > 0) {
            const int m = min(n, after);
            n -= m, after -= m;
            for (int i = 0; i < m; ++i) step(std::integral_constant<int, ST>{});
        }
        for (int i = 0; i < n; ++i) step(H0{});
        if (c_left == 0) next_item();
        if (left == 0) {
            const bool last = ++j == count;
            if (last) wait_vm<0>();  // the repeated copies land before the workgroup ends
            tile_out(it);
            if (last) break;
            after = S - 2;
            clear();
            it = item_at(j);
            left = nk;
        }
    }
}

template <bool SWIGLU, int MI>
__global__ __launch_bounds__(64 * NW, 1) void tiled_a4_kernel(GemmProblem p, int nN) {
    __shared__ __attribute__((aligned(1024))) uint8_t lds[RingA4<MI>::lds > RingA4<1>::lds ? RingA4<MI>::lds : RingA4<1>::lds];
    const int n_tiles = scalar(*p.n_tiles);
    const int n_work = n_tiles * nN;
    const int per = (n_work + kXcds - 1) / kXcds;
    const int xcd = blockIdx.x % kXcds, slots = gridDim.x / kXcds;
    const int mine = min(per, n_work - xcd * per);
    if (mine <= 0) return;
    const int first = xcd * per, slot = blockIdx.x / kXcds;
    // The items of the last round are cut into pieces of 64 rows where those are one round of
    // the XCD's workgroups. 8 experts, 8192 rows (4.5 tiles an expert), whole and cut: H 8192,
    // F 2048 330 and 319 us, H 2048, F 8192 288 and 271, H 1024, F 1024 48 and 46; with two
    // rounds of pieces (H 1024, F 4096) 96.5 and 98. 32 experts of 7168 x 2048, 6 to 592 rows:
    // gate/up 172 us with pieces counted as if tiles were full, 166 with those that have rows
    // (fastest calls of one run; other runs of the latter begin at 172).
    // (Equal parts over K, their sums joined through memory: as fast at K 14336, and nothing
    // below 12 steps a part.)
    int tail = MI > 1 && slots == kBlocksPerXcd ? scalar(mine % slots) : 0;
    Share cut{0, 0, 0};
    if (tail > 0) {
        const int lane = threadIdx.x & 63;
        int rows = MI * 64;  // a single round: as if all tiles were full, which needs no lookup
        if (mine > slots && lane < tail) {
            int g, r0, r1, nt;
            item_rows(p, nN, n_tiles, slots, first + mine - tail + lane, g, r0, r1, nt);
            rows = r1 - r0;
        }
        const int n = lane < tail ? (rows + 63) / 64 : 0;
        int end = n;  // pieces up to this item's last
#pragma unroll
        for (int x = 1; x < kBlocksPerXcd; x <<= 1) {
            const int y = __shfl_up(end, x);
            if (lane >= x) end += y;
        }
        const unsigned long long mine_is = __ballot(slot < end && slot >= end - n);
        if (scalar(__shfl(end, kBlocksPerXcd - 1)) > slots) {
            tail = 0;
        } else if (mine_is) {
            const int i = scalar(__ffsll((long long)mine_is) - 1);
            cut = Share{first + mine - tail + i, 1, scalar(slot - __shfl(end - n, i))};
        }
    }
    run_items<SWIGLU, MI>(p, nN, n_tiles, Share{first, mine - tail, -1}, lds);
    if (tail == 0) return;
    __syncthreads();
    run_items<SWIGLU, 1>(p, nN, n_tiles, cut, lds);
}

int column_tiles(int N, bool swiglu) { return (N + (swiglu ? 127 : 255)) / (swiglu ? 128 : 256); }
// Workgroups of an XCD: one round of resident ones, or as many as keep to the item table
long long slots_for(long long max_tiles, int nN) {
    const long long items = (max_tiles * nN + kXcds - 1) / kXcds;  // at most
    const long long rounds = (items + (long long)kA4Items * kBlocksPerXcd - 1) / (kA4Items * kBlocksPerXcd);
    return kBlocksPerXcd * (rounds > 1 ? rounds : 1);
}

template <bool SWIGLU, int MI>
hipError_t launch(const GemmProblem &p, hipStream_t s) {
    const int nN = column_tiles(p.N, SWIGLU);
    if (!tiled_a4_fits(p.max_tiles, p.N, SWIGLU)) return hipErrorInvalidValue;
    const long long slots = slots_for(p.max_tiles, nN);
    hipLaunchKernelGGL((tiled_a4_kernel<SWIGLU, MI>), dim3((unsigned)(slots * kXcds)), dim3(64 * NW), 0, s, p, nN);
    return hipGetLastError();
}

}  // namespace
}  // namespace tiled

// Tall tiles read the weights less often from LDS and L2, short ones multiply fewer
// rows that are not there. 32 experts of 7168 x 2048, the whole FFN in us, tiles of 64 /
// 128 / 192 / 256 rows: 24 rows an expert 180 / 189 / 218 / 231, 64: 254 / 201 / 232 / 232,
// 128: 313 / 265 / 241 / 254, 256: 481 / 375 / 369 / 336, 384: 579 / 488 / 458 / 442. Narrow
// experts (2048 x 1024) lean to shorter tiles, 64 rows an expert 42 / 41 / 44 / 48, 160:
// 57 / 56 / 51 / 55, 512: 144 / 123 / 106 / 116; with the rows unevenly spread 256 there
// again (116 against 123 for 192).
int tiled_a4_bm(long long rows, int groups) {
    const long long avg = rows / groups;
    return avg > 160 ? 256 : avg > 96 ? 192 : avg > 40 ? 128 : 64;
}

// fewer than 2^32 threads, and (then) tiles counted in ints
bool tiled_a4_fits(long long max_tiles, int N, bool swiglu) {
    using namespace tiled;
    return slots_for(max_tiles, column_tiles(N, swiglu)) * kXcds * (64 * NW) <= 0xffffffffLL;
}

hipError_t launch_tiled_a4(const GemmProblem &p, bool swiglu, int bm, hipStream_t s) {
    if (p.N < 32 || p.N % 32 || p.K < 32 || p.K % 32 || !p.tiles || !p.n_tiles || !p.A || !p.As || p.as_ld < p.M + 256LL ||
        !p.B0 || !p.S0 || (swiglu && (!p.B1 || !p.S1 || !p.Cq || !p.Cqs || p.cqs_ld < p.M)) || (!swiglu && !p.C))
        return hipErrorInvalidValue;
    if (p.extra_group >= 0 && (!p.Bx0 || !p.Sx0 || (swiglu && (!p.Bx1 || !p.Sx1)))) return hipErrorInvalidValue;
    if (p.max_tiles < 1) return hipSuccess;
    switch (bm) {
    case 256: return swiglu ? tiled::launch<true, 4>(p, s) : tiled::launch<false, 4>(p, s);
    case 192: return swiglu ? tiled::launch<true, 3>(p, s) : tiled::launch<false, 3>(p, s);
    case 128: return swiglu ? tiled::launch<true, 2>(p, s) : tiled::launch<false, 2>(p, s);
    case 64: return swiglu ? tiled::launch<true, 1>(p, s) : tiled::launch<false, 1>(p, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace moe
