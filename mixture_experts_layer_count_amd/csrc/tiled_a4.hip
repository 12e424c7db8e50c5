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
// Tile: BM rows x 256 B-columns x 128 deep; WR x 4 wavefronts, each BM / WR
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

template <int WR, int MI>
struct RingA4 {
    static constexpr int waves = 4 * WR;
    static constexpr int threads = 64 * waves;
    static constexpr int BM = 32 * MI * WR;
    static constexpr int a_bytes = BM * 64;
    static constexpr int b_bytes = 64 * 256;
    static constexpr int sa_bytes = BM * 4;
    static constexpr int sb_bytes = 4 * 256;
    static constexpr int sb_at = a_bytes + b_bytes + sa_bytes;
    static constexpr int stage = sb_at + sb_bytes;
    static constexpr int per_cu = WR == 1 ? 2 : 1;  // workgroups a CU
    static constexpr int budget = 160 * 1024 / per_cu - kA4Items * 16;
    static constexpr int S = budget / stage < 6 ? budget / stage : 6;
    static constexpr int a_chunks = a_bytes / 1024;  // 1 KB copies, 16 rows each
    static constexpr int nA = (a_chunks + waves - 1) / waves;
    static constexpr int nB = 16 / waves;            // 1 KB copies, 8 byte rows of a half each
    static constexpr int slots = BM / 64 + 4;        // 256-byte scale copies
    static constexpr int nS = (slots + waves - 1) / waves;
    static constexpr int per_step = nA + nB + nS;
    static constexpr int table = S * stage;
    static constexpr int lds = table + kA4Items * 16;
    static_assert(S >= 3 && BM % 64 == 0 && (S - 2) * per_step < 64, "ring");
};

struct ItemA4 {
    int g, row0, row_end, n0;
};

template <bool SWIGLU, int WR, int MI>
__global__ __launch_bounds__(256 * WR, WR == 1 ? 2 : 1) void tiled_a4_kernel(GemmProblem p, int nN) {
    typedef RingA4<WR, MI> R;
    constexpr int S = R::S, NW = R::waves;
    constexpr int W = SWIGLU ? 128 : 256;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[R::lds];
    int *table = reinterpret_cast<int *>(lds + R::table);

    const int tid = threadIdx.x;
    const int lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), wr = w / 4, wc = w % 4;
    const int l32 = lane & 31, hb = lane >> 5;
    const int nk = (p.K + kA4BK - 1) / kA4BK;

    // ---- this workgroup's items ----
    const int n_tiles = *p.n_tiles;
    const int n_work = n_tiles * nN;
    const int per = (n_work + kXcds - 1) / kXcds;
    const int xcd = blockIdx.x % kXcds, slot = blockIdx.x / kXcds, slots = gridDim.x / kXcds;
    const int mine = min(per, n_work - xcd * per);
    if (slot >= mine) return;
    const int count = (mine - slot + slots - 1) / slots;
    if (MOE_BOUNDS_FAIL(count <= kA4Items, BOUNDS_TILE)) return;
    if (w == 0 && lane < count) {
        int mt, nt;
        tile_of(p, nN, n_tiles, xcd * per + slot + slots * lane, mt, nt);
        const bool ok = mt < p.max_tiles;
        int g = ok ? p.tiles[4 * mt] : 0, r0 = ok ? p.tiles[4 * mt + 1] : 0, r1 = ok ? p.tiles[4 * mt + 2] : 0;
        if (MOE_BOUNDS_FAIL(ok && g >= 0 && g < p.n_groups && r0 >= 0 && r0 < r1 && r1 <= p.M, BOUNDS_TILE)) {
            g = 0;
            r0 = 0;
            r1 = 1;
        }
        *reinterpret_cast<i32x4 *>(table + 4 * lane) = i32x4{g, r0, r1, nt * W};
    }
    __syncthreads();
    auto item_at = [&](int j) {
        const i32x4 t = *reinterpret_cast<const i32x4 *>(table + 4 * j);
        ItemA4 it;
        it.g = __builtin_amdgcn_readfirstlane(t[0]);
        it.row0 = __builtin_amdgcn_readfirstlane(t[1]);
        it.row_end = __builtin_amdgcn_readfirstlane(t[2]);
        it.n0 = __builtin_amdgcn_readfirstlane(t[3]);
        return it;
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
    auto set_sources = [&](const ItemA4 &it) {
        int ln = lane;  // re-read: its multiples need not live through the K loop
        asm volatile("" : "+v"(ln));
        const bool extra = it.g == p.extra_group;
        a_base = reinterpret_cast<const uint8_t *>(p.A) + (long long)it.row0 * 64;
        const long long go = extra ? 0 : (long long)it.g * p.b_stride, so = extra ? 0 : (long long)it.g * p.s_stride;
        const uint8_t *B0 = reinterpret_cast<const uint8_t *>(extra ? p.Bx0 : p.B0) + go;
        const uint8_t *S0 = reinterpret_cast<const uint8_t *>(extra ? p.Sx0 : p.S0) + so;
        b_base[0] = B0;
        b_base[1] = SWIGLU ? reinterpret_cast<const uint8_t *>(extra ? p.Bx1 : p.B1) + go : B0;
        const uint8_t *S1 = SWIGLU ? reinterpret_cast<const uint8_t *>(extra ? p.Sx1 : p.S1) + so : S0;
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
    int c_item = 0, c_kt = 0;  // what the next copies are of
    auto copy = [&](int q, int stage) {
        uint8_t *st = lds + stage * R::stage;
        const bool last = ragged && c_kt == nk - 1;
        if (q < R::nA) {
            copy16(a_base + (a_off + 1024u * (uint32_t)a_chunk(q)), st + a_chunk(q) * 1024);
        } else if (q < R::nA + R::nB) {
            const int i = w + NW * (q - R::nA);
            uint32_t o = b_off[q - R::nA];
            if (last) o -= (uint32_t)max(8 * (i & 7) + (lane >> 3) - (k_rows - 1), 0) * (uint32_t)p.N;
            copy16(b_base[(NW * (q - R::nA)) >> 3] + o, st + R::a_bytes + i * 1024);
        } else {
            const int i = s_slot(q - R::nA - R::nB);
            uint32_t o = s_off[q - R::nA - R::nB];
            if (last && i >= R::BM / 64)
                o -= (uint32_t)max(2 * ((i - R::BM / 64) & 1) + (lane >> 5) - (k_groups - 1), 0) * (uint32_t)p.N;
            copy4(s_base[q - R::nA - R::nB] + o, st + R::a_bytes + R::b_bytes + i * 256);
        }
    };
    // on to the next step, or the next item; past the last item its last step's
    // copies are repeated (into stages that nobody reads)
    auto advance = [&]() {
        if (c_kt + 1 < nk) {
            ++c_kt;
            a_base += p.as_ld * 64;
            b_base[0] += 64LL * p.N;
            b_base[1] += 64LL * p.N;
#pragma unroll
            for (int q = 0; q < R::nS; ++q) s_base[q] += s_slot(q) < R::BM / 64 ? p.as_ld * 4 : 4LL * p.N;
        } else if (c_item + 1 < count) {
            ++c_item;
            c_kt = 0;
            set_sources(item_at(c_item));
        }
    };

    // ---- operand reads of half kh (64 deep) of a stage ----
    struct Frag {
        i32x4 a[MI], b[2];
        u32x2 raw[2][2];
        int sa[MI], sb[2];
    };
    const int i16 = lane & 15;
    uint32_t tr_at[2];  // column block j: byte row 16 hb + i16 / 2 of the first half
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int col = SWIGLU ? 32 * wc : 64 * (wc & 1) + 32 * j, half = SWIGLU ? j : wc >> 1;
        const int c = (col >> 4) + ((lane >> 4) & 1), row = 16 * hb + (i16 >> 1);
        tr_at[j] = R::a_bytes + half * 8192 + row * 128 + 16 * (c ^ (2 * ((row >> 1) & 3))) + 8 * (i16 & 1);
    }
    const int a_row = wr * 32 * MI + l32;
    const int a_at = a_row * 64 + 16 * (hb ^ ((a_row >> 2) & 3));  // first half; the second: ^ 32
    const int sa_at = R::a_bytes + R::b_bytes + a_row * 4 + hb;
    const int sb_at = R::sb_at + (SWIGLU ? 32 * wc : (wc >> 1) * 512 + 64 * (wc & 1)) + l32 + 128 * hb;
    constexpr int NR = 4 + 2 + 2 * MI;
    auto read = [&](Frag &f, int r, int stage, auto kh_) {
        constexpr int kh = decltype(kh_)::value;
        const uint8_t *st = lds + stage * R::stage;
        if (r < 4) {
            const int j = r >> 1;
            const uint32_t at = lds_addr(st) + tr_at[j];
            if (r & 1) f.raw[j][1] = ds_tr8_at<4096 * kh + 1024>(at);
            else f.raw[j][0] = ds_tr8_at<4096 * kh>(at);
        } else if (r < 4 + MI) {
            f.a[r - 4] = *reinterpret_cast<const i32x4 *>(st + (a_at ^ (32 * kh)) + 2048 * (r - 4));
        } else if (r < 6 + MI) {
            const int j = r - 4 - MI;
            f.sb[j] = st[sb_at + 256 * kh + (SWIGLU ? 512 : 32) * j];
        } else {
            f.sa[r - 6 - MI] = st[sa_at + 2 * kh + 128 * (r - 6 - MI)];
        }
    };
    auto land = [&](Frag &f) {
        wait_lds();
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            fence(f.raw[j][0]);
            fence(f.raw[j][1]);
            f.b[j] = i32x4{(int)f.raw[j][0][0], (int)f.raw[j][0][1], (int)f.raw[j][1][0], (int)f.raw[j][1][1]};
        }
    };

    f32x16 acc[MI][2];
    auto clear = [&]() {
#pragma unroll
        for (int m = 0; m < MI; ++m)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[m][j][i] = 0.0f;
    };
    clear();
    // the weights are the first operand: a lane's sixteen results are one row
    // (lane % 32 of its block) and columns 8 q + 4 (lane / 32) + 0..3, q < 4
    auto mma = [&](const Frag &f, int m) {
        __builtin_amdgcn_sched_barrier(0);
        const i32x4 a = f.a[m];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const i32x4 b = f.b[j];
            acc[m][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                i32x8{b[0], b[1], b[2], b[3], 0, 0, 0, 0}, i32x8{a[0], a[1], a[2], a[3], 0, 0, 0, 0}, acc[m][j], 4, 4,
                0, f.sb[j], 0, f.sa[m]);
        }
        __builtin_amdgcn_sched_barrier(0);
    };

    // ---- a finished tile ----
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
        const bool pad = it.n0 + 32 * wc >= p.N;  // columns past the end: zero codes, scale 1
        uint8_t *Hs = reinterpret_cast<uint8_t *>(p.Cqs);
        const long long at = (long long)(it.n0 >> 7) * p.cqs_ld;
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
                const f32x16 &g = acc[m + u][0], &x = acc[m + u][1];
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
            const int row = it.row0 + wr * 32 * MI + 32 * (up ? m + 1 : m) + (ln & 31);
            if (row < it.row_end && (!up || m + 1 < MI)) {
                *reinterpret_cast<u32x4 *>(p.Cq + (at + row) * 64 + 16 * wc) = out;
                Hs[(at + row) * 4 + wc] = (uint8_t)(up ? byte[1] : byte[0]);
            }
        }
    };
    // bf16 rows: of two 8-column pieces the lower lanes store the first, the
    // upper ones the second
    auto down_out = [&](const ItemA4 &it) {
        int ln = lane;
        asm volatile("" : "+v"(ln));
        uint16_t *C = reinterpret_cast<uint16_t *>(p.C);
#pragma unroll
        for (int m = 0; m < MI; ++m) {
            const int row = it.row0 + wr * 32 * MI + 32 * m + (ln & 31);
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int q = 0; q < 4; q += 2) {
                    const f32x16 &x = acc[m][j];
                    uint32_t a0 = pack_bf16x2(x[4 * q], x[4 * q + 1]), a1 = pack_bf16x2(x[4 * q + 2], x[4 * q + 3]);
                    uint32_t b0 = pack_bf16x2(x[4 * q + 4], x[4 * q + 5]),
                             b1 = pack_bf16x2(x[4 * q + 6], x[4 * q + 7]);
                    swap32(a0, b0);
                    swap32(a1, b1);
                    const int col = it.n0 + 64 * wc + 32 * j + 8 * (q + (ln >> 5));
                    if (row < it.row_end && col < p.N)
                        *reinterpret_cast<u32x4 *>(C + (long long)row * p.ldc + col) = u32x4{a0, a1, b0, b1};
                }
        }
    };

    // ---- fill the ring, then the steps of every item ----
    typedef std::integral_constant<int, 0> H0;
    typedef std::integral_constant<int, 1> H1;
    constexpr int NC = R::per_step;
    set_sources(item_at(0));
#pragma unroll
    for (int t = 0; t < S; ++t) {
#pragma unroll
        for (int q = 0; q < NC; ++q) copy(q, t);
        advance();
    }
    wait_vm<(S - 1) * NC>();
    __builtin_amdgcn_s_barrier();
    Frag f0, f1;
#pragma unroll
    for (int r = 0; r < NR; ++r) read(f0, r, 0, H0{});
    land(f0);
    constexpr int PRE = MI > 1 ? 1 : 0, SL = MI - PRE;  // row blocks multiplied before the barrier
    int stage = 0;
    for (int j = 0; j < count; ++j) {
        for (int kt = 0; kt < nk; ++kt) {
            const int nstage = stage + 1 == S ? 0 : stage + 1;
#pragma unroll
            for (int m = 0; m < MI; ++m) {
#pragma unroll
                for (int r = m * NR / MI; r < (m + 1) * NR / MI; ++r) read(f1, r, stage, H1{});
                mma(f0, m);
            }
            land(f1);  // the stage is read: its reads are done before anyone refills it
#pragma unroll
            for (int m = 0; m < PRE; ++m) mma(f1, m);
            wait_vm<(S - 2) * NC>();
            __builtin_amdgcn_s_barrier();
#pragma unroll
            for (int c = 0; c < SL; ++c) {
#pragma unroll
                for (int r = c * NR / SL; r < (c + 1) * NR / SL; ++r) read(f0, r, nstage, H0{});
#pragma unroll
                for (int q = c * NC / SL; q < (c + 1) * NC / SL; ++q) copy(q, stage);
                mma(f1, c + PRE);
            }
            advance();
            land(f0);
            stage = nstage;
        }
        const ItemA4 it = item_at(j);
        if constexpr (SWIGLU) gate_up_out(it);
        else down_out(it);
        clear();
    }
    wait_vm<0>();  // the repeated copies land before the workgroup ends
}

template <bool SWIGLU, int WR, int MI>
hipError_t launch(const GemmProblem &p, hipStream_t s) {
    typedef RingA4<WR, MI> R;
    const int nN = (p.N + (SWIGLU ? 127 : 255)) / (SWIGLU ? 128 : 256);
    const long long items = ((long long)p.max_tiles * nN + kXcds - 1) / kXcds;  // of an XCD, at most
    if (items > 0x0fffffffLL) return hipErrorInvalidValue;
    // one round of resident workgroups, or as many as keep to the item table
    long long slots = kBlocksPerXcd * R::per_cu;
    while ((items + slots - 1) / slots > kA4Items) slots += kBlocksPerXcd * R::per_cu;
    if (slots > items) slots = items;
    hipLaunchKernelGGL((tiled_a4_kernel<SWIGLU, WR, MI>), dim3((unsigned)(slots * kXcds)), dim3(R::threads), 0, s, p, nN);
    return hipGetLastError();
}

}  // namespace
}  // namespace tiled

int tiled_a4_bm(long long rows, int groups) {
    const long long avg = rows / groups;
    return avg > 160 ? 256 : avg > 96 ? 192 : avg > 40 ? 128 : 64;
}

hipError_t launch_tiled_a4(const GemmProblem &p, bool swiglu, int bm, hipStream_t s) {
    if (p.N < 32 || p.N % 32 || p.K < 32 || p.K % 32 || !p.tiles || !p.n_tiles || !p.A || !p.As || p.as_ld < p.M + 256LL ||
        !p.B0 || !p.S0 || (swiglu && (!p.B1 || !p.S1 || !p.Cq || !p.Cqs || p.cqs_ld < p.M)) || (!swiglu && !p.C))
        return hipErrorInvalidValue;
    if (p.extra_group >= 0 && (!p.Bx0 || !p.Sx0 || (swiglu && (!p.Bx1 || !p.Sx1)))) return hipErrorInvalidValue;
    if (p.max_tiles < 1) return hipSuccess;
    switch (bm) {
    case 256: return swiglu ? tiled::launch<true, 2, 4>(p, s) : tiled::launch<false, 2, 4>(p, s);
    case 192: return swiglu ? tiled::launch<true, 2, 3>(p, s) : tiled::launch<false, 2, 3>(p, s);
    case 128: return swiglu ? tiled::launch<true, 2, 2>(p, s) : tiled::launch<false, 2, 2>(p, s);
    case 64: return swiglu ? tiled::launch<true, 2, 1>(p, s) : tiled::launch<false, 2, 1>(p, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace moe
