// build-flags: -mllvm -amdgpu-mfma-vgpr-form
// Weight gradients of the grouped FFN: for every expert g,
//   dW_g[m][n] = sum over its rows r of A(r)[m] B(r)[n]
// in one launch: dW1 and dW3 (A = the token rows read back from their
// checkpoint, B = [dg | du]), then dW2 (A = w h, B = dY), the token operand
// gathered by row. The sum runs over rows, so both operands are contiguous
// across it: LDS tiles keep the matrices' [row][column] layout and both MFMA
// operands are read with ds_read_b64_tr_b16.
//
// A work item is one 256 x 256 tile of one expert's output; its K loop is that
// expert's rows, 32 a step (rows past the end read zeros, so NaN or infinite
// rows of another expert never enter; an expert without rows is one step of
// zeros). 8 wavefronts in 2 x 4 (128 x 64 each), a ring of S = 4 stages.
//
// Persistent: one workgroup per CU walks its items with one copy ring that
// never drains. Three positions move along the same sequence of (item, step):
// the multiplied step; the copied one, S steps ahead, already in the next
// item while the last steps of this one are multiplied; and, for the gathered
// operand, a window of 16 steps whose row numbers are copied to LDS (each
// wavefront its own rows) one window ahead of the copies. Finished tiles are
// stored from the registers while the next item's copies are in flight. (One
// workgroup per item took 7 us of each 23 us, 16-step item for finding its
// rows, filling the ring and storing.) dW2's items follow in the same launch:
// its own launch took 33 us of 117 (8 experts, T 1536, k 2, H 640, F 416).
//
// Measured, all three gradients in bf16 (medians): 128 experts, 65536 rows,
// H 2048, F 768: 801 us (772 TFLOP/s; at best 746); 8 experts, 8192 rows, H 4096,
// F 14336: 2765 us (1044 TFLOP/s; 0.52 of the matrix cores' cycles at 2.0 of 2.4
// GHz, the power limit's clock); 32 experts, 4096 rows, H 7168, F 2048: 775 us,
// 3.4 GB of memory traffic at 4.4 TB/s. A step takes 0.97 to 1.2 us, a tile's
// stores 2.4. In fp32: 945, 3280 and 1217 us. Added to what C holds: in bf16
// 1054, 3569 and 1700, in fp32 1406, 4320 and 2513: each 16-row block waits for
// its values of C, and the copy ring for the tile's stores.
//
// Work order: experts by falling row count, an expert's tiles in bands of
// kBand tile rows, column by column; consecutive runs of 32 tiles (one per CU)
// go to the XCDs in turn, forth and back. So a run reads about 4 panels of A
// and 8 of B through its XCD's L2 (tile rows one by one read 33: 5 % slower),
// and workgroups differ by at most about one item's work whatever the
// experts' row counts.
#include <type_traits>

#include "train_kernel.h"

namespace moe {

MOE_BOUNDS_FILE(train_weights)

namespace tiled {
namespace {

constexpr int kBand = 4;         // tile rows per band of the work order
constexpr int kMaxGroups = 1024;
constexpr uint32_t kNoRow = gather_max_bytes;  // a column's offset added, it stays below 2^32

struct WRing {
    static constexpr int tile = 32 * 512;  // one operand: 32 rows of 256 bf16
    static constexpr int stage = 2 * tile;
    static constexpr int S = 4;
    static constexpr int nC = 4;           // copies per wavefront and step (2 of each operand)
    static constexpr int MI = 8, NB = 4;
    static constexpr int window = 16;      // steps per window of row numbers (4 rows a wavefront and step)
    static constexpr int rows = S * stage, rows_bytes = 4 * 4 * window;
    // experts by falling row count: index (uint16), first row and end (int)
    static constexpr int order = rows + 8 * 2 * rows_bytes;
    static constexpr int range = order + 2 * kMaxGroups;
    static constexpr int lds = range + 8 * kMaxGroups;
    static_assert(lds <= 160 * 1024 && rows_bytes == 256 && 4 * kMaxGroups <= S * stage, "LDS");
};

// n / d for 0 <= n < 2^31 as (n mul) >> shift, exact: with shift = 31 +
// ceil(log2 d) and mul = ceil(2^shift / d), n (mul d - 2^shift) < 2^shift
struct Divisor {
    uint32_t mul;
    int shift;
    Divisor(int d) : shift(31) {
        while ((1LL << (shift - 31)) < d) ++shift;
        mul = (uint32_t)(((1ULL << shift) + d - 1) / d);
    }
    __device__ __forceinline__ uint32_t operator()(uint32_t n) const { return (uint32_t)(((uint64_t)n * mul) >> shift); }
};

// which operand's rows are gathered
enum Gather { GATHER_NONE, GATHER_A, GATHER_B };

// one work item (all uniform)
struct WItem {
    int lo, hi;       // its expert's rows
    int m0, n0;       // first row and column of the tile
    int half, g;      // output matrix, expert
    __device__ __forceinline__ int steps() const { return hi > lo ? (hi - lo + 31) >> 5 : 1; }
};

// one product and its tile counts; its runs follow those of the one before it
struct WWork {
    WeightsProblem p;
    int nM, nN, items, first_run;
    Divisor group_tiles, band_tiles;
};
struct WPair {
    WWork w[2];
    Divisor gk;
};

// ---- experts by falling row count (equal counts by index), to LDS ----
__device__ __forceinline__ void sort_experts(const WeightsProblem &p, uint8_t *lds) {
    uint16_t *order = reinterpret_cast<uint16_t *>(lds + WRing::order);
    int *range = reinterpret_cast<int *>(lds + WRing::range);
    const int tid = threadIdx.x;
    int *count = reinterpret_cast<int *>(lds);
    int lo[kMaxGroups / 512], hi[kMaxGroups / 512];
#pragma unroll
    for (int i = 0; i < kMaxGroups / 512; ++i) {
        const int g = tid + 512 * i;
        if (g < p.G) {
            lo[i] = min(max(p.offsets[g], 0), p.M);
            hi[i] = min(max(p.offsets[g + 1], lo[i]), p.M);
            count[g] = hi[i] - lo[i];
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kMaxGroups / 512; ++i) {
        const int g = tid + 512 * i;
        if (g < p.G) {
            const int mine = hi[i] - lo[i];
            int rank = 0;
            for (int o = 0; o < p.G; ++o) {
                const int c = count[o];
                rank += (c > mine) | ((c == mine) & (o < g));
            }
            order[rank] = (uint16_t)g;
            range[2 * rank] = lo[i];
            range[2 * rank + 1] = hi[i];
        }
    }
    __syncthreads();
}

template <bool F32, bool ACC, Gather GATHER>
__device__ __forceinline__ void weights_gemm(const WWork &work, const Divisor &gk, uint8_t *lds) {
    typedef WRing R;
    constexpr int S = R::S, MI = R::MI, NB = R::NB, NC = R::nC, NR = 2 * (MI + NB);
    constexpr int kStores = F32 ? MI * NB : MI * NB / 2;  // a finished tile's, per wavefront
    const WeightsProblem &p = work.p;
    const uint16_t *order = reinterpret_cast<const uint16_t *>(lds + R::order);
    const int *range = reinterpret_cast<const int *>(lds + R::range);

    const int tid = threadIdx.x;
    const int lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), wr = w / 4, wc = w % 4;
    const int i16 = lane & 15, gq = lane >> 4;

    // ---- this workgroup's items: number `slot` of every run that its XCD takes ----
    const int nM = work.nM, nN = work.nN, nT = nN * (p.C1 ? 2 : 1), per_group = nM * nT, items = work.items;
    const int xcd = blockIdx.x % kXcds, slot = blockIdx.x / kXcds;
    auto run_of = [&](int j) { return j * kXcds + ((j & 1) ? kXcds - 1 - xcd : xcd) - work.first_run; };
    const int j0 = work.first_run / kXcds + (run_of(work.first_run / kXcds) < 0);  // its first of this product
    auto item_id = [&](int j) { return (long long)run_of(j0 + j) * kBlocksPerXcd + slot; };
    if (item_id(0) >= items) return;
    // 64 items from `base` on, one a lane (read back lane by lane: through LDS
    // and scalar divisions each change of items took 0.8 us); past the last one
    // items without rows (copied, never multiplied)
    int base = 0, l_lo, l_hi, l_tile, l_g;
    auto load_items = [&]() {
        l_lo = l_hi = l_tile = l_g = 0;
        const long long id = item_id(base + lane);
        if (id < items) {
            const int e = (int)work.group_tiles((uint32_t)id), t = (int)id - e * per_group;
            const int band = (int)work.band_tiles(t), in = t - band * kBand * nT, deep = min(kBand, nM - kBand * band);
            static_assert(kBand == 4, "in / deep");
            const int n = deep == 4 ? in >> 2 : deep == 3 ? (int)(((uint64_t)in * 0xaaaaaaabu) >> 33) : in >> (deep - 1);
            l_g = order[e];
            l_lo = range[2 * e];
            l_hi = range[2 * e + 1];
            l_tile = (kBand * band + in - n * deep) << 16 | n;
        }
    };
    auto item_at = [&](int j) {
        WItem it;
        it.lo = __builtin_amdgcn_readlane(l_lo, j - base);
        it.hi = __builtin_amdgcn_readlane(l_hi, j - base);
        it.g = __builtin_amdgcn_readlane(l_g, j - base);
        const uint32_t tile = __builtin_amdgcn_readlane(l_tile, j - base);
        const int n = tile & 0xffff;
        it.half = n >= nN ? 1 : 0;
        it.m0 = 256 * (int)(tile >> 16);
        it.n0 = 256 * (n - it.half * nN);
        return it;
    };
    load_items();
    int mj = 0;  // number of the multiplied item

    // ---- the copied position: copy q of an operand and wavefront w fills rows
    // 4 w + 2 q + lane / 32 of the step, the lane's 16-byte chunk being the one
    // the swizzle puts there. Buffer loads, whose range check gives zeros for
    // rows past the expert's end: an operand in row order has a descriptor that
    // starts at the step's first row and ends with the expert's last, so its
    // copies need no address arithmetic but the scalar descriptor's; the
    // gathered one has a descriptor of the whole matrix, and rows past the end
    // get the offset kNoRow, past any range ----
    WItem ci = item_at(0), cn = item_at(1);  // the item being copied, and the one after it
    int cj = 0, ck = 0, cnk = ci.steps();
    const uint32_t lda2 = 2u * p.lda, ldb2 = 2u * p.ldb;
    uint32_t a_off[2], b_off[2];  // the lane's byte offset within the step (gathered: within its row)
    const char *a_ptr, *b_ptr;    // the step's first row at the tile's first column (gathered: row 0)
    uint32_t a_bytes, b_bytes;    // from there to the end of the step's rows (gathered: of the matrix)
    // the scalar unit's descriptors: the rows left in the step, as a scalar
    auto set_bytes = [&]() {
        const uint32_t n = __builtin_amdgcn_readfirstlane(min(max(ci.hi - ci.lo - 32 * ck, 0), 32));
        if (GATHER != GATHER_A) a_bytes = n * lda2;
        if (GATHER != GATHER_B) b_bytes = n * ldb2;
    };
    auto set_item = [&]() {
        // the lane, re-read so that this rare path's offsets do not stay live
        int ln = lane;
        asm volatile("" : "+v"(ln));
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int k = 4 * w + 2 * q + (ln >> 5), c = 8 * ((ln & 31) ^ bswz16(k));
            // columns past the matrix read its last ones (never stored)
            a_off[q] = 2 * min(c, p.MD - 8 - ci.m0) + (GATHER == GATHER_A ? 0 : k * lda2);
            b_off[q] = 2 * min(c, p.ND - 8 - ci.n0) + (GATHER == GATHER_B ? 0 : k * ldb2);
        }
        a_ptr = reinterpret_cast<const char *>(p.A + ci.m0) + (GATHER == GATHER_A ? 0LL : (long long)ci.lo * lda2);
        b_ptr = reinterpret_cast<const char *>(p.B + (long long)ci.half * p.ND + ci.n0) +
                (GATHER == GATHER_B ? 0LL : (long long)ci.lo * ldb2);
        if (GATHER == GATHER_A) a_bytes = (uint32_t)p.src_rows * lda2 - 2u * ci.m0;
        if (GATHER == GATHER_B) b_bytes = (uint32_t)p.src_rows * ldb2 - 2u * ci.n0;
    };
    // the gathered operand's rows: byte offsets of the current window's rows
    // (16 steps x the wavefront's 4), one a lane; the next window's row numbers
    // are on their way to LDS. newer: vector-memory operations since they were
    // sent for
    const int32_t *src = GATHER == GATHER_A ? p.a_src : p.b_src;
    int buf = 0, newer = 0;
    uint8_t *my_rows = lds + R::rows + w * 2 * R::rows_bytes;
    auto fetch_rows = [&](const WItem &it, int k, int b) {
        if (GATHER == GATHER_NONE || it.hi == it.lo) return;
        const int r = it.lo + 32 * (k + (lane >> 2)) + 4 * w + (lane & 3);
        copy4(src + min(r, it.hi - 1), my_rows + b * R::rows_bytes);
    };
    uint32_t l_row = kNoRow;
    auto take_rows = [&]() {
        if (GATHER == GATHER_NONE) return;
        uint32_t got = *(reinterpret_cast<const uint32_t *>(my_rows + buf * R::rows_bytes) + lane);
        const int r = ci.lo + 32 * ((ck & -R::window) + (lane >> 2)) + 4 * w + (lane & 3);
        if (r < ci.hi && MOE_BOUNDS_FAIL(got < (uint32_t)p.src_rows * p.gk, BOUNDS_A_ROW)) got = 0;
        l_row = r < ci.hi ? gk(got) * (GATHER == GATHER_A ? lda2 : ldb2) : kNoRow;
    };
    uint32_t row_off[2] = {0, 0};  // of the gathered operand's two copies of the step
    auto step_rows = [&]() {
        if (GATHER == GATHER_NONE) return;
        const int first = 4 * (ck & (R::window - 1));
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const uint32_t lo = __builtin_amdgcn_readlane(l_row, first + 2 * q);
            const uint32_t hi = __builtin_amdgcn_readlane(l_row, first + 2 * q + 1);
            row_off[q] = lane < 32 ? lo : hi;
        }
    };
    // to the next step: at a window's end the next window becomes current and
    // the one after it is sent for
    auto advance = [&]() {
        ++ck;
        newer += NC;
        a_ptr += GATHER == GATHER_A ? 0 : 32 * lda2;
        b_ptr += GATHER == GATHER_B ? 0 : 32 * ldb2;
        const bool next_item = ck == cnk;
        if (next_item || (ck & (R::window - 1)) == 0) {
            if (GATHER != GATHER_NONE) {
                // the window has landed when no more than `newer` operations
                // are outstanding: the S - 1 steps in flight, and a finished
                // tile's stores where they are among them (waiting for those
                // took 1 us of each 4-step item)
                if (newer >= (S - 1) * NC + kStores) wait_vm<(S - 1) * NC + kStores>();
                else if (newer >= (S - 1) * NC) wait_vm<(S - 1) * NC>();
                else wait_vm<0>();
            }
            newer = 0;
            buf ^= 1;
            if (next_item) {
                ci = cn;
                ++cj;
                ck = 0;
                cnk = ci.steps();
                if (cj + 1 - base >= 64) {
                    base = mj;  // at most S + 1 items behind
                    load_items();
                }
                cn = item_at(cj + 1);
                set_item();
            }
            take_rows();
            if (ck + R::window < cnk) fetch_rows(ci, ck + R::window, buf ^ 1);
            else fetch_rows(cn, 0, buf ^ 1);
        }
        set_bytes();
        step_rows();
    };
    auto copy = [&](int q, int stage) {
        const bool is_a = q < 2;
        uint32_t off = (is_a ? a_off : b_off)[q & 1];
        if (GATHER == (is_a ? GATHER_A : GATHER_B)) off += row_off[q & 1];
        copy16_buffer(is_a ? a_ptr : b_ptr, is_a ? a_bytes : b_bytes, off,
                      lds + stage * R::stage + (is_a ? 0 : R::tile) + (2 * w + (q & 1)) * 1024);
    };

    // ---- fragment reads: r = 2 block + half; blocks 0..MI-1 of A, then B.
    // The lane's K rows are 8 gq + 4 half + i16 / 4, whose chunk swizzle does
    // not depend on the half; column block b moves the chunk index by 2 b in
    // bits that the other terms leave to the swizzle's XOR, so its address is
    // the lane's first address XOR 32 b ----
    struct Frag {
        bf16x8 a[MI], b[NB];
        u32x2 raw[MI + NB][2];
    };
    const int k0 = 8 * gq + (i16 >> 2), b0 = (i16 & 3) >> 1;
    const uint32_t a_base = k0 * 512 + 16 * ((16 * wr + b0) ^ bswz16(k0)) + 8 * (i16 & 1);
    const uint32_t b_base = R::tile + k0 * 512 + 16 * ((8 * wc + b0) ^ bswz16(k0)) + 8 * (i16 & 1);
    auto read = [&](Frag &f, int r, int stage) {
        const int blk = r >> 1;
        const uint32_t st = lds_addr(lds + stage * R::stage);
        const uint32_t addr = (st + (blk < MI ? a_base : b_base)) ^ (32 * (blk < MI ? blk : blk - MI));
        if (r & 1) f.raw[blk][1] = ds_tr16_at<2048>(addr);
        else f.raw[blk][0] = ds_tr16_at<0>(addr);
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
    // FIRST: an item's first step, whose sums begin at zero
    auto mma_rows = [&](auto first, const Frag &f, int m) {
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < NB; ++j)
            acc[m][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f.b[j], f.a[m], decltype(first)::value ? f32x4{} : acc[m][j],
                                                                0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
    };

    // ---- a finished tile, straight from the accumulators: 16-byte pieces of
    // whole 128-byte lines after two exchanges between lanes (through LDS the
    // epilogue took as long). VALU-bound, so the addresses are left to the
    // scalar unit: a lane's offset holds for the whole tile, the rows move the
    // descriptor. MD and ND are multiples of 32: a block of 16 rows
    // is inside the matrix or outside (a descriptor of length 0), a lane's
    // columns likewise (an offset past the range), and the hardware drops
    // those stores, so every wavefront issues exactly kStores of them ----
    constexpr int kOut = 0x7fffffff;
    auto tile_out = [&](const WItem &it) {
        constexpr int size = F32 ? 4 : 2, NP = F32 ? NB / 2 : 1;  // NP: 128-byte pieces of a wavefront's row
        const long long first = (((long long)it.g * p.MD + it.m0 + 128 * wr) * p.ND + it.n0 + 64 * wc) * size;
        const char *held = reinterpret_cast<const char *>(it.half ? p.C1 : p.C0) + first;
        // uniform, which the compiler does not see (it would loop over the lanes)
        const uint64_t at = reinterpret_cast<uint64_t>(held);
        char *C = reinterpret_cast<char *>((uint64_t)__builtin_amdgcn_readfirstlane((uint32_t)(at >> 32)) << 32 |
                                           (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)at));
        // re-read here, so that the offsets are not kept through the K loop
        int ln = lane;
        asm volatile("" : "+v"(ln));
        const int l16 = ln & 15, lq = ln >> 4;
        const int rows = p.MD - it.m0 - 128 * wr, cols = p.ND - it.n0 - 64 * wc;
        int off[NP];
#pragma unroll
        for (int q = 0; q < NP; ++q) {
            const int col = 32 * q + (F32 ? 16 * (l16 >> 3) + 4 * lq : 32 * (l16 >> 3) + pair_column(lq));
            off[q] = ((l16 & 7) * p.ND + col) * size;
            asm volatile("" : "+v"(off[q]));  // formed first: the choice is then no branch
            off[q] = col < cols ? off[q] : kOut;
        }
#pragma unroll
        for (int m = 0; m < MI; ++m) {
            __builtin_amdgcn_sched_barrier(0);
            // rows 16 m .. + 7, and the 8 after them. (Not by the stores' scalar
            // offset: with one, a store of 16 bytes read a data register that
            // the next instruction had already overwritten)
            const int len = 16 * m < rows ? kOut : 0;
            const __amdgpu_buffer_rsrc_t lines[2] = {
                __builtin_amdgcn_make_buffer_rsrc(C + 16LL * m * p.ND * size, 0, len, kBufferWord3),
                __builtin_amdgcn_make_buffer_rsrc(C + (16LL * m + 8) * p.ND * size, 0, len, kBufferWord3)};
            f32x4 v[NB];
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                v[j] = acc[m][j];
                if (!ACC) continue;
                // what C holds, in the accumulators' layout
                const int row = 16 * m + l16, c = 16 * j + 4 * lq;
                if (row < rows && c < cols) {
                    const char *old = held + (row * p.ND + c) * size;
                    if constexpr (F32) {
                        v[j] += *reinterpret_cast<const f32x4 *>(old);
                    } else {
                        const u32x2 o = *reinterpret_cast<const u32x2 *>(old);
                        v[j] += f32x4{bf16_lo(o[0]), bf16_hi(o[0]), bf16_lo(o[1]), bf16_hi(o[1])};
                    }
                }
            }
#pragma unroll
            for (int q = 0; q < NP; ++q) {
                u32x4 x0, x1;
                if constexpr (F32) {
                    x0 = __builtin_bit_cast(u32x4, v[2 * q]);
                    x1 = __builtin_bit_cast(u32x4, v[2 * q + 1]);
                } else {
                    x0 = pair_columns(v[0], v[1]);
                    x1 = pair_columns(v[2], v[3]);
                }
                whole_lines(x0, x1);
                __builtin_amdgcn_raw_buffer_store_b128(x0, lines[0], off[q], 0, 0);
                __builtin_amdgcn_raw_buffer_store_b128(x1, lines[1], off[q], 0, 0);
            }
        }
    };

    // ---- fill the ring ----
    Frag fa, fb;
    set_item();
    fetch_rows(ci, 0, 0);
    if (R::window < cnk) fetch_rows(ci, R::window, 1);
    else fetch_rows(cn, 0, 1);
    if (GATHER != GATHER_NONE) wait_vm<0>();
    take_rows();
    set_bytes();
    step_rows();
#pragma unroll 1
    for (int s = 0; s < S; ++s) {
#pragma unroll
        for (int q = 0; q < NC; ++q) copy(q, s);
        advance();
    }
    wait_vm<(S - 1) * NC>();
    __builtin_amdgcn_s_barrier();
#pragma unroll
    for (int r = 0; r < NR; ++r) read(fa, r, 0);
    land(fa);

    // ---- the multiplied position ----
    WItem mi = item_at(0), mn = item_at(1);
    int left = mi.steps(), stage = 0;
    int relax = 0;  // steps whose awaited copies are older than a finished tile's stores
    auto step = [&](auto first, Frag &cur, Frag &nxt) {
        const int nstage = stage + 1 == S ? 0 : stage + 1;
        mma_rows(first, cur, 0);
        mma_rows(first, cur, 1);
        // the next step's copies have landed when no more than the S - 2 newer
        // steps' (and, for S - 1 steps after a tile, its stores) are outstanding
        if (relax > 0) {
            --relax;
            wait_vm<(S - 2) * NC + kStores>();
        } else {
            wait_vm<(S - 2) * NC>();
        }
        __builtin_amdgcn_s_barrier();
        // copies and reads spread between the MFMA groups; the next copies'
        // descriptors and row offsets formed before the last group
        constexpr int SLOTS = MI - 2;
#pragma unroll
        for (int c = 0; c < SLOTS; ++c) {
#pragma unroll
            for (int q = c * (NC + 1) / SLOTS; q < (c + 1) * (NC + 1) / SLOTS && q < NC; ++q) copy(q, stage);
#pragma unroll
            for (int r = c * NR / SLOTS; r < (c + 1) * NR / SLOTS; ++r) read(nxt, r, nstage);
            if (c == SLOTS - 1) advance();
            mma_rows(first, cur, c + 2);
        }
        land(nxt);
        stage = nstage;
    };
    for (;;) {
        step(std::true_type{}, fa, fb);
        int k = left - 1;
        for (; k > 1; k -= 2) {
            step(std::false_type{}, fb, fa);
            step(std::false_type{}, fa, fb);
        }
        if (k > 0) {
            step(std::false_type{}, fb, fa);
        } else {
            // once per item: the fragment sets change roles by a copy
#pragma unroll
            for (int m = 0; m < MI; ++m) fa.a[m] = fb.a[m];
#pragma unroll
            for (int j = 0; j < NB; ++j) fa.b[j] = fb.b[j];
        }
        if (!ACC || mi.lo < mi.hi) {
            tile_out(mi);
            newer += kStores;
            relax = ACC ? 0 : S - 1;
        }
        ++mj;
        if (item_id(mj) >= items) break;
        mi = mn;
        left = mi.steps();
        mn = item_at(mj + 1);
    }
    wait_vm<0>();  // the copies past the last item land before the ring is used again or the workgroup ends
}

template <bool F32, bool ACC, bool GATHERED>
__global__ __launch_bounds__(512, 1) void weights_gemm_kernel(WPair q) {
    __shared__ __attribute__((aligned(1024))) uint8_t lds[WRing::lds];
    sort_experts(q.w[0].p, lds);
    weights_gemm<F32, ACC, GATHERED ? GATHER_A : GATHER_NONE>(q.w[0], q.gk, lds);
    __syncthreads();
    weights_gemm<F32, ACC, GATHERED ? GATHER_B : GATHER_NONE>(q.w[1], q.gk, lds);
}

}  // namespace
}  // namespace tiled

hipError_t launch_weights_gemm(const WeightsProblem &w13, const WeightsProblem &w2, hipStream_t s) {
    using namespace tiled;
    WPair q{{{w13, 0, 0, 0, 0, 1, 1}, {w2, 0, 0, 0, 0, 1, 1}}, w13.gk};
    long long runs = 0;
    for (WWork &w : q.w) {
        const WeightsProblem &p = w.p;
        if (!p.offsets || p.offsets != w13.offsets || p.G != w13.G || p.M != w13.M || p.gk != w13.gk ||
            p.c_dt != w13.c_dt || p.accumulate != w13.accumulate)
            return hipErrorInvalidValue;
        w.first_run = (int)runs;
        if (!p.C0) continue;  // not asked for: no items
        if (!p.A || !p.B || p.G < 1 || p.G > kMaxGroups || p.M < 0 || p.MD < 32 || p.MD % 32 || p.ND < 32 ||
            p.ND % 32 || p.gk < 1 || p.gk > 64 || p.lda < p.MD || p.ldb < (p.C1 ? 2 : 1) * p.ND ||
            (p.c_dt != MOE_F32 && p.c_dt != MOE_BF16))
            return hipErrorInvalidValue;
        // the gathered operand: A of the first product, B of the second
        const bool first = &w == q.w;
        if ((first ? p.b_src : p.a_src) || (w13.a_src == nullptr) != (w2.b_src == nullptr) ||
            (w13.a_src && (p.src_rows < 1 || 2LL * p.src_rows * (first ? p.lda : p.ldb) > gather_max_bytes)))
            return hipErrorInvalidValue;
        const int nT = (p.ND + 255) / 256 * (p.C1 ? 2 : 1);
        w.nM = (p.MD + 255) / 256;
        w.nN = (p.ND + 255) / 256;
        const long long items = (long long)p.G * w.nM * nT;
        if (items > 0x7fffffffLL) return hipErrorInvalidValue;
        w.items = (int)items;
        w.group_tiles = Divisor(w.nM * nT);
        w.band_tiles = Divisor(kBand * nT);
        runs += (items + kBlocksPerXcd - 1) / kBlocksPerXcd;
    }
    if (runs == 0) return hipSuccess;
    auto launch = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3(kXcds * kBlocksPerXcd), dim3(512), 0, s, q);
    };
#define MOE_WEIGHTS(F32, ACC)                                                         \
    (w13.a_src ? launch(weights_gemm_kernel<F32, ACC, true>) : launch(weights_gemm_kernel<F32, ACC, false>))
    if (w13.c_dt == MOE_F32) {
        if (w13.accumulate) MOE_WEIGHTS(true, true);
        else MOE_WEIGHTS(true, false);
    } else {
        if (w13.accumulate) MOE_WEIGHTS(false, true);
        else MOE_WEIGHTS(false, false);
    }
#undef MOE_WEIGHTS
    return hipGetLastError();
}

}  // namespace moe
