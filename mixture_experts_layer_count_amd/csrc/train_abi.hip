// libmoe public entry points of the layer's training step: router losses and
// gradients, 8-bit activation checkpoints, and the expert FFN's checkpointing
// forward and backward. Argument validation, workspace layout and launch
// order; nothing here synchronises with the device or allocates.
#include "abi_util.h"
#include "train.h"

using namespace moe;

namespace {

constexpr int kMaxSeqs = 65535;
// Tokens of the router's calls: up to 64 of them for each 256-thread workgroup,
// fewer than 2^32 threads
constexpr int kMaxRouterTokens = (1 << 30) - 64;

// Values of a checkpoint: one launch of 256 threads per 4096 values, and a
// grid's dimension holds fewer than 2^32 threads
constexpr long long kMaxCheckpoint = (1LL << 36) - 4096;

// null, or not on the 16-byte boundary that the kernels' wide accesses need
bool bad16(const void *p) { return !p || (reinterpret_cast<uintptr_t>(p) & 15) != 0; }
bool off16(const void *p) { return p && bad16(p); }

moe_status check_router(int T, int E, int k, int B, const int32_t *seq_offsets) {
    if (T < 0 || E < 1 || k < 1 || k > E || B < 1 || (!seq_offsets && B != 1)) return MOE_ERR_INVALID_ARG;
    if (E > 1024 || k > 64 || B > kMaxSeqs || T > kMaxRouterTokens) return MOE_ERR_UNSUPPORTED;
    if ((long long)T * E > 0x7fffffffLL || (long long)T * k > 0x7fffffffLL) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

// gathered: row_src is given (without tokens it may be null)
moe_status check_train_ffn(bool gathered, int k, int T, int G, int H, int F, moe_dtype dt) {
    if (T < 0 || k < 1 || G < 1 || H < 1 || F < 1 || (!gathered && k != 1)) return MOE_ERR_INVALID_ARG;
    if (dt != MOE_BF16 || H % 32 || F % 32 || H > kMaxDim || F > kMaxDim || G > 1024 || k > 64) return MOE_ERR_UNSUPPORTED;
    if ((long long)T * k > 0x7fffffffLL || 2LL * T * H > gather_max_bytes) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

struct Tiles {
    int bm, max_tiles;
    int32_t *tiles, *n_tiles, *start;
    void carve(Carver &c, long long M, int G, int rows_per_tile) {
        bm = rows_per_tile;
        max_tiles = (int)max_tiles_for(M, G, bm);
        tiles = static_cast<int32_t *>(c.take(sizeof(int32_t) * 4 * max_tiles));
        n_tiles = static_cast<int32_t *>(c.take(sizeof(int32_t)));
        start = static_cast<int32_t *>(c.take(sizeof(int32_t) * (G + 1)));
    }
    TilesJob job(const int32_t *offsets, int G, int32_t *zero, int n_zero) const {
        return {offsets, G, bm, tiles, n_tiles, start, zero, n_zero};
    }
};

// room for split items of two row products: sums (shared: one runs after the
// other) and a set of counters each
struct Parts {
    size_t bytes[2];
    float *sums;
    int32_t *count;
    void carve(Carver &c, const Tiles &t, int K0, RowsUse use0, int K1, RowsUse use1) {
        bytes[0] = rows_gemm_part_bytes(t.bm, use0, K0);
        bytes[1] = rows_gemm_part_bytes(t.bm, use1, K1);
        sums = static_cast<float *>(c.take(bytes[0] > bytes[1] ? bytes[0] : bytes[1]));
        count = static_cast<int32_t *>(c.take(sizeof(int32_t) * 2 * rows_gemm_counters));
    }
};

RowsProblem rows_problem(const Tiles &t, const Parts &parts, int which, int G, int M, int k) {
    RowsProblem p{};
    p.gk = k;
    p.tiles = t.tiles;
    p.n_tiles = t.n_tiles;
    p.group_tile_start = t.start;
    p.n_groups = G;
    p.max_tiles = t.max_tiles;
    p.M = M;
    if (parts.bytes[which]) {
        p.part = parts.sums;
        p.part_cnt = parts.count + which * rows_gemm_counters;
    }
    return p;
}

// the fewer of two row products' column tiles
int columns(int N0, RowsUse use0, int N1, RowsUse use1) {
    const int a = rows_gemm_columns(N0, use0), b = rows_gemm_columns(N1, use1);
    return a < b ? a : b;
}

// Yp = h W2 on the inference path's persistent kernel
GemmProblem down_problem(const Tiles &t, int M, int G, int H, int F) {
    GemmProblem g{};
    g.tiles = t.tiles;
    g.n_tiles = t.n_tiles;
    g.group_tile_start = t.start;
    g.n_groups = G;
    g.max_tiles = t.max_tiles;
    g.M = M;
    g.gk = 1;
    g.ksplit = 1;
    g.lda = F;
    g.a_rows = M;
    g.N = g.ldc = H;
    g.K = g.kchunk = F;
    g.b_stride = (long long)F * H;
    return g;
}

// down projections of at most this depth take the persistent kernel where it
// fits: its items overlap, which counts while they are short. Whole forwards,
// row product against persistent (us): 65536 rows, 128 experts, H 2048, F 512
// 559 to 529, 768 762 to 734, 1024 957 to 934, 1536 1396 to 1389, 2048 1802 to
// 1800; 32768 rows, 16 experts, H 2048, F 512 265 to 256, 1024 446 to 436, 2048
// 799 to 801; 32 experts, H 4096, F 512 515 to 491, 1024 841 to 825, 2048 1526
// to 1506. Deeper ones are as fast either way, and the row product splits its
// last round where that is short
constexpr int kPersistDepth = 1024;

struct ForwardWs {
    Tiles t;
    bool persist;  // the down projection's kernel
    Parts parts;
    uint16_t *h;  // [M][F]
    size_t carve(void *ws, long long M, int G, int H, int F) {
        Carver c(ws);
        t.carve(c, M, G, rows_gemm_bm(ROWS_FORWARD, M, G, columns(F, ROWS_GATE_UP, H, ROWS_DOWN)));
        parts.carve(c, t, H, ROWS_GATE_UP, F, ROWS_DOWN);
        persist = F <= kPersistDepth && tiled_persist_fits(down_problem(t, (int)M, G, H, F), W_BF16, false, t.bm);
        h = static_cast<uint16_t *>(c.take(2 * (size_t)M * F));
        return c.used;
    }
};

struct BackwardWs {
    Tiles t;
    Parts parts;
    uint16_t *x;    // [T][H] the token rows, read back from their checkpoint
    uint16_t *dgu;  // [M][2F]
    uint16_t *hw;   // [M][F]
    float *rows;    // [M][H] row gradients at the token rows
    float *dw_part; // [column tiles of F][M]
    size_t carve(void *ws, long long T, long long M, int G, int H, int F) {
        Carver c(ws);
        t.carve(c, M, G, rows_gemm_bm(ROWS_BACKWARD, M, G, columns(F, ROWS_BACK, H, ROWS_DX)));
        parts.carve(c, t, H, ROWS_BACK, F, ROWS_DX);
        x = static_cast<uint16_t *>(c.take(2 * (size_t)T * H));
        dgu = static_cast<uint16_t *>(c.take(4 * (size_t)M * F));
        hw = static_cast<uint16_t *>(c.take(2 * (size_t)M * F));
        rows = static_cast<float *>(c.take(4 * (size_t)M * H));
        dw_part = static_cast<float *>(c.take(4 * (size_t)M * rows_gemm_columns(F, ROWS_BACK)));
        return c.used;
    }
};

bool ckpt_ok(const moe_ffn_checkpoint *c) {
    return c && !bad16(c->xq) && c->xs && !bad16(c->gq) && c->gs && !bad16(c->uq) && c->us;
}

}  // namespace

extern "C" {

// ---------------------------------------------------------------------------
size_t moe_balance_loss_workspace_bytes(int T, int E, int B) {
    if (T < 0 || E < 1 || E > 1024 || B < 1 || B > kMaxSeqs) return 0;
    return balance_ws_bytes(T, E, B);
}

moe_status moe_balance_loss(const float *logits, const int32_t *topk_idx, int T, int E, int k,
                            const int32_t *seq_offsets, int B, float alpha, float beta, float *loss, int32_t *counts,
                            int32_t *seq_counts, void *ws, size_t ws_bytes, hipStream_t stream) {
    const moe_status st = check_router(T, E, k, B, seq_offsets);
    if (st != MOE_OK) return st;
    if ((T > 0 && (!logits || !topk_idx)) || !loss || !counts || !seq_counts) return MOE_ERR_INVALID_ARG;
    // 4-byte aligned: it holds a counter
    if (!ws || (reinterpret_cast<uintptr_t>(ws) & 3) || ws_bytes < balance_ws_bytes(T, E, B))
        return MOE_ERR_WORKSPACE_TOO_SMALL;
    return hip_status(launch_balance_loss(logits, topk_idx, T, E, k, seq_offsets, B, alpha, beta, loss, counts,
                                          seq_counts, ws, stream));
}

moe_status moe_route_backward(const float *logits, const int32_t *topk_idx, const float *topk_w, const float *dtopk_w,
                              int T, int E, int k, const int32_t *seq_offsets, int B, const int32_t *seq_counts,
                              float alpha, float beta, const float *dloss, float *dlogits, hipStream_t stream) {
    const moe_status st = check_router(T, E, k, B, seq_offsets);
    if (st != MOE_OK) return st;
    if (T == 0) return MOE_OK;
    if (!dtopk_w && !seq_counts) return MOE_ERR_INVALID_ARG;
    if (!dlogits || (seq_counts && !logits) || (dtopk_w && (!topk_w || !topk_idx))) return MOE_ERR_INVALID_ARG;
    return hip_status(launch_route_backward(logits, topk_idx, topk_w, dtopk_w, T, E, k, seq_offsets, B, seq_counts,
                                            alpha, beta, dloss, dlogits, stream));
}

// ---------------------------------------------------------------------------
moe_status moe_checkpoint_pack(const void *X, moe_dtype x_dt, long long ldx, long long R, int C, uint8_t *Q, uint8_t *S,
                               hipStream_t stream) {
    if (R < 0 || C < 1 || ldx < C) return MOE_ERR_INVALID_ARG;
    if ((x_dt != MOE_F32 && x_dt != MOE_BF16) || C % 32 || C > kMaxDim || R > kMaxCheckpoint / C ||
        ldx % (x_dt == MOE_F32 ? 4 : 8))
        return MOE_ERR_UNSUPPORTED;
    if (R == 0) return MOE_OK;
    if (bad16(X) || bad16(Q) || !S) return MOE_ERR_INVALID_ARG;
    return hip_status(launch_mx8_pack(X, x_dt, ldx, R, C, Q, S, stream));
}

moe_status moe_checkpoint_unpack(const uint8_t *Q, const uint8_t *S, long long R, int C, moe_dtype y_dt, void *Y,
                                 hipStream_t stream) {
    if (R < 0 || C < 1) return MOE_ERR_INVALID_ARG;
    if ((y_dt != MOE_F32 && y_dt != MOE_BF16) || C % 32 || C > kMaxDim || R > kMaxCheckpoint / C)
        return MOE_ERR_UNSUPPORTED;
    if (R == 0) return MOE_OK;
    if (bad16(Q) || !S || bad16(Y)) return MOE_ERR_INVALID_ARG;
    return hip_status(launch_mx8_unpack(Q, S, R, C, y_dt, Y, stream));
}

// ---------------------------------------------------------------------------
size_t moe_ffn_train_forward_workspace_bytes(int T, int k, int G, int H, int F) {
    if (check_train_ffn(true, k, T, G, H, F, MOE_BF16) != MOE_OK) return 0;
    ForwardWs w;
    return w.carve(nullptr, (long long)T * k, G, H, F);
}

moe_status moe_ffn_train_forward(const void *X, const int32_t *row_src, int k, int T, const int32_t *offsets, int G,
                                 int H, int F, const void *W1, const void *W3, const void *W2, moe_dtype dt, void *Yp,
                                 const moe_ffn_checkpoint *ckpt, void *ws, size_t ws_bytes, hipStream_t stream) {
    const moe_status st = check_train_ffn(row_src || T == 0, k, T, G, H, F, dt);
    if (st != MOE_OK) return st;
    if (T == 0) return MOE_OK;
    if (bad16(X) || !offsets || bad16(W1) || bad16(W3) || bad16(W2) || bad16(Yp) || !ckpt_ok(ckpt))
        return MOE_ERR_INVALID_ARG;
    const int M = T * k;
    ForwardWs w;
    if (bad16(ws) || ws_bytes < w.carve(ws, M, G, H, F)) return MOE_ERR_WORKSPACE_TOO_SMALL;

    MOE_TRY(launch_mx8_pack_tiles(X, T, H, ckpt->xq, ckpt->xs,
                                  w.t.job(offsets, G, w.parts.count, 2 * rows_gemm_counters), stream));
    RowsProblem up = rows_problem(w.t, w.parts, 0, G, M, k);
    up.A = static_cast<const uint16_t *>(X);
    up.row_src = row_src;
    up.lda = H;
    up.a_rows = T;
    up.N = F;
    up.K0 = H;
    up.B0 = static_cast<const uint16_t *>(W1);
    up.B1 = static_cast<const uint16_t *>(W3);
    up.C = w.h;
    up.gq_out = ckpt->gq;
    up.gs_out = ckpt->gs;
    up.uq_out = ckpt->uq;
    up.us_out = ckpt->us;
    MOE_TRY(launch_rows_gemm(up, ROWS_GATE_UP, w.t.bm, stream));
    if (w.persist) {
        GemmProblem d = down_problem(w.t, M, G, H, F);
        d.A = w.h;
        d.B0 = W2;
        d.C = Yp;
        return hip_status(launch_tiled_persist(d, false, stream));
    }
    RowsProblem down = rows_problem(w.t, w.parts, 1, G, M, k);
    down.A = w.h;
    down.lda = F;
    down.N = H;
    down.K0 = F;
    down.B0 = static_cast<const uint16_t *>(W2);
    down.C = Yp;
    return hip_status(launch_rows_gemm(down, ROWS_DOWN, w.t.bm, stream));
}

// ---------------------------------------------------------------------------
moe_status moe_ffn_train_plan(int T, int k, int G, int H, int F, int *forward_rows, int *backward_rows,
                              int *persistent_down) {
    const moe_status st = check_train_ffn(true, k, T, G, H, F, MOE_BF16);
    if (st != MOE_OK) return st;
    if (!forward_rows || !backward_rows || !persistent_down) return MOE_ERR_INVALID_ARG;
    const long long M = (long long)T * k;
    ForwardWs f;
    BackwardWs b;
    f.carve(nullptr, M, G, H, F);
    b.carve(nullptr, T, M, G, H, F);
    *forward_rows = f.t.bm;
    *backward_rows = b.t.bm;
    *persistent_down = f.persist;
    return MOE_OK;
}

// ---------------------------------------------------------------------------
size_t moe_ffn_train_backward_workspace_bytes(int T, int k, int G, int H, int F) {
    if (check_train_ffn(true, k, T, G, H, F, MOE_BF16) != MOE_OK) return 0;
    BackwardWs w;
    return w.carve(nullptr, T, (long long)T * k, G, H, F);
}

moe_status moe_ffn_train_backward(const void *dY, const float *topk_w, const int32_t *row_src,
                                  const int32_t *assign_row, int k, int T, const int32_t *offsets, int G, int H, int F,
                                  const void *W1, const void *W3, const void *W2, moe_dtype dt,
                                  const moe_ffn_checkpoint *ckpt, const void *dX_add, void *dX, float *dtopk_w,
                                  void *dW1, void *dW3, void *dW2, moe_dtype dw_dt, int accumulate, void *ws,
                                  size_t ws_bytes, hipStream_t stream) {
    const moe_status st = check_train_ffn(row_src || T == 0, k, T, G, H, F, dt);
    if (st != MOE_OK) return st;
    if (dw_dt != MOE_BF16 && dw_dt != MOE_F32) return MOE_ERR_UNSUPPORTED;
    if (accumulate != 0 && accumulate != 1) return MOE_ERR_INVALID_ARG;
    if ((row_src == nullptr) != (assign_row == nullptr) || (dW1 == nullptr) != (dW3 == nullptr) || (dX_add && !dX))
        return MOE_ERR_INVALID_ARG;
    if (!offsets || off16(dX_add) || off16(dX) || off16(dW1) || off16(dW3) || off16(dW2)) return MOE_ERR_INVALID_ARG;
    if (T > 0 && (bad16(dY) || bad16(W1) || bad16(W3) || bad16(W2) || !ckpt_ok(ckpt))) return MOE_ERR_INVALID_ARG;
    const int M = T * k;
    BackwardWs w;
    if (bad16(ws) || ws_bytes < w.carve(ws, T, M, G, H, F)) return MOE_ERR_WORKSPACE_TOO_SMALL;

    if (T > 0) {
        MOE_TRY(launch_build_tiles(offsets, G, 0, w.t.bm, w.t.tiles, w.t.n_tiles, w.t.start, stream, w.parts.count,
                                   2 * rows_gemm_counters));
        // p = dY W2^T, then dg, du, w h and the routing weights' partial sums
        RowsProblem b = rows_problem(w.t, w.parts, 0, G, M, k);
        b.A = static_cast<const uint16_t *>(dY);
        b.row_src = row_src;
        b.lda = H;
        b.a_rows = T;
        b.N = F;
        b.K0 = H;
        b.B0 = static_cast<const uint16_t *>(W2);
        b.gq = ckpt->gq;
        b.gs = ckpt->gs;
        b.uq = ckpt->uq;
        b.us = ckpt->us;
        b.topk_w = topk_w;
        b.w_src = row_src;
        b.dGU = w.dgu;
        b.Hw = w.hw;
        b.dw_part = dtopk_w ? w.dw_part : nullptr;
        MOE_TRY(launch_rows_gemm(b, ROWS_BACK, w.t.bm, stream));
        if (dX) {
            RowsProblem d = rows_problem(w.t, w.parts, 1, G, M, k);
            d.A = w.dgu;
            d.lda = 2 * F;
            d.N = H;
            d.K0 = F;
            d.B0 = static_cast<const uint16_t *>(W1);
            d.B1 = static_cast<const uint16_t *>(W3);
            d.C = w.rows;
            MOE_TRY(launch_rows_gemm(d, ROWS_DX, w.t.bm, stream));
        }
        GatherProblem g{};
        g.assign_row = assign_row;
        g.n_rows = offsets + G;
        g.T = T;
        g.k = k;
        g.M = M;
        g.H = H;
        g.rows = w.rows;
        g.add = static_cast<const uint16_t *>(dX_add);
        g.dX = static_cast<uint16_t *>(dX);
        g.dw_part = w.dw_part;
        g.n_part = rows_gemm_columns(F, ROWS_BACK);
        g.dw = dtopk_w;
        g.xq = ckpt->xq;
        g.xs = ckpt->xs;
        g.x = dW1 ? w.x : nullptr;
        MOE_TRY(launch_gather_grads(g, stream));
    }
    // with T == 0 every expert is empty: zeros (or, accumulating, nothing)
    WeightsProblem q{};
    q.gk = k;
    q.src_rows = T;
    q.offsets = offsets;
    q.G = G;
    q.M = M;
    q.c_dt = dw_dt;
    q.accumulate = accumulate;
    q.a_src = T > 0 ? row_src : nullptr;
    q.A = w.x;
    q.lda = H;
    q.MD = H;
    q.B = w.dgu;
    q.ldb = 2 * F;
    q.ND = F;
    q.C0 = dW1;
    q.C1 = dW3;
    WeightsProblem q2 = q;
    q2.a_src = nullptr;
    q2.b_src = q.a_src;
    q2.A = w.hw;
    q2.lda = F;
    q2.MD = F;
    q2.B = T > 0 ? static_cast<const uint16_t *>(dY) : w.hw;
    q2.ldb = H;
    q2.ND = H;
    q2.C0 = dW2;
    q2.C1 = nullptr;
    return hip_status(launch_weights_gemm(q, q2, stream));
}

// ---------------------------------------------------------------------------
namespace {

moe_status check_dispatch(int T, int k, int H, moe_dtype dt) {
    if (T < 0 || k < 1 || H < 1) return MOE_ERR_INVALID_ARG;
    if ((dt != MOE_F32 && dt != MOE_BF16) || H % 4 || H > kMaxDim || k > 64) return MOE_ERR_UNSUPPORTED;
    if ((long long)T * k > 0x7fffffffLL || T > kCombineBackTokens || (long long)T * H > kPermuteBackValues)
        return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}
// the boundary that rows of H values allow: 16 bytes, or 8 for bf16 of H % 8 = 4
bool off_rows(const void *p, int H, moe_dtype dt) {
    return (reinterpret_cast<uintptr_t>(p) & (dt == MOE_BF16 && H % 8 ? 7 : 15)) != 0;
}

}  // namespace

moe_status moe_combine_backward(const void *dY, const void *Yp, const int32_t *assign_row, const float *topk_w,
                                const int32_t *n_rows, int T, int k, int H, moe_dtype dt, void *dYp, float *dtopk_w,
                                hipStream_t stream) {
    const moe_status st = check_dispatch(T, k, H, dt);
    if (st != MOE_OK) return st;
    if (T == 0) return MOE_OK;
    if (!dYp && !dtopk_w) return MOE_ERR_INVALID_ARG;
    if (!dY || !assign_row || (dYp && !topk_w) || (dtopk_w && !Yp)) return MOE_ERR_INVALID_ARG;
    if (off_rows(dY, H, dt) || off_rows(Yp, H, dt) || off_rows(dYp, H, dt)) return MOE_ERR_UNSUPPORTED;
    return hip_status(launch_combine_back({dY, Yp, assign_row, topk_w, n_rows, T, k, H, dYp, dtopk_w}, dt, stream));
}

moe_status moe_permute_backward(const void *dXp, const int32_t *assign_row, const int32_t *n_rows, int T, int k, int H,
                                moe_dtype dt, const void *dX_add, void *dX, hipStream_t stream) {
    const moe_status st = check_dispatch(T, k, H, dt);
    if (st != MOE_OK) return st;
    if (T == 0) return MOE_OK;
    if (!dXp || !assign_row || !dX) return MOE_ERR_INVALID_ARG;
    if (off_rows(dXp, H, dt) || off_rows(dX_add, H, dt) || off_rows(dX, H, dt)) return MOE_ERR_UNSUPPORTED;
    return hip_status(launch_permute_back({dXp, assign_row, n_rows, dX_add, T, k, H, dX}, dt, stream));
}

}  // extern "C"
