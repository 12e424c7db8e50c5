// libmoe public entry points of the layer's training step: router losses and
// gradients, 8-bit activation checkpoints, and the expert FFN's checkpointing
// forward and backward. Argument validation, workspace layout and launch
// order; nothing here synchronises with the device or allocates.
#include "abi_util.h"

using namespace moe;

namespace {

constexpr int kMaxSeqs = 65535;

// null, or not on the 16-byte boundary that the kernels' wide accesses need
bool bad16(const void *p) { return !p || (reinterpret_cast<uintptr_t>(p) & 15) != 0; }
bool off16(const void *p) { return p && bad16(p); }

moe_status check_router(int T, int E, int k, int B, const int32_t *seq_offsets) {
    if (T < 0 || E < 1 || k < 1 || k > E || B < 1 || (!seq_offsets && B != 1)) return MOE_ERR_INVALID_ARG;
    if (E > 1024 || k > 64 || B > kMaxSeqs) return MOE_ERR_UNSUPPORTED;
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
    hipError_t build(const int32_t *offsets, int G, hipStream_t s, int32_t *zero = nullptr, int n_zero = 0) const {
        return launch_build_tiles(offsets, G, 0, bm, tiles, n_tiles, start, s, zero, n_zero);
    }
};

struct ForwardWs {
    Tiles t;
    uint16_t *h;  // [M][F]
    float *tail_part;
    int32_t *tail_cnt;
    size_t carve(void *ws, long long M, int G, int F) {
        Carver c(ws);
        t.carve(c, M, G, tiled_gemm_bm(W_BF16, M, G));
        h = static_cast<uint16_t *>(c.take(2 * (size_t)M * F));
        tail_part = static_cast<float *>(c.take(tiled_tail_bytes(t.bm)));
        tail_cnt = static_cast<int32_t *>(c.take(sizeof(int32_t) * tiled_tail_counters));
        return c.used;
    }
};

struct BackwardWs {
    Tiles t;
    uint16_t *x;    // [T][H] the token rows, read back from their checkpoint
    uint16_t *dgu;  // [M][2F]
    uint16_t *hw;   // [M][F]
    float *rows;    // [M][H] row gradients at the token rows
    float *dw_part; // [column tiles of F][M]
    float *part;    // sums of split items, and their counters (one set per launch)
    int32_t *part_cnt;
    int parts_f, parts_h;
    size_t carve(void *ws, long long T, long long M, int G, int H, int F) {
        Carver c(ws);
        t.carve(c, M, G, rows_gemm_bm(M, G));
        x = static_cast<uint16_t *>(c.take(2 * (size_t)T * H));
        dgu = static_cast<uint16_t *>(c.take(4 * (size_t)M * F));
        hw = static_cast<uint16_t *>(c.take(2 * (size_t)M * F));
        rows = static_cast<float *>(c.take(4 * (size_t)M * H));
        dw_part = static_cast<float *>(c.take(4 * (size_t)M * ((F + rows_gemm_bn - 1) / rows_gemm_bn)));
        parts_f = rows_gemm_xcd_parts(t.max_tiles, F);
        parts_h = rows_gemm_xcd_parts(t.max_tiles, H);
        part = static_cast<float *>(c.take(rows_gemm_part_bytes(t.bm, parts_f > parts_h ? parts_f : parts_h)));
        part_cnt = static_cast<int32_t *>(c.take(sizeof(int32_t) * 2 * rows_gemm_counters));
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
    if (!ws || ws_bytes < balance_ws_bytes(T, E, B)) return MOE_ERR_WORKSPACE_TOO_SMALL;
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
    if ((x_dt != MOE_F32 && x_dt != MOE_BF16) || C % 32 || C > kMaxDim || R > 0x7fffffffLL ||
        ldx % (x_dt == MOE_F32 ? 4 : 8) || R * (C / 16) > 0x7fffffffLL * 256)
        return MOE_ERR_UNSUPPORTED;
    if (R == 0) return MOE_OK;
    if (bad16(X) || bad16(Q) || !S) return MOE_ERR_INVALID_ARG;
    return hip_status(launch_mx8_pack(X, x_dt, ldx, R, C, Q, S, stream));
}

moe_status moe_checkpoint_unpack(const uint8_t *Q, const uint8_t *S, long long R, int C, moe_dtype y_dt, void *Y,
                                 hipStream_t stream) {
    if (R < 0 || C < 1) return MOE_ERR_INVALID_ARG;
    if ((y_dt != MOE_F32 && y_dt != MOE_BF16) || C % 32 || C > kMaxDim || R > 0x7fffffffLL ||
        R * (C / 16) > 0x7fffffffLL * 256)
        return MOE_ERR_UNSUPPORTED;
    if (R == 0) return MOE_OK;
    if (bad16(Q) || !S || bad16(Y)) return MOE_ERR_INVALID_ARG;
    return hip_status(launch_mx8_unpack(Q, S, R, C, y_dt, Y, stream));
}

// ---------------------------------------------------------------------------
size_t moe_ffn_train_forward_workspace_bytes(int T, int k, int G, int H, int F) {
    if (check_train_ffn(true, k, T, G, H, F, MOE_BF16) != MOE_OK) return 0;
    ForwardWs w;
    return w.carve(nullptr, (long long)T * k, G, F);
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
    if (bad16(ws) || ws_bytes < w.carve(ws, M, G, F)) return MOE_ERR_WORKSPACE_TOO_SMALL;

    MOE_TRY(launch_mx8_pack(X, MOE_BF16, H, T, H, ckpt->xq, ckpt->xs, stream));
    MOE_TRY(w.t.build(offsets, G, stream, w.tail_cnt, tiled_tail_counters));
    GemmProblem g{};
    g.tiles = w.t.tiles;
    g.n_tiles = w.t.n_tiles;
    g.group_tile_start = w.t.start;
    g.n_groups = G;
    g.max_tiles = w.t.max_tiles;
    g.M = M;
    g.gk = k;
    g.ksplit = 1;
    GemmProblem up = g;
    up.A = X;
    up.row_src = row_src;
    up.lda = H;
    up.a_rows = T;
    up.N = F;
    up.K = up.kchunk = H;
    up.B0 = W1;
    up.B1 = W3;
    up.b_stride = (long long)H * F;
    up.C = w.h;
    up.ldc = F;
    up.ckpt[0] = ckpt->gq;
    up.ckpt[1] = ckpt->gs;
    up.ckpt[2] = ckpt->uq;
    up.ckpt[3] = ckpt->us;
    MOE_TRY(launch_tiled_ckpt(up, w.t.bm, stream));
    GemmProblem down = g;
    down.A = w.h;
    down.lda = F;
    down.a_rows = M;
    down.N = H;
    down.K = down.kchunk = F;
    down.B0 = W2;
    down.b_stride = (long long)F * H;
    down.C = Yp;
    down.ldc = H;
    down.tail_part = w.tail_part;
    down.tail_cnt = w.tail_cnt;
    return hip_status(launch_tiled_gemm(down, W_BF16, false, true, w.t.bm, stream));
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
        MOE_TRY(w.t.build(offsets, G, stream, w.part_cnt, 2 * rows_gemm_counters));
        RowsProblem p{};
        p.gk = k;
        p.tiles = w.t.tiles;
        p.n_tiles = w.t.n_tiles;
        p.group_tile_start = w.t.start;
        p.n_groups = G;
        p.max_tiles = w.t.max_tiles;
        p.M = M;
        p.part = w.part;
        // p = dY W2^T, then dg, du, w h and the routing weights' partial sums
        RowsProblem b = p;
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
        b.part_cnt = w.part_cnt;
        b.xcd_parts = w.parts_f;
        b.dw_part = dtopk_w ? w.dw_part : nullptr;
        MOE_TRY(launch_rows_gemm(b, true, w.t.bm, stream));
        if (dX) {
            RowsProblem d = p;
            d.A = w.dgu;
            d.lda = 2 * F;
            d.a_rows = M;
            d.N = H;
            d.K0 = F;
            d.B0 = static_cast<const uint16_t *>(W1);
            d.B1 = static_cast<const uint16_t *>(W3);
            d.C = w.rows;
            d.part_cnt = w.part_cnt + rows_gemm_counters;
            d.xcd_parts = w.parts_h;
            MOE_TRY(launch_rows_gemm(d, false, w.t.bm, stream));
        }
        MOE_TRY(launch_gather_grads(w.rows, w.dw_part, (F + rows_gemm_bn - 1) / rows_gemm_bn, assign_row, T, k,
                                    offsets + G, M, H, dX_add, dX, dtopk_w, stream));
        if (dW1) MOE_TRY(launch_mx8_unpack(ckpt->xq, ckpt->xs, T, H, MOE_BF16, w.x, stream));
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
    if (dW1) {
        q.A = w.x;
        q.a_src = row_src;
        q.lda = H;
        q.MD = H;
        q.B = w.dgu;
        q.ldb = 2 * F;
        q.ND = F;
        q.C0 = dW1;
        q.C1 = dW3;
        MOE_TRY(launch_weights_gemm(q, stream));
    }
    if (dW2) {
        q.A = w.hw;
        q.a_src = nullptr;
        q.lda = F;
        q.MD = F;
        q.B = T > 0 ? static_cast<const uint16_t *>(dY) : w.hw;
        q.b_src = row_src;
        q.ldb = H;
        q.ND = H;
        q.C0 = dW2;
        q.C1 = nullptr;
        MOE_TRY(launch_weights_gemm(q, stream));
    }
    return MOE_OK;
}

}  // extern "C"
