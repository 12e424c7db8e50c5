// The layer's training operators: problem descriptions and launchers.
#pragma once

#include "common.h"

namespace moe {

unsigned bounds_take_train_rows();
unsigned bounds_take_train_weights();

// Between LDS writes and reads by other lanes of the same wavefront, whose LDS
// operations complete in order: no instruction, but without it the compiler
// may hand a lane back the value it wrote itself.
__device__ __forceinline__ void wave_lds_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// MXFP8 activation checkpoints (mx8.hip): rows of C values (a multiple of 32),
// codes Q [R][C] and scale bytes S [R][C/32]
hipError_t launch_mx8_pack(const void *X, moe_dtype x_dt, long long ldx, long long R, int C, uint8_t *Q, uint8_t *S,
                           hipStream_t s);
// dense bf16 rows packed, and in the same launch a tile list as
// launch_build_tiles forms it
struct TilesJob {
    const int32_t *offsets;
    int G, bm;
    int32_t *tiles, *n_tiles, *start, *zero;
    int n_zero;
};
hipError_t launch_mx8_pack_tiles(const void *X, long long R, int C, uint8_t *Q, uint8_t *S, const TilesJob &tiles,
                                 hipStream_t s);
hipError_t launch_mx8_unpack(const uint8_t *Q, const uint8_t *S, long long R, int C, moe_dtype y_dt, void *Y,
                             hipStream_t s);

// Router losses and the gradient at its logits (balance.hip). seq: device
// [B + 1] token offsets or NULL (then B == 1).
size_t balance_ws_bytes(int T, int E, int B);
hipError_t launch_balance_loss(const float *logits, const int32_t *idx, int T, int E, int k, const int32_t *seq, int B,
                               float alpha, float beta, float *loss, int32_t *counts, int32_t *seq_counts, void *ws,
                               hipStream_t s);
hipError_t launch_route_backward(const float *logits, const int32_t *idx, const float *w, const float *dw, int T, int E,
                                 int k, const int32_t *seq, int B, const int32_t *seq_counts, float alpha, float beta,
                                 const float *dloss, float *dlogits, hipStream_t s);

// ---------------------------------------------------------------------------
// The grouped FFN in training (train_rows.hip, train_weights.hip)
// ---------------------------------------------------------------------------

// C[r] = A(r) B_g, A(r) = A[row_src[r] / gk] (A[r] if NULL), K0 deep:
//  GATE_UP  B0, B1 = W1, W3 [G][K0][N]: C = silu(A B0) (A B1) bf16 [M][N], and
//           both products as MXFP8 checkpoints
//  DOWN     B0 = W2 [G][K0][N]: C bf16 [M][N]
//  BACK     B0 = W2 [G][N][K0]: p = A B0^T, and with the checkpointed g, u and
//           the row's routing weight w (1 if topk_w is NULL): dGU [M][2 N] (dg
//           then du), Hw [M][N] = w h, and dw_part[column tile][M] = sum over
//           the tile's columns of p h
//  DX       B0, B1 = W1, W3 [G][N][K0]: C = A[:, :K0] B0^T + A[:, K0:] B1^T,
//           fp32 [M][N]
enum RowsUse { ROWS_GATE_UP, ROWS_DOWN, ROWS_BACK, ROWS_DX };
struct RowsProblem {
    const uint16_t *A;
    const int32_t *row_src;
    int gk, lda;
    int a_rows;               // rows of A, when gathered (in at most gather_max_bytes)
    const int32_t *tiles, *n_tiles, *group_tile_start;
    int n_groups, max_tiles;
    int M, N, K0;
    const uint16_t *B0, *B1;
    void *C;
    uint8_t *gq_out, *gs_out, *uq_out, *us_out;
    const uint8_t *gq, *gs, *uq, *us;
    const float *topk_w;
    const int32_t *w_src;     // row_src for topk_w (NULL: row r)
    uint16_t *dGU, *Hw;
    float *dw_part;
    // split of the last, partial round: rows_gemm_part_bytes bytes for the
    // parts' sums and rows_gemm_counters counters, zero at launch and used by
    // one launch. NULL: no split
    float *part = nullptr;
    int32_t *part_cnt = nullptr;
};
// rows per tile of a pass's products; columns: the fewer of their column tiles
enum RowsPass { ROWS_FORWARD, ROWS_BACKWARD };
int rows_gemm_bm(RowsPass pass, long long rows, int groups, int columns);
constexpr int rows_gemm_bn = 256;  // B columns per tile
constexpr int rows_gemm_counters = 256;
int rows_gemm_columns(int N, RowsUse use);  // column tiles
size_t rows_gemm_part_bytes(int bm, RowsUse use, int K0);  // 0: never split
constexpr uint32_t gather_max_bytes = 0xfffff000u;  // of a gathered matrix: 32-bit offsets
hipError_t launch_rows_gemm(const RowsProblem &p, RowsUse use, int bm, hipStream_t s);

// dW_g[m][n] = sum over rows r of group g of A(r)[m] B(r)[n], for one or two
// output matrices (the second of B's columns ND .. 2 ND - 1).
struct WeightsProblem {
    const uint16_t *A, *B;
    int lda, ldb;
    const int32_t *a_src, *b_src;  // row r is A[a_src[r] / gk]; NULL: A[r] (at most one given)
    int gk, src_rows;              // rows of the gathered operand (in at most gather_max_bytes)
    const int32_t *offsets;        // [G + 1]
    int G, M, MD, ND;              // M rows in all; output MD x ND
    void *C0, *C1;                 // [G][MD][ND]; C1 NULL: one output
    moe_dtype c_dt;
    int accumulate;                // add to what C holds
};
// dW1 and dW3 (w13), then dW2, in one launch; C0 NULL: that product is left out
hipError_t launch_weights_gemm(const WeightsProblem &w13, const WeightsProblem &w2, hipStream_t s);

// What the backward pass does token by token; each of dX, dw and x may be NULL.
// dX[t] = sum_j rows[assign_row[t k + j]] (+ add[t]); dw[t k + j] = sum over
// column tiles of dw_part[tile][assign_row[t k + j]]; x = the values of the
// checkpoint xq, xs. assign_row NULL: row t (k == 1). Rows outside
// [0, min(M, *n_rows)) contribute nothing.
struct GatherProblem {
    const int32_t *assign_row, *n_rows;
    int T, k, M, H;
    const float *rows;     // [M][H]
    const uint16_t *add;   // [T][H] or NULL
    uint16_t *dX;          // [T][H]
    const float *dw_part;  // [n_part][M]
    int n_part;
    float *dw;             // [T][k]
    const uint8_t *xq, *xs;
    uint16_t *x;           // [T][H]
};
hipError_t launch_gather_grads(const GatherProblem &p, hipStream_t s);

// Gradients of the sorted rows and of the weighted sum back (dispatch_grad.hip),
// for rows of dt (MOE_F32, MOE_BF16). n_rows: device, NULL for T * k.
struct CombineBack {
    const void *dY, *Yp;        // [T][H], [M][H]
    const int32_t *assign_row;  // [T * k]
    const float *w;             // [T][k]
    const int32_t *n_rows;
    int T, k, H;
    void *dYp;                  // [M][H] or NULL
    float *dw;                  // [T][k] or NULL
};
struct PermuteBack {
    const void *dXp;            // [M][H]
    const int32_t *assign_row, *n_rows;
    const void *add;            // [T][H] or NULL
    int T, k, H;
    void *dX;                   // [T][H]
};
// fewer than 2^32 threads a launch: a workgroup of up to 256 a token, a thread
// for 4 values at least
constexpr int kCombineBackTokens = (1 << 24) - 1;
constexpr long long kPermuteBackValues = (1LL << 34) - 1024;
hipError_t launch_combine_back(const CombineBack &p, moe_dtype dt, hipStream_t s);
hipError_t launch_permute_back(const PermuteBack &p, moe_dtype dt, hipStream_t s);

}  // namespace moe
