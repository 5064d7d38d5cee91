/*
 * dsmoe_experts.h -- the routed experts' feed-forward products outside FP8, for
 * AMD Instinct MI355X (gfx950): in bf16 with their gradients (training, or the
 * precision that FP8 is compared with), and in 8-bit integers with a scale for
 * each token and each output channel (serving).
 *
 * Rows are grouped by expert as dsmoe_route lays them out, in ragged groups:
 *     [g | u] = x[perm] W13_e^T,  a = gate * act(g) * u,  o = a W2_e^T,
 *     y[t] = sum over k of o[inv[t][k]]                    (dsmoe_combine_rows)
 * W13 and W2 are laid out as the FP8 layer's: an expert's gate rows, then its up
 * rows.  The gate enters with the activation, so o needs no factor, and the
 * gate's gradient comes with the activation's.
 *
 * The calls are part of libdsmoe.so and follow the conventions of dsmoe.h
 * (device pointers owned by the caller, asynchronous on `stream`, host
 * validation before anything is enqueued, status codes), except that:
 * - Matrices are row-major with a row stride in elements (ld..., at least the
 *   row length); columns are contiguous.  Any size and any element-aligned
 *   pointer is accepted.  Operands whose rows are not 16-byte aligned or not a
 *   multiple of 16 bytes long may be copied into the workspace first, weights
 *   as a whole: of all G experts, also those without rows.  Operands that the
 *   caller keeps widened by columns of zeros (K 1008 for 1001) need no copy.
 * - NaN and infinities propagate as in the formulas.
 * - offsets [G+1] int32 on the device: group g owns rows offsets[g] ..
 *   offsets[g+1]-1, 0 <= offsets[g] <= offsets[g+1] <= R.  NULL: one group of
 *   all R rows (G must be 1).  A group may be empty.  Results of rows outside
 *   every group are left untouched, and such rows enter no sum.  Offsets that
 *   break the rule give unspecified results but no access outside the buffers.
 * - rows [R] int32 on the device, or NULL: row r of the operand is its source
 *   row rows[r] (NULL: r), of n source rows (NULL: n must be R, unless R is 0).
 *   An index outside [0, n) reads as a row of zeros.
 * - Weights of G experts are one matrix of all their rows, expert by expert.
 * - Sizes: 1 <= G <= DSMOE_MAX_EXPERTS; row lengths and row strides are in [1,
 *   DSMOE_DENSE_MAX_DIM]; R and n in [0, 2^31), n > 0 where R > 0; the weights and
 *   either side's R rows have at most 2^40 elements.  No rows:
 *   outputs per row are not touched, weight gradients are written as 0.
 * - The workspace is 256-byte aligned; its size comes from the
 *   ..._workspace_bytes call with the same arguments (0: NULL is accepted).
 *   Those calls look only at a pointer's alignment and whether it is NULL.
 *   The contents need no initialisation and mean nothing after the call.
 * - Outputs must not overlap inputs or one another.
 * - All sums are float32 (int32 for integers) in a fixed order: equal calls give
 *   equal bits.
 */
#ifndef DSMOE_EXPERTS_H
#define DSMOE_EXPERTS_H

#include "dsmoe_dense.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * dsmoe_grouped_linear -- y[r] = x[rows[r]] W_g^T for the rows of each group.
 *   x   [n][K] bf16, rows as above
 *   w   [G*N][K] bf16
 *   y   [R][N], type yt (bf16 or f32)
 */
size_t dsmoe_grouped_linear_workspace_bytes(const void* x, int64_t ldx, int64_t n, const int32_t* rows,
                                            const void* w, int64_t ldw, int32_t G, int64_t R, int64_t N, int64_t K);
dsmoe_status dsmoe_grouped_linear(const void* x, int64_t ldx, int64_t n, const int32_t* rows, const void* w,
                                  int64_t ldw, const int32_t* offsets, int32_t G, int64_t R, int64_t N, int64_t K,
                                  void* y, int64_t ldy, int yt, void* workspace, size_t ws_bytes, void* stream);

/*
 * dsmoe_grouped_linear_backward -- with dy[r] = dy[dy_rows[r]], x[r] = x[rows[r]]:
 *   dx[r] = dy[r] W_g,   dW_g = sum over the group's rows of dy[r]^T x[r]
 *   dy  [n_dy][N] bf16, dy_rows as rows above
 *   x   [n][K], rows, w [G*N][K] bf16: the forward's
 *   dx  [R][K], type dxt, or NULL: one row per routed row (where rows repeat,
 *       the caller adds them up, e.g. with dsmoe_combine_rows)
 *   dw  [G*N][K], type dwt, or NULL; 0 for a group without rows
 */
size_t dsmoe_grouped_linear_backward_workspace_bytes(const void* dy, int64_t lddy, int64_t n_dy,
                                                     const int32_t* dy_rows, const void* x, int64_t ldx, int64_t n,
                                                     const int32_t* rows, const void* w, int64_t ldw, int32_t G,
                                                     int64_t R, int64_t N, int64_t K);
dsmoe_status dsmoe_grouped_linear_backward(const void* dy, int64_t lddy, int64_t n_dy, const int32_t* dy_rows,
                                           const void* x, int64_t ldx, int64_t n, const int32_t* rows, const void* w,
                                           int64_t ldw, const int32_t* offsets, int32_t G, int64_t R, int64_t N,
                                           int64_t K, void* dx, int64_t lddx, int dxt, void* dw, int64_t lddw,
                                           int dwt, void* workspace, size_t ws_bytes, void* stream);

/*
 * dsmoe_grouped_gated_linear -- [g | u] = x[rows[r]] W13_g^T, a = s act(g) u, in
 * one product: h is written only where the caller wants it.
 *   x          [n][H] bf16, rows as above
 *   w13        [G*2I][H] bf16: I gate rows, then I up rows of each expert
 *   row_scale  [R] f32, or NULL (1): s, the row's gate
 *   a          [R][I], type at (bf16 or f32)
 *   h          [R][2I] bf16, or NULL: the pre-activations, for the backward
 * act is one of SILU, GELU, RELU or NONE (a bilinear gate).  a is formed in
 * float32 from the float32 sums and rounded once.
 */
size_t dsmoe_grouped_gated_linear_workspace_bytes(const void* x, int64_t ldx, int64_t n, const int32_t* rows,
                                                  const void* w13, int64_t ldw, int32_t G, int64_t R, int64_t H,
                                                  int64_t I);
dsmoe_status dsmoe_grouped_gated_linear(const void* x, int64_t ldx, int64_t n, const int32_t* rows, const void* w13,
                                        int64_t ldw, const float* row_scale, int act, const int32_t* offsets,
                                        int32_t G, int64_t R, int64_t H, int64_t I, void* a, int64_t lda, int at,
                                        void* h, int64_t ldh, void* workspace, size_t ws_bytes, void* stream);

/*
 * dsmoe_grouped_gated_linear_backward -- with f = act(g):
 *   dscale[r] = sum over columns of da f u
 *   dh = s [da u act'(g) | da f],  dx[r] = dh[r] W13_g,
 *   dW13_g = sum over the group's rows of dh[r]^T x[rows[r]]
 *   da      [R][I] bf16
 *   x, rows, w13, row_scale, h: the forward's
 *   dx      [R][H], type dxt, or NULL (one row per routed row)
 *   dw13    [G*2I][H], type dwt, or NULL; 0 for a group without rows
 *   dscale  [R] f32, or NULL
 * dh is formed in float32.  It enters a bf16 gradient rounded to bf16, an error
 * as large as the result's own rounding, and a float32 gradient as the sum of
 * two bf16 values, which keeps 16 significant bits and takes a product for each,
 * the second added to the first (8192 tokens x 2 of 32 experts, H 7168, I 2048: dw13
 * in float32 4.8 ms instead of 2.5).  With act | DSMOE_DZ_BF16 it is rounded to bf16
 * for float32 gradients too.  A bf16 gradient of more bits is a float32 one that
 * the caller rounds.  The workspace's size holds dh and its rest for any of these.
 */
size_t dsmoe_grouped_gated_linear_backward_workspace_bytes(const void* x, int64_t ldx, int64_t n,
                                                           const int32_t* rows, const void* w13, int64_t ldw,
                                                           int32_t G, int64_t R, int64_t H, int64_t I);
dsmoe_status dsmoe_grouped_gated_linear_backward(const void* da, int64_t ldda, const void* x, int64_t ldx, int64_t n,
                                                 const int32_t* rows, const void* w13, int64_t ldw, const void* h,
                                                 int64_t ldh, const float* row_scale, int act, const int32_t* offsets,
                                                 int32_t G, int64_t R, int64_t H, int64_t I, void* dx, int64_t lddx,
                                                 int dxt, void* dw13, int64_t lddw, int dwt, float* dscale,
                                                 void* workspace, size_t ws_bytes, void* stream);

/*
 * dsmoe_router_backward -- gradients of the router logits from the gates'.
 *   dgate     [T][K] f32 (dscale of row inv[t][k])
 *   topk_idx  [T][K] int32, logits [T][E] f32: the routing's
 *   dlogits   [T][E] f32 (output): with s = sigmoid(z), S = sum of the chosen
 *             s, gate = s / S: s_k (1 - s_k) (dgate_k - sum_j dgate_j gate_j) / S
 *             at the chosen experts, 0 elsewhere (routing held fixed); evaluated
 *             in double and rounded once (an expert chosen twice gets the sum)
 * An index outside [0, E) is left out.  Requires 1 <= K <= DSMOE_MAX_TOPK,
 * K <= E <= DSMOE_MAX_EXPERTS, T in [0, 2^31).
 */
dsmoe_status dsmoe_router_backward(const float* dgate, const int32_t* topk_idx, const float* logits, int64_t T,
                                   int32_t E, int32_t K, float* dlogits, void* stream);

/*
 * dsmoe_quant_rows_int8 -- 8-bit integers with one scale per row: per token for
 * activations [tokens][channels], per output channel for a weight [N][K].
 *   x      [rows][cols], type xt (bf16 or f32)
 *   q      [rows][cols] int8 (output)
 *   scale  [rows] f32 (output)
 * Per row: s = fl32(max |x| / 127) by IEEE division (1 where that is 0), q = the
 * whole number nearest to fl32(x / s) by IEEE division, ties to even, within
 * +-127.  A row with a NaN or an infinity has scale NaN and codes 0, so every
 * product of it is NaN.
 */
dsmoe_status dsmoe_quant_rows_int8(const void* x, int64_t ldx, int xt, int64_t rows, int64_t cols, int8_t* q,
                                   int64_t ldq, float* scale, void* stream);

/* The contraction length of the 8-bit products is below this, so that a sum of
 * products of any codes fits 32 bits. */
#define DSMOE_INT8_MAX_K 131072

/*
 * dsmoe_int8_linear -- y[r][c] = xs[rows[r]] ws_g[c] (sum over k of x[rows[r]][k] w_g[c][k]).
 *   x        [n][K] int8, x_scale [n] f32, rows as above
 *   w        [G*N][K] int8, w_scale [G*N] f32
 *   y        [R][N], type yt (bf16 or f32)
 * The sum is exact in int32; it is rounded to float32, multiplied by x's scale,
 * then w's, and rounded to y's type.  With offsets NULL and G = 1 it is a dense
 * product.  Requires K < DSMOE_INT8_MAX_K.
 */
size_t dsmoe_int8_linear_workspace_bytes(const int8_t* x, int64_t ldx, int64_t n, const int32_t* rows,
                                         const int8_t* w, int64_t ldw, int32_t G, int64_t R, int64_t N, int64_t K);
dsmoe_status dsmoe_int8_linear(const int8_t* x, int64_t ldx, const float* x_scale, int64_t n, const int32_t* rows,
                               const int8_t* w, int64_t ldw, const float* w_scale, const int32_t* offsets, int32_t G,
                               int64_t R, int64_t N, int64_t K, void* y, int64_t ldy, int yt, void* workspace,
                               size_t ws_bytes, void* stream);

/*
 * dsmoe_int8_gated_linear -- a = s act(g) u with [g | u] as dsmoe_int8_linear
 * gives them in float32.
 *   w13      [G*2I][H] int8, w13_scale [G*2I] f32
 *   the rest as there and in dsmoe_grouped_gated_linear.
 */
size_t dsmoe_int8_gated_linear_workspace_bytes(const int8_t* x, int64_t ldx, int64_t n, const int32_t* rows,
                                               const int8_t* w13, int64_t ldw, int32_t G, int64_t R, int64_t H,
                                               int64_t I);
dsmoe_status dsmoe_int8_gated_linear(const int8_t* x, int64_t ldx, const float* x_scale, int64_t n,
                                     const int32_t* rows, const int8_t* w13, int64_t ldw, const float* w13_scale,
                                     const float* row_scale, int act, const int32_t* offsets, int32_t G, int64_t R,
                                     int64_t H, int64_t I, void* a, int64_t lda, int at, void* workspace,
                                     size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* DSMOE_EXPERTS_H */
