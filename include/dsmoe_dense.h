/*
 * dsmoe_dense.h -- the dense (not routed) feed-forward sub-layer beside the
 * MoE layer, in bf16: layer norm, gated linear and linear with an epilogue,
 * each with its backward pass, for AMD Instinct MI355X (gfx950).
 *
 * They make the feed-forward sub-layer of the leading dense layers, or a
 * shared expert kept out of FP8:
 *     n = layer_norm(x),  a = act(n Wg^T) * (n Wu^T),  y = x + a W2^T
 * W13 = [Wg; Wu] is laid out as the MoE layer's gate/up weight (gate rows
 * first), W2 as its down weight.
 *
 * The calls are part of libdsmoe.so and follow the conventions of dsmoe.h
 * (device pointers owned by the caller, asynchronous on `stream`, host
 * validation before anything is enqueued, status codes), except that:
 * - Matrices are row-major with a row stride in elements (ld..., at least the
 *   row length); columns are contiguous.  Any size and any element-aligned
 *   pointer is accepted.  Operands of products whose rows are not 16-byte
 *   aligned or whose length is not a multiple of 8 may be copied into the
 *   workspace first.
 * - NaN and infinities propagate as in the formulas.
 * - Sizes: every row length and row stride is in [1, DSMOE_DENSE_MAX_DIM];
 *   rows / tokens in [0, 2^31).  No rows: outputs per row are not touched,
 *   gradients summed over rows are written as 0.
 * - The workspace is 256-byte aligned; its size comes from the
 *   ..._workspace_bytes call with the same arguments (0: NULL is accepted).
 *   Those calls look only at a pointer's alignment and whether it is NULL.
 *   The contents need no initialisation and mean nothing after the call.
 * - All sums are float32 in a fixed order: equal calls give equal bits.
 */
#ifndef DSMOE_DENSE_H
#define DSMOE_DENSE_H

#include "dsmoe.h"

#ifdef __cplusplus
extern "C" {
#endif

#define DSMOE_DENSE_MAX_DIM 4194304

typedef enum dsmoe_act {
  DSMOE_ACT_NONE = 0,
  DSMOE_ACT_SILU = 1,   /* z / (1 + e^-z) */
  DSMOE_ACT_GELU = 2,   /* z (1 + erf(z / sqrt 2)) / 2 */
  DSMOE_ACT_RELU = 3    /* max(z, 0), derivative 0 at 0 */
} dsmoe_act;

/*
 * dsmoe_layer_norm -- y = (s - mean(s)) rstd * gamma + beta per row, with
 * s = x + residual, rstd = 1 / sqrt(var(s) + eps), var the mean square
 * deviation (not the sample variance).
 *   x, residual  [rows][cols], type xt (bf16 or f32); residual may be NULL
 *   gamma, beta  [cols], type pt; either may be NULL (1, 0)
 *   y            [rows][cols], type xt
 *   sum          [rows][cols], type xt, or NULL: s, rounded to xt
 *   mean, rstd   [rows] f32, or NULL
 * s is formed and normalised in float32 (y does not see the rounding of
 * sum).  y or sum may be x or residual itself (same pointer and stride).
 * Requires eps >= 0 and finite (DSMOE_ERR_SHAPE otherwise).
 */
dsmoe_status dsmoe_layer_norm(const void* x, int64_t ldx, const void* residual, int64_t ldr, int xt,
                              const void* gamma, const void* beta, int pt, int64_t rows, int64_t cols,
                              float eps, void* y, int64_t ldy, void* sum, int64_t lds, float* mean,
                              float* rstd, void* stream);

/*
 * dsmoe_layer_norm_backward -- with n = (x - mean) rstd, g = dy * gamma:
 *   dx = rstd (g - mean(g) - n mean(g n)) + dsum
 *   dgamma = sum over rows of dy n,  dbeta = sum over rows of dy
 *   dy, x, dsum  [rows][cols], type xt; x is the s of the forward; dsum (the
 *                gradient that reaches s past the norm) may be NULL
 *   mean, rstd   [rows] f32, the forward's
 *   gamma        [cols], type pt, or NULL (1)
 *   dx           [rows][cols], type xt; may be dy, x or dsum itself
 *   dgamma, dbeta [cols] f32, both or neither NULL
 */
size_t dsmoe_layer_norm_backward_workspace_bytes(int64_t rows, int64_t cols);
dsmoe_status dsmoe_layer_norm_backward(const void* dy, int64_t lddy, const void* x, int64_t ldx,
                                       const void* dsum, int64_t ldds, int xt, const void* gamma, int pt,
                                       const float* mean, const float* rstd, int64_t rows, int64_t cols,
                                       void* dx, int64_t lddx, float* dgamma, float* dbeta,
                                       void* workspace, size_t ws_bytes, void* stream);

/*
 * dsmoe_linear -- z = x W^T + bias, y = act(z) + residual.
 *   x         [M][K] bf16
 *   w         [N][K] bf16
 *   bias      [N], type bt, or NULL
 *   residual  [M][N], type yt, or NULL
 *   y         [M][N], type yt (bf16 or f32); may be residual itself
 *   z         [M][N], type yt, or NULL: the pre-activation, for the backward
 * Products of bf16 values are exact and summed in float32; the epilogue is
 * float32 and each output is rounded once.
 */
size_t dsmoe_linear_workspace_bytes(const void* x, int64_t ldx, const void* w, int64_t ldw, int64_t M,
                                    int64_t N, int64_t K);
dsmoe_status dsmoe_linear(const void* x, int64_t ldx, const void* w, int64_t ldw, const void* bias, int bt,
                          const void* residual, int64_t ldr, int act, int64_t M, int64_t N, int64_t K,
                          void* y, int64_t ldy, int yt, void* z, int64_t ldz, void* workspace,
                          size_t ws_bytes, void* stream);

/*
 * dsmoe_linear_backward -- with dz = dy * act'(z):
 *   dx = dz W,  dw = dz^T x,  dbias = sum over rows of dz
 *   (the residual's gradient is dy itself)
 *   dy     [M][N] bf16
 *   x      [M][K], w [N][K] bf16: the forward's
 *   z      [M][N], type zt: the forward's; NULL only for DSMOE_ACT_NONE
 *   dx     [M][K], type dxt, or NULL
 *   dw     [N][K], type dwt, or NULL
 *   dbias  [N] f32, or NULL
 * Without an activation dz is dy and its products are exact.  With one dz is
 * formed in float32 (and dbias sums it so).  It enters a bf16 gradient rounded
 * to bf16, and a float32 gradient as the sum of two bf16 values, which keeps
 * 16 significant bits and takes a product for each.  With act |
 * DSMOE_DZ_BF16 it is rounded to bf16 for float32 gradients too.
 */
#define DSMOE_DZ_BF16 16
size_t dsmoe_linear_backward_workspace_bytes(const void* dy, int64_t lddy, const void* x, int64_t ldx,
                                             const void* w, int64_t ldw, int act, int64_t M, int64_t N,
                                             int64_t K);
dsmoe_status dsmoe_linear_backward(const void* dy, int64_t lddy, const void* x, int64_t ldx, const void* w,
                                   int64_t ldw, const void* z, int64_t ldz, int zt, int act, int64_t M,
                                   int64_t N, int64_t K, void* dx, int64_t lddx, int dxt, void* dw,
                                   int64_t lddw, int dwt, float* dbias, void* workspace, size_t ws_bytes,
                                   void* stream);

/*
 * dsmoe_gated_linear -- h = x W13^T = [g | u], a = act(g) * u, in one product:
 * h is written only where the caller wants it.
 *   x    [M][H] bf16
 *   w13  [2I][H] bf16: I gate rows, then I up rows
 *   a    [M][I], type at
 *   h    [M][2I] bf16, or NULL: the pre-activations, for the backward
 * act is one of SILU, GELU, RELU or NONE (a bilinear gate).
 */
size_t dsmoe_gated_linear_workspace_bytes(const void* x, int64_t ldx, const void* w13, int64_t ldw, int64_t M,
                                          int64_t H, int64_t I);
dsmoe_status dsmoe_gated_linear(const void* x, int64_t ldx, const void* w13, int64_t ldw, int act, int64_t M,
                                int64_t H, int64_t I, void* a, int64_t lda, int at, void* h, int64_t ldh,
                                void* workspace, size_t ws_bytes, void* stream);

/*
 * dsmoe_gated_linear_backward -- with dh = [da u act'(g) | da act(g)]:
 *   dx = dh W13,  dw13 = dh^T x
 *   da    [M][I] bf16
 *   x     [M][H], w13 [2I][H], h [M][2I] bf16: the forward's
 *   dx    [M][H], type dxt, or NULL
 *   dw13  [2I][H], type dwt, or NULL
 * dh is formed in float32 and enters the products as dz in
 * dsmoe_linear_backward, act | DSMOE_DZ_BF16 included.
 */
size_t dsmoe_gated_linear_backward_workspace_bytes(const void* x, int64_t ldx, const void* w13, int64_t ldw,
                                                   int64_t M, int64_t H, int64_t I);
dsmoe_status dsmoe_gated_linear_backward(const void* da, int64_t ldda, const void* x, int64_t ldx,
                                         const void* w13, int64_t ldw, const void* h, int64_t ldh, int act,
                                         int64_t M, int64_t H, int64_t I, void* dx, int64_t lddx, int dxt,
                                         void* dw13, int64_t lddw, int dwt, void* workspace, size_t ws_bytes,
                                         void* stream);

#ifdef __cplusplus
}
#endif

#endif /* DSMOE_DENSE_H */
