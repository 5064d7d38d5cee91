// Internal launchers of the routed experts' products outside FP8 (bf16 with
// gradients, 8-bit integers).  Called by experts_abi.hip after it has validated
// every argument.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dsmoe {

// Rows of an operand: row r is index[r] (null: r) of the n rows at p.
struct RowsOf {
  const void* p;
  int64_t ld;
  int64_t n;
  const int32_t* index;
  bool padded;               // rows are readable, and zero, up to a multiple of 16 bytes
};

// The groups: group g owns rows offsets[g] .. offsets[g + 1] - 1 of R (null: one
// group of all rows).
struct Groups {
  const int32_t* offsets;
  int32_t n;
  int64_t R;
};

enum class GroupedKind : int {
  kLinear = 0,   // y[r] = a[r] W_g^T, W_g [N][K]
  kGated = 1,    // [g | u] = a[r] W_g^T, W_g [2N][K]: y = scale act(g) u, z = [g | u]
  kDx = 2,       // y[r] = a[r] W_g, W_g [K][N]
  kDw = 3,       // y_g [N][K] = sum over the group's rows of a[r]^T b[r]
};

// N result columns (kDw: result rows), K the contraction (kDw: result columns)
struct GroupedGemm {
  GroupedKind kind;
  bool i8;                   // kLinear, kGated: integers with scales
  RowsOf a, b;               // b: kDw only
  const void* w;             // groups one after the other; not kDw
  int64_t ldw;
  Groups groups;
  int64_t N, K;
  int act;
  const float* row_scale;    // [R] or null; kGated
  const float* a_scale;      // i8: [a.n]
  const float* w_scale;      // i8: [groups][N] (kGated: [2N])
  // y (float32) += the result where y is finite (plus_rest); kDx, kDw.  The call
  // before had the same operands but for a's values, and a needs no copy: the other
  // operand's is in the workspace.
  bool add;
  void* y;
  int64_t ldy;
  bool y_f32;
  void* z;                   // kGated: [R][2N] bf16, or null
  int64_t ldz;
  void* workspace;           // grouped_gemm_workspace_bytes() bytes
};
size_t grouped_gemm_workspace_bytes(const GroupedGemm& p);
hipError_t launch_grouped_gemm(const GroupedGemm& p, hipStream_t s);
// The tile shape that a product takes (the index in kShapes; 4: the first, y by a
// block for each tile).
int grouped_gemm_shape(const GroupedGemm& p);

// Whether a row of `cols` values is made of whole aligned groups of 16 bytes.
bool rows_copyable(const RowsOf& o, int64_t cols, int bytes);

// grouped_grad.hip -------------------------------------------------------------
// dh = [s da u act'(g) | s da act(g)] as bf16 [R][lddh] from h = [g | u], what
// that rounding leaves of it in dh_lo (null: not wanted), and dscale[r] = sum over
// columns of da act(g) u (null: not wanted); dh null: only dscale.  s = scale[r]
// (null: 1).
struct GroupedGatedGrad {
  const uint16_t* da;
  int64_t ldda;
  const uint16_t* h;
  int64_t ldh;
  const float* scale;
  int act;
  Groups groups;
  int64_t I;
  uint16_t* dh;
  uint16_t* dh_lo;
  int64_t lddh;
  float* dscale;
};
hipError_t launch_grouped_gated_grad(const GroupedGatedGrad& p, hipStream_t s);

// dlogits [T][E] from the gates' gradients
hipError_t launch_router_grad(const float* dgate, const int32_t* topk, const float* logits, int64_t T, int32_t E,
                              int32_t K, float* dlogits, hipStream_t s);

// int8_quant.hip ---------------------------------------------------------------
hipError_t launch_quant_rows_int8(const void* x, int64_t ldx, bool f32, int64_t rows, int64_t cols, int8_t* q,
                                  int64_t ldq, float* scale, hipStream_t s);

}  // namespace dsmoe
