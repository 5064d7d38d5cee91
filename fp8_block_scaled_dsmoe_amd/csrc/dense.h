// Internal launchers of the dense feed-forward operators (layer norm, gated
// linear, linear).  Called by dense_abi.hip after it has validated every
// argument.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dsmoe {

// norm.hip -------------------------------------------------------------------
struct NormFwd {
  const void* x;
  int64_t ldx;
  const void* residual;   // or null
  int64_t ldr;
  bool x_f32;
  const void* gamma;      // or null
  const void* beta;       // or null
  bool p_f32;
  int64_t rows, cols;
  float eps;
  void* y;
  int64_t ldy;
  void* sum;              // or null
  int64_t lds;
  float* mean;            // or null
  float* rstd;            // or null
};
hipError_t launch_layer_norm(const NormFwd& p, hipStream_t s);

struct NormBwd {
  const void* dy;
  int64_t lddy;
  const void* x;
  int64_t ldx;
  const void* dsum;       // or null
  int64_t ldds;
  bool x_f32;
  const void* gamma;      // or null
  bool p_f32;
  const float* mean;
  const float* rstd;
  int64_t rows, cols;
  void* dx;
  int64_t lddx;
  float* dgamma;          // both or neither null
  float* dbeta;
  float* partial;         // layer_norm_backward_partial_floats() floats
};
size_t layer_norm_backward_partial_floats(int64_t rows, int64_t cols);
hipError_t launch_layer_norm_backward(const NormBwd& p, hipStream_t s);

// out[c] = sum over r < n of partial[r * cols + c], in a fixed order
hipError_t launch_sum_partials(const float* partial, int64_t n, int64_t cols, float* out, hipStream_t s);

// dense_gemm.hip -------------------------------------------------------------
// A bf16 matrix operand: element (r, k) -- r a row of the result's dimension,
// k the contraction index -- is p[r * ld + k], or p[k * ld + r] when k_rows.
struct Operand {
  const uint16_t* p;
  int64_t ld;
  bool k_rows;
  bool padded;            // rows are readable, and zero, up to a multiple of 8 values
};
// whether a row of `cols` values is made of whole aligned groups of 8
bool operand_copyable(const Operand& o, int64_t cols);

enum class DenseEpi : int {
  kLinear = 0,   // z = acc + bias, y = act(z) + residual
  kGated = 1,    // acc over [gate | up] rows of B: y = act(g) * u, z = [g | u]
};

struct DenseGemm {
  Operand a, b;           // a: M rows, b: N rows (kGated: 2 N rows, gate rows first)
  int64_t M, N, K;
  int64_t gate_n;         // kGated: rows of b (columns of z) from a gate to its up row: N of the whole product
  DenseEpi epi;
  int act;
  const void* bias;       // [N] or null
  bool bias_f32;
  const void* residual;   // [M][N], type of y, or null
  int64_t ldr;
  // the residual is the product of a's other part (vec8.h, plus_rest); no act, z or bias
  bool rest;
  void* y;                // [M][N]
  int64_t ldy;
  bool y_f32;
  void* z;                // or null.  kLinear: [M][N], type of y; kGated: [M][2N] bf16
  int64_t ldz;
  void* workspace;        // dense_gemm_workspace_bytes() bytes
};
size_t dense_gemm_workspace_bytes(const DenseGemm& p);
// The kernels that a product of at most 2^28 rows takes: few tokens (1) or
// tiles (0), then of its one or two launches of tiles the shape (the index in
// kShapes) and splits of K, and the first column of the second (0: none).
struct DenseKernels {
  int64_t few_tokens, shape, splits, cut, rest_shape, rest_splits;
};
DenseKernels dense_gemm_kernels(const DenseGemm& p);
hipError_t launch_dense_gemm(const DenseGemm& p, hipStream_t s);

// dense_skinny.hip: the same products for p.M <= 64 and both operands by rows;
// no workspace
hipError_t launch_dense_skinny(const DenseGemm& p, hipStream_t s);

// dst [M][N] (row stride ldd, type f32 / bf16) = 0
hipError_t launch_zero_matrix(void* dst, int64_t ldd, bool f32, int64_t m, int64_t n, hipStream_t s);

// dense_grad.hip -------------------------------------------------------------
// dz = dy * act'(z) as bf16 [M][lddz] (dz null: not wanted), what that rounding
// leaves of it as bf16 in dz_lo (null: not wanted), and its column sums over
// each of bias_partial_rows() strips of rows, partial [strips][N] (null: not
// wanted); z null: act' = 1
int64_t bias_partial_rows(int64_t M, int64_t N);
hipError_t launch_act_backward(const uint16_t* dy, int64_t lddy, const void* z, int64_t ldz, bool z_f32, int act,
                               int64_t M, int64_t N, uint16_t* dz, uint16_t* dz_lo, int64_t lddz, float* partial,
                               hipStream_t s);
// dh = [da u act'(g) | da act(g)] as bf16 [M][lddh] from h = [g | u], and in
// dh_lo as above
hipError_t launch_gated_backward(const uint16_t* da, int64_t ldda, const uint16_t* h, int64_t ldh, int act,
                                 int64_t M, int64_t I, uint16_t* dh, uint16_t* dh_lo, int64_t lddh, hipStream_t s);

}  // namespace dsmoe
