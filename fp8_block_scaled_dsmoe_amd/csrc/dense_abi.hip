// The extern "C" boundary of the dense feed-forward operators
// (dsmoe_dense.h): host-side validation, workspace layout and the order of
// the launches.  Nothing here allocates device memory.
#include <hip/hip_runtime.h>

#include <cmath>

#include "dense.h"
#include "dsmoe_dense.h"
#include "host.h"

namespace {

using dsmoe::aligned;
using dsmoe::check_device;
using dsmoe::DenseEpi;
using dsmoe::DenseGemm;
using dsmoe::kI32Max;
using dsmoe::launch_status;
using dsmoe::Operand;
using dsmoe::round_up;
using dsmoe::valid_dtype;

size_t esize(int t) { return t == DSMOE_F32 ? 4 : 2; }
bool rows_ok(int64_t n) { return n >= 0 && n <= kI32Max; }
bool dim_ok(int64_t n) { return n >= 1 && n <= DSMOE_DENSE_MAX_DIM; }
bool half_dim_ok(int64_t n) { return n >= 1 && n <= DSMOE_DENSE_MAX_DIM / 2; }
// a row stride, looked at only where its matrix is given
bool ld_ok(const void* p, int64_t ld, int64_t cols) { return !p || (ld >= cols && ld <= DSMOE_DENSE_MAX_DIM); }
bool el_aligned(const void* p, int t) { return !p || aligned(p, esize(t)); }
bool act_ok(int act) { return act >= DSMOE_ACT_NONE && act <= DSMOE_ACT_RELU; }
// act of a backward call
bool grad_act_ok(int act) { return act_ok(act & ~DSMOE_DZ_BF16); }
Operand operand(const void* p, int64_t ld, bool k_rows, bool padded = false) {
  return Operand{static_cast<const uint16_t*>(p), ld, k_rows, padded};
}

// Regions of a workspace, each 256-byte aligned.
struct Carver {
  size_t off = 0;
  size_t take(size_t bytes) {
    const size_t at = off;
    off = round_up(off + bytes, 256);
    return at;
  }
};

dsmoe_status check_workspace(const void* ws, size_t have, size_t need) {
  if (need == 0) return DSMOE_OK;
  if (!ws || have < need) return DSMOE_ERR_WORKSPACE;
  return aligned(ws, 256) ? DSMOE_OK : DSMOE_ERR_ALIGN;
}

// The products of the calls, without outputs and workspace.
DenseGemm forward_product(const void* x, int64_t ldx, const void* w, int64_t ldw, int64_t M, int64_t N, int64_t K,
                          DenseEpi epi) {
  DenseGemm g{};
  g.a = operand(x, ldx, false);
  g.b = operand(w, ldw, false);
  g.M = M, g.N = N, g.K = K, g.gate_n = N, g.epi = epi;
  return g;
}
// dx [M][K] = dz [M][N] w [N][K]
DenseGemm dx_product(const void* dz, int64_t lddz, bool padded, const void* w, int64_t ldw, int64_t M, int64_t N, int64_t K) {
  DenseGemm g{};
  g.a = operand(dz, lddz, false, padded);
  g.b = operand(w, ldw, true);
  g.M = M, g.N = K, g.K = N;
  return g;
}
// dw [N][K] = dz [M][N]^T x [M][K]
DenseGemm dw_product(const void* dz, int64_t lddz, bool padded, const void* x, int64_t ldx, int64_t M, int64_t N, int64_t K) {
  DenseGemm g{};
  g.a = operand(dz, lddz, true, padded);
  g.b = operand(x, ldx, true);
  g.M = N, g.N = K, g.K = M;
  return g;
}
void set_output(DenseGemm& g, void* y, int64_t ldy, int yt) {
  g.y = y;
  g.ldy = ldy;
  g.y_f32 = yt == DSMOE_F32;
}

// Workspace of the products of a backward pass, whose dz has N columns: dz
// (when it is not dy itself: an activation, or rows the products cannot copy),
// where `two` what its rounding to bf16 leaves, the bias partials, one
// product's scratch (they run one after the other).
struct BackwardLayout {
  size_t dz, dz_lo, partial, product, total;
  int64_t lddz;
  bool own_dz;
};
BackwardLayout backward_layout(const void* dy, int64_t lddy, bool act, bool two, bool bias, const void* x, int64_t ldx,
                               const void* w, int64_t ldw, int64_t M, int64_t N, int64_t K) {
  BackwardLayout L{};
  if (M == 0) return L;
  Carver c;
  const bool own_dz = L.own_dz = act || !dsmoe::operand_copyable(operand(dy, lddy, false), N);
  L.lddz = own_dz ? (N + 7) / 8 * 8 : lddy;
  if (own_dz) {
    L.dz = c.take(static_cast<size_t>(M) * L.lddz * 2);
    if (two) L.dz_lo = c.take(static_cast<size_t>(M) * L.lddz * 2);
    dy = nullptr;   // the workspace's own rows are aligned
  }
  if (bias && dsmoe::bias_partial_rows(M, N) > 1)
    L.partial = c.take(static_cast<size_t>(dsmoe::bias_partial_rows(M, N)) * N * 4);
  const size_t a = dsmoe::dense_gemm_workspace_bytes(dx_product(dy, L.lddz, own_dz, w, ldw, M, N, K));
  const size_t b = dsmoe::dense_gemm_workspace_bytes(dw_product(dy, L.lddz, own_dz, x, ldx, M, N, K));
  L.product = c.take(a > b ? a : b);
  L.total = c.off;
  return L;
}

// dx and dw from dz; M = 0 leaves dx alone and clears dw.  dz_lo: what dz's
// rounding left of it, or null; a float32 gradient adds its product.
dsmoe_status run_products(const void* dz, const void* dz_lo, int64_t lddz, bool padded, const void* x, int64_t ldx,
                          const void* w, int64_t ldw, int64_t M, int64_t N, int64_t K, void* dx, int64_t lddx, int dxt,
                          void* dw, int64_t lddw, int dwt, void* scratch, hipStream_t st) {
  if (M == 0) return dw ? launch_status(dsmoe::launch_zero_matrix(dw, lddw, dwt == DSMOE_F32, N, K, st)) : DSMOE_OK;
  auto gradient = [&](DenseGemm g, void* y, int64_t ldy, int yt) {
    set_output(g, y, ldy, yt);
    g.workspace = scratch;
    const hipError_t e = dsmoe::launch_dense_gemm(g, st);
    if (e != hipSuccess || yt != DSMOE_F32 || !dz_lo) return e;
    g.a.p = static_cast<const uint16_t*>(dz_lo);
    g.residual = y, g.ldr = ldy;
    return dsmoe::launch_dense_gemm(g, st);
  };
  hipError_t e = hipSuccess;
  if (dx) e = gradient(dx_product(dz, lddz, padded, w, ldw, M, N, K), dx, lddx, dxt);
  if (e == hipSuccess && dw) e = gradient(dw_product(dz, lddz, padded, x, ldx, M, N, K), dw, lddw, dwt);
  return launch_status(e);
}

// Whether a float32 gradient is wanted, whose dz keeps what its rounding leaves.
bool f32_gradient(const void* dx, int dxt, const void* dw, int dwt) {
  return (dx && dxt == DSMOE_F32) || (dw && dwt == DSMOE_F32);
}

}  // namespace

extern "C" {

// Not part of the interface: lets tests hold the sizes they use to the kernels
// they are for.  The kernels of one product of 16-byte rows: 0 y of
// dsmoe_linear, 1 its dx, 2 its dw (M, N, K as there), 3 dsmoe_gated_linear (N
// its I, K its H); the gated backward's are those of 1 and 2 with N = 2 I.
int dsmoe_dense_kernels(int product, int64_t M, int64_t N, int64_t K, int64_t out[6]) {
  if (product < 0 || product > 3 || M < 1 || M > (1 << 28) || !half_dim_ok(N) || !dim_ok(K)) return DSMOE_ERR_SHAPE;
  const int64_t ldn = round_up(N, 8), ldk = round_up(K, 8);
  DenseGemm g = product == 0   ? forward_product(nullptr, ldk, nullptr, ldk, M, N, K, DenseEpi::kLinear)
                : product == 1 ? dx_product(nullptr, ldn, true, nullptr, ldk, M, N, K)
                : product == 2 ? dw_product(nullptr, ldn, true, nullptr, ldk, M, N, K)
                               : forward_product(nullptr, ldk, nullptr, ldk, M, N, K, DenseEpi::kGated);
  g.a.padded = g.b.padded = true;
  const dsmoe::DenseKernels k = dsmoe::dense_gemm_kernels(g);
  const int64_t v[6] = {k.few_tokens, k.shape, k.splits, k.cut, k.rest_shape, k.rest_splits};
  for (int i = 0; i < 6; ++i) out[i] = v[i];
  return DSMOE_OK;
}

dsmoe_status dsmoe_layer_norm(const void* x, int64_t ldx, const void* residual, int64_t ldr, int xt,
                              const void* gamma, const void* beta, int pt, int64_t rows, int64_t cols,
                              float eps, void* y, int64_t ldy, void* sum, int64_t lds, float* mean,
                              float* rstd, void* stream) {
  if (!valid_dtype(xt) || !valid_dtype(pt)) return DSMOE_ERR_DTYPE;
  if (!rows_ok(rows) || !dim_ok(cols) || !(eps >= 0.0f) || !std::isfinite(eps)) return DSMOE_ERR_SHAPE;
  if (!ld_ok(x, ldx, cols) || !ld_ok(residual, ldr, cols) || !ld_ok(y, ldy, cols) || !ld_ok(sum, lds, cols))
    return DSMOE_ERR_SHAPE;
  if (rows == 0) return DSMOE_OK;
  if (!x || !y) return DSMOE_ERR_NULL;
  if (!el_aligned(x, xt) || !el_aligned(residual, xt) || !el_aligned(y, xt) || !el_aligned(sum, xt) ||
      !el_aligned(gamma, pt) || !el_aligned(beta, pt) || !aligned(mean, 4) || !aligned(rstd, 4))
    return DSMOE_ERR_ALIGN;
  const dsmoe_status ds = check_device();
  if (ds != DSMOE_OK) return ds;
  const dsmoe::NormFwd p{x,    ldx,  residual, ldr, xt == DSMOE_F32, gamma, beta, pt == DSMOE_F32, rows,
                         cols, eps, y,        ldy, sum,             lds,   mean, rstd};
  return launch_status(dsmoe::launch_layer_norm(p, static_cast<hipStream_t>(stream)));
}

size_t dsmoe_layer_norm_backward_workspace_bytes(int64_t rows, int64_t cols) {
  if (!rows_ok(rows) || !dim_ok(cols)) return 0;
  return round_up(dsmoe::layer_norm_backward_partial_floats(rows, cols) * 4, 256);
}

dsmoe_status dsmoe_layer_norm_backward(const void* dy, int64_t lddy, const void* x, int64_t ldx,
                                       const void* dsum, int64_t ldds, int xt, const void* gamma, int pt,
                                       const float* mean, const float* rstd, int64_t rows, int64_t cols,
                                       void* dx, int64_t lddx, float* dgamma, float* dbeta,
                                       void* workspace, size_t ws_bytes, void* stream) {
  if (!valid_dtype(xt) || !valid_dtype(pt)) return DSMOE_ERR_DTYPE;
  if (!rows_ok(rows) || !dim_ok(cols)) return DSMOE_ERR_SHAPE;
  if (!ld_ok(dy, lddy, cols) || !ld_ok(x, ldx, cols) || !ld_ok(dsum, ldds, cols) || !ld_ok(dx, lddx, cols))
    return DSMOE_ERR_SHAPE;
  if ((dgamma == nullptr) != (dbeta == nullptr)) return DSMOE_ERR_NULL;
  if (rows > 0 && (!dy || !x || !mean || !rstd || !dx)) return DSMOE_ERR_NULL;
  if (!el_aligned(dy, xt) || !el_aligned(x, xt) || !el_aligned(dsum, xt) || !el_aligned(dx, xt) ||
      !el_aligned(gamma, pt) || !aligned(mean, 4) || !aligned(rstd, 4) || !aligned(dgamma, 4) || !aligned(dbeta, 4))
    return DSMOE_ERR_ALIGN;
  if (rows == 0 && !dgamma) return DSMOE_OK;
  if (dgamma) {
    const dsmoe_status ws = check_workspace(workspace, ws_bytes, dsmoe_layer_norm_backward_workspace_bytes(rows, cols));
    if (ws != DSMOE_OK) return ws;
  }
  const dsmoe_status ds = check_device();
  if (ds != DSMOE_OK) return ds;
  const dsmoe::NormBwd p{dy,   lddy, x,    ldx,  dsum, ldds,   xt == DSMOE_F32, gamma,
                         pt == DSMOE_F32, mean, rstd, rows, cols, dx,     lddx,            dgamma,
                         dbeta, dgamma ? static_cast<float*>(workspace) : nullptr};
  return launch_status(dsmoe::launch_layer_norm_backward(p, static_cast<hipStream_t>(stream)));
}

size_t dsmoe_linear_workspace_bytes(const void* x, int64_t ldx, const void* w, int64_t ldw, int64_t M,
                                    int64_t N, int64_t K) {
  if (!rows_ok(M) || !dim_ok(N) || !dim_ok(K) || M == 0) return 0;
  return dsmoe::dense_gemm_workspace_bytes(forward_product(x, ldx, w, ldw, M, N, K, DenseEpi::kLinear));
}

dsmoe_status dsmoe_linear(const void* x, int64_t ldx, const void* w, int64_t ldw, const void* bias, int bt,
                          const void* residual, int64_t ldr, int act, int64_t M, int64_t N, int64_t K,
                          void* y, int64_t ldy, int yt, void* z, int64_t ldz, void* workspace,
                          size_t ws_bytes, void* stream) {
  if (!valid_dtype(yt) || !valid_dtype(bt)) return DSMOE_ERR_DTYPE;
  if (!rows_ok(M) || !dim_ok(N) || !dim_ok(K) || !act_ok(act)) return DSMOE_ERR_SHAPE;
  if (!ld_ok(x, ldx, K) || !ld_ok(w, ldw, K) || !ld_ok(residual, ldr, N) || !ld_ok(y, ldy, N) || !ld_ok(z, ldz, N))
    return DSMOE_ERR_SHAPE;
  if (M == 0) return DSMOE_OK;
  if (!x || !w || !y) return DSMOE_ERR_NULL;
  if (!aligned(x, 2) || !aligned(w, 2) || !el_aligned(bias, bt) || !el_aligned(residual, yt) || !el_aligned(y, yt) ||
      !el_aligned(z, yt))
    return DSMOE_ERR_ALIGN;
  DenseGemm g = forward_product(x, ldx, w, ldw, M, N, K, DenseEpi::kLinear);
  const dsmoe_status ws = check_workspace(workspace, ws_bytes, dsmoe::dense_gemm_workspace_bytes(g));
  if (ws != DSMOE_OK) return ws;
  const dsmoe_status ds = check_device();
  if (ds != DSMOE_OK) return ds;
  g.act = act;
  g.bias = bias, g.bias_f32 = bt == DSMOE_F32;
  g.residual = residual, g.ldr = ldr;
  set_output(g, y, ldy, yt);
  g.z = z, g.ldz = ldz;
  g.workspace = workspace;
  return launch_status(dsmoe::launch_dense_gemm(g, static_cast<hipStream_t>(stream)));
}

size_t dsmoe_linear_backward_workspace_bytes(const void* dy, int64_t lddy, const void* x, int64_t ldx,
                                             const void* w, int64_t ldw, int act, int64_t M, int64_t N,
                                             int64_t K) {
  if (!rows_ok(M) || !dim_ok(N) || !dim_ok(K) || !grad_act_ok(act) || M == 0) return 0;
  const bool has_act = (act & ~DSMOE_DZ_BF16) != DSMOE_ACT_NONE;
  return backward_layout(dy, lddy, has_act, has_act && !(act & DSMOE_DZ_BF16), true, x, ldx, w, ldw, M, N, K).total;
}

dsmoe_status dsmoe_linear_backward(const void* dy, int64_t lddy, const void* x, int64_t ldx, const void* w,
                                   int64_t ldw, const void* z, int64_t ldz, int zt, int act, int64_t M,
                                   int64_t N, int64_t K, void* dx, int64_t lddx, int dxt, void* dw,
                                   int64_t lddw, int dwt, float* dbias, void* workspace, size_t ws_bytes,
                                   void* stream) {
  if (!valid_dtype(zt) || !valid_dtype(dxt) || !valid_dtype(dwt)) return DSMOE_ERR_DTYPE;
  if (!rows_ok(M) || !dim_ok(N) || !dim_ok(K) || !grad_act_ok(act)) return DSMOE_ERR_SHAPE;
  const bool bf16_dz = act & DSMOE_DZ_BF16;
  act &= ~DSMOE_DZ_BF16;
  const bool has_act = act != DSMOE_ACT_NONE, two = has_act && !bf16_dz;
  if (!has_act) z = nullptr;
  if (!ld_ok(dy, lddy, N) || !ld_ok(x, ldx, K) || !ld_ok(w, ldw, K) || !ld_ok(z, ldz, N) || !ld_ok(dx, lddx, K) ||
      !ld_ok(dw, lddw, K))
    return DSMOE_ERR_SHAPE;
  if (M > 0 && (!dy || (has_act && !z) || (dx && !w) || (dw && !x))) return DSMOE_ERR_NULL;
  if (!aligned(dy, 2) || !aligned(x, 2) || !aligned(w, 2) || !el_aligned(z, zt) || !el_aligned(dx, dxt) ||
      !el_aligned(dw, dwt) || !aligned(dbias, 4))
    return DSMOE_ERR_ALIGN;
  if (!dx && !dw && !dbias) return DSMOE_OK;
  if (M == 0 && !dw && !dbias) return DSMOE_OK;
  const BackwardLayout L = backward_layout(dy, lddy, has_act, two, true, x, ldx, w, ldw, M, N, K);
  if (M > 0) {
    const dsmoe_status ws = check_workspace(workspace, ws_bytes, L.total);
    if (ws != DSMOE_OK) return ws;
  }
  const dsmoe_status ds = check_device();
  if (ds != DSMOE_OK) return ds;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  uint8_t* base = static_cast<uint8_t*>(workspace);
  const uint16_t* dz = static_cast<const uint16_t*>(dy);
  uint16_t* lo = two && f32_gradient(dx, dxt, dw, dwt) ? reinterpret_cast<uint16_t*>(base + L.dz_lo) : nullptr;
  if (M == 0) {
    if (dbias) {
      const hipError_t e = dsmoe::launch_zero_matrix(dbias, N, true, 1, N, st);
      if (e != hipSuccess) return launch_status(e);
    }
  } else if (dbias || L.own_dz) {
    uint16_t* to = L.own_dz && (dx || dw) ? reinterpret_cast<uint16_t*>(base + L.dz) : nullptr;
    const int64_t strips = dsmoe::bias_partial_rows(M, N);
    float* partial = dbias && strips > 1 ? reinterpret_cast<float*>(base + L.partial) : dbias;
    hipError_t e = dsmoe::launch_act_backward(dz, lddy, z, ldz, zt == DSMOE_F32, act, M, N, to, lo, L.lddz, partial, st);
    if (e == hipSuccess && partial != dbias) e = dsmoe::launch_sum_partials(partial, strips, N, dbias, st);
    if (e != hipSuccess) return launch_status(e);
    if (to) dz = to;
  }
  return run_products(dz, lo, L.lddz, L.own_dz, x, ldx, w, ldw, M, N, K, dx, lddx, dxt, dw, lddw, dwt, base + L.product,
                      st);
}

size_t dsmoe_gated_linear_workspace_bytes(const void* x, int64_t ldx, const void* w13, int64_t ldw, int64_t M,
                                          int64_t H, int64_t I) {
  if (!rows_ok(M) || !dim_ok(H) || !half_dim_ok(I) || M == 0) return 0;
  return dsmoe::dense_gemm_workspace_bytes(forward_product(x, ldx, w13, ldw, M, I, H, DenseEpi::kGated));
}

dsmoe_status dsmoe_gated_linear(const void* x, int64_t ldx, const void* w13, int64_t ldw, int act, int64_t M,
                                int64_t H, int64_t I, void* a, int64_t lda, int at, void* h, int64_t ldh,
                                void* workspace, size_t ws_bytes, void* stream) {
  if (!valid_dtype(at)) return DSMOE_ERR_DTYPE;
  if (!rows_ok(M) || !dim_ok(H) || !half_dim_ok(I) || !act_ok(act)) return DSMOE_ERR_SHAPE;
  if (!ld_ok(x, ldx, H) || !ld_ok(w13, ldw, H) || !ld_ok(a, lda, I) || !ld_ok(h, ldh, 2 * I)) return DSMOE_ERR_SHAPE;
  if (M == 0) return DSMOE_OK;
  if (!x || !w13 || !a) return DSMOE_ERR_NULL;
  if (!aligned(x, 2) || !aligned(w13, 2) || !el_aligned(a, at) || !aligned(h, 2)) return DSMOE_ERR_ALIGN;
  DenseGemm g = forward_product(x, ldx, w13, ldw, M, I, H, DenseEpi::kGated);
  const dsmoe_status ws = check_workspace(workspace, ws_bytes, dsmoe::dense_gemm_workspace_bytes(g));
  if (ws != DSMOE_OK) return ws;
  const dsmoe_status ds = check_device();
  if (ds != DSMOE_OK) return ds;
  g.act = act;
  set_output(g, a, lda, at);
  g.z = h, g.ldz = ldh;
  g.workspace = workspace;
  return launch_status(dsmoe::launch_dense_gemm(g, static_cast<hipStream_t>(stream)));
}

size_t dsmoe_gated_linear_backward_workspace_bytes(const void* x, int64_t ldx, const void* w13, int64_t ldw,
                                                   int64_t M, int64_t H, int64_t I) {
  if (!rows_ok(M) || !dim_ok(H) || !half_dim_ok(I) || M == 0) return 0;
  return backward_layout(nullptr, 0, true, true, false, x, ldx, w13, ldw, M, 2 * I, H).total;
}

dsmoe_status dsmoe_gated_linear_backward(const void* da, int64_t ldda, const void* x, int64_t ldx,
                                         const void* w13, int64_t ldw, const void* h, int64_t ldh, int act,
                                         int64_t M, int64_t H, int64_t I, void* dx, int64_t lddx, int dxt,
                                         void* dw13, int64_t lddw, int dwt, void* workspace, size_t ws_bytes,
                                         void* stream) {
  if (!valid_dtype(dxt) || !valid_dtype(dwt)) return DSMOE_ERR_DTYPE;
  if (!rows_ok(M) || !dim_ok(H) || !half_dim_ok(I) || !grad_act_ok(act)) return DSMOE_ERR_SHAPE;
  const bool two = !(act & DSMOE_DZ_BF16);
  act &= ~DSMOE_DZ_BF16;
  if (!ld_ok(da, ldda, I) || !ld_ok(x, ldx, H) || !ld_ok(w13, ldw, H) || !ld_ok(h, ldh, 2 * I) ||
      !ld_ok(dx, lddx, H) || !ld_ok(dw13, lddw, H))
    return DSMOE_ERR_SHAPE;
  if (M > 0 && (!da || !h || (dx && !w13) || (dw13 && !x))) return DSMOE_ERR_NULL;
  if (!aligned(da, 2) || !aligned(x, 2) || !aligned(w13, 2) || !aligned(h, 2) || !el_aligned(dx, dxt) ||
      !el_aligned(dw13, dwt))
    return DSMOE_ERR_ALIGN;
  if ((!dx && !dw13) || (M == 0 && !dw13)) return DSMOE_OK;
  const BackwardLayout L = backward_layout(nullptr, 0, true, two, false, x, ldx, w13, ldw, M, 2 * I, H);
  if (M > 0) {
    const dsmoe_status ws = check_workspace(workspace, ws_bytes, L.total);
    if (ws != DSMOE_OK) return ws;
  }
  const dsmoe_status ds = check_device();
  if (ds != DSMOE_OK) return ds;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  uint8_t* base = static_cast<uint8_t*>(workspace);
  uint16_t* dh = reinterpret_cast<uint16_t*>(base + L.dz);
  uint16_t* lo = two && f32_gradient(dx, dxt, dw13, dwt) ? reinterpret_cast<uint16_t*>(base + L.dz_lo) : nullptr;
  const hipError_t e = dsmoe::launch_gated_backward(static_cast<const uint16_t*>(da), ldda,
                                                    static_cast<const uint16_t*>(h), ldh, act, M, I, dh, lo, L.lddz, st);
  if (e != hipSuccess) return launch_status(e);
  return run_products(dh, lo, L.lddz, true, x, ldx, w13, ldw, M, 2 * I, H, dx, lddx, dxt, dw13, lddw, dwt,
                      base + L.product, st);
}

}  // extern "C"
