// The extern "C" boundary of the routed experts' products outside FP8
// (dsmoe_experts.h): host-side validation, workspace layout and the order of the
// launches.  Nothing here allocates device memory.
#include <hip/hip_runtime.h>

#include "dense.h"
#include "dsmoe_experts.h"
#include "grouped.h"
#include "grouped_walk.h"
#include "host.h"

namespace {

using dsmoe::aligned;
using dsmoe::check_device;
using dsmoe::GroupedGemm;
using dsmoe::GroupedKind;
using dsmoe::Groups;
using dsmoe::kI32Max;
using dsmoe::launch_status;
using dsmoe::round_up;
using dsmoe::RowsOf;
using dsmoe::valid_dtype;

size_t esize(int t) { return t == DSMOE_F32 ? 4 : 2; }
bool rows_ok(int64_t n) { return n >= 0 && n <= kI32Max; }
bool dim_ok(int64_t n) { return n >= 1 && n <= DSMOE_DENSE_MAX_DIM; }
bool half_dim_ok(int64_t n) { return n >= 1 && n <= DSMOE_DENSE_MAX_DIM / 2; }
bool groups_ok(int32_t G) { return G >= 1 && G <= DSMOE_MAX_EXPERTS; }
// source rows of an operand of R rows
bool source_ok(int64_t n, const int32_t* rows, int64_t R) { return rows_ok(n) && (R == 0 || (rows ? n > 0 : n == R)); }
// a row stride, looked at only where its matrix is given
bool ld_ok(const void* p, int64_t ld, int64_t cols) { return !p || (ld >= cols && ld <= DSMOE_DENSE_MAX_DIM); }
bool el_aligned(const void* p, int t) { return !p || aligned(p, esize(t)); }
// no more elements than a card can hold, which keeps the numbers of tiles in 32 bits
bool fits(int64_t G, int64_t R, int64_t N, int64_t K) {
  constexpr int64_t kMost = int64_t{1} << 40;
  return G * N <= kMost / K && (R == 0 || (N <= kMost / R && K <= kMost / R));
}
bool act_ok(int act) { return act >= DSMOE_ACT_NONE && act <= DSMOE_ACT_RELU; }
bool grad_act_ok(int act) { return act_ok(act & ~DSMOE_DZ_BF16); }

dsmoe_status check_workspace(const void* ws, size_t have, size_t need) {
  if (need == 0) return DSMOE_OK;
  if (!ws || have < need) return DSMOE_ERR_WORKSPACE;
  return aligned(ws, 256) ? DSMOE_OK : DSMOE_ERR_ALIGN;
}

RowsOf rows_of(const void* p, int64_t ld, int64_t n, const int32_t* index, bool padded = false) {
  return RowsOf{p, ld, n, index, padded};
}

// The products of the calls, without outputs and workspace.
GroupedGemm row_product(GroupedKind kind, bool i8, const RowsOf& a, const void* w, int64_t ldw, const Groups& g,
                        int64_t N, int64_t K) {
  GroupedGemm p{};
  p.kind = kind;
  p.i8 = i8;
  p.a = a;
  p.w = w, p.ldw = ldw;
  p.groups = g;
  p.N = N, p.K = K;
  return p;
}
GroupedGemm dw_product(const RowsOf& a, const RowsOf& b, const Groups& g, int64_t N, int64_t K) {
  GroupedGemm p{};
  p.kind = GroupedKind::kDw;
  p.a = a, p.b = b;
  p.groups = g;
  p.N = N, p.K = K;
  return p;
}
void set_output(GroupedGemm& p, void* y, int64_t ldy, int yt) {
  p.y = y;
  p.ldy = ldy;
  p.y_f32 = yt == DSMOE_F32;
}

// dx = dy W and dw = dy^T x by the groups; lo: what the rounding of dy to bf16
// left, or null: a float32 gradient adds its product.
dsmoe_status run_gradients(const RowsOf& dy, const void* lo, const RowsOf& x, const void* w, int64_t ldw,
                           const Groups& g, int64_t N, int64_t K, void* dx, int64_t lddx, int dxt, void* dw,
                           int64_t lddw, int dwt, void* scratch, hipStream_t st) {
  auto run = [&](GroupedGemm p, void* y, int64_t ldy, int yt) {
    set_output(p, y, ldy, yt);
    p.workspace = scratch;
    const hipError_t e = dsmoe::launch_grouped_gemm(p, st);
    if (e != hipSuccess || yt != DSMOE_F32 || !lo) return e;
    p.a.p = lo;
    p.add = true;
    return dsmoe::launch_grouped_gemm(p, st);
  };
  hipError_t e = hipSuccess;
  if (dx) e = run(row_product(GroupedKind::kDx, false, dy, w, ldw, g, K, N), dx, lddx, dxt);
  if (e == hipSuccess && dw) e = run(dw_product(dy, x, g, N, K), dw, lddw, dwt);
  return launch_status(e);
}
size_t gradients_bytes(const RowsOf& dy, const RowsOf& x, const void* w, int64_t ldw, const Groups& g, int64_t N,
                       int64_t K) {
  const size_t a = dsmoe::grouped_gemm_workspace_bytes(row_product(GroupedKind::kDx, false, dy, w, ldw, g, K, N));
  const size_t b = dsmoe::grouped_gemm_workspace_bytes(dw_product(dy, x, g, N, K));
  return a > b ? a : b;
}

// Workspace of the gated backward: dh, what its rounding leaves, a product's.
struct GatedLayout {
  size_t dh, lo, product, total;
  int64_t lddh;
};
GatedLayout gated_layout(const void* x, int64_t ldx, int64_t n, const int32_t* rows, const void* w13, int64_t ldw,
                         int32_t G, int64_t R, int64_t H, int64_t I) {
  GatedLayout L{};
  if (R == 0) return L;
  L.lddh = static_cast<int64_t>(round_up(2 * I, 8));
  const size_t one = round_up(static_cast<size_t>(R) * L.lddh * 2, 256);
  L.lo = one;
  L.product = 2 * one;
  const Groups g{nullptr, G, R};
  L.total = L.product + gradients_bytes(rows_of(nullptr, L.lddh, R, nullptr, true), rows_of(x, ldx, n, rows), w13, ldw,
                                        g, 2 * I, H);
  return L;
}

dsmoe_status linear_call(bool i8, const void* x, int64_t ldx, const float* x_scale, int64_t n, const int32_t* rows,
                         const void* w, int64_t ldw, const float* w_scale, bool gated, const float* row_scale, int act,
                         const int32_t* offsets, int32_t G, int64_t R, int64_t N, int64_t K, void* y, int64_t ldy,
                         int yt, void* z, int64_t ldz, void* workspace, size_t ws_bytes, void* stream) {
  if (!valid_dtype(yt)) return DSMOE_ERR_DTYPE;
  if (!groups_ok(G) || !rows_ok(R) || !source_ok(n, rows, R) || !(gated ? half_dim_ok(N) : dim_ok(N)) || !dim_ok(K) ||
      !act_ok(act) || (i8 && K >= DSMOE_INT8_MAX_K) || (!offsets && G != 1) || !fits(G, R, gated ? 2 * N : N, K))
    return DSMOE_ERR_SHAPE;
  if (!ld_ok(x, ldx, K) || !ld_ok(w, ldw, K) || !ld_ok(y, ldy, N) || !ld_ok(z, ldz, 2 * N)) return DSMOE_ERR_SHAPE;
  if (R == 0) return DSMOE_OK;
  if (!x || !w || !y || (i8 && (!x_scale || !w_scale))) return DSMOE_ERR_NULL;
  const size_t es = i8 ? 1 : 2;
  if (!aligned(x, es) || !aligned(w, es) || !el_aligned(y, yt) || !aligned(z, 2) || !aligned(rows, 4) ||
      !aligned(offsets, 4) || !aligned(row_scale, 4) || !aligned(x_scale, 4) || !aligned(w_scale, 4))
    return DSMOE_ERR_ALIGN;
  GroupedGemm p = row_product(gated ? GroupedKind::kGated : GroupedKind::kLinear, i8, rows_of(x, ldx, n, rows), w, ldw,
                              Groups{offsets, G, R}, N, K);
  const dsmoe_status ws = check_workspace(workspace, ws_bytes, dsmoe::grouped_gemm_workspace_bytes(p));
  if (ws != DSMOE_OK) return ws;
  const dsmoe_status ds = check_device();
  if (ds != DSMOE_OK) return ds;
  p.act = act;
  p.row_scale = row_scale;
  p.a_scale = x_scale, p.w_scale = w_scale;
  set_output(p, y, ldy, yt);
  p.z = z, p.ldz = ldz;
  p.workspace = workspace;
  return launch_status(dsmoe::launch_grouped_gemm(p, static_cast<hipStream_t>(stream)));
}

size_t linear_bytes(bool i8, bool gated, const void* x, int64_t ldx, int64_t n, const int32_t* rows, const void* w,
                    int64_t ldw, int32_t G, int64_t R, int64_t N, int64_t K) {
  if (!groups_ok(G) || !rows_ok(R) || !source_ok(n, rows, R) || !(gated ? half_dim_ok(N) : dim_ok(N)) || !dim_ok(K) ||
      !fits(G, R, gated ? 2 * N : N, K))
    return 0;
  return dsmoe::grouped_gemm_workspace_bytes(row_product(gated ? GroupedKind::kGated : GroupedKind::kLinear, i8,
                                                         rows_of(x, ldx, n, rows), w, ldw, Groups{nullptr, G, R}, N, K));
}

}  // namespace

extern "C" {

// Not part of the interface: lets tests hold the sizes they use to the kernels
// they are for.  The tile shape (0: 256 x 256, 1: 128 x 128, 2: 64 x 64, 3: 32 x 128,
// 4: 256 x 256 where y takes a block for each tile instead of blocks that stay)
// of R aligned rows in G groups: product 0 y of dsmoe_grouped_linear, 1 its dx, 2
// its dw (N, K as there), 3 dsmoe_grouped_gated_linear (N its I, K its H), 4 and 5
// the 8-bit forms of 0 and 3.
int dsmoe_grouped_shape(int product, int32_t G, int64_t R, int64_t N, int64_t K) {
  if (product < 0 || product > 5 || !groups_ok(G) || R < 1 || !rows_ok(R) || !half_dim_ok(N) || !dim_ok(K) ||
      !fits(G, R, 2 * N, K))
    return -1;
  const RowsOf a = rows_of(nullptr, round_up(product == 1 || product == 2 ? N : K, 16), R, nullptr, true);
  const RowsOf b = rows_of(nullptr, round_up(K, 16), R, nullptr, true);
  const Groups g{nullptr, G, R};
  const int64_t ld = round_up(K, 16);
  switch (product) {
    case 1: return dsmoe::grouped_gemm_shape(row_product(GroupedKind::kDx, false, a, nullptr, ld, g, K, N));
    case 2: return dsmoe::grouped_gemm_shape(dw_product(a, b, g, N, K));
    case 0:
    case 4: return dsmoe::grouped_gemm_shape(row_product(GroupedKind::kLinear, product == 4, a, nullptr, ld, g, N, K));
    default: return dsmoe::grouped_gemm_shape(row_product(GroupedKind::kGated, product == 5, a, nullptr, ld, g, N, K));
  }
}

// Not part of the interface: the tiles that block `block` of `blocks` blocks that stay
// takes, in their order, for y [R][N] (dw 0) or dw [N][K] of bf16 operands, from
// offsets in host memory (NULL: one group): group, m0, m_end, n0, k0, k1 and chunks of
// the first `most`.  Returns their number, or -1.
int64_t dsmoe_grouped_walk(int dw, const int32_t* offsets, int32_t G, int64_t R, int64_t N, int64_t K, uint32_t block,
                           uint32_t blocks, int32_t* out, int64_t most) {
  constexpr int kRows = 256, kCols = 256, kChunk = 64;
  constexpr uint32_t kXcds = 8;
  if (!groups_ok(G) || !rows_ok(R) || !dim_ok(N) || !dim_ok(K) || !fits(G, R, N, K) || (!offsets && G != 1) ||
      blocks == 0 || blocks % kXcds != 0 || block >= blocks)
    return -1;
  int32_t begin[DSMOE_MAX_EXPERTS], end[DSMOE_MAX_EXPERTS], first[DSMOE_MAX_EXPERTS + 1];
  auto clamped = [&](int32_t v) { return v < 0 ? 0 : v > R ? static_cast<int32_t>(R) : v; };
  uint32_t before = 0;
  for (int32_t g = 0; g < G; ++g) {
    begin[g] = offsets ? clamped(offsets[g]) : 0;
    end[g] = offsets ? clamped(offsets[g + 1]) : static_cast<int32_t>(R);
    if (end[g] < begin[g]) end[g] = begin[g];
    first[g] = static_cast<int32_t>(before);
    before += (static_cast<uint32_t>(end[g] - begin[g]) + kRows - 1) / kRows;
  }
  first[G] = static_cast<int32_t>(before);
  const int64_t cols = dw ? K : N;
  const dsmoe::StreamSizes s{G, static_cast<int32_t>(N), static_cast<int32_t>((K + kChunk - 1) / kChunk),
                             static_cast<uint32_t>((N + kRows - 1) / kRows), static_cast<uint32_t>((cols + kCols - 1) / kCols)};
  auto read = [](const int32_t& v) { return v; };
  uint32_t tile = dsmoe::first_stream_tile(block, blocks, kXcds);
  int32_t walk = 0;
  dsmoe::StreamTile d{};
  int64_t n = 0;
  while (dw ? dsmoe::next_stream_tile<true, kRows, kCols, kChunk>(s, begin, end, first, blocks, tile, walk, read, d)
            : dsmoe::next_stream_tile<false, kRows, kCols, kChunk>(s, begin, end, first, blocks, tile, walk, read, d)) {
    const int32_t v[7] = {d.group, d.m0, d.m_end, d.n0, d.k0, d.k1, d.chunks};
    if (n < most)
      for (int i = 0; i < 7; ++i) out[7 * n + i] = v[i];
    ++n;
  }
  return n;
}
// Not part of the interface: the tiles that the copies may have entered past the
// products' tile, which the queue of those blocks is sized by.
int dsmoe_grouped_walk_ahead(void) { return dsmoe::kStreamAhead; }

size_t dsmoe_grouped_linear_workspace_bytes(const void* x, int64_t ldx, int64_t n, const int32_t* rows,
                                            const void* w, int64_t ldw, int32_t G, int64_t R, int64_t N, int64_t K) {
  return linear_bytes(false, false, x, ldx, n, rows, w, ldw, G, R, N, K);
}
dsmoe_status dsmoe_grouped_linear(const void* x, int64_t ldx, int64_t n, const int32_t* rows, const void* w,
                                  int64_t ldw, const int32_t* offsets, int32_t G, int64_t R, int64_t N, int64_t K,
                                  void* y, int64_t ldy, int yt, void* workspace, size_t ws_bytes, void* stream) {
  return linear_call(false, x, ldx, nullptr, n, rows, w, ldw, nullptr, false, nullptr, DSMOE_ACT_NONE, offsets, G, R,
                     N, K, y, ldy, yt, nullptr, 0, workspace, ws_bytes, stream);
}

size_t dsmoe_grouped_linear_backward_workspace_bytes(const void* dy, int64_t lddy, int64_t n_dy,
                                                     const int32_t* dy_rows, const void* x, int64_t ldx, int64_t n,
                                                     const int32_t* rows, const void* w, int64_t ldw, int32_t G,
                                                     int64_t R, int64_t N, int64_t K) {
  if (!groups_ok(G) || !rows_ok(R) || !source_ok(n, rows, R) || !source_ok(n_dy, dy_rows, R) || !dim_ok(N) ||
      !dim_ok(K) || !fits(G, R, N, K) || R == 0)
    return 0;
  return gradients_bytes(rows_of(dy, lddy, n_dy, dy_rows), rows_of(x, ldx, n, rows), w, ldw, Groups{nullptr, G, R}, N,
                         K);
}
dsmoe_status dsmoe_grouped_linear_backward(const void* dy, int64_t lddy, int64_t n_dy, const int32_t* dy_rows,
                                           const void* x, int64_t ldx, int64_t n, const int32_t* rows, const void* w,
                                           int64_t ldw, const int32_t* offsets, int32_t G, int64_t R, int64_t N,
                                           int64_t K, void* dx, int64_t lddx, int dxt, void* dw, int64_t lddw,
                                           int dwt, void* workspace, size_t ws_bytes, void* stream) {
  if (!valid_dtype(dxt) || !valid_dtype(dwt)) return DSMOE_ERR_DTYPE;
  if (!groups_ok(G) || !rows_ok(R) || !source_ok(n, rows, R) || !source_ok(n_dy, dy_rows, R) || !dim_ok(N) ||
      !dim_ok(K) || (!offsets && G != 1) || !fits(G, R, N, K))
    return DSMOE_ERR_SHAPE;
  if (!ld_ok(dy, lddy, N) || !ld_ok(x, ldx, K) || !ld_ok(w, ldw, K) || !ld_ok(dx, lddx, K) || !ld_ok(dw, lddw, K))
    return DSMOE_ERR_SHAPE;
  if (R > 0 && (!dy || (dx && !w) || (dw && !x))) return DSMOE_ERR_NULL;
  if (!aligned(dy, 2) || !aligned(x, 2) || !aligned(w, 2) || !el_aligned(dx, dxt) || !el_aligned(dw, dwt) ||
      !aligned(rows, 4) || !aligned(dy_rows, 4) || !aligned(offsets, 4))
    return DSMOE_ERR_ALIGN;
  if ((!dx && !dw) || (R == 0 && !dw)) return DSMOE_OK;
  const Groups g{offsets, G, R};
  const RowsOf d = rows_of(dy, lddy, n_dy, dy_rows), xr = rows_of(x, ldx, n, rows);
  if (R > 0) {
    const dsmoe_status ws = check_workspace(workspace, ws_bytes, gradients_bytes(d, xr, w, ldw, g, N, K));
    if (ws != DSMOE_OK) return ws;
  }
  const dsmoe_status ds = check_device();
  if (ds != DSMOE_OK) return ds;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  if (R == 0) return launch_status(dsmoe::launch_zero_matrix(dw, lddw, dwt == DSMOE_F32, G * N, K, st));
  return run_gradients(d, nullptr, xr, w, ldw, g, N, K, dx, lddx, dxt, dw, lddw, dwt, workspace, st);
}

size_t dsmoe_grouped_gated_linear_workspace_bytes(const void* x, int64_t ldx, int64_t n, const int32_t* rows,
                                                  const void* w13, int64_t ldw, int32_t G, int64_t R, int64_t H,
                                                  int64_t I) {
  return linear_bytes(false, true, x, ldx, n, rows, w13, ldw, G, R, I, H);
}
dsmoe_status dsmoe_grouped_gated_linear(const void* x, int64_t ldx, int64_t n, const int32_t* rows, const void* w13,
                                        int64_t ldw, const float* row_scale, int act, const int32_t* offsets,
                                        int32_t G, int64_t R, int64_t H, int64_t I, void* a, int64_t lda, int at,
                                        void* h, int64_t ldh, void* workspace, size_t ws_bytes, void* stream) {
  return linear_call(false, x, ldx, nullptr, n, rows, w13, ldw, nullptr, true, row_scale, act, offsets, G, R, I, H, a,
                     lda, at, h, ldh, workspace, ws_bytes, stream);
}

size_t dsmoe_grouped_gated_linear_backward_workspace_bytes(const void* x, int64_t ldx, int64_t n,
                                                           const int32_t* rows, const void* w13, int64_t ldw,
                                                           int32_t G, int64_t R, int64_t H, int64_t I) {
  if (!groups_ok(G) || !rows_ok(R) || !source_ok(n, rows, R) || !dim_ok(H) || !half_dim_ok(I) || !fits(G, R, 2 * I, H))
    return 0;
  return gated_layout(x, ldx, n, rows, w13, ldw, G, R, H, I).total;
}
dsmoe_status dsmoe_grouped_gated_linear_backward(const void* da, int64_t ldda, const void* x, int64_t ldx, int64_t n,
                                                 const int32_t* rows, const void* w13, int64_t ldw, const void* h,
                                                 int64_t ldh, const float* row_scale, int act, const int32_t* offsets,
                                                 int32_t G, int64_t R, int64_t H, int64_t I, void* dx, int64_t lddx,
                                                 int dxt, void* dw13, int64_t lddw, int dwt, float* dscale,
                                                 void* workspace, size_t ws_bytes, void* stream) {
  if (!valid_dtype(dxt) || !valid_dtype(dwt)) return DSMOE_ERR_DTYPE;
  if (!groups_ok(G) || !rows_ok(R) || !source_ok(n, rows, R) || !dim_ok(H) || !half_dim_ok(I) || !grad_act_ok(act) ||
      (!offsets && G != 1) || !fits(G, R, 2 * I, H))
    return DSMOE_ERR_SHAPE;
  const bool two = !(act & DSMOE_DZ_BF16);
  act &= ~DSMOE_DZ_BF16;
  if (!ld_ok(da, ldda, I) || !ld_ok(x, ldx, H) || !ld_ok(w13, ldw, H) || !ld_ok(h, ldh, 2 * I) ||
      !ld_ok(dx, lddx, H) || !ld_ok(dw13, lddw, H))
    return DSMOE_ERR_SHAPE;
  if (R > 0 && (!da || !h || (dx && !w13) || (dw13 && !x))) return DSMOE_ERR_NULL;
  if (!aligned(da, 2) || !aligned(x, 2) || !aligned(w13, 2) || !aligned(h, 2) || !el_aligned(dx, dxt) ||
      !el_aligned(dw13, dwt) || !aligned(rows, 4) || !aligned(offsets, 4) || !aligned(row_scale, 4) ||
      !aligned(dscale, 4))
    return DSMOE_ERR_ALIGN;
  if ((!dx && !dw13 && !dscale) || (R == 0 && !dw13)) return DSMOE_OK;
  const Groups g{offsets, G, R};
  const GatedLayout L = gated_layout(x, ldx, n, rows, w13, ldw, G, R, H, I);
  const bool products = dx || dw13;
  if (R > 0 && products) {
    const dsmoe_status ws = check_workspace(workspace, ws_bytes, L.total);
    if (ws != DSMOE_OK) return ws;
  }
  const dsmoe_status ds = check_device();
  if (ds != DSMOE_OK) return ds;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  if (R == 0) return launch_status(dsmoe::launch_zero_matrix(dw13, lddw, dwt == DSMOE_F32, G * 2 * I, H, st));
  uint8_t* base = static_cast<uint8_t*>(workspace);
  const bool f32 = (dx && dxt == DSMOE_F32) || (dw13 && dwt == DSMOE_F32);
  uint16_t* dh = products ? reinterpret_cast<uint16_t*>(base + L.dh) : nullptr;
  uint16_t* lo = products && two && f32 ? reinterpret_cast<uint16_t*>(base + L.lo) : nullptr;
  const hipError_t e = dsmoe::launch_grouped_gated_grad(
      dsmoe::GroupedGatedGrad{static_cast<const uint16_t*>(da), ldda, static_cast<const uint16_t*>(h), ldh, row_scale,
                              act, g, I, dh, lo, L.lddh, dscale},
      st);
  if (e != hipSuccess || !products) return launch_status(e);
  return run_gradients(rows_of(dh, L.lddh, R, nullptr, true), lo, rows_of(x, ldx, n, rows), w13, ldw, g, 2 * I, H, dx,
                       lddx, dxt, dw13, lddw, dwt, base + L.product, st);
}

dsmoe_status dsmoe_router_backward(const float* dgate, const int32_t* topk_idx, const float* logits, int64_t T,
                                   int32_t E, int32_t K, float* dlogits, void* stream) {
  if (!rows_ok(T) || E < 1 || E > DSMOE_MAX_EXPERTS || K < 1 || K > DSMOE_MAX_TOPK || K > E) return DSMOE_ERR_SHAPE;
  if (T == 0) return DSMOE_OK;
  if (!dgate || !topk_idx || !logits || !dlogits) return DSMOE_ERR_NULL;
  if (!aligned(dgate, 4) || !aligned(topk_idx, 4) || !aligned(logits, 4) || !aligned(dlogits, 4))
    return DSMOE_ERR_ALIGN;
  const dsmoe_status ds = check_device();
  if (ds != DSMOE_OK) return ds;
  return launch_status(dsmoe::launch_router_grad(dgate, topk_idx, logits, T, E, K, dlogits,
                                                 static_cast<hipStream_t>(stream)));
}

dsmoe_status dsmoe_quant_rows_int8(const void* x, int64_t ldx, int xt, int64_t rows, int64_t cols, int8_t* q,
                                   int64_t ldq, float* scale, void* stream) {
  if (!valid_dtype(xt)) return DSMOE_ERR_DTYPE;
  if (!rows_ok(rows) || !dim_ok(cols) || !ld_ok(x, ldx, cols) || !ld_ok(q, ldq, cols)) return DSMOE_ERR_SHAPE;
  if (rows == 0) return DSMOE_OK;
  if (!x || !q || !scale) return DSMOE_ERR_NULL;
  if (!el_aligned(x, xt) || !aligned(scale, 4)) return DSMOE_ERR_ALIGN;
  const dsmoe_status ds = check_device();
  if (ds != DSMOE_OK) return ds;
  return launch_status(dsmoe::launch_quant_rows_int8(x, ldx, xt == DSMOE_F32, rows, cols, q, ldq, scale,
                                                     static_cast<hipStream_t>(stream)));
}

size_t dsmoe_int8_linear_workspace_bytes(const int8_t* x, int64_t ldx, int64_t n, const int32_t* rows,
                                         const int8_t* w, int64_t ldw, int32_t G, int64_t R, int64_t N, int64_t K) {
  return linear_bytes(true, false, x, ldx, n, rows, w, ldw, G, R, N, K);
}
dsmoe_status dsmoe_int8_linear(const int8_t* x, int64_t ldx, const float* x_scale, int64_t n, const int32_t* rows,
                               const int8_t* w, int64_t ldw, const float* w_scale, const int32_t* offsets, int32_t G,
                               int64_t R, int64_t N, int64_t K, void* y, int64_t ldy, int yt, void* workspace,
                               size_t ws_bytes, void* stream) {
  return linear_call(true, x, ldx, x_scale, n, rows, w, ldw, w_scale, false, nullptr, DSMOE_ACT_NONE, offsets, G, R, N,
                     K, y, ldy, yt, nullptr, 0, workspace, ws_bytes, stream);
}

size_t dsmoe_int8_gated_linear_workspace_bytes(const int8_t* x, int64_t ldx, int64_t n, const int32_t* rows,
                                               const int8_t* w13, int64_t ldw, int32_t G, int64_t R, int64_t H,
                                               int64_t I) {
  return linear_bytes(true, true, x, ldx, n, rows, w13, ldw, G, R, I, H);
}
dsmoe_status dsmoe_int8_gated_linear(const int8_t* x, int64_t ldx, const float* x_scale, int64_t n,
                                     const int32_t* rows, const int8_t* w13, int64_t ldw, const float* w13_scale,
                                     const float* row_scale, int act, const int32_t* offsets, int32_t G, int64_t R,
                                     int64_t H, int64_t I, void* a, int64_t lda, int at, void* workspace,
                                     size_t ws_bytes, void* stream) {
  return linear_call(true, x, ldx, x_scale, n, rows, w13, ldw, w13_scale, true, row_scale, act, offsets, G, R, I, H, a,
                     lda, at, nullptr, 0, workspace, ws_bytes, stream);
}

}  // extern "C"
