// Matrix products of the dense feed-forward operators in bf16 with float32
// sums: c[m][n] = sum_k a(m, k) b(n, k) and a fused epilogue, in the tiles and
// loops of tile.h.  Row operands are x and W forward and dz in dx; k-row operands
// W in dx, dz and x in dW.
// The matrix cores bound the large products: 8192^3 takes 0.74 to 0.76 ms, 1.45
// to 1.49 PFLOP/s, the matrix cores busy 76% of the launch's cycles (80% of
// those with a block on the CU), and the card lowers its clock under this load
// (to 1.7 GHz of 2.4), so LDS and memory traffic cost time through power as
// well.  For 256 x 256, four phases per
// chunk (A0 B0, A0 B1, A1 B1, A1 B0) took 10% longer, with twice the barriers
// and reads crowded into two of the phases; four waves of 128 x 128 with the
// reads between their own products 9%.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "act.h"
#include "common.h"
#include "dense.h"
#include "tile.h"
#include "vec8.h"

namespace dsmoe {
namespace {

constexpr int kChunk = 64;   // K per chunk

// ---------------------------------------------------------------------------
// Epilogue: 8 adjacent columns of one row.
// ---------------------------------------------------------------------------

struct TileArgs {
  DenseGemm p;
  int64_t a_k, b_k;       // contraction length readable along a row (row operands: a multiple of 8)
  int64_t a_r, b_r;       // rows readable (k-row operands: a multiple of 8; kGated: of one half of b)
  bool plain;             // kLinear: one split, no activation or z
  float* partial;         // splits > 1: [split][M][ldp] partial sums, no epilogue
  int64_t ldp;            // (kGated: gate sums, then up sums at + N rounded up to 8)
  int32_t splits;
  int32_t chunks;         // chunks of K in all
  int32_t tiles_m, tiles_n;
};

// y = act(acc + bias) + residual, z = acc + bias
__device__ __forceinline__ void finish_linear(const DenseGemm& p, int64_t m, int64_t n, float* v, const float* bias) {
  const int64_t left = p.N - n;
  float r[8];
  if (p.residual) load8(p.residual, m * p.ldr + n, p.y_f32, left, r);
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] += bias[e];
  if (p.z) store8(p.z, m * p.ldz + n, p.y_f32, left, v);
  if (p.act != DSMOE_ACT_NONE) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = act_f32(p.act, v[e]);
  }
  if (p.rest) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = plus_rest(r[e], v[e]);
  } else if (p.residual) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += r[e];
  }
  store8(p.y, m * p.ldy + n, p.y_f32, left, v);
}

// a = act(g) u, h = [g | u]
__device__ __forceinline__ void finish_gated(const DenseGemm& p, int64_t m, int64_t n, const float* g, const float* u) {
  const int64_t left = p.N - n;
  if (p.z) {
    store8(p.z, m * p.ldz + n, false, left, g);
    store8(p.z, m * p.ldz + p.gate_n + n, false, left, u);
  }
  float v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = act_f32(p.act, g[e]) * u[e];
  store8(p.y, m * p.ldy + n, p.y_f32, left, v);
}

__device__ __forceinline__ void load_bias(const DenseGemm& p, int64_t n, float* o) {
  if (p.bias) {
    load8(p.bias, n, p.bias_f32, p.N - n, o);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = 0.0f;
  }
}

// Blocks are dispatched round-robin over the 8 XCDs: give each XCD a run of
// consecutive tiles, and number the tiles in bands of 4 row tiles, column by
// column, so that the tiles an XCD works on at once (about 4 x 8) share their
// operand rows in its L2.
__device__ __forceinline__ void tile_of_block(uint32_t b, uint32_t n, int32_t tiles_m, int32_t tiles_n, int32_t& tm,
                                              int32_t& tn) {
  const uint32_t x = b % kXcds, q = n / kXcds, r = n % kXcds;
  const uint32_t t = x * q + min(x, r) + b / kXcds;
  constexpr uint32_t kBand = 4;
  const uint32_t band = t / (kBand * tiles_n), in = t % (kBand * tiles_n);
  const uint32_t rows = min(kBand, tiles_m - band * kBand);
  tm = static_cast<int32_t>(band * kBand + in % rows);
  tn = static_cast<int32_t>(in / rows);
}

// What a block and its waves work on (TileCore), its part of the problem and its
// epilogue.
template <int HM, int HN, int WM, int WN, bool AT, bool BT, DenseEpi EPI>
struct Tile : TileCore<Elem::kBf16, HM, HN, WM, WN, AT, BT, EPI == DenseEpi::kGated, false> {
  using Core = TileCore<Elem::kBf16, HM, HN, WM, WN, AT, BT, EPI == DenseEpi::kGated, false>;
  using typename Core::Acc;
  using typename Core::SA;
  using typename Core::SB;
  using Core::a0, Core::a1, Core::b0, Core::b1, Core::c0, Core::c1, Core::get, Core::kGated, Core::kRowsAtOnce,
      Core::kRuns, Core::m0, Core::n0, Core::put;

  const TileArgs& t;
  const DenseGemm& p;
  int32_t split;   // of K

  __device__ __forceinline__ Tile(const TileArgs& args, const uint8_t* mem) : Core(mem), t(args), p(args.p) {
    const uint32_t per_split = static_cast<uint32_t>(t.tiles_m) * t.tiles_n;
    split = blockIdx.x / per_split;
    int32_t tm, tn;
    tile_of_block(blockIdx.x % per_split, per_split, t.tiles_m, t.tiles_n, tm, tn);
    m0 = static_cast<int64_t>(tm) * 2 * HM;
    n0 = static_cast<int64_t>(tn) * (kGated ? HN : 2 * HN);
    c0 = static_cast<int32_t>(static_cast<int64_t>(t.chunks) * split / t.splits);
    c1 = static_cast<int32_t>(static_cast<int64_t>(t.chunks) * (split + 1) / t.splits);
    const int64_t k0 = static_cast<int64_t>(c0) * kChunk;
    const int64_t ka = min(t.a_k, static_cast<int64_t>(c1) * kChunk);
    const int64_t kb = min(t.b_k, static_cast<int64_t>(c1) * kChunk);
    a0 = SA(p.a.p, p.a.ld, m0, t.a_r, k0, ka, this->wave, this->lane);
    a1 = SA(p.a.p, p.a.ld, m0 + HM, t.a_r, k0, ka, this->wave, this->lane);
    // kGated: the up rows are rows gate_n + n of b
    const uint16_t* up = kGated ? p.b.p + p.gate_n * p.b.ld : p.b.p;
    b0 = SB(p.b.p, p.b.ld, n0, t.b_r, k0, kb, this->wave, this->lane);
    b1 = SB(up, p.b.ld, kGated ? n0 : n0 + HN, t.b_r, k0, kb, this->wave, this->lane);
  }

  // y = acc + bias + residual.  The residual of all of
  // a thread's rows is on its way before the results are in LDS (bf16: of both
  // halves; a batch of four rows at a time between the stores cost 4096 x 7168
  // x 2048 with a residual 27 us over the same without).
  template <bool F32, bool REST>
  __device__ __forceinline__ void finish_plain(const Acc& acc) const {
    constexpr int R = HM / kRowsAtOnce, ES = F32 ? 4 : 2;
    const int run = threadIdx.x % kRuns, r0 = threadIdx.x / kRuns;
    const int64_t n = n0 + run * 8;
    const bool in = n < p.N && r0 < kRowsAtOnce;
    float bias[8];
    load_bias(p, n, bias);
    Raw8<F32> res[2][R];
    auto fetch = [&](int ha) {
#pragma unroll
      for (int q = 0; q < R; ++q) {
        const int64_t m = m0 + ha * HM + r0 + q * kRowsAtOnce;
        const bool some = p.residual && in && m < p.M;
        res[ha][q] = fetch8<F32>(static_cast<const char*>(p.residual) + (m * p.ldr + n) * ES, some ? p.N - n : 0);
      }
    };
    fetch(0);
    if constexpr (!F32) fetch(1);
#pragma unroll
    for (int ha = 0; ha < 2; ++ha) {
      if (F32 && ha == 1) fetch(1);
      put(acc[ha]);
      if (!in) continue;
#pragma unroll
      for (int q = 0; q < R; ++q) {
        const int r = r0 + q * kRowsAtOnce;
        const int64_t m = m0 + ha * HM + r;
        if (m >= p.M) break;
        float v[8], x[8];
        get(r, run * 8, v);
        unpack8<F32>(res[ha][q], x);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = REST ? plus_rest(x[e], v[e]) : v[e] + bias[e] + x[e];
        store8(p.y, m * p.ldy + n, F32, p.N - n, v);
      }
    }
  }

  __device__ __forceinline__ void finish(const Acc& acc) const {
    if constexpr (!kGated) {
      if (t.plain) {
        if (!p.y_f32)
          finish_plain<false, false>(acc);
        else if (p.rest)
          finish_plain<true, true>(acc);
        else
          finish_plain<true, false>(acc);
        return;
      }
    }
    const int64_t half_n = (p.N + 7) / 8 * 8;   // columns of partial sums of a kind, padded
    const int run = threadIdx.x % kRuns;
    const int64_t n = n0 + run * 8;
    float bias[8] = {};
    if (!kGated && t.splits == 1) load_bias(p, n, bias);
#pragma unroll
    for (int ha = 0; ha < 2; ++ha) {
      put(acc[ha]);
      if (static_cast<int>(threadIdx.x) >= kRowsAtOnce * kRuns) continue;
#pragma unroll 1
      for (int r = threadIdx.x / kRuns; r < HM; r += kRowsAtOnce) {
        const int64_t m = m0 + ha * HM + r;
        if (m >= p.M || n >= half_n) break;
        float v[8], u[8];
        get(r, run * 8, v);
        if constexpr (kGated) get(r, HN + run * 8, u);
        if (t.splits > 1) {
          put8<true>(t.partial + (split * p.M + m) * t.ldp + n, 8, v);
          if constexpr (kGated) put8<true>(t.partial + (split * p.M + m) * t.ldp + half_n + n, 8, u);
        } else if constexpr (kGated) {
          finish_gated(p, m, n, v, u);
        } else {
          finish_linear(p, m, n, v, bias);
        }
      }
    }
  }
};

template <int HM, int HN, int WM, int WN, bool AT, bool BT, DenseEpi EPI>
__global__ __launch_bounds__(64 * WM * WN) void dense_phased_kernel(TileArgs args) {
  using T = Tile<HM, HN, WM, WN, AT, BT, EPI>;
  __shared__ __attribute__((aligned(1024))) uint8_t s_mem[T::lds_bytes(2)];
  T w(args, s_mem);
  typename T::Acc acc;
  phased_loop(w, acc);
  w.finish(acc);
}

template <int HM, int HN, int WM, int WN, int S, bool AT, bool BT, DenseEpi EPI>
__global__ __launch_bounds__(64 * WM * WN) void dense_paired_kernel(TileArgs args) {
  using T = Tile<HM, HN, WM, WN, AT, BT, EPI>;
  __shared__ __attribute__((aligned(1024))) uint8_t s_mem[T::lds_bytes(S)];
  T w(args, s_mem);
  typename T::Acc acc;
  paired_loop<S>(w, acc);
  w.finish(acc);
}

template <int HM, int HN, int WM, int WN, int S, bool AT, bool BT, DenseEpi EPI>
__global__ __launch_bounds__(64 * WM * WN) void dense_ring_kernel(TileArgs args) {
  using T = Tile<HM, HN, WM, WN, AT, BT, EPI>;
  __shared__ __attribute__((aligned(1024))) uint8_t s_mem[T::lds_bytes(S)];
  T w(args, s_mem);
  typename T::Acc acc;
  ring_loop<S>(w, acc);
  w.finish(acc);
}

// Sum of the splits' partial results in order, then the epilogue: 8 columns
// of a row per thread, four splits' loads in flight (64 x 2 x 2048, 8 splits:
// 8.4 MB from L2 in 4.1 us, mostly the launch).
constexpr int kJoinThreads = 64;
template <DenseEpi EPI>
__global__ __launch_bounds__(kJoinThreads) void join_splits_kernel(TileArgs t) {
  const DenseGemm& p = t.p;
  const int64_t runs = (p.N + 7) / 8;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kJoinThreads + threadIdx.x;
  if (i >= p.M * runs) return;
  const int64_t m = i / runs, n = i % runs * 8;
  constexpr int kKinds = EPI == DenseEpi::kGated ? 2 : 1;
  float v[kKinds][8] = {};
  for (int s = 0; s < t.splits; s += 4) {
    float o[4][kKinds][8];
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int k = 0; k < kKinds; ++k)
        if (s + q < t.splits) load8(t.partial + ((s + q) * p.M + m) * t.ldp + k * runs * 8, n, true, 8, o[q][k]);
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (s + q < t.splits) {
#pragma unroll
        for (int k = 0; k < kKinds; ++k)
#pragma unroll
          for (int e = 0; e < 8; ++e) v[k][e] += o[q][k][e];
      }
  }
  if constexpr (EPI == DenseEpi::kGated) {
    finish_gated(p, m, n, v[0], v[1]);
  } else {
    float bias[8];
    load_bias(p, n, bias);
    finish_linear(p, m, n, v[0], bias);
  }
}

// Up to two copies of operands into rows of whole groups of 8, for rows the
// copies to LDS cannot take (16-byte aligned ones only):
// dst [rows][ldd] = src [rows][cols], the row's padding up to ldd zeroed.  HBM
// bounds it (640 x 6030 and 7256 x 6030, 190 MB in all: about 40 us).
struct PackArgs {
  const uint16_t* src[2];
  uint16_t* dst[2];
  int64_t lds[2], rows[2], cols[2];
};
__global__ __launch_bounds__(256) void pack_rows_kernel(PackArgs a) {
  const int w = blockIdx.y;
  const uint16_t* src = w ? a.src[1] : a.src[0];
  uint16_t* dst = w ? a.dst[1] : a.dst[0];
  const int64_t lds = w ? a.lds[1] : a.lds[0], rows = w ? a.rows[1] : a.rows[0], cols = w ? a.cols[1] : a.cols[0];
  const int64_t segs = (cols + 7) / 8, n = rows * segs;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t r = i >> 32 ? i / segs : static_cast<uint32_t>(i) / static_cast<uint32_t>(segs);
    const int64_t c = (i - r * segs) * 8;
    *reinterpret_cast<u32x4*>(dst + r * segs * 8 + c) = fetch8<false>(src + r * lds + c, cols - c).q[0];
  }
}

__global__ __launch_bounds__(256) void zero_matrix_kernel(void* dst, int64_t ldd, bool f32, int64_t m, int64_t n) {
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < m * n;
       i += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t at = i / n * ldd + i % n;
    if (f32)
      static_cast<float*>(dst)[at] = 0.0f;
    else
      static_cast<uint16_t*>(dst)[at] = 0;
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

// The tile shapes.  chunk_us: time of one chunk (64 of K) of one block, alone
// on its CU and with a second block beside it; end_us: a block's start and
// epilogue.  Measured on products of 2048^3 to 8192^3 (the blocks per CU of a
// shape are what its LDS stages allow).
//   256 x 256  phased, 128 KB of LDS: 4096^3 in 103 us, where 128 x 128 takes
//              134 (two per CU) or 154 (one per CU, four stages)
//   128 x 128  four stages, one per CU: when there is at most one tile per CU
//              (1024 x 4096 x 4096 in 38 us; with two stages 45, 256 x 256 80)
//   128 x 128  two stages, two per CU: a few tiles per CU and few chunks
//              (16384 x 512 x 256 in 11.5 us, 128 x 256 11.9; from 6 chunks on
//              the two are within 3%: 16384 x 512 x 512 15.9 and 16.2)
//   256 x 192  phased: what is left over when 256 x 256 tiles fill the card a
//              whole number of times (see make_plan), and sizes it fits better
//   128 x 256  three stages, one per CU: when 256 x 256 leaves CUs without a
//              tile (4096 x 2048 x 7168 in 92 us; 128 x 128 117, 256 x 256 173)
//   64 x 64    four stages, two per CU: small products
//              (1024^3 in 9.5 us; 128 x 128 12.8)
enum class Shape { k256, k256x192, k128x256, k128x4, k128x2, k64 };
struct ShapeInfo {
  int64_t rows, cols;
  int per_cu;
  double chunk_us, shared_us, end_us;
};
constexpr ShapeInfo kShapes[] = {
    {256, 256, 1, 1.42, 0.0, 5.0}, {256, 192, 1, 1.12, 0.0, 4.5},  {128, 256, 1, 0.79, 0.0, 4.0},
    {128, 128, 1, 0.50, 0.0, 3.0}, {128, 128, 2, 0.60, 1.00, 3.0}, {64, 64, 2, 0.30, 0.42, 2.0}};
constexpr int64_t kCus = 256;
constexpr double kHbm = 4.8e6;   // bytes per us of a long read

struct Grid {   // a launch of dense_*_kernel
  Shape shape;
  int splits;
  int64_t tiles_m, tiles_n;
  double us;    // estimated time
};
struct Plan {
  Grid first, rest;
  int64_t cut;    // columns of the result in the first launch; 0: all, there is no other
  int64_t chunks;
  bool pack_a, pack_b;
  int64_t a_rows, a_cols, b_rows, b_cols;   // of the stored matrices
  size_t a_bytes, b_bytes, partial_bytes;
  double us;      // estimated time
};

int64_t up8(int64_t v) { return (v + 7) / 8 * 8; }
size_t up256(size_t v) { return (v + 255) / 256 * 256; }

// whether the tile kernel can copy an operand whose rows hold `cols` values
bool copyable(const Operand& o, int64_t cols) {
  return (reinterpret_cast<uintptr_t>(o.p) & 15) == 0 && o.ld % 8 == 0 && (cols % 8 == 0 || o.padded);
}

// Time of n blocks of `chunks` chunks: full rounds of the card, then the rest.
double blocks_us(const ShapeInfo& s, int64_t n, int64_t chunks) {
  const double full = static_cast<double>(chunks) * (s.per_cu > 1 ? s.shared_us : s.chunk_us) + s.end_us;
  const double alone = static_cast<double>(chunks) * s.chunk_us + s.end_us;
  const int64_t slots = kCus * s.per_cu, rest = n % slots;
  return static_cast<double>(n / slots) * full + (rest == 0 ? 0.0 : rest <= kCus ? alone : full);
}

// Shape and number of splits of K for m rows and nb rows of b by the estimated
// time: the blocks, and with splits the launch that joins them and the partial
// sums' way to memory and back.
Grid best_grid(int64_t m, int64_t nb, int64_t chunks, int max_splits) {
  Grid g{};
  g.us = 1e30;
  for (int i = 0; i < 6; ++i) {
    const ShapeInfo& s = kShapes[i];
    const int64_t tm = (m + s.rows - 1) / s.rows, tn = (nb + s.cols - 1) / s.cols;
    for (int sp = 1; sp <= max_splits && sp <= chunks; sp *= 2) {
      double us = blocks_us(s, tm * tn * sp, (chunks + sp - 1) / sp);
      if (sp > 1) us += 4.0 + 2.0 * sp * static_cast<double>(m) * nb * 4 / 4e6;
      if (us < g.us) g = Grid{static_cast<Shape>(i), sp, tm, tn, us};
    }
  }
  return g;
}

Plan make_plan(const DenseGemm& p) {
  Plan pl{};
  const bool gated = p.epi == DenseEpi::kGated;
  const int64_t nb = gated ? 2 * p.N : p.N;   // rows of b
  pl.a_rows = p.a.k_rows ? p.K : p.M, pl.a_cols = p.a.k_rows ? p.M : p.K;
  pl.b_rows = p.b.k_rows ? p.K : nb, pl.b_cols = p.b.k_rows ? nb : p.K;
  pl.pack_a = !copyable(p.a, pl.a_cols);
  pl.pack_b = !copyable(p.b, pl.b_cols);
  pl.a_bytes = pl.pack_a ? up256(static_cast<size_t>(pl.a_rows) * up8(pl.a_cols) * 2) : 0;
  pl.b_bytes = pl.pack_b ? up256(static_cast<size_t>(pl.b_rows) * up8(pl.b_cols) * 2) : 0;
  pl.chunks = (p.K + kChunk - 1) / kChunk;

  pl.first = best_grid(p.M, nb, pl.chunks, 32);
  // Tiles of 256 x 256 that fill the card a whole number of times, and another
  // launch for the columns left over: 4096 x 7168 is one round of 256 such
  // tiles and one of 256 tiles of 256 x 192, instead of two rounds of which
  // the second has 192.
  const ShapeInfo& big = kShapes[static_cast<int>(Shape::k256)];
  const int64_t tm = (p.M + big.rows - 1) / big.rows, tn = (nb + big.cols - 1) / big.cols;
  for (int64_t rounds = 1; rounds * kCus < tm * tn && rounds <= 8; ++rounds) {
    const int64_t c = rounds * kCus / tm;   // tile columns of the first launch
    if (c < 1 || c >= tn) continue;
    const Grid rest = best_grid(p.M, nb - c * big.cols, pl.chunks, 1);
    const double first_us = blocks_us(big, tm * c, pl.chunks), us = first_us + rest.us + 3.0;
    if (us < pl.first.us + (pl.cut ? pl.rest.us + 3.0 : 0.0)) {
      pl.cut = c * (gated ? big.cols / 2 : big.cols);
      pl.first = Grid{Shape::k256, 1, tm, c, first_us};
      pl.rest = rest;
    }
  }
  const double work = pl.first.us + (pl.cut ? pl.rest.us + 3.0 : 0.0);
  // launches, W's way from memory, copies of operands
  const double bytes = static_cast<double>(nb) * p.K * 2;
  pl.us = 3.5 + (work > bytes / kHbm ? work + 0.25 * bytes / kHbm : bytes / kHbm + 0.25 * work);
  if (pl.pack_a) pl.us += 3.0 + 2.0 * pl.a_bytes / kHbm;
  if (pl.pack_b) pl.us += 3.0 + 2.0 * pl.b_bytes / kHbm;
  if (pl.first.splits > 1)
    pl.partial_bytes = static_cast<size_t>(pl.first.splits) * p.M * (gated ? 2 * up8(p.N) : up8(p.N)) * 4;
  return pl;
}

template <int HM, int HN, int WM, int WN, int S, bool AT, bool BT, DenseEpi EPI>
hipError_t launch_kernel(const TileArgs& t, hipStream_t s) {
  const uint32_t grid = static_cast<uint32_t>(static_cast<int64_t>(t.tiles_m) * t.tiles_n * t.splits);
  constexpr int threads = 64 * WM * WN;
  if constexpr (HM == 128)
    dense_phased_kernel<HM, HN, WM, WN, AT, BT, EPI><<<grid, threads, 0, s>>>(t);
  else if constexpr (HN == 128)
    dense_paired_kernel<HM, HN, WM, WN, S, AT, BT, EPI><<<grid, threads, 0, s>>>(t);
  else
    dense_ring_kernel<HM, HN, WM, WN, S, AT, BT, EPI><<<grid, threads, 0, s>>>(t);
  return hipGetLastError();
}

template <int HM, int HN, int WM, int WN, int S>
hipError_t launch_shape(const TileArgs& t, hipStream_t s) {
  if (t.p.epi == DenseEpi::kGated)   // forward only: both operands by rows
    return launch_kernel<HM, HN, WM, WN, S, false, false, DenseEpi::kGated>(t, s);
  if (!t.p.b.k_rows) return launch_kernel<HM, HN, WM, WN, S, false, false, DenseEpi::kLinear>(t, s);
  if (!t.p.a.k_rows) return launch_kernel<HM, HN, WM, WN, S, false, true, DenseEpi::kLinear>(t, s);
  return launch_kernel<HM, HN, WM, WN, S, true, true, DenseEpi::kLinear>(t, s);
}

// Whether the kernel for few tokens takes a product.  Its time is W's way from
// memory or x's way from L2 to every block (about 35 KB per us and CU),
// whichever is longer, and some of the other; wide loads of rows off 4 bytes
// take 2.3 times as long (7168 x 2047 17.8 us, 7168 x 2044 8.1).  4096 x 7168:
// 1 token 12 us (tiles 18), 16 tokens 16 (19), 32 tokens 22 (19); 1000 x 1000:
// 64 tokens 6.5 (9).
bool few_tokens(const DenseGemm& p, const Plan& pl) {
  if (p.M > 64 || p.a.k_rows || p.b.k_rows) return false;
  const bool gated = p.epi == DenseEpi::kGated;
  const int64_t blocks = gated ? (p.N + 7) / 8 : (p.N + 15) / 16, groups = (p.M + 15) / 16;
  auto even = [](const Operand& o) { return reinterpret_cast<uintptr_t>(o.p) % 4 == 0 && o.ld % 2 == 0; };
  const double slow = even(p.a) && even(p.b) ? 1.0 : 2.3;
  const double w = slow * (gated ? 2.0 : 1.0) * p.N * p.K * 2 / kHbm;
  const double rounds = blocks > kCus ? static_cast<double>(blocks) / kCus : 1.0;
  const double x = p.M == 1 ? 0.0 : slow * rounds * groups * 16 * p.K * 2 / 35e3;
  return 4.0 + (w > x ? w + 0.3 * x : x + 0.3 * w) < pl.us;
}

hipError_t launch_range(const DenseGemm& p, hipStream_t s) {
  const Plan pl = make_plan(p);
  if (few_tokens(p, pl)) return launch_dense_skinny(p, s);
  uint8_t* ws = static_cast<uint8_t*>(p.workspace);
  TileArgs t{};
  t.p = p;
  hipError_t e = hipSuccess;
  PackArgs pk{};
  int packs = 0;
  auto pack = [&](Operand& o, size_t at, int64_t rows, int64_t cols) {
    pk.src[packs] = o.p, pk.lds[packs] = o.ld, pk.rows[packs] = rows, pk.cols[packs] = cols;
    pk.dst[packs] = reinterpret_cast<uint16_t*>(ws + at);
    o = Operand{pk.dst[packs++], up8(cols), o.k_rows, true};
  };
  if (pl.pack_a) pack(t.p.a, 0, pl.a_rows, pl.a_cols);
  if (pl.pack_b) pack(t.p.b, pl.a_bytes, pl.b_rows, pl.b_cols);
  if (packs) {
    const int64_t n0 = pk.rows[0] * (up8(pk.cols[0]) / 8), n1 = pk.rows[1] * (up8(pk.cols[1]) / 8);
    const int64_t blocks = ((n0 > n1 ? n0 : n1) + 255) / 256;
    pack_rows_kernel<<<dim3(static_cast<uint32_t>(blocks < 8192 ? blocks : 8192), packs), 256, 0, s>>>(pk);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  const bool gated = p.epi == DenseEpi::kGated;
  // padded rows read as zeros up to a multiple of 8
  t.a_k = p.a.k_rows ? p.K : up8(p.K);
  t.b_k = p.b.k_rows ? p.K : up8(p.K);
  t.a_r = p.a.k_rows ? up8(p.M) : p.M;
  t.b_r = p.b.k_rows ? up8(p.N) : p.N;
  t.chunks = static_cast<int32_t>(pl.chunks);
  auto run = [&](const Grid& g) {
    t.splits = g.splits;
    t.plain = g.splits == 1 && p.act == DSMOE_ACT_NONE && !p.z;
    t.tiles_m = static_cast<int32_t>(g.tiles_m);
    t.tiles_n = static_cast<int32_t>(g.tiles_n);
    switch (g.shape) {
      case Shape::k256: return launch_shape<128, 128, 2, 4, 2>(t, s);
      case Shape::k256x192: return launch_shape<128, 96, 4, 2, 2>(t, s);
      case Shape::k128x256: return launch_shape<64, 128, 2, 4, 3>(t, s);
      case Shape::k128x4: return launch_shape<64, 64, 2, 4, 4>(t, s);
      case Shape::k128x2: return launch_shape<64, 64, 2, 4, 2>(t, s);
      case Shape::k64: break;
    }
    return launch_shape<32, 32, 2, 2, 4>(t, s);
  };
  if (pl.cut) {
    DenseGemm& q = t.p;
    q.N = pl.cut;
    t.b_r = q.b.k_rows ? up8(q.N) : q.N;
    if ((e = run(pl.first)) != hipSuccess) return e;
    // the columns from cut on
    q.N = p.N - pl.cut;
    t.b_r = q.b.k_rows ? up8(q.N) : q.N;
    q.b.p += q.b.k_rows ? pl.cut : pl.cut * q.b.ld;
    const int64_t es = q.y_f32 ? 4 : 2;
    auto move = [&](const void* m, int64_t size) {
      return m ? static_cast<const void*>(static_cast<const char*>(m) + pl.cut * size) : nullptr;
    };
    q.y = const_cast<void*>(move(q.y, es));
    q.residual = move(q.residual, es);
    q.bias = move(q.bias, q.bias_f32 ? 4 : 2);
    q.z = const_cast<void*>(move(q.z, gated ? 2 : es));
    return run(pl.rest);
  }
  if (pl.first.splits > 1) {
    t.partial = reinterpret_cast<float*>(ws + pl.a_bytes + pl.b_bytes);
    t.ldp = gated ? 2 * up8(p.N) : up8(p.N);
  }
  e = run(pl.first);
  if (e != hipSuccess || pl.first.splits == 1) return e;
  const int64_t blocks = (p.M * (up8(p.N) / 8) + kJoinThreads - 1) / kJoinThreads;
  if (gated)
    join_splits_kernel<DenseEpi::kGated><<<static_cast<uint32_t>(blocks), kJoinThreads, 0, s>>>(t);
  else
    join_splits_kernel<DenseEpi::kLinear><<<static_cast<uint32_t>(blocks), kJoinThreads, 0, s>>>(t);
  return hipGetLastError();
}

// A launch holds fewer than 2^32 threads: f with ranges of at most 2^28 of the
// result's rows (2^30 threads in tiles of 64 x 64; wider results take larger
// tiles).  dW's rows are a dimension of the weights.
template <typename F>
hipError_t by_row_ranges(const DenseGemm& p, F f) {
  constexpr int64_t kRows = int64_t{1} << 28;
  if (p.a.k_rows || p.M <= kRows) return f(p);
  const int64_t ys = p.y_f32 ? 4 : 2, zs = p.epi == DenseEpi::kGated ? 2 : ys;
  for (int64_t r = 0; r < p.M; r += kRows) {
    DenseGemm q = p;
    q.M = p.M - r < kRows ? p.M - r : kRows;
    if (p.a.p) q.a.p += r * p.a.ld;
    if (p.y) q.y = static_cast<char*>(p.y) + r * p.ldy * ys;
    if (p.residual) q.residual = static_cast<const char*>(p.residual) + r * p.ldr * ys;
    if (p.z) q.z = static_cast<char*>(p.z) + r * p.ldz * zs;
    const hipError_t e = f(q);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

bool operand_copyable(const Operand& o, int64_t cols) { return copyable(o, cols); }

size_t dense_gemm_workspace_bytes(const DenseGemm& p) {
  size_t most = 0;
  (void)by_row_ranges(p, [&](const DenseGemm& q) {
    const Plan pl = make_plan(q);
    const size_t n = few_tokens(q, pl) ? 0 : pl.a_bytes + pl.b_bytes + up256(pl.partial_bytes);
    most = n > most ? n : most;
    return hipSuccess;
  });
  return most;
}

DenseKernels dense_gemm_kernels(const DenseGemm& p) {
  const Plan pl = make_plan(p);
  return DenseKernels{few_tokens(p, pl),  static_cast<int>(pl.first.shape), pl.first.splits, pl.cut,
                      pl.cut ? static_cast<int>(pl.rest.shape) : 0, pl.cut ? pl.rest.splits : 0};
}

hipError_t launch_dense_gemm(const DenseGemm& p, hipStream_t s) {
  return by_row_ranges(p, [&](const DenseGemm& q) { return launch_range(q, s); });
}

hipError_t launch_zero_matrix(void* dst, int64_t ldd, bool f32, int64_t m, int64_t n, hipStream_t s) {
  if (m * n == 0) return hipSuccess;
  const int64_t blocks = (m * n + 1023) / 1024;
  zero_matrix_kernel<<<static_cast<uint32_t>(blocks < 4096 ? blocks : 4096), 256, 0, s>>>(dst, ldd, f32, m, n);
  return hipGetLastError();
}

}  // namespace dsmoe
