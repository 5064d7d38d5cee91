// Products over rows grouped by expert with ragged sizes, outside FP8: y, dx and
// dW of the grouped linear and gated linear operators in bf16, and y of their
// 8-bit forms.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <cmath>

#include "common.h"
#include "grouped.h"
#include "grouped_stream.h"
#include "grouped_tile.h"
#include "vec8.h"

namespace dsmoe {
namespace {

// Copies of operand rows into aligned rows of whole 16 bytes: dst [rows][segs]
// segments = src [rows][cols] or its rows index[r] (an index outside [0, n):
// zeros), the padding zeroed.  Bound by memory: 16384 rows of 7168 by index, 235 MB
// written, in 73 us.
struct PackArgs {
  const char* src;
  char* dst;
  const int32_t* index;
  int64_t ld, rows, cols, n;   // ld, cols in bytes
};
// Both operands of a product in one launch: blocks [0, blocks0) copy the first, the
// others the second.
__global__ __launch_bounds__(256) void pack_grouped_kernel(PackArgs first, PackArgs second, uint32_t blocks0) {
  const bool one = blockIdx.x < blocks0;
  const PackArgs a = one ? first : second;
  const uint32_t block = one ? blockIdx.x : blockIdx.x - blocks0, blocks = one ? blocks0 : gridDim.x - blocks0;
  const int64_t segs = (a.cols + 15) / 16, all = a.rows * segs;
  for (int64_t i = static_cast<int64_t>(block) * 256 + threadIdx.x; i < all; i += static_cast<int64_t>(blocks) * 256) {
    const int64_t r = i >> 32 ? i / segs : static_cast<uint32_t>(i) / static_cast<uint32_t>(segs);
    const int64_t c = (i - r * segs) * 16;
    const int64_t row = a.index ? a.index[r] : r;
    u32x4 v{0, 0, 0, 0};
    if (row >= 0 && row < a.n) {
      const char* p = a.src + row * a.ld + c;
      if (a.cols - c >= 16) {
        v = *reinterpret_cast<const u32x4_at1*>(p);
      } else {
#pragma unroll
        for (int e = 0; e < 15; ++e)
          if (e < a.cols - c) v[e / 4] |= static_cast<uint32_t>(static_cast<uint8_t>(p[e])) << (e % 4 * 8);
      }
    }
    *reinterpret_cast<u32x4*>(a.dst + (r * segs + (c >> 4)) * 16) = v;
  }
}

int64_t up(int64_t v, int64_t a) { return (v + a - 1) / a * a; }
size_t up256(size_t v) { return (v + 255) / 256 * 256; }

// What the copies of an operand before the product take.
struct PackPlan {
  bool pack, gather;   // gather: R rows by index, else the source rows
  int64_t rows, cols, bytes;
};

constexpr int64_t kIndexed = int64_t{1} << 31;   // bytes that rows by index may span

// An operand by rows: in place where its rows are whole aligned 16 bytes and
// the lanes' offsets reach all of them.  Otherwise a copy: of the source rows
// where they are fewer than R and the offsets then reach them, else of the
// R rows taken by index.
PackPlan plan_rows(const RowsOf& o, int64_t R, int64_t cols, int es) {
  PackPlan q{};
  q.cols = cols;
  const int64_t ld = up(cols * es, 16);
  const bool fits = !o.index || o.n * o.ld * es < kIndexed;
  if (rows_copyable(o, cols, es) && fits) return q;
  q.pack = true;
  q.gather = o.index && (o.n > R || o.n * ld >= kIndexed);
  q.rows = q.gather ? R : o.n;
  q.bytes = static_cast<int64_t>(up256(static_cast<size_t>(q.rows) * ld));
  return q;
}
// An operand across its rows (dW): rows by index are gathered first.
PackPlan plan_k_rows(const RowsOf& o, int64_t R, int64_t cols) {
  PackPlan q{};
  q.cols = cols;
  if (!o.index && rows_copyable(o, cols, 2)) return q;
  q.pack = true;
  q.gather = o.index != nullptr;
  q.rows = q.gather ? R : o.n;
  q.bytes = static_cast<int64_t>(up256(static_cast<size_t>(q.rows) * up(cols * 2, 16)));
  return q;
}

// The tile shapes and the times they are chosen by: chunk_us of one chunk (128
// bytes of K) of a block alone on its CU, shared_us with a second block beside it,
// end_us a block's start and end.  For y, and dx in whole tiles, fitted to 143
// measured sizes (1 to 2048 rows per expert, 16 to 128 experts, 512 x 256 to 4096 x
// 7168, bf16 and 8 bits): the shape taken is 1.5% from the best on average, 17% at
// worst.
//   256 x 256  64 experts of 7168 x 2048 with 1024 rows each: 1.73 ms, 128 x 128
//              2.23, 64 x 64 3.96; with 128 rows 458 us, 486, 673
//   128 x 128  two stages, two blocks per CU: 16 experts of 2 x 1024 x 1024 with 512
//              rows: 54 us, 256 x 256 71, 64 x 64 101
//   64 x 64    16 experts of 1024 x 1024 with 16 rows: 11 us, 128 x 128 15, 256 x
//              256 25
//   32 x 128   128 experts of 512 x 512 with 4 rows: 14 us, 64 x 64 17.8, 128 x 128
//              15.5; 64 of 7168 x 2048 with 8-bit codes: 160 us, 185, 176
// dW's tiles of 128 and 64 rows, whose results go through LDS, end later: 64
// experts of 7168 x 2048 with 128 rows 630 us, 128 x 128 869, 64 x 64 1927; 16 of
// 512 x 256 with 1024 rows 33 us, 15, 13.
struct ShapeInfo {
  int64_t rows, cols;
  int per_cu;
  double chunk_us, shared_us, end_us, dw_end_us;
};
constexpr ShapeInfo kShapes[] = {{256, 256, 1, 1.42, 1.42, 7.0, 4.0},
                                 {128, 128, 2, 0.40, 1.02, 2.9, 8.0},
                                 {64, 64, 2, 0.37, 0.40, 2.8, 5.0},
                                 {32, 128, 2, 0.41, 0.52, 2.5, 0.0}};
// A block for each 256-row tile computes one of few rows in 1/2 or 3/4 of the height
// (grouped_tile.h) and takes longer to start and end: with up to `rows` rows per
// group, a tile each, a chunk takes chunk_us.  For the gated product and dx fitted
// to 108 measured sizes (16 to 320 rows per expert, 16 and 64 experts, 1024 x 512 to
// 7168 x 2048, bf16 and 8 bits): the shape taken is 1.0% from the best on average,
// 20% at worst (16 rows of 2048 x 1024, 29 us); by whole tiles' times 3.9%, 52% at
// worst.  Where the groups are uneven, which the host does not know, more is lost:
// with popularities falling as the rank's square root 3.8% on average over 315 sizes
// (4 to 768 rows per expert, every product; even popularities 1.2% over the same), 5%
// of the sizes lose more than 23%, and small products most (64 experts of 1024 -> 512
// with 192 rows in 8 bits 51 us, in 128 x 128 tiles 32).
// 64 experts of 7168 x 2048 with 48 rows, dx: 647 us, 128 x 128 677, 64 x 64 883; with
// 96 rows gated 653 us, 768, 1047.
// y takes these blocks up to 192 rows per group, and up to 224 where there are at most
// kFewTiles tiles, so that the start of a tile's copies under the tile before matters
// less; past that those that stay (grouped_stream.h).  Their time by that of blocks that
// stay, on average over 7 sizes of 1024 x 512 to 2048 x 7168 with 8 to 256 experts, in
// both types, and in brackets with more than kFewTiles tiles: 160 rows 0.91 (0.99), 192
// 0.92 (1.00, at worst 1.09), 224 0.95 (1.03, at worst 1.14), 240 0.97 (1.03).  256
// experts of 7168 x 2048 with 192 rows 1.82 ms, 1.80 by blocks that stay, in 8 bits 1.07,
// 1.05; with 224 1.91, 1.85 and 1.13, 1.10.  64 of 1024 x 512 with 192 rows 24 us, 30
// and 22, 29; with 224 38, 42 and 34, 38.
struct ShortTile {
  double rows, chunk_us;
};
constexpr ShortTile kShort[] = {{128, 0.8}, {192, 1.1}, {224, 1.42}};
constexpr double kShortEnd = 9.0;
constexpr int64_t kCus = 256;
constexpr double kFewTiles = 4.0 * kCus;
constexpr double kRead = 6.1e6, kWrite = 4.0e6;   // bytes per us of weights, of their gradients

// Time of `tiles` tiles of `chunks` chunks: rounds of the card.
double tiles_us(const ShapeInfo& s, double tiles, double chunks, double end_us) {
  const double alone = chunks * s.chunk_us + end_us, full = chunks * s.shared_us + end_us;
  const double slots = static_cast<double>(kCus * s.per_cu), rounds = tiles / slots;
  if (tiles <= kCus) return alone;
  if (rounds <= 1.0) return alone + (full - alone) * (tiles - kCus) / kCus;
  return (rounds < 4.0 ? std::ceil(rounds) : rounds + 0.5) * full;
}

struct GroupedPlan {
  GroupedShape shape;
  bool few_rows;         // per group: a block for each 256-row tile, of less height
  PackPlan a, b;         // b: w, or kDw's b
  uint32_t tiles_m, tiles_n;
  uint64_t tiles;        // at most
};

GroupedPlan make_plan(const GroupedGemm& p) {
  GroupedPlan q{};
  const int64_t R = p.groups.R, G = p.groups.n;
  const int es = p.i8 ? 1 : 2;
  const bool dw = p.kind == GroupedKind::kDw, dx = p.kind == GroupedKind::kDx, gated = p.kind == GroupedKind::kGated;
  const int64_t cols = dw ? p.K : p.N * (gated ? 2 : 1);   // the tiles' columns
  const int64_t busy = R < G ? R : G;                      // groups with rows, at most
  // the launch's time: memory's or the tiles', whichever is longer, and some of the
  // other.  The sizes of the groups are on the device: tiles of rows are counted
  // as for groups of equal sizes that end anywhere in their last tile.
  double best = 1e300;
  for (int i = 0; i < 4; ++i) {
    ShapeInfo s = kShapes[i];
    if (dw && i == 3) break;
    const double tn = static_cast<double>((cols + s.cols - 1) / s.cols), per_group = static_cast<double>(R) / busy;
    double tiles, chunks, mem;
    if (dw) {
      tiles = static_cast<double>((p.N + s.rows - 1) / s.rows) * tn * G;
      chunks = static_cast<double>(R) / G * 2 / kChunkBytes + 0.5;
      mem = static_cast<double>(G) * p.N * p.K * 2 / kWrite;
    } else {
      double tm = G == 1 ? static_cast<double>((R + s.rows - 1) / s.rows) : per_group / s.rows + 0.5;
      if (i == 0) {
        q.few_rows = per_group <= kShort[busy * tn <= kFewTiles ? 2 : 1].rows;
        if (gated || dx || q.few_rows) s.end_us = kShortEnd;
        for (const ShortTile& t : kShort) {
          if (per_group > t.rows) continue;
          s.chunk_us = s.shared_us = t.chunk_us;
          tm = 1.0;
          break;
        }
      }
      tiles = busy * (tm > 1.0 ? tm : 1.0) * tn;
      chunks = static_cast<double>((p.K * es + kChunkBytes - 1) / kChunkBytes);
      mem = static_cast<double>(busy) * cols * p.K * es / kRead;
    }
    const double work = tiles_us(s, tiles, chunks, dw ? s.dw_end_us : s.end_us);
    const double us = work > mem ? work + 0.2 * mem : mem + 0.2 * work;
    if (us < best) best = us, q.shape = static_cast<GroupedShape>(i);
  }
  const ShapeInfo& s = kShapes[static_cast<int>(q.shape)];
  q.tiles_n = static_cast<uint32_t>((cols + s.cols - 1) / s.cols);
  if (dw) {
    q.a = plan_k_rows(p.a, R, p.N);
    q.b = plan_k_rows(p.b, R, p.K);
    q.tiles_m = static_cast<uint32_t>((p.N + s.rows - 1) / s.rows);
    q.tiles = static_cast<uint64_t>(q.tiles_m) * q.tiles_n * G;
    return q;
  }
  q.a = plan_rows(p.a, R, p.K, es);
  const RowsOf w{p.w, p.ldw, G * (dx ? p.K : cols), nullptr, false};
  q.b = plan_rows(w, w.n, dx ? p.N : p.K, es);
  // at most: a group with rows has at most one tile that is not full
  q.tiles = static_cast<uint64_t>((R + (s.rows - 1) * busy) / s.rows) * q.tiles_n;
  return q;
}

PackArgs pack_args(const RowsOf& o, const PackPlan& q, int es, void* dst) {
  return PackArgs{static_cast<const char*>(o.p), static_cast<char*>(dst), q.gather ? o.index : nullptr, o.ld * es,
                  q.pack ? q.rows : 0, q.cols * es, o.n};
}
uint32_t pack_blocks(const PackArgs& a) {
  const int64_t blocks = (a.rows * ((a.cols + 15) / 16) + 255) / 256;
  return static_cast<uint32_t>(blocks < 8192 ? blocks : 8192);
}
hipError_t pack(const PackArgs& a, const PackArgs& b, hipStream_t s) {
  const uint32_t na = pack_blocks(a), nb = pack_blocks(b);
  if (na + nb == 0) return hipSuccess;
  pack_grouped_kernel<<<na + nb, 256, 0, s>>>(a, b, na);
  return hipGetLastError();
}

// The operand after its copy.
RowsOf packed(const RowsOf& o, const PackPlan& q, int es, void* dst) {
  return RowsOf{dst, up(q.cols * es, 16) / es, q.rows, q.gather ? nullptr : o.index, true};
}

}  // namespace

bool rows_copyable(const RowsOf& o, int64_t cols, int bytes) {
  return (reinterpret_cast<uintptr_t>(o.p) & 15) == 0 && o.ld * bytes % 16 == 0 && (cols * bytes % 16 == 0 || o.padded);
}

int grouped_gemm_shape(const GroupedGemm& p) {
  const GroupedPlan q = make_plan(p);
  const bool each = q.shape == GroupedShape::k256 && p.kind == GroupedKind::kLinear && q.few_rows;
  return each ? 4 : static_cast<int>(q.shape);
}

size_t grouped_gemm_workspace_bytes(const GroupedGemm& p) {
  if (p.groups.R == 0) return 0;
  const GroupedPlan q = make_plan(p);
  return static_cast<size_t>(q.a.bytes + q.b.bytes);
}

hipError_t launch_grouped_gemm(const GroupedGemm& p, hipStream_t s) {
  const GroupedPlan q = make_plan(p);
  const int es = p.i8 ? 1 : 2;
  const bool dw = p.kind == GroupedKind::kDw, dx = p.kind == GroupedKind::kDx;
  GroupedArgs t{};
  t.p = p;
  t.scale_index = p.a.index, t.scale_n = p.a.n;
  char* const to_a = static_cast<char*>(p.workspace);
  char* const to_b = to_a + q.a.bytes;
  const RowsOf b = dw ? p.b : RowsOf{p.w, p.ldw, q.b.rows, nullptr, false};
  PackPlan copy_b = q.b;
  copy_b.pack = q.b.pack && !p.add;   // the product that is added finds it there
  const hipError_t e = pack(pack_args(p.a, q.a, es, to_a), pack_args(b, copy_b, es, to_b), s);
  if (e != hipSuccess) return e;
  if (q.a.pack) t.p.a = packed(p.a, q.a, es, to_a);
  if (q.b.pack) {
    const RowsOf c = packed(b, q.b, es, to_b);
    if (dw)
      t.p.b = c;
    else
      t.p.w = c.p, t.p.ldw = c.ld;
  }
  // a row operand's padding reads as zeros up to whole 16 bytes
  const int64_t per16 = 16 / es;
  t.a_k = up(p.K, per16);
  t.b_k = dx ? p.K : up(p.K, per16);
  t.a_r = up(p.N, per16);
  t.b_r = dw ? up(p.K, per16) : dx ? up(p.N, per16) : p.N;
  t.chunks = static_cast<int32_t>((p.K * es + kChunkBytes - 1) / kChunkBytes);
  t.tiles_m = q.tiles_m;
  t.few_rows = q.few_rows;
  t.tiles_n = q.tiles_n;
  const uint64_t run = (q.tiles + kXcds - 1) / kXcds;
  t.run = static_cast<uint32_t>(run < 32 ? run : 32);
  if (p.i8) return launch_grouped_int8(q.shape, t, q.tiles, s);
  switch (p.kind) {
    case GroupedKind::kLinear: return launch_grouped_tiles<Elem::kBf16, GroupedKind::kLinear>(q.shape, t, q.tiles, s);
    case GroupedKind::kGated: return launch_grouped_tiles<Elem::kBf16, GroupedKind::kGated>(q.shape, t, q.tiles, s);
    case GroupedKind::kDx: return launch_grouped_tiles<Elem::kBf16, GroupedKind::kDx>(q.shape, t, q.tiles, s);
    case GroupedKind::kDw: break;
  }
  return launch_grouped_tiles<Elem::kBf16, GroupedKind::kDw>(q.shape, t, q.tiles, s);
}

}  // namespace dsmoe
