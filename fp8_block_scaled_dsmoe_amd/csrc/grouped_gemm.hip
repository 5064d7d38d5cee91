// Products over rows grouped by expert with ragged sizes, outside FP8: y, dx and
// dW of the grouped linear and gated linear operators in bf16, and y of their
// 8-bit forms.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.h"
#include "grouped.h"
#include "grouped_tile.h"
#include "vec8.h"

namespace dsmoe {
namespace {

// Copies of operand rows into aligned rows of whole 16 bytes: dst [rows][segs]
// segments = src [rows][cols] or its rows index[r] (an index outside [0, n):
// zeros), the padding zeroed.
struct PackArgs {
  const char* src;
  char* dst;
  const int32_t* index;
  int64_t ld, rows, cols, n;   // ld, cols in bytes
};
__global__ __launch_bounds__(256) void pack_grouped_kernel(PackArgs a) {
  const int64_t segs = (a.cols + 15) / 16, all = a.rows * segs;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < all;
       i += static_cast<int64_t>(gridDim.x) * 256) {
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

struct GroupedPlan {
  PackPlan a, b;         // b: w, or kDw's b
  uint32_t tiles_m, tiles_n;
  uint64_t tiles;        // at most
};

GroupedPlan make_plan(const GroupedGemm& p) {
  GroupedPlan q{};
  const int64_t R = p.groups.R, G = p.groups.n;
  const int es = p.i8 ? 1 : 2;
  constexpr int64_t rows = 64, cols = 64;
  if (p.kind == GroupedKind::kDw) {
    q.a = plan_k_rows(p.a, R, p.N);
    q.b = plan_k_rows(p.b, R, p.K);
    q.tiles_m = static_cast<uint32_t>((p.N + rows - 1) / rows);
    q.tiles_n = static_cast<uint32_t>((p.K + cols - 1) / cols);
    q.tiles = static_cast<uint64_t>(q.tiles_m) * q.tiles_n * G;
    return q;
  }
  q.a = plan_rows(p.a, R, p.K, es);
  const bool dx = p.kind == GroupedKind::kDx, gated = p.kind == GroupedKind::kGated;
  const RowsOf w{p.w, p.ldw, G * (dx ? p.K : gated ? 2 * p.N : p.N), nullptr, false};
  q.b = plan_rows(w, w.n, dx ? p.N : p.K, es);
  q.tiles_n = static_cast<uint32_t>((p.N * (gated ? 2 : 1) + cols - 1) / cols);
  const int64_t busy = R < G ? R : G;   // groups with rows; each has at most one tile that is not full
  q.tiles = static_cast<uint64_t>((R + (rows - 1) * busy) / rows) * q.tiles_n;
  return q;
}

hipError_t pack(const RowsOf& o, const PackPlan& q, int es, void* dst, hipStream_t s) {
  const int64_t ld = up(q.cols * es, 16), all = q.rows * (ld / 16);
  if (all == 0) return hipSuccess;
  const int64_t blocks = (all + 255) / 256;
  pack_grouped_kernel<<<static_cast<uint32_t>(blocks < 8192 ? blocks : 8192), 256, 0, s>>>(
      PackArgs{static_cast<const char*>(o.p), static_cast<char*>(dst), q.gather ? o.index : nullptr, o.ld * es, q.rows,
               q.cols * es, o.n});
  return hipGetLastError();
}

// The operand after its copy.
RowsOf packed(const RowsOf& o, const PackPlan& q, int es, void* dst) {
  return RowsOf{dst, up(q.cols * es, 16) / es, q.rows, q.gather ? nullptr : o.index, true};
}

template <Elem E, GroupedKind KIND>
hipError_t launch_tiles(GroupedArgs t, uint64_t tiles, hipStream_t s) {
  // a launch holds fewer than 2^32 threads
  constexpr uint64_t kMost = 1u << 22;
  for (uint64_t t0 = 0; t0 < tiles; t0 += kMost) {
    const uint64_t n = tiles - t0 < kMost ? tiles - t0 : kMost;
    t.tile0 = t0;
    const uint64_t round = static_cast<uint64_t>(kXcds) * t.run;
    const uint32_t grid = static_cast<uint32_t>((n + round - 1) / round * round);
    grouped_ring_kernel<E, 32, 32, 2, 2, 4, KIND><<<grid, 256, 0, s>>>(t);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

bool rows_copyable(const RowsOf& o, int64_t cols, int bytes) {
  return (reinterpret_cast<uintptr_t>(o.p) & 15) == 0 && o.ld * bytes % 16 == 0 && (cols * bytes % 16 == 0 || o.padded);
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
  char* ws = static_cast<char*>(p.workspace);
  hipError_t e = hipSuccess;
  if (q.a.pack) {
    if ((e = pack(p.a, q.a, es, ws, s)) != hipSuccess) return e;
    t.p.a = packed(p.a, q.a, es, ws);
  }
  if (q.b.pack) {
    const RowsOf b = dw ? p.b : RowsOf{p.w, p.ldw, q.b.rows, nullptr, false};
    char* to = ws + q.a.bytes;
    if ((e = pack(b, q.b, es, to, s)) != hipSuccess) return e;
    const RowsOf c = packed(b, q.b, es, to);
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
  t.tiles_n = q.tiles_n;
  const uint64_t run = (q.tiles + kXcds - 1) / kXcds;
  t.run = static_cast<uint32_t>(run < 32 ? run : 32);
  switch (p.kind) {
    case GroupedKind::kLinear:
      return p.i8 ? launch_tiles<Elem::kI8, GroupedKind::kLinear>(t, q.tiles, s)
                  : launch_tiles<Elem::kBf16, GroupedKind::kLinear>(t, q.tiles, s);
    case GroupedKind::kGated:
      return p.i8 ? launch_tiles<Elem::kI8, GroupedKind::kGated>(t, q.tiles, s)
                  : launch_tiles<Elem::kBf16, GroupedKind::kGated>(t, q.tiles, s);
    case GroupedKind::kDx: return launch_tiles<Elem::kBf16, GroupedKind::kDx>(t, q.tiles, s);
    case GroupedKind::kDw: break;
  }
  return launch_tiles<Elem::kBf16, GroupedKind::kDw>(t, q.tiles, s);
}

}  // namespace dsmoe
