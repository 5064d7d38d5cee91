// The tile kernels of the products over ragged groups, in the tiles and loops of
// tile.h.  A tile lies in one group: of the rows (y, dx: the groups' row tiles
// follow one another, the group of a tile is found on the device) or of the
// contraction (dW: every group has the same tiles and its own length of K).
// Rows taken by index are gathered by the copies themselves, through the lanes'
// offsets.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "act.h"
#include "grouped.h"
#include "tile.h"

namespace dsmoe {

struct GroupedArgs {
  GroupedGemm p;
  int64_t a_k, b_k;        // contraction length readable along a row (row operands: whole 16 bytes)
  int64_t a_r, b_r;        // kDw, kDx: columns of a, of w or b readable (whole 16 bytes)
  const int32_t* scale_index;   // i8: row r has scale scale_index[r] (null: r) of scale_n,
  int64_t scale_n;              // also where the rows were gathered before
  int32_t chunks;          // of K; not kDw
  uint32_t tiles_m;        // kDw: of a group
  uint32_t tiles_n;
  uint32_t run;            // consecutive tiles of an XCD
  uint64_t tile0;          // first tile of the launch
  bool few_rows;           // k256: most tiles have few rows (grouped_gemm.hip)
};

// Blocks are dispatched round-robin over the XCDs.  In a round of kXcds * run
// blocks each XCD takes a run of consecutive tiles, which share operand rows
// in its L2; the tiles in use are a prefix of the grid, which is sized for the
// worst case, so they are spread over all XCDs.
__device__ __forceinline__ uint64_t tile_of_block(const GroupedArgs& t) {
  const uint32_t slot = blockIdx.x / kXcds;
  return t.tile0 + (slot / t.run) * (kXcds * t.run) + (blockIdx.x % kXcds) * t.run + slot % t.run;
}

// Inclusive prefix sum over the lanes of a wave: within rows of 16 lanes by DPP
// shifts, then the totals of the rows before.
__device__ __forceinline__ uint32_t wave_scan(uint32_t v, int lane) {
  auto shr = [](uint32_t x, auto ctrl) {
    return static_cast<uint32_t>(
        __builtin_amdgcn_update_dpp(0, static_cast<int>(x), decltype(ctrl)::value, 0xF, 0xF, false));
  };
  v += shr(v, std::integral_constant<int, 0x111>{});   // row_shr:1
  v += shr(v, std::integral_constant<int, 0x112>{});   // row_shr:2
  v += shr(v, std::integral_constant<int, 0x114>{});   // row_shr:4
  v += shr(v, std::integral_constant<int, 0x118>{});   // row_shr:8
  auto total = [&](int l) { return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), l)); };
  const uint32_t t0 = total(15), t1 = total(31), t2 = total(47);
  const int row = lane >> 4;
  return v + (row >= 1 ? t0 : 0) + (row >= 2 ? t1 : 0) + (row >= 3 ? t2 : 0);
}

__device__ __forceinline__ int32_t group_begin(const Groups& g, int32_t i) {
  if (!g.offsets) return 0;
  return min(max(g.offsets[i], 0), static_cast<int32_t>(g.R));
}
__device__ __forceinline__ int32_t group_end(const Groups& g, int32_t i) {
  if (!g.offsets) return static_cast<int32_t>(g.R);
  return min(max(g.offsets[i + 1], 0), static_cast<int32_t>(g.R));
}

struct RowTile {
  int32_t group;
  int32_t r0, end;   // the tile's first row, the end of its group
  int32_t tn;        // its column tile
};

// The group, rows and columns of a tile; false past the last one.  A group's row
// tiles form bands of 4, a band is numbered column by column, so that the
// tiles an XCD works on at once share rows of both operands in its L2.  Every
// wave looks by itself, without LDS or barriers: 256 groups' offsets in flight,
// their tiles counted by prefix sums.
template <int ROWS>
__device__ __forceinline__ bool find_tile(const Groups& g, uint64_t tile, uint32_t tiles_n, RowTile& t) {
  const int lane = threadIdx.x & 63;
  uint64_t local = 0;
  int32_t lo = 0, hi = 0;
  bool found = false;
  if (!g.offsets) {
    hi = static_cast<int32_t>(g.R);
    t.group = 0;
    local = tile;
    found = tile < static_cast<uint64_t>((static_cast<uint32_t>(hi) + ROWS - 1) / ROWS) * tiles_n;
  } else {
    uint32_t before = 0;   // row tiles of the groups before
    constexpr int kBatch = 4;
    for (int32_t g0 = 0; g0 < g.n && !found; g0 += 64 * kBatch) {
      int32_t b[kBatch], e[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int32_t i = g0 + 64 * j + lane;
        b[j] = i < g.n ? g.offsets[i] : 0;
        e[j] = i < g.n ? g.offsets[i + 1] : 0;
      }
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        if (found) continue;
        b[j] = min(max(b[j], 0), static_cast<int32_t>(g.R));
        e[j] = min(max(e[j], 0), static_cast<int32_t>(g.R));
        const uint32_t n = e[j] > b[j] ? (static_cast<uint32_t>(e[j] - b[j]) + ROWS - 1) / ROWS : 0;
        const uint32_t sum = before + wave_scan(n, lane);
        const uint64_t first = static_cast<uint64_t>(sum - n) * tiles_n;
        const uint64_t mask = __ballot(tile >= first && tile < static_cast<uint64_t>(sum) * tiles_n);
        if (mask) {
          const int l = __builtin_ctzll(mask);
          lo = __builtin_amdgcn_readlane(b[j], l);
          hi = __builtin_amdgcn_readlane(e[j], l);
          t.group = g0 + 64 * j + l;
          const uint32_t at = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(sum - n), l));
          local = tile - static_cast<uint64_t>(at) * tiles_n;
          found = true;
        }
        before = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(sum), 63));
      }
    }
  }
  if (!found) return false;
  constexpr uint32_t kBand = 4;
  const uint32_t rows = (static_cast<uint32_t>(hi - lo) + ROWS - 1) / ROWS;
  const uint64_t per_band = static_cast<uint64_t>(kBand) * tiles_n;
  const uint32_t band = static_cast<uint32_t>(local / per_band), in = static_cast<uint32_t>(local % per_band);
  const uint32_t high = min(kBand, rows - band * kBand);
  t.r0 = lo + static_cast<int32_t>((band * kBand + in % high) * ROWS);
  t.end = hi;
  t.tn = static_cast<int32_t>(in / high);
  return true;
}

template <Elem E, int HM, int HN, int WM, int WN, GroupedKind KIND>
struct GroupedTile : TileCore<E, HM, HN, WM, WN, KIND == GroupedKind::kDw,
                              KIND == GroupedKind::kDw || KIND == GroupedKind::kDx, KIND == GroupedKind::kGated, true> {
  using Core = TileCore<E, HM, HN, WM, WN, KIND == GroupedKind::kDw,
                        KIND == GroupedKind::kDw || KIND == GroupedKind::kDx, KIND == GroupedKind::kGated, true>;
  using typename Core::Acc;
  using typename Core::SA;
  using typename Core::SB;
  using Core::a0, Core::a1, Core::b0, Core::b1, Core::c0, Core::c1, Core::get, Core::kGated, Core::kRowsAtOnce,
      Core::kRuns, Core::m0, Core::n0, Core::put;
  static constexpr bool kDw = KIND == GroupedKind::kDw, kI8 = E == Elem::kI8;
  static constexpr int kCols = kGated ? HN : 2 * HN;

  const GroupedArgs& t;
  const GroupedGemm& p;
  int32_t group;
  int64_t m_end;   // end of the rows of the result (kDw: within its group)
  bool found;

  __device__ __forceinline__ GroupedTile(const GroupedArgs& args, const uint8_t* mem) : Core(mem), t(args), p(args.p) {
    const uint64_t tile = tile_of_block(t);
    c0 = 0;
    if constexpr (kDw) {
      const uint32_t per_group = t.tiles_m * t.tiles_n;
      found = tile < static_cast<uint64_t>(per_group) * p.groups.n;
      if (!found) return;
      group = static_cast<int32_t>(tile / per_group);
      const uint32_t in = static_cast<uint32_t>(tile % per_group);
      constexpr uint32_t kBand = 4;
      const uint32_t band = in / (kBand * t.tiles_n), at = in % (kBand * t.tiles_n);
      const uint32_t rows = min(kBand, t.tiles_m - band * kBand);
      m0 = static_cast<int64_t>(band * kBand + at % rows) * 2 * HM;
      n0 = static_cast<int64_t>(at / rows) * 2 * HN;
      m_end = p.N;
      const int32_t lo = __builtin_amdgcn_readfirstlane(group_begin(p.groups, group));
      const int32_t hi = max(lo, __builtin_amdgcn_readfirstlane(group_end(p.groups, group)));
      c1 = static_cast<int32_t>((static_cast<uint32_t>(hi - lo) + Core::kChunk - 1) / Core::kChunk);
      a0 = SA(p.a.p, p.a.ld, m0, t.a_r, lo, hi, this->wave, this->lane);
      a1 = SA(p.a.p, p.a.ld, m0 + HM, t.a_r, lo, hi, this->wave, this->lane);
      b0 = SB(p.b.p, p.b.ld, n0, t.b_r, lo, hi, this->wave, this->lane);
      b1 = SB(p.b.p, p.b.ld, n0 + HN, t.b_r, lo, hi, this->wave, this->lane);
    } else {
      RowTile r;
      found = find_tile<2 * HM>(p.groups, tile, t.tiles_n, r);
      if (found) take(r);
    }
  }
  // y, dx: a tile found by its caller
  __device__ __forceinline__ GroupedTile(const GroupedArgs& args, const uint8_t* mem, const RowTile& r)
      : Core(mem), t(args), p(args.p), found(true) {
    c0 = 0;
    take(r);
  }
  __device__ __forceinline__ void take(const RowTile& r) {
    if constexpr (!kDw) {
      group = __builtin_amdgcn_readfirstlane(r.group);
      m0 = __builtin_amdgcn_readfirstlane(r.r0);
      m_end = __builtin_amdgcn_readfirstlane(r.end);
      n0 = static_cast<int64_t>(__builtin_amdgcn_readfirstlane(r.tn)) * kCols;
      c1 = t.chunks;
      if (p.a.index) {
        const int32_t n = static_cast<int32_t>(p.a.n);
        a0 = SA(p.a.p, p.a.ld, n, p.a.index + m0, m_end - m0, 0, t.a_k, this->wave, this->lane);
        a1 = SA(p.a.p, p.a.ld, n, p.a.index + m0 + HM, m_end - m0 - HM, 0, t.a_k, this->wave, this->lane);
      } else {
        a0 = SA(p.a.p, p.a.ld, m0, m_end, 0, t.a_k, this->wave, this->lane);
        a1 = SA(p.a.p, p.a.ld, m0 + HM, m_end, 0, t.a_k, this->wave, this->lane);
      }
      // the group's rows of w: N (kGated: 2 N), kDx: K
      const int64_t w_rows = KIND == GroupedKind::kDx ? p.K : kGated ? 2 * p.N : p.N;
      const char* w = static_cast<const char*>(p.w) + group * w_rows * p.ldw * Core::El::kBytes;
      const char* up = kGated ? w + p.N * p.ldw * Core::El::kBytes : w;
      b0 = SB(w, p.ldw, n0, t.b_r, 0, t.b_k, this->wave, this->lane);
      b1 = SB(up, p.ldw, kGated ? n0 : n0 + HN, t.b_r, 0, t.b_k, this->wave, this->lane);
    }
  }

  // The results, 8 columns of a row at a time.
  __device__ __forceinline__ void finish(const Acc& acc) const {
    const int run = threadIdx.x % kRuns;
    const int64_t n = n0 + run * 8;
    const int64_t cols = kDw ? p.K : p.N, left = cols - n;
    float ws[8], us[8];   // i8: scales of the columns
    if constexpr (kI8) {
      const int64_t at = static_cast<int64_t>(group) * (kGated ? 2 : 1) * p.N + n;
      load8(p.w_scale, at, true, left, ws);
      if constexpr (kGated) load8(p.w_scale, at + p.N, true, left, us);
    }
#pragma unroll
    for (int ha = 0; ha < 2; ++ha) {
      put(acc[ha]);
      if (static_cast<int>(threadIdx.x) >= kRowsAtOnce * kRuns) continue;
#pragma unroll 1
      for (int r = threadIdx.x / kRuns; r < HM; r += kRowsAtOnce) {
        const int64_t m = m0 + ha * HM + r;
        if (m >= m_end || left <= 0) break;
        float v[8], u[8];
        get(r, run * 8, v);
        if constexpr (kGated) get(r, HN + run * 8, u);
        if constexpr (kI8) {
          const int64_t row = t.scale_index ? t.scale_index[m] : m;
          const float xs = row >= 0 && row < t.scale_n ? p.a_scale[row] : 0.0f;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            v[e] = v[e] * xs * ws[e];
            if constexpr (kGated) u[e] = u[e] * xs * us[e];
          }
        }
        const int64_t y = (kDw ? static_cast<int64_t>(group) * p.N + m : m) * p.ldy + n;
        if constexpr (kGated) {
          if (p.z) {
            store8(p.z, m * p.ldz + n, false, left, v);
            store8(p.z, m * p.ldz + p.N + n, false, left, u);
          }
          const float s = p.row_scale ? p.row_scale[m] : 1.0f;
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = s * (act_f32(p.act, v[e]) * u[e]);
        }
        if (!kGated && !kI8 && p.add) {
          float o[8];
          load8(p.y, y, true, left, o);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = plus_rest(o[e], v[e]);
        }
        store8(p.y, y, p.y_f32, left, v);
      }
    }
  }
};

// A tile of few rows (a group's last one, or its only one) is computed in half the
// height, or in 3/4 of it.  4096 tokens to 8 of 256 experts, 128 rows each: gated
// in bf16 2.78 ms (whole tiles only 3.02, with the half 2.87), in 8 bits 1.53 (1.64,
// 1.59).
template <Elem E, int HM, int HN, int WM, int WN, GroupedKind KIND>
__global__ __launch_bounds__(64 * WM * WN) void grouped_phased_kernel(GroupedArgs args) {
  using T = GroupedTile<E, HM, HN, WM, WN, KIND>;
  using T3 = GroupedTile<E, HM / 4 * 3, HN, WM, WN, KIND>;
  using T2 = GroupedTile<E, HM / 2, HN, WM, WN, KIND>;
  constexpr int kStages = 3;
  constexpr int kBytes = T::lds_bytes(2) > T2::lds_bytes(kStages) ? T::lds_bytes(2) : T2::lds_bytes(kStages);
  __shared__ __attribute__((aligned(1024))) uint8_t s_mem[kBytes];
  RowTile r;
  if (!find_tile<2 * HM>(args.p.groups, tile_of_block(args), args.tiles_n, r)) return;   // the whole block
  const int32_t rows = __builtin_amdgcn_readfirstlane(r.end - r.r0);
  if (rows <= HM) {
    T2 w(args, s_mem, r);
    typename T2::Acc acc;
    paired_loop<kStages>(w, acc);
    w.finish(acc);
  } else if (rows <= HM / 2 * 3) {
    T3 w(args, s_mem, r);
    typename T3::Acc acc;
    phased_loop(w, acc);
    w.finish(acc);
  } else {
    T w(args, s_mem, r);
    typename T::Acc acc;
    phased_loop(w, acc);
    w.finish(acc);
  }
}

template <Elem E, int HM, int HN, int WM, int WN, int S, GroupedKind KIND>
__global__ __launch_bounds__(64 * WM * WN) void grouped_ring_kernel(GroupedArgs args) {
  using T = GroupedTile<E, HM, HN, WM, WN, KIND>;
  __shared__ __attribute__((aligned(1024))) uint8_t s_mem[T::lds_bytes(S)];
  T w(args, s_mem);
  if (!w.found) return;
  typename T::Acc acc;
  ring_loop<S>(w, acc);
  w.finish(acc);
}

// The tile shapes (grouped_gemm.hip).
enum class GroupedShape : int { k256, k128, k64, k32x128 };

// The tiles of a launch after another, which holds fewer than 2^32 threads.
template <typename F>
hipError_t by_tiles(GroupedArgs t, uint64_t tiles, F f) {
  constexpr uint64_t kMost = 1u << 22;
  const uint64_t round = static_cast<uint64_t>(kXcds) * t.run;
  for (uint64_t t0 = 0; t0 < tiles; t0 += kMost) {
    const uint64_t n = tiles - t0 < kMost ? tiles - t0 : kMost;
    t.tile0 = t0;
    f(t, static_cast<uint32_t>((n + round - 1) / round * round));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// 256 x 256 tiles: blocks that stay (grouped_stream.h) for dW, and for y of more than
// few rows per group (grouped_gemm.hip); a block for each tile for the gated product,
// whose longer epilogue would not stay in the instruction cache (one token 200 us
// instead of 134; 4096 tokens to 256 experts, in whole tiles, 3.30 ms instead of
// 3.08), and for dx, where the two are equal in whole tiles.
template <Elem E, GroupedKind KIND>
hipError_t launch_grouped_256(const GroupedArgs& t, uint64_t tiles, hipStream_t s);

template <Elem E, GroupedKind KIND>
hipError_t launch_grouped_tiles(GroupedShape shape, const GroupedArgs& t, uint64_t tiles, hipStream_t s) {
  if (shape == GroupedShape::k256) return launch_grouped_256<E, KIND>(t, tiles, s);
  return by_tiles(t, tiles, [&](const GroupedArgs& q, uint32_t grid) {
    if (shape == GroupedShape::k128)
      grouped_ring_kernel<E, 64, 64, 2, 4, 2, KIND><<<grid, 512, 0, s>>>(q);
    else if (shape == GroupedShape::k64 || KIND == GroupedKind::kDw)
      grouped_ring_kernel<E, 32, 32, 2, 2, 4, KIND><<<grid, 256, 0, s>>>(q);
    else if constexpr (KIND != GroupedKind::kDw)
      grouped_ring_kernel<E, 16, 64, 1, 4, 4, KIND><<<grid, 256, 0, s>>>(q);
  });
}
hipError_t launch_grouped_int8(GroupedShape shape, const GroupedArgs& t, uint64_t tiles, hipStream_t s);

}  // namespace dsmoe
