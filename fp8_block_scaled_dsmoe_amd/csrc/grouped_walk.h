// The order in which the blocks that stay (grouped_stream.h) take their tiles: whole
// numbers only, the same on the device and on the host.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dsmoe {

// What of the problem a tile is: rows [m0, m_end) of the result at most (dW: of
// the group's), columns from n0 on.
struct StreamTile {
  int32_t group;
  int32_t m0, m_end, n0;
  int32_t k0, k1;        // dW: the group's rows
  int32_t chunks;        // at least 1: a group without rows has one of zeros
};

struct StreamSizes {
  int32_t groups;
  int32_t m_end;         // dW: rows of a group's result
  int32_t chunks;        // y: of K
  uint32_t tiles_m;      // dW: of a group
  uint32_t tiles_n;
};

// A block's tile of number `tile`, which becomes that of its next one, `step` further;
// false past the last.  Group g's rows are [begin[g], end[g]); y: first[g] row tiles come before them
// (first[groups]: all), and walk is a group that tile's is not before.  read: of
// a table's value.
template <bool DW, int ROWS, int COLS, int CHUNK, typename Read>
__host__ __device__ __forceinline__ bool next_stream_tile(const StreamSizes& s, const int32_t* begin, const int32_t* end,
                                                          const int32_t* first, uint32_t step, uint32_t& tile, int32_t& walk,
                                                          Read read, StreamTile& d) {
  constexpr uint32_t kBand = DW ? 8 : 4;   // row tiles that share their columns' rows in L2
  uint32_t local, rows;
  if constexpr (DW) {
    const uint32_t per_group = s.tiles_m * s.tiles_n;
    const uint32_t g = tile / per_group;
    if (g >= static_cast<uint32_t>(s.groups)) return false;
    d.group = static_cast<int32_t>(g);
    local = tile - g * per_group;
    rows = s.tiles_m;
  } else {
    // tile >= first[walk] * tiles_n
    int32_t f0 = read(first[walk]), f1 = f0;
    while (walk < s.groups) {
      f1 = read(first[walk + 1]);
      if (tile < static_cast<uint32_t>(f1) * s.tiles_n) break;
      f0 = f1;
      ++walk;
    }
    if (walk >= s.groups) return false;
    d.group = walk;
    local = tile - static_cast<uint32_t>(f0) * s.tiles_n;
    rows = static_cast<uint32_t>(f1 - f0);
  }
  // past the group only where offsets that break the rule let a count wrap
  if (local >= rows * s.tiles_n) return false;
  const int32_t lo = read(begin[d.group]);
  const int32_t hi = read(end[d.group]);
  const uint32_t per_band = kBand * s.tiles_n, band = local / per_band, in = local - band * per_band;
  const uint32_t behind = rows - band * kBand, high = kBand < behind ? kBand : behind;
  const uint32_t tn = in / high, tm = band * kBand + (in - tn * high);
  d.n0 = static_cast<int32_t>(tn) * COLS;
  d.m0 = static_cast<int32_t>(tm) * ROWS;
  if constexpr (DW) {
    const int32_t n = static_cast<int32_t>((static_cast<uint32_t>(hi - lo) + CHUNK - 1) / CHUNK);
    d.m_end = s.m_end;
    d.k0 = lo, d.k1 = hi;
    d.chunks = n > 1 ? n : 1;
  } else {
    d.m0 += lo;
    d.m_end = hi;
    d.k0 = d.k1 = 0;
    d.chunks = s.chunks;
  }
  tile += step;
  return true;
}

// The first tile of a block: each XCD has a run of consecutive tiles at a time.
__host__ __device__ __forceinline__ uint32_t first_stream_tile(uint32_t block, uint32_t blocks, uint32_t xcds) {
  return block % xcds * (blocks / xcds) + block / xcds;
}

// The tiles that the copies may have entered past the products': they are two chunks
// ahead, and a tile has at least one.
constexpr int kStreamAhead = 2;

}  // namespace dsmoe
