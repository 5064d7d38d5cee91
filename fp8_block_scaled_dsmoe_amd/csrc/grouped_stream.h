// The 256-row tiles of the grouped products by blocks that stay: a block takes
// every gridDim-th tile, and its copies run on over the borders of tiles, so that
// the next tile's first chunks arrive while the last one's products run and
// its results are written.  The results leave from the registers, since LDS holds
// the next chunks: turned among the lanes so that a quad has 64 bytes of a row; a
// wave's 64 columns are whole 128-byte lines.  The two waves of a SIMD are half a phase
// apart (phased_loop); at a tile's end both write at once.
//
// Bound by the copies and LDS reads beside the matrix instructions, 1.42 us a chunk
// (64 KB copied, 192 KB read from LDS by the waves; without the products 1.3), and
// by the tile's border, 5 to 7 us of first chunks from memory, turning and storing
// 128 KB of results.  A block for each tile, against these, on one card: y of 256
// experts, 262144 rows of uneven groups, 7168 x 2048 (grouped_phased_kernel): 7.13 ms,
// 6.70; dW of 32 experts with 512 rows each, 7168 x 2048 (this kernel with as many blocks
// as tiles): 671 us, 568 in bf16, 795, 755 in float32, in uneven groups 748, 585 and
// 988, 778; 8-bit 4096 x 7168 x 2048: 70 us, 67.  Writing in two halves, each while the
// SIMD's other wave multiplies: dW 598 instead of 575 in bf16.
#pragma once

#include "dsmoe.h"
#include "grouped_tile.h"
#include "grouped_walk.h"

namespace dsmoe {

// The kernel's arguments, read again: what is read through it does not stay in
// scalar registers over the loop.
__device__ __forceinline__ const GroupedArgs& arguments_again() {
  auto q = __builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(q));
  return *(const GroupedArgs*)q;
}
// The lane, so that what depends on it is computed where it is used.
__device__ __forceinline__ int lane_again(int lane) {
  asm volatile("" : "+v"(lane));
  return lane;
}

// y = a W^T (kLinear) or dW.  A wave's columns of the two halves of B lie side by
// side in the result (PAIR).
template <Elem E, int HM, int HN, int WM, int WN, GroupedKind KIND>
using StreamCore = TileCore<E, HM, HN, WM, WN, KIND == GroupedKind::kDw, KIND == GroupedKind::kDw, false, true, HN / WN>;

template <Elem E, int HM, int HN, int WM, int WN, GroupedKind KIND>
struct Stream : StreamCore<E, HM, HN, WM, WN, KIND> {
  using Core = StreamCore<E, HM, HN, WM, WN, KIND>;
  using typename Core::Acc;
  using typename Core::SA;
  using typename Core::SB;
  using typename Core::Sums;
  using Core::a0, Core::a1, Core::b0, Core::b1, Core::lane, Core::TM, Core::TN, Core::wave, Core::wm,
      Core::wn;
  static constexpr bool kDw = KIND == GroupedKind::kDw, kI8 = E == Elem::kI8;
  static_assert(kDw || KIND == GroupedKind::kLinear, "y or dW");
  static constexpr int kCols = 2 * HN, W = HN / WN;   // of a tile; of a wave in either half
  static constexpr int kWide = 2 * W;                 // a wave's columns in the result, side by side
  static constexpr int kMaxGroups = DSMOE_MAX_EXPERTS;
  // The queue: tiles (a power of 2), integers of one.  It holds the products' tile,
  // whose entry is free once the next one is popped, and those that the copies have
  // entered past it.
  static constexpr int kQueue = 4, kEntry = 8;
  static_assert(kQueue >= 1 + kStreamAhead && (kQueue & (kQueue - 1)) == 0, "an entered tile's entry may not be in use");

  const GroupedArgs& t;
  const GroupedGemm& p;
  struct Table;
  const Table& table;
  uint32_t tile;             // the copies' next
  int32_t walk;              // its group at least
  // The tiles whose products are not done: a queue of the wave's own in LDS.
  int32_t* const queue;
  int32_t entered, done;
  StreamTile pt;             // the products' tile
  int32_t cl, pl;            // chunks left of the copies', the products' tile

  // What the walk over the groups needs, in LDS (a load from memory would wait for
  // every copy and store on the way): their rows, and for g <= G the row tiles
  // before them.  Every wave scans, wave 0 writes.
  struct Table {
    int32_t begin[kMaxGroups], end[kMaxGroups], first[kDw ? 1 : kMaxGroups + 1];
    int32_t queue[Core::NW * kQueue * kEntry];
  };
  __device__ __forceinline__ Stream(const GroupedArgs& args, const uint8_t* mem, Table& s)
      : Core(mem), t(args), p(args.p), table(s), queue(s.queue + wave * kQueue * kEntry) {
    int32_t before = 0;
    for (int32_t g0 = 0; g0 < p.groups.n; g0 += 64) {
      const int32_t g = g0 + lane;
      int32_t n = 0;
      if (g < p.groups.n) {
        const int32_t lo = group_begin(p.groups, g), hi = max(lo, group_end(p.groups, g));
        n = static_cast<int32_t>((static_cast<uint32_t>(hi - lo) + 2 * HM - 1) / (2 * HM));
        if (wave == 0) s.begin[g] = lo, s.end[g] = hi;
      }
      if constexpr (!kDw) {
        const int32_t sum = before + static_cast<int32_t>(wave_scan(static_cast<uint32_t>(n), lane));
        if (wave == 0 && g < p.groups.n) s.first[g] = sum - n;
        before = __builtin_amdgcn_readlane(sum, 63);
      }
    }
    if constexpr (!kDw)
      if (wave == 0 && lane == 0) s.first[p.groups.n] = before;
    __syncthreads();
    tile = first_stream_tile(blockIdx.x, gridDim.x, kXcds);
    walk = 0;
    entered = done = 0;
  }

  // The copies' next tile; false past the last.
  __device__ __forceinline__ bool next(StreamTile& d) {
    const StreamSizes z{p.groups.n, static_cast<int32_t>(p.N), t.chunks, t.tiles_m, t.tiles_n};
    return next_stream_tile<kDw, 2 * HM, kCols, Core::kChunk>(
        z, table.begin, table.end, table.first, gridDim.x, tile, walk,
        [](const int32_t& v) { return __builtin_amdgcn_readfirstlane(v); }, d);
  }
  // The products' tile: the queue's head.
  __device__ __forceinline__ void head() {
    const int32_t* q = queue + (done & (kQueue - 1)) * kEntry;
    pt.group = __builtin_amdgcn_readfirstlane(q[0]);
    pt.m0 = __builtin_amdgcn_readfirstlane(q[1]);
    pt.m_end = __builtin_amdgcn_readfirstlane(q[2]);
    pt.n0 = __builtin_amdgcn_readfirstlane(q[3]);
    pl = __builtin_amdgcn_readfirstlane(q[4]);
  }
  // The next one; false past the last (the copies enter a tile two chunks before
  // its first products).
  __device__ __forceinline__ bool pop() {
    if (++done >= entered) return false;
    head();
    return true;
  }

  static __device__ __forceinline__ SA source_a(const GroupedArgs& t, const StreamTile& d, int half, int wave, int lane) {
    const GroupedGemm& p = t.p;
    const int64_t m = static_cast<int64_t>(d.m0) + half * HM;
    if constexpr (kDw) {
      return SA(p.a.p, p.a.ld, m, t.a_r, d.k0, d.k1, wave, lane);
    } else {
      if (p.a.index)
        return SA(p.a.p, p.a.ld, static_cast<int32_t>(p.a.n), p.a.index + m, d.m_end - m, 0, t.a_k, wave, lane);
      return SA(p.a.p, p.a.ld, m, d.m_end, 0, t.a_k, wave, lane);
    }
  }
  // The copies enter the next tile; past the last one they bring zeros, as of no
  // rows (without a branch: the compiler would keep what both sides write in
  // memory).
  __device__ __forceinline__ void enter() {
    StreamTile d;
    const bool some = next(d);
    if (!some) {
      d.group = 0;
      d.m0 = d.m_end = d.n0 = 0;
      d.k0 = d.k1 = 0;
      d.chunks = 0x7fffffff;
    }
    cl = d.chunks;
    if (some && lane == 0) {
      int32_t* q = queue + (entered & (kQueue - 1)) * kEntry;
      q[0] = d.group, q[1] = d.m0, q[2] = d.m_end, q[3] = d.n0, q[4] = d.chunks;
    }
    entered += some;
    const GroupedArgs& t = arguments_again();
    const GroupedGemm& p = t.p;
    const int lane = lane_again(this->lane);
    a0 = source_a(t, d, 0, wave, lane);
    a1 = source_a(t, d, 1, wave, lane);
    const int64_t rows = some ? t.b_r : 0;
    if constexpr (kDw) {
      b0 = SB(p.b.p, p.b.ld, d.n0, rows, d.k0, d.k1, wave, lane);
      b1 = SB(p.b.p, p.b.ld, d.n0 + W, rows, d.k0, d.k1, wave, lane);
    } else {
      const char* w = static_cast<const char*>(p.w) + d.group * p.N * p.ldw * Core::El::kBytes;
      b0 = SB(w, p.ldw, d.n0, rows, 0, t.b_k, wave, lane);
      b1 = SB(w, p.ldw, d.n0 + W, rows, 0, t.b_k, wave, lane);
    }
  }

  __device__ __forceinline__ void load4(const float* q, int32_t left, float* v) const {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = 0.0f;
    if (left >= 4) {
      const f32x4 w = *reinterpret_cast<const f32x4_at4*>(q);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = w[e];
    } else {
#pragma unroll
      for (int e = 0; e < 3; ++e)
        if (e < left) v[e] = q[e];
    }
  }

  // A fragment pair's 32 columns of 16 rows go to memory with a store for every 64
  // bytes of a row, 16 bytes a lane.  Stores run at full rate only where the lanes
  // of a quad are neighbours in their row (38 GB/s of a CU with a row for each of
  // 16 lanes, 135 with whole lines), so lane 4 m + s takes segment s of row m.
  template <bool F32>
  struct Out {
    u32x4 w[F32 ? 2 : 1];
  };
  // v: the lane's 4 columns of either fragment.  bf16: first the lanes of rows 16
  // apart exchange halves of their fragments, so that lanes 0-15 have columns 0-7
  // of the pair, 16-31 columns 16-23, 32-47 columns 8-15 and 48-63 columns 24-31.
  template <bool F32>
  static __device__ __forceinline__ Out<F32> turn(const float (&v)[2][4], int lane) {
    const int s = lane & 3;
    const int from = 4 * ((lane >> 2) + 16 * (F32 ? s : (s & 1) << 1 | s >> 1));
    auto get = [&](uint32_t x) {
      return static_cast<uint32_t>(__builtin_amdgcn_ds_bpermute(from, static_cast<int>(x)));
    };
    Out<F32> o;
    if constexpr (F32) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o.w[j][e] = get(__float_as_uint(v[j][e]));
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const auto q = __builtin_amdgcn_permlane16_swap(f32x2_to_bf16x2(v[0][2 * h], v[0][2 * h + 1]),
                                                        f32x2_to_bf16x2(v[1][2 * h], v[1][2 * h + 1]), false, false);
        o.w[0][h] = get(q[0]), o.w[0][2 + h] = get(q[1]);
      }
    }
    return o;
  }
  // row: that the lane writes, from the pair's first column on.  FULL: all 32
  // columns are in the result, else `left` of them.
  template <bool FULL, bool F32>
  static __device__ __forceinline__ void pair_out(char* row, int32_t left, const Out<F32>& o, int lane) {
    constexpr int ES = F32 ? 4 : 2, kPer = 16 / ES;
#pragma unroll
    for (int j = 0; j < (F32 ? 2 : 1); ++j) {
      const int c = 16 * j + kPer * (lane & 3);
      if (FULL || left - c >= kPer) {
        *reinterpret_cast<u32x4_at2*>(row + ES * c) = o.w[j];
      } else {
#pragma unroll
        for (int e = 0; e < kPer - 1; ++e) {
          if (e >= left - c) break;
          if constexpr (F32)
            reinterpret_cast<uint32_t*>(row)[c + e] = o.w[j][e];
          else
            reinterpret_cast<uint16_t*>(row)[c + e] = static_cast<uint16_t>(o.w[j][e / 2] >> (e % 2 * 16));
        }
      }
    }
  }

  // The results of the products' tile, then zeros for the next one's.  A lane
  // holds row l % 16 of its A fragment and columns 4 (l / 16) + [0, 4) of its B
  // fragment.  FULL: all of the wave's columns are in the result.
  template <bool FULL, bool F32>
  __device__ __forceinline__ void finish_as(Acc& acc) const {
    constexpr int ES = F32 ? 4 : 2;
    static_assert(TN == 2, "fragment pairs");
    const GroupedArgs& t = arguments_again();
    const GroupedGemm& p = t.p;
    const int lane = lane_again(this->lane);
    const int32_t n = pt.n0 + wn * kWide;   // the wave's first column
    const int32_t left = static_cast<int32_t>((kDw ? p.K : p.N) - n);
    const int32_t rows = pt.m_end - pt.m0 - wm * (HM / WM);   // from the wave's first on
    const int64_t row0 = (kDw ? static_cast<int64_t>(pt.group) * p.N : 0) + pt.m0 + wm * (HM / WM);
    const int64_t ld = p.ldy * ES;
    char* const y = static_cast<char*>(p.y) + row0 * ld + static_cast<int64_t>(n) * ES;
    const uint32_t y_lane = static_cast<uint32_t>(lane >> 2) * static_cast<uint32_t>(ld);   // of the row it writes
    // the factors, before the first store: a wait for a load would wait for the
    // stores before it
    float ws[2][TN][4];   // i8: scales of the columns
    if constexpr (kI8) {
      const float* s = p.w_scale + static_cast<int64_t>(pt.group) * p.N + n;
#pragma unroll
      for (int hb = 0; hb < 2; ++hb)
#pragma unroll
        for (int j = 0; j < TN; ++j) {
          const int c = hb * W + 16 * j + 4 * (lane >> 4);
          load4(s + c, left - c, ws[hb][j]);
        }
    }
    float xs[2][TM];      // and of the rows
    if constexpr (kI8) {
#pragma unroll
      for (int ha = 0; ha < 2; ++ha)
#pragma unroll
        for (int i = 0; i < TM; ++i) {
          const int32_t r = ha * HM + 16 * i + (lane & 15);
          const int64_t m = row0 + r;
          const int64_t row = r >= rows ? -1 : t.scale_index ? t.scale_index[m] : m;
          xs[ha][i] = row >= 0 && row < t.scale_n ? p.a_scale[row] : 0.0f;
        }
    }
#pragma unroll
    for (int ha = 0; ha < 2; ++ha)
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        const int32_t r = ha * HM + 16 * i;   // the fragment's rows from the wave's first on
        if (r < rows) {
          const bool in = r + (lane >> 2) < rows;   // the row it writes
          char* const yr = y + r * ld + y_lane;
          auto value = [&](int hb, int j, float* v) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              v[e] = static_cast<float>(acc[ha][hb][i][j][e]);
              if constexpr (kI8) v[e] = v[e] * xs[ha][i] * ws[hb][j][e];
            }
          };
          Out<F32> o[2];
#pragma unroll
          for (int hb = 0; hb < 2; ++hb) {
            float v[2][4];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              value(hb, j, v[j]);
              if constexpr (F32 && !kI8) {
                if (p.add && r + (lane & 15) < rows) {
                  float add[4];
                  const int32_t at = hb * W + 16 * j + 4 * (lane >> 4);
                  load4(reinterpret_cast<const float*>(y + (r + (lane & 15)) * ld) + at, left - at, add);
#pragma unroll
                  for (int e = 0; e < 4; ++e) v[j][e] = plus_rest(add[e], v[j][e]);
                }
              }
            }
            o[hb] = turn<F32>(v, lane);
          }
          if (in) {
#pragma unroll
            for (int hb = 0; hb < 2; ++hb) pair_out<FULL, F32>(yr + hb * W * ES, left - hb * W, o[hb], lane);
          }
        }
#pragma unroll
        for (int hb = 0; hb < 2; ++hb)
#pragma unroll
          for (int j = 0; j < TN; ++j) acc[ha][hb][i][j] = Sums{};
      }
  }
  // Returns the number of stores, at least, that were made: kStores, or kStoresF32
  // of float32, where the wave's part of the tile is full, else 0.
  static constexpr int kStores = 4 * TM, kStoresF32 = 2 * kStores;
  __device__ __forceinline__ int finish(Acc& acc) const {
    const GroupedArgs& t = arguments_again();
    const bool f32 = t.p.y_f32, full = pt.n0 + (wn + 1) * kWide <= (kDw ? t.p.K : t.p.N);
    if (f32)
      full ? finish_as<true, true>(acc) : finish_as<false, true>(acc);
    else
      full ? finish_as<true, false>(acc) : finish_as<false, false>(acc);
    if (!full || (wm + 1) * (HM / WM) + HM > pt.m_end - pt.m0) return 0;
    return f32 ? kStoresF32 : kStores;
  }
};

// The loop is phased_loop's, over all chunks of the block's tiles.
template <Elem E, int HM, int HN, int WM, int WN, GroupedKind KIND>
__global__ __launch_bounds__(64 * WM * WN) void grouped_stream_kernel(GroupedArgs args) {
  using T = Stream<E, HM, HN, WM, WN, KIND>;
  constexpr int TM = T::TM, TN = T::TN, LA = T::LA, LB = T::LB;
  static_assert(T::NW == 8, "two waves per SIMD");
  __shared__ __attribute__((aligned(1024))) uint8_t s_mem[2 * T::kStage];
  __shared__ typename T::Table s_table;
  T w(args, s_mem, s_table);
  w.enter();
  if (w.entered == 0) return;   // the whole block
  w.head();
  typename T::Acc acc;
  T::clear(acc);
  typename T::Frag fa[TM][2], fb[3][TN][2];

  uint32_t st = w.lds, nx = w.lds + T::kStage;
  w.copy_b0(st);
  w.copy_a0(st);
  w.copy_b1(st);
  w.copy_a1(st);
  if (--w.cl == 0) w.enter();
  w.copy_b0(nx);
  w.copy_a0(nx);
  w.copy_b1(nx);
  --w.cl;
  wait_copies<0>();
  block_barrier();
#define DSMOE_READ_A(stage, half)                                                                 \
  _Pragma("unroll") for (int i = 0; i < TM; ++i)                                                  \
      _Pragma("unroll") for (int kk = 0; kk < 2; ++kk) fa[i][kk] = w.ra.read(stage, half, i, kk)
#define DSMOE_READ_B(f, stage, half)                                                              \
  _Pragma("unroll") for (int j = 0; j < TN; ++j)                                                  \
      _Pragma("unroll") for (int kk = 0; kk < 2; ++kk) fb[f][j][kk] = w.rb.read(stage, half, j, kk)
  // The end of a phase's reads and copies, then its products (phased_loop).  The
  // stores of finish() are counted with the copies, in the order of their issue;
  // in the two phases after it the copies that have to be there were issued before
  // them, so that the stores may still be on their way.  Other loads and stores in
  // between make a wait longer, never shorter.
  int after = 0, stores = 0;
#define DSMOE_PHASE(ha)                                                                               \
  do {                                                                                                \
    if (after == 0)                                                                                   \
      wait_copies<2 * LA + 2 * LB>();                                                                 \
    else if (--after, stores == T::kStoresF32)                                                        \
      wait_copies<2 * LA + 2 * LB + T::kStoresF32>();                                                 \
    else                                                                                              \
      wait_copies<2 * LA + 2 * LB + T::kStores>();                                                    \
    wait_lds();                                                                                       \
    block_barrier();                                                                                  \
    __builtin_amdgcn_sched_barrier(0);                                                                \
    __builtin_amdgcn_s_setprio(1);                                                                    \
    _Pragma("unroll") for (int kk = 0; kk < 2; ++kk)                                                  \
        _Pragma("unroll") for (int hb = 0; hb < 2; ++hb)                                              \
            _Pragma("unroll") for (int i = 0; i < TM; ++i)                                            \
                _Pragma("unroll") for (int j = 0; j < TN; ++j) acc[ha][hb][i][j] =                    \
                    T::El::mfma(fb[hb][j][kk], fa[i][kk], acc[ha][hb][i][j]);                         \
    __builtin_amdgcn_s_setprio(0);                                                                    \
    __builtin_amdgcn_sched_barrier(0);                                                                \
  } while (0)
  DSMOE_READ_B(0, st, T::kB0);
  wait_lds();
  block_barrier();
  if (w.wave >= 4) block_barrier();

  while (true) {
    DSMOE_READ_A(st, T::kA0);
    DSMOE_READ_B(1, st, T::kB1);
    __builtin_amdgcn_sched_barrier(0);
    w.copy_a1(nx);                // the last half of a chunk, before the next tile's first
    if (w.cl == 0) w.enter();
    w.copy_b0(st);
    DSMOE_PHASE(0);
    block_barrier();
    DSMOE_READ_A(st, T::kA1);
    DSMOE_READ_B(2, nx, T::kB0);
    __builtin_amdgcn_sched_barrier(0);
    w.copy_a0(st);
    w.copy_b1(st);
    --w.cl;
    DSMOE_PHASE(1);
    const bool last = --w.pl == 0;
    // waves 4 to 7 write their results before the barrier, at the same time as waves
    // 0 to 3, which are half a phase ahead, write theirs
    if (!last || w.wave < 4) block_barrier();
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) fb[0][j][kk] = fb[2][j][kk];
    const uint32_t sw = st;
    st = nx;
    nx = sw;
    if (last) {
      stores = w.finish(acc);
      after = stores ? 2 : 0;
      if (w.wave >= 4) block_barrier();
      if (!w.pop()) break;
    }
  }
  if (w.wave < 4) block_barrier();
#undef DSMOE_READ_A
#undef DSMOE_READ_B
#undef DSMOE_PHASE
  wait_copies<0>();   // copies past the last chunk land before the block ends
}

template <Elem E, GroupedKind KIND>
hipError_t launch_grouped_256(const GroupedArgs& t, uint64_t tiles, hipStream_t s) {
  if constexpr (KIND == GroupedKind::kLinear || KIND == GroupedKind::kDw) {
    if (KIND == GroupedKind::kDw || !t.few_rows) {
      const uint32_t grid = static_cast<uint32_t>(tiles < 256 ? (tiles + kXcds - 1) / kXcds * kXcds : 256);   // of 256 CUs
      grouped_stream_kernel<E, 128, 128, 2, 4, KIND><<<grid, 512, 0, s>>>(t);
      return hipGetLastError();
    }
  }
  if constexpr (KIND != GroupedKind::kDw) {
    return by_tiles(t, tiles, [&](const GroupedArgs& q, uint32_t n) {
      grouped_phased_kernel<E, 128, 128, 2, 4, KIND><<<n, 512, 0, s>>>(q);
    });
  }
  return hipSuccess;
}

}  // namespace dsmoe
