// Building blocks of the matrix products on v_mfma 16x16 tiles: bf16 operands
// with float32 sums, or 8-bit integers with int32 sums.  A block computes a tile
// c[m][n] = sum_k a(m, k) b(n, k) in chunks of 128 bytes of K per row (64 bf16
// values, 128 integers).  Either bf16 operand may be stored with the contraction
// index along its rows ("row" operands) or across them ("k-row" operands);
// integers are row operands.
//
// Both operand tiles are split in two halves (rows [0, BM/2) and [BM/2, BM), and
// so for B), and every wave owns an equal part of each half.  Chunks come by
// asynchronous copies (buffer loads straight to LDS, 16 bytes a lane) one to
// three chunks ahead; operands leave LDS as whole fragments, k-row operands by
// the transposing read.  Three loops differ in how reads, copies and products
// meet:
//   phased_loop  256 rows: a chunk in two phases (A0, A1), the two waves of a
//                SIMD half a phase apart, one multiplying while the other reads
//   paired_loop  128 x 256: the same with whole chunks
//   ring_loop    smaller tiles: reads between a wave's own products
// A fragment of either kind is 16 bytes of a lane: v_mfma_f32_16x16x32_bf16 and
// v_mfma_i32_16x16x64_i8 take the same rows and bytes, so the loops do not differ.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "common.h"
#include "vec8.h"

namespace dsmoe {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x2 u32x2_at2 __attribute__((aligned(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
#define DSMOE_LDS __attribute__((address_space(3)))
template <typename T>
__device__ __forceinline__ DSMOE_LDS T* lds_ptr(uint32_t at) {
  return (DSMOE_LDS T*)static_cast<uintptr_t>(at);
}

constexpr int kXcds = 8;
constexpr int kChunkBytes = 128;   // of K per row and chunk

enum class Elem { kBf16, kI8 };
template <Elem E>
struct ElemOf;
template <>
struct ElemOf<Elem::kBf16> {
  static constexpr int kBytes = 2;
  typedef bf16x8 Frag;
  typedef f32x4 Acc;
  static __device__ __forceinline__ Acc mfma(const Frag& a, const Frag& b, const Acc& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
};
template <>
struct ElemOf<Elem::kI8> {
  static constexpr int kBytes = 1;
  typedef i32x4 Frag;
  typedef i32x4 Acc;
  static __device__ __forceinline__ Acc mfma(const Frag& a, const Frag& b, const Acc& c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
  }
};

// ---------------------------------------------------------------------------
// Operand halves: from memory to LDS, from LDS to MFMA operands.
// ---------------------------------------------------------------------------

// Asynchronous copy of 16 bytes per lane to lds + 16 lane (wave-uniform lds):
// offset voff from the resource's base; past its range zeros are written.
// Issued from assembly so that the compiler neither waits for it nor counts
// it; the kernel waits for vmcnt itself.  A copy to LDS must not follow a
// write of M0 directly (one wait state, which the compiler cannot add inside
// assembly).
__device__ __forceinline__ void copy16(const i32x4& rsrc, uint32_t voff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds" ::"v"(voff), "s"(rsrc),
               "s"(lds)
               : "memory", "m0");
}
template <int N>
__device__ __forceinline__ void wait_copies() {
  static_assert(N < 64, "vmcnt range");
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }
__device__ __forceinline__ void block_barrier() { asm volatile("s_barrier" ::: "memory"); }

// One half (HR rows x 128 bytes of K) of an operand tile in LDS, HR * 128 bytes.
//
// Row operand: row r is 128 bytes of 8 16-byte segments, segment s stored in
// place s ^ (r % 8), so that the 16 rows an operand read touches at one
// segment spread over all banks.
// K-row operand: k is a row of HR * 2 bytes of HR / 16 32-byte blocks (16
// columns), block b stored in place b ^ key(k); operands are read with the
// transposing LDS read, which takes four rows of k x 16 columns per 16 lanes
// and gives each lane its column: the key separates the rows that one read
// touches.
template <int HR, bool KROWS, int NW>
struct Half {
  static constexpr int kBytes = HR * 128;
  static constexpr int kAll = HR / 8;                      // copies of 1 KB
  static constexpr int kCopies = (kAll + NW - 1) / NW;     // of a wave
  static constexpr int kSegs = HR / 8;                     // k-row operand: 16-byte segments of a row
  // the wave's i-th copy; where they do not come out even the last one is
  // made more than once (the same bytes to the same place)
  static __device__ __forceinline__ int index(int wave, int i) { return min(wave * kCopies + i, kAll - 1); }

  static __device__ __forceinline__ int key(int k) {
    if constexpr (HR == 128) return (k & 3) | ((k >> 3) & 1) << 2;
    if constexpr (HR == 64) return ((k >> 1) & 1) | ((k >> 3) & 1) << 1;
    return (k >> 3) & 1;
  }
};

// What a wave copies of one half, chunk by chunk: a buffer resource that starts
// at the half's chunk and ends with its last valid element, and the lane's
// offsets in it.  advance() is a few scalar instructions while whole chunks
// are left; the offsets and the range change only from the last one on.
// (Masking every copy by its k, and a range computed anew per chunk, cost the
// multiplies of a one-wave-per-SIMD loop 8 to 10 cycles per vector
// instruction.)
// WAIT: see copy().  PAIR: 0, or the half holds every other run of PAIR rows, from
// its first row on (both halves then lie side by side, run by run).
template <Elem E, int HR, bool KROWS, int NW, bool WAIT, int PAIR = 0>
struct Source {
  using H = Half<HR, KROWS, NW>;
  static constexpr int ES = ElemOf<E>::kBytes;
  static constexpr int kChunk = kChunkBytes / ES;   // K per chunk
  static_assert(!KROWS || E == Elem::kBf16, "integers are row operands");
  static constexpr int kSpan = PAIR ? 2 * HR - PAIR : HR;   // rows from the first to past the last
  static __device__ __forceinline__ int place(int r) {
    if constexpr (PAIR > 0) return r / PAIR * (2 * PAIR) + r % PAIR;
    return r;
  }
  uint64_t base;                  // byte address of the half's (row 0, chunk's first k)
  int32_t range;                  // bytes from base that may be read
  uint32_t ld2;                   // row stride in bytes
  int32_t k_left;                 // valid k from base on
  int32_t cols2;                  // k-row operand: bytes of a row's valid columns
  int32_t lane_k;                 // row operand: first k of the lane's segment
  uint32_t voff[H::kCopies];

  __device__ __forceinline__ Source() {}
  // rows from r0 on of `rows` rows at p, chunks from k0 on, k_end: end of valid k
  __device__ __forceinline__ Source(const void* p, int64_t ld, int64_t r0, int64_t rows, int64_t k0, int64_t k_end,
                                    int wave, int lane) {
    ld2 = static_cast<uint32_t>(ld * ES);
    const int64_t left = min(static_cast<int64_t>(kSpan), rows - r0);
    k_left = left > 0 ? static_cast<int32_t>(k_end - k0) : 0;
    lane_k = 16 / ES * ((lane & 7) ^ (lane >> 3));
    if constexpr (KROWS) {
      base = reinterpret_cast<uint64_t>(p) + static_cast<uint64_t>(k0 * ld + r0) * ES;
      cols2 = left > 0 ? static_cast<int32_t>(left) * ES : 0;
      range = (kChunk - 1) * static_cast<int32_t>(ld2) + cols2;
    } else {
      base = reinterpret_cast<uint64_t>(p) + static_cast<uint64_t>(r0 * ld + k0) * ES;
      range = left > 0 ? static_cast<int32_t>(left - 1) * static_cast<int32_t>(ld2) + ES * k_left : 0;
    }
#pragma unroll
    for (int i = 0; i < H::kCopies; ++i) {
      const int j = H::index(wave, i);
      if constexpr (KROWS) {
        const int k = (j * 64 + lane) / H::kSegs, seg = (j * 64 + lane) % H::kSegs;
        const int col = place(((seg >> 1) ^ H::key(k)) * 16 + (seg & 1) * 8);
        voff[i] = col < left ? static_cast<uint32_t>(k) * ld2 + col * 2 : kOutside;
      } else {
        voff[i] = static_cast<uint32_t>(place(8 * j + lane / 8)) * ld2 + ES * lane_k;
      }
    }
    if (k_left < kChunk) cut();
  }
  // Row operand, rows taken by index: row i of the half is row index[i] of the
  // n rows at p (i < left; rows past it, and indices outside [0, n), read as
  // zeros).  n * ld * ES < 2^31.
  __device__ __forceinline__ Source(const void* p, int64_t ld, int32_t n, const int32_t* index, int64_t left, int64_t k0,
                                    int64_t k_end, int wave, int lane) {
    static_assert(!KROWS && PAIR == 0, "row operands, one after the other");
    ld2 = static_cast<uint32_t>(ld * ES);
    k_left = left > 0 ? static_cast<int32_t>(k_end - k0) : 0;
    lane_k = 16 / ES * ((lane & 7) ^ (lane >> 3));
    base = reinterpret_cast<uint64_t>(p) + static_cast<uint64_t>(k0) * ES;
    range = left > 0 ? (n - 1) * static_cast<int32_t>(ld2) + ES * k_left : 0;
#pragma unroll
    for (int i = 0; i < H::kCopies; ++i) {
      const int r = 8 * H::index(wave, i) + lane / 8;
      const int32_t row = r < left ? index[r] : -1;
      voff[i] = static_cast<uint32_t>(row) < static_cast<uint32_t>(n) ? static_cast<uint32_t>(row) * ld2 + ES * lane_k
                                                                      : kOutside;
    }
    if (k_left < kChunk) cut();
  }
  // past every range (the largest is 224 rows of 2^23 bytes, or 2^31 - 1 by index)
  static constexpr uint32_t kOutside = 0x80000000u;
  // The last chunk, and those past the end: what is past k_left reads as zero.
  __device__ __forceinline__ void cut() {
    asm volatile("");   // a branch around it, not selects in every chunk
    if constexpr (KROWS) {
      range = k_left > 0 ? (k_left - 1) * static_cast<int32_t>(ld2) + cols2 : 0;
    } else {
      if (k_left <= 0) range = 0;
#pragma unroll
      for (int i = 0; i < H::kCopies; ++i)
        if (lane_k >= k_left) voff[i] = kOutside;   // it would read the next row
    }
  }
  __device__ __forceinline__ void advance() {
    if constexpr (KROWS) {
      base += ld2 * kChunk;
    } else {
      base += kChunkBytes;
      range -= kChunkBytes;   // may pass 0 only where cut() makes it 0
    }
    k_left -= kChunk;
    if (k_left < kChunk) cut();
  }
  // Issue this wave's copies of the current chunk to the half at lds.
  __device__ __forceinline__ void copy(uint32_t lds, int wave) const {
    // wave-uniform: into scalar registers
    i32x4 r;
    r.x = __builtin_amdgcn_readfirstlane(static_cast<int>(base & 0xffffffffu));
    r.y = __builtin_amdgcn_readfirstlane(static_cast<int>(base >> 32));   // below bit 48: stride 0, a raw buffer
    r.z = __builtin_amdgcn_readfirstlane(range);
    r.w = 0x00020000;
    // Where the compiler keeps them in vector registers, they are written here:
    // five wait states before the copies, which it does not count for assembly.
    if constexpr (WAIT) asm volatile("s_nop 4" : "+s"(r));
#pragma unroll
    for (int i = 0; i < H::kCopies; ++i)
      copy16(r, voff[i],
             __builtin_amdgcn_readfirstlane(lds + static_cast<uint32_t>(H::index(wave, i)) * 1024));
  }
};

// A wave's reader of T 16-row operand fragments from row0 of a half:
// fragment i, K step kk (of 2): lane l holds 16 bytes of row l % 16, from byte
// 64 kk + 16 (l / 16) of the chunk on.
template <Elem E, int HR, bool KROWS, int T>
struct Reader {
  using Frag = typename ElemOf<E>::Frag;
  uint32_t at[KROWS ? T : 2];
  __device__ __forceinline__ Reader(int row0, int lane) {
    if constexpr (KROWS) {
      const int s = lane & 15, g = lane >> 4;
      const int k = 8 * g + (s >> 2);      // key() ignores the bits the reads below add to k
#pragma unroll
      for (int i = 0; i < T; ++i)
        at[i] = k * HR * 2 + (((row0 / 16 + i) ^ Half<HR, true, 1>::key(k)) << 5) + (s & 3) * 8;
    } else {
#pragma unroll
      for (int kk = 0; kk < 2; ++kk)
        at[kk] = (row0 + (lane & 15)) * 128 + (((kk * 4 + (lane >> 4)) ^ (lane & 7)) << 4);
    }
  }
  // half: the half's place in the stage (a constant: it goes into the
  // instruction's offset)
  __device__ __forceinline__ Frag read(uint32_t stage, uint32_t half, int i, int kk) const {
    if constexpr (KROWS) {
      DSMOE_LDS char* a = lds_ptr<char>(stage + at[i]) + (half + kk * (32 * HR * 2));
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((DSMOE_LDS s16x4*)a);
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((DSMOE_LDS s16x4*)(a + 4 * HR * 2));
      return __builtin_bit_cast(Frag, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
      return *(DSMOE_LDS const Frag*)(lds_ptr<char>(stage + at[kk]) + (half + i * 2048));
    }
  }
};

// What a block and its waves work on.  HM, HN: rows of a half of A and of B;
// WM x WN waves.  GATED: half 0 of B holds gate rows, half 1 the same up
// rows, so a lane has both sums of its columns.
// WAIT and PAIR (of B): see Source.
template <Elem E, int HM, int HN, int WM, int WN, bool AT, bool BT, bool GATED, bool WAIT, int PAIR = 0>
struct TileCore {
  static constexpr bool kGated = GATED;
  static constexpr int NW = WM * WN;
  static constexpr int TM = HM / WM / 16, TN = HN / WN / 16;   // fragments of a wave per half
  static constexpr int kChunk = kChunkBytes / ElemOf<E>::kBytes;
  using El = ElemOf<E>;
  using Frag = typename El::Frag;
  using SA = Source<E, HM, AT, NW, WAIT>;
  using SB = Source<E, HN, BT, NW, WAIT, PAIR>;
  static constexpr int LA = SA::H::kCopies, LB = SB::H::kCopies;
  static constexpr int AB = SA::H::kBytes, BB = SB::H::kBytes;
  // a stage of LDS and the places of the halves in it
  static constexpr uint32_t kStage = 2 * (AB + BB), kA0 = 0, kA1 = AB, kB0 = 2 * AB, kB1 = 2 * AB + BB;
  static constexpr int kOutStride = 2 * HN + 4;   // sums between rows of results in LDS
  static constexpr int lds_bytes(int stages) {
    const int a = stages * kStage, b = HM * kOutStride * 4;
    return a > b ? a : b;
  }
  typedef typename El::Acc Sums;
  typedef Sums Acc[2][2][TM][TN];   // [half of A][half of B]

  const int lane, wave, wm, wn;
  int32_t c0, c1;   // chunks of K
  int64_t m0, n0;
  SA a0, a1;
  SB b0, b1;
  const Reader<E, HM, AT, TM> ra;
  const Reader<E, HN, BT, TN> rb;
  const uint32_t lds;

  __device__ __forceinline__ explicit TileCore(const uint8_t* mem)
      : lane(threadIdx.x & 63),
        wave(__builtin_amdgcn_readfirstlane(threadIdx.x >> 6)),
        wm(wave / WN),
        wn(wave % WN),
        ra(wm * (HM / WM), lane),
        rb(wn * (HN / WN), lane),
        lds(static_cast<uint32_t>(reinterpret_cast<uintptr_t>(mem))) {}

  // the wave's copies of the next chunk of a half into a stage
  __device__ __forceinline__ void copy_a0(uint32_t stage) { a0.copy(stage + kA0, wave), a0.advance(); }
  __device__ __forceinline__ void copy_a1(uint32_t stage) { a1.copy(stage + kA1, wave), a1.advance(); }
  __device__ __forceinline__ void copy_b0(uint32_t stage) { b0.copy(stage + kB0, wave), b0.advance(); }
  __device__ __forceinline__ void copy_b1(uint32_t stage) { b1.copy(stage + kB1, wave), b1.advance(); }

  static __device__ __forceinline__ void clear(Acc& acc) {
#pragma unroll
    for (int h = 0; h < 4; ++h)
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[h >> 1][h & 1][i][j] = Sums{};
  }

  // The results pass through LDS, half of the tile's rows at a time, so that a
  // thread finishes runs of 8 columns and a wave writes whole lines.
  static constexpr int kRuns = (kGated ? HN : 2 * HN) / 8;   // of 8 columns
  // rows that the block's threads take at once, a power of 2 (with 24 runs a
  // quarter of the threads stay out)
  static constexpr int rows_at_once(int per_row) {
    int r = 1;
    while (2 * r * per_row <= 64 * NW && 2 * r <= HM) r *= 2;
    return r;
  }
  static constexpr int kRowsAtOnce = rows_at_once(kRuns);

  // Half ha of the results to LDS.  A result lane holds row l % 16 of its A
  // fragment and columns 4 (l / 16) + [0, 4) of its B fragment; rows 16 bytes
  // off a multiple of 256 apart keep the writes of 16 rows on separate banks.
  __device__ __forceinline__ void put(const Sums (&acc)[2][TM][TN]) const {
    wait_lds();        // this wave's reads of LDS are done, and past the barrier
    block_barrier();   // everyone's
#pragma unroll
    for (int hb = 0; hb < 2; ++hb)
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) {
          const int r = wm * (HM / WM) + 16 * i + (lane & 15);
          const int c = hb * HN + wn * (HN / WN) + 16 * j + 4 * (lane >> 4);
          *lds_ptr<Sums>(lds + (r * kOutStride + c) * 4) = acc[hb][i][j];
        }
    wait_lds();
    block_barrier();
  }
  __device__ __forceinline__ void get(int r, int col, float* v) const {
    const uint32_t at = lds + (r * kOutStride + col) * 4;
    const Sums v0 = *lds_ptr<const Sums>(at), v1 = *lds_ptr<const Sums>(at + 16);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = static_cast<float>(v0[e]), v[4 + e] = static_cast<float>(v1[e]);
  }
};

// ---------------------------------------------------------------------------
// The loops: the products of chunks [w.c0, w.c1) of the tile w into acc.  The
// times are those of bf16 products.
// ---------------------------------------------------------------------------

// The 256-row tiles: two stages of LDS refilled half by half.  A chunk falls
// into two phases, A0 with both halves of B and A1 with both, each half of the
// tile's products.  Once every wave has read a half into registers, its place
// takes the same half of the chunk two ahead; the copies have a whole chunk to
// arrive, and only two chunks are ever in LDS.  Waves w and w + 4 share a SIMD.
// 4096^3 takes 100 us, by W's columns 102, both by columns 106.
template <typename T>
__device__ __forceinline__ void phased_loop(T& w, typename T::Acc& acc) {
  constexpr int TM = T::TM, TN = T::TN, LA = T::LA, LB = T::LB;
  static_assert(T::NW == 8, "two waves per SIMD");
  T::clear(acc);
  typename T::Frag fa[TM][2], fb[3][TN][2];

  const uint32_t s0 = w.lds, s1 = w.lds + T::kStage;
  w.copy_b0(s0);
  w.copy_a0(s0);
  w.copy_b1(s0);
  w.copy_a1(s0);
  w.copy_b0(s1);
  w.copy_a0(s1);
  w.copy_b1(s1);
  wait_copies<2 * LA + 2 * LB>();   // this wave's part of B0, A0 and B1 of the first chunk
  block_barrier();
#define DSMOE_READ_A(stage, half)                \
  _Pragma("unroll") for (int i = 0; i < TM; ++i) \
      _Pragma("unroll") for (int kk = 0; kk < 2; ++kk) fa[i][kk] = w.ra.read(stage, half, i, kk)
#define DSMOE_READ_B(f, stage, half)             \
  _Pragma("unroll") for (int j = 0; j < TN; ++j) \
      _Pragma("unroll") for (int kk = 0; kk < 2; ++kk) fb[f][j][kk] = w.rb.read(stage, half, j, kk)
  // The end of a phase's reads and copies: the reads are done (the halves may
  // be refilled once all waves are past the barrier), and what the next phase
  // reads is there (at most the copies of this phase and the last may still be
  // on the way).  Then the phase's products: both halves of B with A's half
  // ha, B0 in fb[0], B1 in fb[1].
#define DSMOE_PHASE(ha)                                                            \
  do {                                                                             \
    wait_copies<2 * LA + 2 * LB>();                                                \
    wait_lds();                                                                    \
    block_barrier();                                                               \
    __builtin_amdgcn_sched_barrier(0);                                             \
    __builtin_amdgcn_s_setprio(1);                                                 \
    _Pragma("unroll") for (int kk = 0; kk < 2; ++kk)                               \
        _Pragma("unroll") for (int hb = 0; hb < 2; ++hb)                           \
            _Pragma("unroll") for (int i = 0; i < TM; ++i)                         \
                _Pragma("unroll") for (int j = 0; j < TN; ++j) acc[ha][hb][i][j] = \
                    T::El::mfma(fb[hb][j][kk], fa[i][kk], acc[ha][hb][i][j]);      \
    __builtin_amdgcn_s_setprio(0);                                                 \
    __builtin_amdgcn_sched_barrier(0);                                             \
    block_barrier();                                                               \
  } while (0)
  DSMOE_READ_B(0, s0, T::kB0);
  wait_lds();
  block_barrier();
  if (w.wave >= 4) block_barrier();

  // The next chunk's B0 is read in the second phase, to even out the phases'
  // reads; it has registers of its own and moves at the end.
  uint32_t st = s0, nx = s1;
  for (int32_t c = w.c0; c < w.c1; ++c) {
    DSMOE_READ_A(st, T::kA0);
    DSMOE_READ_B(1, st, T::kB1);
    __builtin_amdgcn_sched_barrier(0);
    w.copy_a1(nx);
    w.copy_b0(st);
    DSMOE_PHASE(0);
    DSMOE_READ_A(st, T::kA1);
    DSMOE_READ_B(2, nx, T::kB0);
    __builtin_amdgcn_sched_barrier(0);
    w.copy_a0(st);
    w.copy_b1(st);
    DSMOE_PHASE(1);
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) fb[0][j][kk] = fb[2][j][kk];
    const uint32_t sw = st;
    st = nx;
    nx = sw;
  }
  if (w.wave < 4) block_barrier();
#undef DSMOE_READ_A
#undef DSMOE_READ_B
#undef DSMOE_PHASE
  wait_copies<0>();   // copies past the last chunk (zeros) land before LDS is used again
}

// 128 x 256: S stages of LDS, whole chunks.  The two waves of a SIMD run half a
// chunk apart, one multiplying while the other reads all of its part of the
// chunk; the stage that both have read takes the chunk S - 1 ahead.  Reads and
// products of a chunk are about as long (16 reads, 32 products a wave), so
// this beats reads between a wave's own products: 4096 x 2048 x 7168 in 92 us
// instead of 103, by W's columns 97 instead of 122.  With 128 x 128, half the
// products per barrier, it loses (2048^3 24.2 us instead of 22.9).
template <int S, typename T>
__device__ __forceinline__ void paired_loop(T& w, typename T::Acc& acc) {
  constexpr int TM = T::TM, TN = T::TN, L = 2 * T::LA + 2 * T::LB;
  static_assert(T::NW == 8, "two waves per SIMD");
  T::clear(acc);
  typename T::Frag fa[2][TM][2], fb[2][TN][2];

#define DSMOE_COPY(stage) w.copy_a0(stage), w.copy_b0(stage), w.copy_b1(stage), w.copy_a1(stage)
  for (int i = 0; i < S - 1; ++i) DSMOE_COPY(w.lds + i * T::kStage);
  wait_copies<(S - 2) * L>();
  block_barrier();
  if (w.wave >= 4) block_barrier();
  uint32_t st = w.lds, free = w.lds + (S - 1) * T::kStage;
  for (int32_t c = w.c0; c < w.c1; ++c) {
#pragma unroll
    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int i = 0; i < TM; ++i) fa[h][i][kk] = w.ra.read(st, h ? T::kA1 : T::kA0, i, kk);
#pragma unroll
        for (int j = 0; j < TN; ++j) fb[h][j][kk] = w.rb.read(st, h ? T::kB1 : T::kB0, j, kk);
      }
    __builtin_amdgcn_sched_barrier(0);
    // The last barrier was the other wave's end of reading the chunk before.
    DSMOE_COPY(free);
    wait_copies<(S - 2) * L>();   // this wave's part of the next chunk is there
    wait_lds();
    block_barrier();
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
      for (int h = 0; h < 4; ++h)
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
          for (int j = 0; j < TN; ++j)
            acc[h >> 1][h & 1][i][j] = T::El::mfma(fb[h & 1][j][kk], fa[h >> 1][i][kk], acc[h >> 1][h & 1][i][j]);
    __builtin_amdgcn_s_setprio(0);
    __builtin_amdgcn_sched_barrier(0);
    block_barrier();
    free = st;
    st = st + T::kStage == w.lds + S * T::kStage ? w.lds : st + T::kStage;
  }
#undef DSMOE_COPY
  if (w.wave < 4) block_barrier();
  wait_copies<0>();   // copies past the last chunk (zeros) land before LDS is used again
}

// Smaller tiles: S stages of LDS, latency and the copies' way bound them (2048^3
// 21.5 to 24 us, 1000^3 8.6).  A chunk's fragments are read in two steps of
// 64 bytes, each while the products of the step before run; once a chunk's
// second step is in registers in every wave, its stage is refilled with the
// chunk S ahead.
template <int S, typename T>
__device__ __forceinline__ void ring_loop(T& w, typename T::Acc& acc) {
  constexpr int TM = T::TM, TN = T::TN, L = 2 * T::LA + 2 * T::LB;
  T::clear(acc);
  typename T::Frag fa[2][2][TM], fb[2][2][TN];   // [step][half]

#define DSMOE_COPY(stage) w.copy_a0(stage), w.copy_b0(stage), w.copy_b1(stage), w.copy_a1(stage)
#define DSMOE_READ(kk, stage)                                       \
  do {                                                              \
    _Pragma("unroll") for (int h = 0; h < 2; ++h) {                 \
      _Pragma("unroll") for (int i = 0; i < TM; ++i) fa[kk][h][i] = \
          w.ra.read(stage, h ? T::kA1 : T::kA0, i, kk);             \
      _Pragma("unroll") for (int j = 0; j < TN; ++j) fb[kk][h][j] = \
          w.rb.read(stage, h ? T::kB1 : T::kB0, j, kk);             \
    }                                                               \
  } while (0)
#define DSMOE_PRODUCTS(kk)                                                          \
  _Pragma("unroll") for (int h = 0; h < 4; ++h)                                     \
      _Pragma("unroll") for (int i = 0; i < TM; ++i)                                \
          _Pragma("unroll") for (int j = 0; j < TN; ++j) acc[h >> 1][h & 1][i][j] = \
              T::El::mfma(fb[kk][h & 1][j], fa[kk][h >> 1][i], acc[h >> 1][h & 1][i][j])
  for (int i = 0; i < S; ++i) DSMOE_COPY(w.lds + i * T::kStage);
  wait_copies<(S - 1) * L>();
  block_barrier();
  uint32_t st = w.lds;
  DSMOE_READ(0, st);
  for (int32_t c = w.c0; c < w.c1; ++c) {
    const uint32_t nx = st + T::kStage == w.lds + S * T::kStage ? w.lds : st + T::kStage;
    DSMOE_READ(1, st);
    DSMOE_PRODUCTS(0);
    __builtin_amdgcn_sched_barrier(0);
    wait_copies<(S - 2) * L>();   // the next chunk's copies of this wave
    wait_lds();
    block_barrier();
    DSMOE_COPY(st);
    DSMOE_READ(0, nx);
    DSMOE_PRODUCTS(1);
    __builtin_amdgcn_sched_barrier(0);
    st = nx;
  }
#undef DSMOE_COPY
#undef DSMOE_READ
#undef DSMOE_PRODUCTS
  wait_copies<0>();   // copies past the last chunk (zeros) land before LDS is used again
  wait_lds();
}

}  // namespace dsmoe
