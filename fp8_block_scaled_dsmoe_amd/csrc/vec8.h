// Runs of 8 adjacent values of a row, bf16 or float32, as 16-byte accesses at
// any element's address: gfx950 takes wide global accesses of any alignment,
// so rows of odd strides need no other path (with values moved one by one, 4096 x
// 7163 x 2048 with a residual took 243 us, not 115 to 120, the layer norm of 4096
// rows of 4095 33 us, not 19).  Off 4 bytes they are about half as fast, which
// matters only where a row is streamed once.  Only a run that the row's end cuts
// is moved value by value.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.h"

namespace dsmoe {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_at2 __attribute__((aligned(2)));
typedef u32x4 u32x4_at4 __attribute__((aligned(4)));

// 8 values as they are in memory
template <bool F32>
struct Raw8 {
  u32x4 q[F32 ? 2 : 1];
};

// the first `left` (8 or more: all, 0 or less: none) of 8 values at p, the others 0
template <bool F32>
__device__ __forceinline__ Raw8<F32> fetch8(const void* p, int64_t left) {
  Raw8<F32> r;
#pragma unroll
  for (int h = 0; h < (F32 ? 2 : 1); ++h) r.q[h] = u32x4{0, 0, 0, 0};
  if (left >= 8) {
    if constexpr (F32) {
      const u32x4_at4* q = static_cast<const u32x4_at4*>(p);
      r.q[0] = q[0], r.q[1] = q[1];
    } else {
      r.q[0] = *static_cast<const u32x4_at2*>(p);
    }
  } else if (left > 0) {
#pragma unroll
    for (int e = 0; e < 7; ++e) {
      if (e >= left) break;
      if constexpr (F32)
        r.q[e / 4][e % 4] = static_cast<const uint32_t*>(p)[e];
      else
        r.q[0][e / 2] |= static_cast<uint32_t>(static_cast<const uint16_t*>(p)[e]) << (e % 2 * 16);
    }
  }
  return r;
}

template <bool F32>
__device__ __forceinline__ void unpack8(const Raw8<F32>& r, float* o) {
  if constexpr (F32) {
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = __uint_as_float(r.q[e / 4][e % 4]);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      o[2 * e] = __uint_as_float(r.q[0][e] << 16);
      o[2 * e + 1] = __uint_as_float(r.q[0][e] & 0xffff0000u);
    }
  }
}

__device__ __forceinline__ u32x4 pack8(const float* v) {
  u32x4 a;
#pragma unroll
  for (int e = 0; e < 4; ++e) a[e] = f32x2_to_bf16x2(v[2 * e], v[2 * e + 1]);
  return a;
}

// the first `left` of 8 values to p
template <bool F32>
__device__ __forceinline__ void put8(void* p, int64_t left, const float* v) {
  Raw8<F32> r;
  if constexpr (F32) {
#pragma unroll
    for (int e = 0; e < 8; ++e) r.q[e / 4][e % 4] = __float_as_uint(v[e]);
  } else {
    r.q[0] = pack8(v);
  }
  if (left >= 8) {
    if constexpr (F32) {
      u32x4_at4* q = static_cast<u32x4_at4*>(p);
      q[0] = r.q[0], q[1] = r.q[1];
    } else {
      *static_cast<u32x4_at2*>(p) = r.q[0];
    }
  } else {
#pragma unroll
    for (int e = 0; e < 7; ++e) {
      if (e >= left) break;
      if constexpr (F32)
        static_cast<uint32_t*>(p)[e] = r.q[e / 4][e % 4];
      else
        static_cast<uint16_t*>(p)[e] = static_cast<uint16_t>(r.q[0][e / 2] >> (e % 2 * 16));
    }
  }
}

// v less its bf16 rounding q, 0 where q is not finite (infinity less infinity
// would be NaN)
__device__ __forceinline__ void rest8(float* v, const u32x4& q) {
  float r[8];
  unpack8<false>(Raw8<false>{{q}}, r);
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = __builtin_isfinite(r[e]) ? v[e] - r[e] : 0.0f;
}

// The same for values i, i + 1, ... of a matrix or vector whose type is known
// at run time.
__device__ __forceinline__ void load8(const void* base, int64_t i, bool f32, int64_t left, float* o) {
  if (f32)
    unpack8<true>(fetch8<true>(static_cast<const float*>(base) + i, left), o);
  else
    unpack8<false>(fetch8<false>(static_cast<const uint16_t*>(base) + i, left), o);
}
__device__ __forceinline__ void store8(void* base, int64_t i, bool f32, int64_t left, const float* v) {
  if (f32)
    put8<true>(static_cast<float*>(base) + i, left, v);
  else
    put8<false>(static_cast<uint16_t*>(base) + i, left, v);
}

}  // namespace dsmoe
