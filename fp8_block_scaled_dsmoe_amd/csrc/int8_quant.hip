// 8-bit integers with one scale per row.  A row is read once where it fits the
// registers of its threads, and its largest magnitude is found on the bit
// patterns, whose order is the order of the magnitudes with infinity and NaN
// above every number.  Bound by memory and the exact divisions, 8 of a thread at a
// time: 4096 x 7168 bf16 in 24 us (3.6 TB/s read and written), 4096 x 2048 in 10, a
// row of 7168 in 4.3 (the launch, the row's way from memory, one join).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.h"
#include "grouped.h"
#include "vec8.h"

namespace dsmoe {
namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x2 u32x2_at1 __attribute__((aligned(1)));

struct QuantArgs {
  const void* x;
  int64_t ldx, rows, cols;
  int8_t* q;
  int64_t ldq;
  float* scale;
};

__device__ __forceinline__ uint32_t max_bits(const float* v, uint32_t m) {
#pragma unroll
  for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(v[e]) & 0x7fffffffu);
  return m;
}

// the first `left` of 8 codes to p
__device__ __forceinline__ void put_codes(int8_t* p, int64_t left, const float* v, float s) {
  u32x2 w{0, 0};
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float t = __builtin_fminf(__builtin_fmaxf(__builtin_rintf(v[e] / s), -127.0f), 127.0f);
    w[e / 4] |= (static_cast<uint32_t>(static_cast<int32_t>(t)) & 0xffu) << (e % 4 * 8);
  }
  if (left >= 8) {
    *reinterpret_cast<u32x2_at1*>(p) = w;
  } else {
#pragma unroll
    for (int e = 0; e < 7; ++e)
      if (e < left) p[e] = static_cast<int8_t>(w[e / 4] >> (e % 4 * 8));
  }
}

// The scale of a row whose largest magnitude has the bits m.
__device__ __forceinline__ float scale_of(uint32_t m) {
  if (m >= 0x7f800000u) return __uint_as_float(0x7fc00000u);
  const float s = __uint_as_float(m) / 127.0f;
  return s == 0.0f ? 1.0f : s;
}

// TPR threads per row; SLOTS runs of 8 columns of a thread in registers (0: any
// number, the row is read twice).
template <bool F32, int TPR, int SLOTS>
__global__ __launch_bounds__(256) void quant_rows_int8_kernel(QuantArgs a) {
  __shared__ uint32_t s_max[4];
  constexpr int kRows = 256 / TPR, ES = F32 ? 4 : 2;
  const int t = threadIdx.x % TPR;
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * kRows; r0 < a.rows; r0 += static_cast<int64_t>(gridDim.x) * kRows) {
    const int64_t r = r0 + threadIdx.x / TPR;
    const bool in = r < a.rows;
    const char* x = static_cast<const char*>(a.x) + r * a.ldx * ES;
    const int64_t cols = in ? a.cols : 0;
    uint32_t m = 0;
    float v[SLOTS ? SLOTS : 1][8];
    if constexpr (SLOTS > 0) {
      Raw8<F32> raw[SLOTS];
#pragma unroll
      for (int i = 0; i < SLOTS; ++i) {
        const int64_t c = 8 * (t + static_cast<int64_t>(i) * TPR);
        raw[i] = fetch8<F32>(x + c * ES, cols - c);
      }
#pragma unroll
      for (int i = 0; i < SLOTS; ++i) {
        unpack8<F32>(raw[i], v[i]);
        m = max_bits(v[i], m);
      }
    } else {
      for (int64_t c = 8 * t; c < cols; c += 8 * TPR) {
        unpack8<F32>(fetch8<F32>(x + c * ES, cols - c), v[0]);
        m = max_bits(v[0], m);
      }
    }
#pragma unroll
    for (int o = (TPR < 64 ? TPR : 64) >> 1; o > 0; o >>= 1) m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), o, 64)));
    if constexpr (TPR > 64) {
      if ((threadIdx.x & 63) == 0) s_max[threadIdx.x >> 6] = m;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < 4; ++w) m = max(m, s_max[w]);
      __syncthreads();
    }
    const float s = scale_of(m);
    const bool bad = m >= 0x7f800000u;
    if (in && t == 0) a.scale[r] = s;
    int8_t* q = a.q + r * a.ldq;
    if constexpr (SLOTS > 0) {
#pragma unroll
      for (int i = 0; i < SLOTS; ++i) {
        const int64_t c = 8 * (t + static_cast<int64_t>(i) * TPR);
        if (c >= cols) break;
        if (bad) {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[i][e] = 0.0f;
        }
        put_codes(q + c, cols - c, v[i], bad ? 1.0f : s);
      }
    } else {
      for (int64_t c = 8 * t; c < cols; c += 8 * TPR) {
        unpack8<F32>(fetch8<F32>(x + c * ES, cols - c), v[0]);
        if (bad) {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[0][e] = 0.0f;
        }
        put_codes(q + c, cols - c, v[0], bad ? 1.0f : s);
      }
    }
  }
}

template <bool F32>
hipError_t launch(const QuantArgs& a, hipStream_t s) {
  auto blocks = [&](int64_t per) {
    const int64_t n = (a.rows + per - 1) / per;
    return static_cast<uint32_t>(n < (1 << 20) ? n : 1 << 20);
  };
  if (a.cols <= 64)
    quant_rows_int8_kernel<F32, 8, 1><<<blocks(32), 256, 0, s>>>(a);
  else if (a.cols <= 512)
    quant_rows_int8_kernel<F32, 64, 1><<<blocks(4), 256, 0, s>>>(a);
  else if (a.cols <= 2048)
    quant_rows_int8_kernel<F32, 256, 1><<<blocks(1), 256, 0, s>>>(a);
  else if (a.cols <= 4096)
    quant_rows_int8_kernel<F32, 256, 2><<<blocks(1), 256, 0, s>>>(a);
  else if (a.cols <= 8192)
    quant_rows_int8_kernel<F32, 256, 4><<<blocks(1), 256, 0, s>>>(a);
  else
    quant_rows_int8_kernel<F32, 256, 0><<<blocks(1), 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quant_rows_int8(const void* x, int64_t ldx, bool f32, int64_t rows, int64_t cols, int8_t* q,
                                  int64_t ldq, float* scale, hipStream_t s) {
  const QuantArgs a{x, ldx, rows, cols, q, ldq, scale};
  return f32 ? launch<true>(a, s) : launch<false>(a, s);
}

}  // namespace dsmoe
