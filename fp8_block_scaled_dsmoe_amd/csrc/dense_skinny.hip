// The forward products for few tokens (decode): y = epilogue(x W^T) with at
// most 64 rows of x.  W is read once, straight from memory into matrix-core
// operands; nothing but the sums goes through LDS.
//
// A block takes 16 rows of W (gated: 8 gate rows and the same 8 up rows) and
// all of K, split over 8 or 16 waves; its waves' sums are joined in LDS in order
// and finished by the same block, so a product is one launch without partial
// sums in memory.  v_mfma_f32_16x16x32_bf16 has W's rows as its first operand
// and 16 tokens as its second: per 32 of K a wave loads 1 KB of W (16 bytes
// per lane, its row's next 64 bytes) and 1 KB of x per 16 tokens, several
// steps ahead.  HBM bounds it (one token, 7168 x 2048: 29.4 MB in 7.8 us, 3.8
// TB/s with the launch in it); x is read by every block from L2, MT KB per KB of
// W, which is what limits it to a few tokens (16 tokens, 4096 x 2048: 6.7 us).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "act.h"
#include "common.h"
#include "dense.h"
#include "vec8.h"

namespace dsmoe {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ float load1(const void* p, int64_t i, bool f32) {
  return f32 ? static_cast<const float*>(p)[i] : bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
}
__device__ __forceinline__ void store1(void* p, int64_t i, bool f32, float v) {
  if (f32)
    static_cast<float*>(p)[i] = v;
  else
    static_cast<uint16_t*>(p)[i] = static_cast<uint16_t>(f32x2_to_bf16x2(v, 0.0f));
}

// y = act(v + bias) + r, z = v + bias; r: the residual's value, if there is one
__device__ __forceinline__ void finish_linear1(const DenseGemm& p, int64_t m, int64_t n, float v, float r) {
  if (p.bias) v += load1(p.bias, n, p.bias_f32);
  if (p.z) store1(p.z, m * p.ldz + n, p.y_f32, v);
  v = act_f32(p.act, v);
  if (p.residual) v += r;
  store1(p.y, m * p.ldy + n, p.y_f32, v);
}

// a = act(g) u, h = [g | u]
__device__ __forceinline__ void finish_gated1(const DenseGemm& p, int64_t m, int64_t n, float g, float u) {
  if (p.z) {
    store1(p.z, m * p.ldz + n, false, g);
    store1(p.z, m * p.ldz + p.gate_n + n, false, u);
  }
  store1(p.y, m * p.ldy + n, p.y_f32, act_f32(p.act, g) * u);
}

__device__ __forceinline__ u32x4 load_frag(const uint16_t* q) { return *reinterpret_cast<const u32x4_at2*>(q); }

// MT: groups of 16 tokens; DEPTH: steps of K in flight per wave.
template <int MT, int DEPTH, int kWaves, DenseEpi EPI>
__global__ __launch_bounds__(64 * kWaves) void dense_skinny_kernel(DenseGemm p) {
  constexpr bool kGated = EPI == DenseEpi::kGated;
  constexpr int kCols = kGated ? 8 : 16;   // result columns of the block
  __shared__ f32x4 s_sum[kWaves][MT][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * kCols;
  // this lane's row of W, rows of x and first k; rows past the end repeat the
  // last one (their results are not stored)
  const int r = lane & 15;
  int64_t wrow;
  if constexpr (kGated) {
    const int64_t n = min(n0 + (r & 7), p.N - 1);
    wrow = r < 8 ? n : p.gate_n + n;
  } else {
    wrow = min(n0 + r, p.N - 1);
  }
  // whole steps of 64, spread evenly over the waves; the last wave also takes
  // what is left of K.  Lane group g = lane / 16 holds k = 16 g + [0, 16) of a
  // step: the first 8 in one product, the others in the next.
  const int64_t steps = p.K / 64;
  const int64_t s0 = steps * wave / kWaves, s1 = steps * (wave + 1) / kWaves;
  const int64_t k0 = s0 * 64 + 16 * (lane >> 4);
  const uint16_t* wp = p.b.p + wrow * p.b.ld + k0;
  const uint16_t* xp[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) xp[t] = p.a.p + min(static_cast<int64_t>(16 * t + r), p.M - 1) * p.a.ld + k0;

  f32x4 acc[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto product = [&](const u32x4& a, const u32x4& b, f32x4& c) {
    c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
                                                0);
  };
  const int n_steps = static_cast<int>(s1 - s0);
  u32x4 fw[DEPTH][2], fx[DEPTH][MT][2];
  auto fetch = [&](int d, int s) {
    const int64_t at = static_cast<int64_t>(s) * 64;
#pragma unroll
    for (int h = 0; h < 2; ++h) fw[d][h] = load_frag(wp + at + 8 * h);
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int h = 0; h < 2; ++h) fx[d][t][h] = load_frag(xp[t] + at + 8 * h);
  };
  auto multiply = [&](int d) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int t = 0; t < MT; ++t) product(fw[d][h], fx[d][t][h], acc[t]);
  };
#pragma unroll
  for (int d = 0; d < DEPTH; ++d)
    if (d < n_steps) fetch(d, d);
  int s = 0;
  for (; s + DEPTH <= n_steps; s += DEPTH) {
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
      multiply(d);
      if (s + DEPTH + d < n_steps) fetch(d, s + DEPTH + d);
    }
  }
#pragma unroll
  for (int d = 0; d < DEPTH; ++d)
    if (s + d < n_steps) multiply(d);
  if (wave == kWaves - 1 && steps * 64 < p.K) {
    const int64_t at = static_cast<int64_t>(n_steps) * 64;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t left = p.K - k0 - at - 8 * h;   // valid k from this lane's 8 on
      auto load = [&](const uint16_t* q) { return fetch8<false>(q + at + 8 * h, left).q[0]; };
      const u32x4 a = load(wp);
#pragma unroll
      for (int t = 0; t < MT; ++t) product(a, load(xp[t]), acc[t]);
    }
  }

  // acc: lane l holds token l % 16 of its group and rows 4 (l / 16) + [0, 4)
  // of the block's 16
#pragma unroll
  for (int t = 0; t < MT; ++t) s_sum[wave][t][lane] = acc[t];
  __syncthreads();
  auto total = [&](int t, int m, int row) {
    float v = 0.0f;
    const int l = m + 16 * (row >> 2);
#pragma unroll
    for (int w = 0; w < kWaves; ++w) v += s_sum[w][t][l][row & 3];
    return v;
  };
  for (int i = threadIdx.x; i < MT * 16 * kCols; i += 64 * kWaves) {
    const int c = i % kCols, m = i / kCols % 16, t = i / (16 * kCols);
    const int64_t row = 16 * t + m, n = n0 + c;
    if (row >= p.M || n >= p.N) continue;
    if constexpr (kGated)
      finish_gated1(p, row, n, total(t, m, c), total(t, m, c + 8));
    else
      finish_linear1(p, row, n, total(t, m, c), p.residual ? load1(p.residual, row * p.ldr + n, p.y_f32) : 0.0f);
  }
}

template <int MT, int DEPTH, int kWaves>
hipError_t launch_mt(const DenseGemm& p, hipStream_t s) {
  const int cols = p.epi == DenseEpi::kGated ? 8 : 16;
  const uint32_t grid = static_cast<uint32_t>((p.N + cols - 1) / cols);
  if (p.epi == DenseEpi::kGated)
    dense_skinny_kernel<MT, DEPTH, kWaves, DenseEpi::kGated><<<grid, 64 * kWaves, 0, s>>>(p);
  else
    dense_skinny_kernel<MT, DEPTH, kWaves, DenseEpi::kLinear><<<grid, 64 * kWaves, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_dense_skinny(const DenseGemm& p, hipStream_t s) {
  // more token groups need more registers per step: fewer waves, same bytes in
  // flight
  if (p.M <= 16) return launch_mt<1, 4, 16>(p, s);
  if (p.M <= 32) return launch_mt<2, 3, 16>(p, s);
  if (p.M <= 48) return launch_mt<3, 4, 8>(p, s);
  return launch_mt<4, 3, 8>(p, s);
}

}  // namespace dsmoe
