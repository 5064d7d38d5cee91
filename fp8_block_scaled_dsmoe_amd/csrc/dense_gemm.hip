// Matrix products of the dense feed-forward operators in bf16 with float32
// sums: c[m][n] = sum_k a(m, k) b(n, k) and a fused epilogue.  Either operand
// may be stored with the contraction index along its rows (forward: x and W;
// dx: dz) or across them (dx: W; dW: dz and x).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "act.h"
#include "common.h"
#include "dense.h"

namespace dsmoe {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
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

// One result (m, n) of the linear epilogue.
__device__ __forceinline__ void finish_linear(const DenseGemm& p, int64_t m, int64_t n, float acc) {
  if (p.bias) acc += load1(p.bias, n, p.bias_f32);
  if (p.z) store1(p.z, m * p.ldz + n, p.y_f32, acc);
  float y = act_f32(p.act, acc);
  if (p.residual) y += load1(p.residual, m * p.ldr + n, p.y_f32);
  store1(p.y, m * p.ldy + n, p.y_f32, y);
}
// One result (m, n) of the gated epilogue, from its gate and up sums.
__device__ __forceinline__ void finish_gated(const DenseGemm& p, int64_t m, int64_t n, float g, float u) {
  if (p.z) {
    store1(p.z, m * p.ldz + n, false, g);
    store1(p.z, m * p.ldz + p.N + n, false, u);
  }
  store1(p.y, m * p.ldy + n, p.y_f32, act_f32(p.act, g) * u);
}

// 64 x 64 tile (kGated: 32 gate and the same 32 up columns), 4 waves of
// 32 x 32 by v_mfma_f32_16x16x32_bf16, one 32-deep step of K in LDS at a time.
constexpr int kRowPad = 40;   // LDS row of 32 values, 80 bytes apart
template <DenseEpi EPI>
__global__ __launch_bounds__(256) void dense_gemm_kernel(DenseGemm p) {
  constexpr bool kGated = EPI == DenseEpi::kGated;
  constexpr int BN = kGated ? 32 : 64;   // result columns of the tile
  __shared__ __attribute__((aligned(16))) uint16_t s_a[64 * kRowPad], s_b[64 * kRowPad];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t tiles_n = (p.N + BN - 1) / BN;
  const int64_t m0 = blockIdx.x / tiles_n * 64, n0 = blockIdx.x % tiles_n * BN;
  f32x4 acc[2][2] = {};
  for (int64_t k0 = 0; k0 < p.K; k0 += 32) {
    for (int i = tid; i < 64 * 32; i += 256) {
      // consecutive threads along the operand's contiguous index
      const int ra = p.a.k_rows ? i & 63 : i >> 5, ka = p.a.k_rows ? i >> 6 : i & 31;
      const int64_t m = m0 + ra, k = k0 + ka;
      s_a[ra * kRowPad + ka] =
          m < p.M && k < p.K ? p.a.p[p.a.k_rows ? k * p.a.ld + m : m * p.a.ld + k] : static_cast<uint16_t>(0);
      const int rb = p.b.k_rows ? i & 63 : i >> 5, kb = p.b.k_rows ? i >> 6 : i & 31;
      const int64_t nn = n0 + (kGated ? rb & 31 : rb), kk = k0 + kb;
      const int64_t n = kGated && rb >= 32 ? p.N + nn : nn;
      s_b[rb * kRowPad + kb] =
          nn < p.N && kk < p.K ? p.b.p[p.b.k_rows ? kk * p.b.ld + n : n * p.b.ld + kk] : static_cast<uint16_t>(0);
    }
    __syncthreads();
    // operand lane l: row l % 16, k = 8 (l / 16) + [0, 8)
    bf16x8 fa[2], fb[2];
    const int r = lane & 15, q = (lane >> 4) * 8;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int ra = 32 * (wave >> 1) + 16 * i + r;
      // kGated: b fragment 0 holds gate columns, fragment 1 the same up columns
      const int rb = kGated ? 32 * i + 16 * (wave & 1) + r : 32 * (wave & 1) + 16 * i + r;
      fa[i] = *reinterpret_cast<const bf16x8*>(&s_a[ra * kRowPad + q]);
      fb[i] = *reinterpret_cast<const bf16x8*>(&s_b[rb * kRowPad + q]);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[j], fa[i], acc[i][j], 0, 0, 0);
    __syncthreads();
  }
  // result lane l: row l % 16 of a, columns 4 (l / 16) + [0, 4) of b
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t m = m0 + 32 * (wave >> 1) + 16 * i + (lane & 15);
    if (m >= p.M) continue;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      if constexpr (kGated) {
        const int64_t n = n0 + 16 * (wave & 1) + 4 * (lane >> 4) + r;
        if (n < p.N) finish_gated(p, m, n, acc[i][0][r], acc[i][1][r]);
      } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int64_t n = n0 + 32 * (wave & 1) + 16 * j + 4 * (lane >> 4) + r;
          if (n < p.N) finish_linear(p, m, n, acc[i][j][r]);
        }
      }
    }
  }
}

__global__ __launch_bounds__(256) void zero_matrix_kernel(void* dst, int64_t ldd, bool f32, int64_t m, int64_t n) {
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < m * n;
       i += static_cast<int64_t>(gridDim.x) * 256)
    store1(dst, i / n * ldd + i % n, f32, 0.0f);
}

}  // namespace

size_t dense_gemm_workspace_bytes(const DenseGemm& p) { return 0; }

hipError_t launch_dense_gemm(const DenseGemm& p, hipStream_t s) {
  const int bn = p.epi == DenseEpi::kGated ? 32 : 64;
  const int64_t grid = (p.M + 63) / 64 * ((p.N + bn - 1) / bn);
  if (p.epi == DenseEpi::kGated)
    dense_gemm_kernel<DenseEpi::kGated><<<static_cast<uint32_t>(grid), 256, 0, s>>>(p);
  else
    dense_gemm_kernel<DenseEpi::kLinear><<<static_cast<uint32_t>(grid), 256, 0, s>>>(p);
  return hipGetLastError();
}

hipError_t launch_zero_matrix(void* dst, int64_t ldd, bool f32, int64_t m, int64_t n, hipStream_t s) {
  if (m * n == 0) return hipSuccess;
  const int64_t blocks = (m * n + 1023) / 1024;
  zero_matrix_kernel<<<static_cast<uint32_t>(blocks < 4096 ? blocks : 4096), 256, 0, s>>>(dst, ldd, f32, m, n);
  return hipGetLastError();
}

}  // namespace dsmoe
