// Elementwise parts of the dense backward passes: the gradient at the
// pre-activations, as the operand of the two products that follow, and the
// bias gradient's column sums (of the unrounded values).  The matrix cores take
// bf16: the gradient is rounded to it once, as its products' bf16 results
// are, and for float32 results the rounding's rest is kept as a second bf16
// operand, 16 significant bits in all.
// HBM bounds them: dy and z (or da and h) in, dz (dh) out.  Column sums alone of
// 4096 x 7168 (58 MB): 13 us; the gated gradient of 4096 x 2 x 2048 (84 MB in
// all): 20 us, 23 with the second operand (117 MB).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "act.h"
#include "common.h"
#include "dense.h"
#include "vec8.h"

namespace dsmoe {
namespace {

// A block takes `ct` slots of 8 columns (a power of 2, 32 at most) and the rows
// of strip blockIdx.y, 256 / ct of them at a time, two such steps of loads in
// flight; its threads' column sums are joined through LDS.
template <bool ZF32>
__global__ __launch_bounds__(256) void act_backward_kernel(const uint16_t* __restrict__ dy, int64_t lddy,
                                                           const void* __restrict__ z, int64_t ldz, int act,
                                                           int64_t M, int64_t N, int ct, int64_t strip,
                                                           uint16_t* __restrict__ dz, uint16_t* __restrict__ dz_lo,
                                                           int64_t lddz, float* __restrict__ partial) {
  __shared__ float s_sum[256 * 8];
  const int slot = threadIdx.x % ct, rt = 256 / ct;
  const int64_t c = 8 * (static_cast<int64_t>(blockIdx.x) * ct + slot);
  float sum[8] = {};
  const int64_t r1 = min(M, (blockIdx.y + 1) * strip);
  if (c < N) {
#pragma unroll 2
    for (int64_t r = blockIdx.y * strip + threadIdx.x / ct; r < r1; r += rt) {
      float g[8];
      unpack8<false>(fetch8<false>(dy + r * lddy + c, N - c), g);
      if (z) {
        float zz[8];
        unpack8<ZF32>(fetch8<ZF32>(static_cast<const char*>(z) + (r * ldz + c) * (ZF32 ? 4 : 2), N - c), zz);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float f, d;
          act_and_grad_f32(act, zz[e], f, d);
          g[e] *= d;
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] += g[e];
      // dz's rows are padded to a multiple of 8 with zeros (the products read
      // whole groups of 8)
      if (dz) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (c + e >= N) g[e] = 0.0f;
        const u32x4 q = pack8(g);
        *reinterpret_cast<u32x4*>(dz + r * lddz + c) = q;
        if (dz_lo) {
          rest8(g, q);
          *reinterpret_cast<u32x4*>(dz_lo + r * lddz + c) = pack8(g);
        }
      }
    }
  }
  if (!partial) return;
#pragma unroll
  for (int e = 0; e < 8; ++e) s_sum[e * 256 + threadIdx.x] = sum[e];
  __syncthreads();
  // thread i < 8 ct sums column (i / ct) of slot (i % ct), rows in order
  if (static_cast<int>(threadIdx.x) < 8 * ct) {
    const int e = threadIdx.x / ct;
    const int64_t col = 8 * (static_cast<int64_t>(blockIdx.x) * ct + slot) + e;
    float s = 0.0f;
    for (int r = 0; r < rt; ++r) s += s_sum[e * 256 + r * ct + slot];
    if (col < N) partial[blockIdx.y * N + col] = s;
  }
}

// One slot of 8 columns of da per thread and pass over the grid.
__global__ __launch_bounds__(256) void gated_backward_kernel(const uint16_t* __restrict__ da, int64_t ldda,
                                                             const uint16_t* __restrict__ h, int64_t ldh, int act,
                                                             int64_t M, int64_t I,
                                                             uint16_t* __restrict__ dh,
                                                             uint16_t* __restrict__ dh_lo, int64_t lddh) {
  const uint32_t slots = static_cast<uint32_t>((I + 7) / 8);
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < M * slots;
       i += static_cast<int64_t>(gridDim.x) * 256) {
    // 32-bit division where the index allows it
    const int64_t r = i >> 32 ? i / slots : static_cast<uint32_t>(i) / slots;
    const int64_t c = 8 * (i - r * slots);
    float d[8], g[8], u[8], dg[8], du[8];
    unpack8<false>(fetch8<false>(da + r * ldda + c, I - c), d);
    unpack8<false>(fetch8<false>(h + r * ldh + c, I - c), g);
    unpack8<false>(fetch8<false>(h + r * ldh + I + c, I - c), u);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float f, df;
      act_and_grad_f32(act, g[e], f, df);
      dg[e] = d[e] * u[e] * df;
      du[e] = d[e] * f;
    }
    auto store = [&](uint16_t* to) {
      uint16_t* o = to + r * lddh + c;
      put8<false>(o, I - c, dg);
      put8<false>(o + I, I - c, du);
      // the row's padding past 2 I, by the thread that owns the last column
      if (c + 8 >= I)
        for (int64_t j = 2 * I; j < lddh; ++j) to[r * lddh + j] = 0;
    };
    store(dh);
    if (dh_lo) {
      rest8(dg, pack8(dg));
      rest8(du, pack8(du));
      store(dh_lo);
    }
  }
}

constexpr int64_t kMaxBlocks = 1 << 23;   // 2^31 threads; a launch holds fewer than 2^32

// column slots of a block of act_backward_kernel, rows of a strip: about 1024
// blocks, of at least two steps of rows each; few rows are one strip, whose
// sums need no second launch
int column_slots(int64_t N) {
  int ct = 1;
  while (ct < 32 && ct * 8 < N) ct *= 2;
  return ct;
}
int64_t strip_rows(int64_t M, int64_t N) {
  const int ct = column_slots(N);
  const int64_t blocks_n = (N + 8 * ct - 1) / (8 * ct), step = 256 / ct;
  const int64_t strips = (1024 + blocks_n - 1) / blocks_n, least = (M + 65534) / 65535;   // the grid's limit
  const int64_t rows = (M + strips - 1) / strips;
  if (M <= 4 * step) return M;
  const int64_t s = rows < 2 * step ? 2 * step : rows;
  return s < least ? least : s;
}

}  // namespace

int64_t bias_partial_rows(int64_t M, int64_t N) {
  return M == 0 ? 0 : (M + strip_rows(M, N) - 1) / strip_rows(M, N);
}

hipError_t launch_act_backward(const uint16_t* dy, int64_t lddy, const void* z, int64_t ldz, bool z_f32, int act,
                               int64_t M, int64_t N, uint16_t* dz, uint16_t* dz_lo, int64_t lddz, float* partial,
                               hipStream_t s) {
  if (M == 0) return hipSuccess;
  const int ct = column_slots(N);
  const int64_t strip = strip_rows(M, N);
  const dim3 grid(static_cast<uint32_t>((N + 8 * ct - 1) / (8 * ct)), static_cast<uint32_t>((M + strip - 1) / strip));
  if (z_f32)
    act_backward_kernel<true><<<grid, 256, 0, s>>>(dy, lddy, z, ldz, act, M, N, ct, strip, dz, dz_lo, lddz, partial);
  else
    act_backward_kernel<false><<<grid, 256, 0, s>>>(dy, lddy, z, ldz, act, M, N, ct, strip, dz, dz_lo, lddz, partial);
  return hipGetLastError();
}

hipError_t launch_gated_backward(const uint16_t* da, int64_t ldda, const uint16_t* h, int64_t ldh, int act,
                                 int64_t M, int64_t I, uint16_t* dh, uint16_t* dh_lo, int64_t lddh, hipStream_t s) {
  if (M == 0) return hipSuccess;
  const int64_t all = (M * ((I + 7) / 8) + 255) / 256;
  const uint32_t blocks = static_cast<uint32_t>(all < kMaxBlocks ? all : kMaxBlocks);
  gated_backward_kernel<<<blocks, 256, 0, s>>>(da, ldda, h, ldh, act, M, I, dh, dh_lo, lddh);
  return hipGetLastError();
}

}  // namespace dsmoe
