// Elementwise parts of the routed experts' backward pass outside FP8: the gradient
// at the gate and up projections with the gate's own, and the router logits'.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "act.h"
#include "common.h"
#include "grouped.h"
#include "router_grad.h"
#include "vec8.h"

namespace dsmoe {
namespace {

// A row by `per_row` threads (a power of 2, 256 at most), 8 columns each at a
// time, 256 / per_row rows of a block at once; the row's dscale is joined by
// shuffles and, past a wave, through LDS, in a fixed order.
// Bound by memory: 16384 rows of I = 2048, 335 MB read and written, in 79 us (4.3
// TB/s); 999 rows of 343 in 6.4.
// dh leaves rounded to bf16, the type of the products' operands.  In a bf16 gradient
// that is an error as large as the result's own rounding: 1.7e-3 of its norm from
// either, 2.3e-3 together (8192 x 2 tokens of 32 experts), and a second product for the
// rest would more than double the pass (2.2 ms; 4.8 with a float32 dW) for a result that
// is rounded anyway.  A float32 gradient takes the rest too, and one that its caller
// rounds has the 1.7e-3 alone.
__global__ __launch_bounds__(256) void grouped_gated_grad_kernel(GroupedGatedGrad p, int per_row) {
  __shared__ float s_sum[4];
  const int t = threadIdx.x % per_row, per_block = 256 / per_row;
  // rows of the groups; offsets as the products take them
  int32_t lo = 0, hi = static_cast<int32_t>(p.groups.R);
  if (p.groups.offsets) {
    lo = min(max(p.groups.offsets[0], 0), hi);
    hi = min(max(p.groups.offsets[p.groups.n], 0), hi);
  }
  for (int64_t r0 = lo + static_cast<int64_t>(blockIdx.x) * per_block; r0 < hi;
       r0 += static_cast<int64_t>(gridDim.x) * per_block) {
    const int64_t r = r0 + threadIdx.x / per_row;
    const bool in = r < hi;
    const float scale = in && p.scale ? p.scale[r] : 1.0f;
    float sum = 0.0f;
    for (int64_t c = 8 * t; in && c < p.I; c += 8 * per_row) {
      const int64_t left = p.I - c;
      float d[8], g[8], u[8], dg[8], du[8];
      unpack8<false>(fetch8<false>(p.da + r * p.ldda + c, left), d);
      unpack8<false>(fetch8<false>(p.h + r * p.ldh + c, left), g);
      unpack8<false>(fetch8<false>(p.h + r * p.ldh + p.I + c, left), u);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float f, df;
        act_and_grad_f32(p.act, g[e], f, df);
        sum = __builtin_fmaf(d[e] * f, u[e], sum);
        dg[e] = scale * (d[e] * u[e] * df);
        du[e] = scale * (d[e] * f);
      }
      if (!p.dh) continue;
      auto store = [&](uint16_t* to) {
        uint16_t* o = to + r * p.lddh + c;
        put8<false>(o, left, dg);
        put8<false>(o + p.I, left, du);
        // the row's padding past 2 I, by the thread that owns the last column
        if (left <= 8)
          for (int64_t j = 2 * p.I; j < p.lddh; ++j) to[r * p.lddh + j] = 0;
      };
      store(p.dh);
      if (p.dh_lo) {
        rest8(dg, pack8(dg));
        rest8(du, pack8(du));
        store(p.dh_lo);
      }
    }
    if (!p.dscale) continue;
    for (int o = min(per_row, 64) >> 1; o > 0; o >>= 1) sum += __shfl_xor(sum, o, 64);
    if (per_row > 64) {
      if ((threadIdx.x & 63) == 0) s_sum[threadIdx.x >> 6] = sum;
      __syncthreads();
      if (t == 0) {
        const int w = threadIdx.x >> 6;
        for (int i = 1; i < per_row / 64; ++i) sum += s_sum[w + i];
      }
      __syncthreads();
    }
    if (in && t == 0) p.dscale[r] = sum;
  }
}

// A wave per token: the chosen experts' values by lane, then the row of dlogits.
// Bound by the launch, and by writing the rows (256 experts: 1 KB a token): 4096 tokens
// in 6.2 us, 32768 in 25.
__global__ __launch_bounds__(256) void router_grad_kernel(const float* __restrict__ dgate,
                                                          const int32_t* __restrict__ topk,
                                                          const float* __restrict__ logits, int64_t T, int32_t E,
                                                          int32_t K, float* __restrict__ dlogits) {
  const int lane = threadIdx.x & 63;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6); t < T;
       t += static_cast<int64_t>(gridDim.x) * 4) {
    // lane k < K holds the k-th choice
    const int32_t e = lane < K ? topk[t * K + lane] : -1;
    const bool in = e >= 0 && e < E;
    write_router_grad(e, in ? logits[t * E + e] : 0.0f, in ? dgate[t * K + lane] : 0.0f, in, K, E, dlogits + t * E);
  }
}

constexpr int64_t kMaxBlocks = 1 << 20;

}  // namespace

hipError_t launch_grouped_gated_grad(const GroupedGatedGrad& p, hipStream_t s) {
  if (p.groups.R == 0) return hipSuccess;
  int per_row = 8;
  while (per_row < 256 && per_row * 8 < p.I) per_row *= 2;
  const int64_t all = (p.groups.R + 256 / per_row - 1) / (256 / per_row);
  const uint32_t blocks = static_cast<uint32_t>(all < kMaxBlocks ? all : kMaxBlocks);
  grouped_gated_grad_kernel<<<blocks, 256, 0, s>>>(p, per_row);
  return hipGetLastError();
}

hipError_t launch_router_grad(const float* dgate, const int32_t* topk, const float* logits, int64_t T, int32_t E,
                              int32_t K, float* dlogits, hipStream_t s) {
  if (T == 0) return hipSuccess;
  const int64_t all = (T + 3) / 4;
  const uint32_t blocks = static_cast<uint32_t>(all < kMaxBlocks ? all : kMaxBlocks);
  router_grad_kernel<<<blocks, 256, 0, s>>>(dgate, topk, logits, T, E, K, dlogits);
  return hipGetLastError();
}

}  // namespace dsmoe
