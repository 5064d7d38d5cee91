// Layer norm, forward and backward.
//
// Forward, per row of s = x + residual (cols values):
//   mu = sum(s) / cols,  var = sum((s - mu)^2) / cols,  rstd = 1 / sqrt(var + eps)
//   y = (s - mu) rstd gamma + beta
// The deviations are summed from the row held in registers (a second pass
// over registers, not over memory), so the variance does not cancel as
// E[s^2] - mu^2 would.  Backward, with n = (x - mu) rstd and g = dy gamma:
//   dx = rstd (g - mean(g) - n mean(g n)) + dsum
//   dgamma = sum_rows dy n,  dbeta = sum_rows dy
//
// Both move every byte once and do a few operations per byte: HBM bounds them.
// bf16 rows of 7168: forward with residual 32768 rows (1.88 GB) in 330 us, 5.7
// TB/s; backward with dsum 4096 rows (235 MB) in 50 us, 4.7 TB/s.  At few rows
// it is latency: one row takes 5 us in the kernel.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.h"
#include "dense.h"
#include "vec8.h"

namespace dsmoe {
namespace {

__device__ __forceinline__ uint16_t f32_to_bf16(float v) { return static_cast<uint16_t>(f32x2_to_bf16x2(v, 0.0f)); }

__device__ __forceinline__ float load1(const void* p, int64_t i, bool f32) {
  return f32 ? static_cast<const float*>(p)[i] : bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
}

// A row of up to NT * 8 * PER values over NT threads: slot v of thread t holds
// columns 8 (v NT + t) + [0, 8), those past cols 0.
template <bool F32, int NT>
struct Row {
  using Raw = Raw8<F32>;
  static constexpr int ES = F32 ? 4 : 2;
  static __device__ __forceinline__ int64_t col(int v, int t) { return 8 * (static_cast<int64_t>(v) * NT + t); }
  static __device__ __forceinline__ Raw fetch(const void* base, int v, int t, int64_t cols) {
    const int64_t c = col(v, t);
    return fetch8<F32>(static_cast<const char*>(base) + c * ES, cols - c);
  }
  static __device__ __forceinline__ void load(const void* base, int v, int t, int64_t cols, float* o) {
    unpack8<F32>(fetch(base, v, t, cols), o);
  }
  static __device__ __forceinline__ void store(void* base, int v, int t, int64_t cols, const float* o) {
    const int64_t c = col(v, t);
    if (c < cols) put8<F32>(static_cast<char*>(base) + c * ES, cols - c, o);
  }
  static __device__ __forceinline__ bool in(int v, int e, int t, int64_t cols) { return col(v, t) + e < cols; }
};

// slot v of a parameter vector
template <int NT>
__device__ __forceinline__ void load_param(const void* p, bool p_f32, float missing, int v, int t, int64_t cols,
                                           float* o) {
  if (!p) {
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = missing;
  } else if (p_f32) {
    Row<true, NT>::load(p, v, t, cols, o);
  } else {
    Row<false, NT>::load(p, v, t, cols, o);
  }
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// Sums of N values over NT threads (NT / 64 waves from wave w0 of the block),
// left in every thread.  scratch: one slot of N floats per wave of the block.
template <int NT, int N>
__device__ __forceinline__ void group_sum(float* v, float* scratch, int wave) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  if constexpr (NT > 64) {
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) scratch[wave * N + i] = v[i];
    }
    __syncthreads();
    constexpr int W = NT / 64;
    const int w0 = wave / W * W;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < W; ++w) s += scratch[(w0 + w) * N + i];
      v[i] = s;
    }
  }
}

constexpr int kFwdThreads = 256;

// One row per NT threads, as few as hold it at 8 to 32 values each: more rows in
// flight per CU, and up to 64 threads no barrier.
template <bool F32, int NT, int PER>
__global__ __launch_bounds__(NT > kFwdThreads ? NT : kFwdThreads) void layer_norm_kernel(NormFwd p, int64_t row0) {
  constexpr int BT = NT > kFwdThreads ? NT : kFwdThreads;
  constexpr int ES = F32 ? 4 : 2;
  using R = Row<F32, NT>;
  __shared__ float s_red[2][BT / 64];
  const int wave = threadIdx.x >> 6;
  const int t = threadIdx.x % NT;
  const int64_t row = row0 + static_cast<int64_t>(blockIdx.x) * (BT / NT) + threadIdx.x / NT;
  if (NT <= 64 && row >= p.rows) return;   // whole waves; wider groups fill their block
  const int64_t cols = p.cols;
  float s[PER][8];
  const char* xr = static_cast<const char*>(p.x) + row * p.ldx * ES;
#pragma unroll
  for (int v = 0; v < PER; ++v) R::load(xr, v, t, cols, s[v]);
  if (p.residual) {
    const char* rr = static_cast<const char*>(p.residual) + row * p.ldr * ES;
#pragma unroll
    for (int v = 0; v < PER; ++v) {
      float r[8];
      R::load(rr, v, t, cols, r);
#pragma unroll
      for (int e = 0; e < 8; ++e) s[v][e] += r[e];
    }
  }
  if (p.sum) {
    char* sr = static_cast<char*>(p.sum) + row * p.lds * ES;
#pragma unroll
    for (int v = 0; v < PER; ++v) R::store(sr, v, t, cols, s[v]);
  }
  float acc = 0.0f;
#pragma unroll
  for (int v = 0; v < PER; ++v)
#pragma unroll
    for (int e = 0; e < 8; ++e) acc += s[v][e];
  group_sum<NT, 1>(&acc, s_red[0], wave);
  const float mean = acc / static_cast<float>(cols);
  acc = 0.0f;
#pragma unroll
  for (int v = 0; v < PER; ++v)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      s[v][e] -= mean;
      if (R::in(v, e, t, cols)) acc = __builtin_fmaf(s[v][e], s[v][e], acc);
    }
  group_sum<NT, 1>(&acc, s_red[1], wave);
  const float rstd = 1.0f / sqrtf(acc / static_cast<float>(cols) + p.eps);
  char* yr = static_cast<char*>(p.y) + row * p.ldy * ES;
#pragma unroll
  for (int v = 0; v < PER; ++v) {
    float ga[8], be[8], o[8];
    load_param<NT>(p.gamma, p.p_f32, 1.0f, v, t, cols, ga);
    load_param<NT>(p.beta, p.p_f32, 0.0f, v, t, cols, be);
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = __builtin_fmaf(s[v][e] * rstd, ga[e], be[e]);
    R::store(yr, v, t, cols, o);
  }
  if (t == 0) {
    if (p.mean) p.mean[row] = mean;
    if (p.rstd) p.rstd[row] = rstd;
  }
}

// Rows too long for registers (above 32768 columns): one block per row, three
// passes over it, the last two from L2.
constexpr int kLongThreads = 1024;
template <bool F32>
__global__ __launch_bounds__(kLongThreads) void layer_norm_long_kernel(NormFwd p, int64_t row0) {
  constexpr int ES = F32 ? 4 : 2;
  __shared__ float s_red[2][kLongThreads / 64];
  const int64_t row = row0 + blockIdx.x;
  const int wave = threadIdx.x >> 6;
  const char* xr = static_cast<const char*>(p.x) + row * p.ldx * ES;
  const char* rr = p.residual ? static_cast<const char*>(p.residual) + row * p.ldr * ES : nullptr;
  auto at = [&](int64_t c) { return load1(xr, c, F32) + (rr ? load1(rr, c, F32) : 0.0f); };
  float acc = 0.0f;
  for (int64_t c = threadIdx.x; c < p.cols; c += kLongThreads) acc += at(c);
  group_sum<kLongThreads, 1>(&acc, s_red[0], wave);
  const float mean = acc / static_cast<float>(p.cols);
  acc = 0.0f;
  for (int64_t c = threadIdx.x; c < p.cols; c += kLongThreads) {
    const float d = at(c) - mean;
    acc = __builtin_fmaf(d, d, acc);
  }
  group_sum<kLongThreads, 1>(&acc, s_red[1], wave);
  const float rstd = 1.0f / sqrtf(acc / static_cast<float>(p.cols) + p.eps);
  for (int64_t c = threadIdx.x; c < p.cols; c += kLongThreads) {
    const float s = at(c);   // read before either output may overwrite it
    const float y = __builtin_fmaf((s - mean) * rstd, p.gamma ? load1(p.gamma, c, p.p_f32) : 1.0f,
                                   p.beta ? load1(p.beta, c, p.p_f32) : 0.0f);
    if constexpr (F32) {
      if (p.sum) reinterpret_cast<float*>(static_cast<char*>(p.sum) + row * p.lds * ES)[c] = s;
      reinterpret_cast<float*>(static_cast<char*>(p.y) + row * p.ldy * ES)[c] = y;
    } else {
      if (p.sum) reinterpret_cast<uint16_t*>(static_cast<char*>(p.sum) + row * p.lds * ES)[c] = f32_to_bf16(s);
      reinterpret_cast<uint16_t*>(static_cast<char*>(p.y) + row * p.ldy * ES)[c] = f32_to_bf16(y);
    }
  }
  if (threadIdx.x == 0) {
    if (p.mean) p.mean[row] = mean;
    if (p.rstd) p.rstd[row] = rstd;
  }
}

// A launch holds fewer than 2^32 threads: f(first row, rows of the launch) for
// ranges of `rows` that take 2^31 at `threads` per row.
template <typename F>
hipError_t by_row_ranges(int64_t rows, int threads, F f) {
  const int64_t step = (int64_t{1} << 31) / threads;
  for (int64_t r = 0; r < rows; r += step) {
    f(r, rows - r < step ? rows - r : step);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <bool F32>
hipError_t launch_fwd(const NormFwd& p, hipStream_t s) {
#define DSMOE_LN(NT, PER)                                                                                \
  return by_row_ranges(p.rows, NT, [&](int64_t r0, int64_t n) {                                          \
    constexpr int bt = NT > kFwdThreads ? NT : kFwdThreads;                                              \
    const uint32_t grid = static_cast<uint32_t>((n + bt / NT - 1) / (bt / NT));                          \
    layer_norm_kernel<F32, NT, PER><<<grid, bt, 0, s>>>(p, r0);                                          \
  })
  if (p.cols <= 512) DSMOE_LN(64, 1);
  if (p.cols <= 1024) DSMOE_LN(64, 2);
  if (p.cols <= 2048) DSMOE_LN(256, 1);
  if (p.cols <= 4096) DSMOE_LN(256, 2);
  if (p.cols <= 8192) DSMOE_LN(256, 4);
  if (p.cols <= 16384) DSMOE_LN(512, 4);
  if (p.cols <= 32768) DSMOE_LN(1024, 4);
#undef DSMOE_LN
  return by_row_ranges(p.rows, kLongThreads, [&](int64_t r0, int64_t n) {
    layer_norm_long_kernel<F32><<<static_cast<uint32_t>(n), kLongThreads, 0, s>>>(p, r0);
  });
}

// ---------------------------------------------------------------------------
// Backward.  A block walks over rows with stride gridDim; its NT threads per
// row own fixed columns, so the weight gradients accumulate in registers over
// the block's rows and leave as one partial row per block, summed by
// sum_partials_kernel in a fixed order (no atomics: equal calls, equal bits).
// ---------------------------------------------------------------------------
constexpr int kBwdThreads = 512;
// One block per CU: its 160 registers leave no room for a second, and every
// block writes a partial row (512 blocks took 67 us on 4096 x 7168, 256 took 53)
constexpr int64_t kBwdBlocks = 256;

// PER: slots of 8 columns per thread
template <bool F32, int NT, int PER>
__global__ __launch_bounds__(kBwdThreads) void layer_norm_bwd_kernel(NormBwd p) {
  constexpr int BT = kBwdThreads, RG = BT / NT;
  constexpr int ES = F32 ? 4 : 2;
  using R = Row<F32, NT>;
  __shared__ float s_red[2][2 * (BT / 64)];
  __shared__ float s_part[RG > 1 ? BT * PER * 8 : 1];
  const int wave = threadIdx.x >> 6;
  const int t = threadIdx.x % NT, rg = threadIdx.x / NT;
  const int64_t cols = p.cols;
  const float inv = 1.0f / static_cast<float>(cols);
  float ga[PER][8], dga[PER][8], dbe[PER][8];
#pragma unroll
  for (int v = 0; v < PER; ++v) {
    load_param<NT>(p.gamma, p.p_f32, 1.0f, v, t, cols, ga[v]);
#pragma unroll
    for (int e = 0; e < 8; ++e) dga[v][e] = dbe[v][e] = 0.0f;
  }
  // The next row is fetched before this one is finished: with the loads of a
  // row waited for in turn, even two blocks per CU kept too few bytes on the
  // way (4096 x 7168 bf16 with dsum took 103 us, not 50).
  constexpr bool kAhead = PER <= 2;   // beyond, there are no registers left for it
  typename R::Raw nx[PER], ny[PER], nd[PER];
  float nmean = 0.0f, nrstd = 0.0f;
  auto fetch = [&](int64_t row) {
    if (row >= p.rows) return;   // the same for a row's NT threads
    nmean = p.mean[row];
    nrstd = p.rstd[row];
#pragma unroll
    for (int v = 0; v < PER; ++v) {
      nx[v] = R::fetch(static_cast<const char*>(p.x) + row * p.ldx * ES, v, t, cols);
      ny[v] = R::fetch(static_cast<const char*>(p.dy) + row * p.lddy * ES, v, t, cols);
      if (kAhead && p.dsum) nd[v] = R::fetch(static_cast<const char*>(p.dsum) + row * p.ldds * ES, v, t, cols);
    }
  };
  int flip = 0;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * RG;
  if (kAhead) fetch(static_cast<int64_t>(blockIdx.x) * RG + rg);
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * RG; r0 < p.rows; r0 += stride, flip ^= 1) {
    const int64_t row = r0 + rg;
    const bool live = row < p.rows;
    float x[PER][8], dy[PER][8], sums[2] = {0.0f, 0.0f};
    typename R::Raw ds[PER];
    if (!kAhead) fetch(row);
    const float mean = nmean, rstd = nrstd;
#pragma unroll
    for (int v = 0; v < PER; ++v) {
      unpack8<F32>(nx[v], x[v]);
      unpack8<F32>(ny[v], dy[v]);
      if (kAhead) ds[v] = nd[v];
    }
    if (kAhead) fetch(row + stride);
    if (live) {
#pragma unroll
      for (int v = 0; v < PER; ++v)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (!R::in(v, e, t, cols)) continue;
          x[v][e] = (x[v][e] - mean) * rstd;   // n
          const float g = dy[v][e] * ga[v][e];
          sums[0] += g;
          sums[1] = __builtin_fmaf(g, x[v][e], sums[1]);
        }
    }
    group_sum<NT, 2>(sums, s_red[flip], wave);
    if (!live) continue;
    const float c1 = sums[0] * inv, c2 = sums[1] * inv;
#pragma unroll
    for (int v = 0; v < PER; ++v) {
      float o[8], d[8];
      if (p.dsum) {
        unpack8<F32>(kAhead ? ds[v] : R::fetch(static_cast<const char*>(p.dsum) + row * p.ldds * ES, v, t, cols), d);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) d[e] = 0.0f;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        o[e] = __builtin_fmaf(rstd, dy[v][e] * ga[v][e] - c1 - x[v][e] * c2, d[e]);
        dga[v][e] = __builtin_fmaf(dy[v][e], x[v][e], dga[v][e]);
        dbe[v][e] += dy[v][e];
      }
      R::store(static_cast<char*>(p.dx) + row * p.lddx * ES, v, t, cols, o);
    }
  }
  if (!p.partial) return;
  // one partial row [dgamma | dbeta] per block: the row groups' sums are
  // joined in LDS first
  float* out = p.partial + static_cast<int64_t>(blockIdx.x) * 2 * cols;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    float(&acc)[PER][8] = which ? dbe : dga;
    if constexpr (RG > 1) {
      __syncthreads();
#pragma unroll
      for (int v = 0; v < PER; ++v)
#pragma unroll
        for (int e = 0; e < 8; ++e) s_part[(rg * PER * 8 + v * 8 + e) * NT + t] = acc[v][e];
      __syncthreads();
      if (rg == 0) {
#pragma unroll
        for (int v = 0; v < PER; ++v)
#pragma unroll
          for (int e = 0; e < 8; ++e)
#pragma unroll
            for (int g = 1; g < RG; ++g) acc[v][e] += s_part[(g * PER * 8 + v * 8 + e) * NT + t];
      }
    }
    if (rg == 0) {
#pragma unroll
      for (int v = 0; v < PER; ++v) Row<true, NT>::store(out + which * cols, v, t, cols, acc[v]);
    }
  }
}

// Rows too long for registers: dx by one block per row, two passes over it...
template <bool F32>
__global__ __launch_bounds__(kLongThreads) void layer_norm_bwd_long_kernel(NormBwd p, int64_t row0) {
  constexpr int ES = F32 ? 4 : 2;
  __shared__ float s_red[2 * (kLongThreads / 64)];
  const int64_t row = row0 + blockIdx.x;
  const char* xr = static_cast<const char*>(p.x) + row * p.ldx * ES;
  const char* yr = static_cast<const char*>(p.dy) + row * p.lddy * ES;
  const char* sr = p.dsum ? static_cast<const char*>(p.dsum) + row * p.ldds * ES : nullptr;
  char* dr = static_cast<char*>(p.dx) + row * p.lddx * ES;
  const float mean = p.mean[row], rstd = p.rstd[row];
  auto gam = [&](int64_t c) { return p.gamma ? load1(p.gamma, c, p.p_f32) : 1.0f; };
  float sums[2] = {0.0f, 0.0f};
  for (int64_t c = threadIdx.x; c < p.cols; c += kLongThreads) {
    const float g = load1(yr, c, F32) * gam(c);
    sums[0] += g;
    sums[1] = __builtin_fmaf(g, (load1(xr, c, F32) - mean) * rstd, sums[1]);
  }
  group_sum<kLongThreads, 2>(sums, s_red, threadIdx.x >> 6);
  const float inv = 1.0f / static_cast<float>(p.cols);
  const float c1 = sums[0] * inv, c2 = sums[1] * inv;
  for (int64_t c = threadIdx.x; c < p.cols; c += kLongThreads) {
    const float n = (load1(xr, c, F32) - mean) * rstd;
    const float o = __builtin_fmaf(rstd, load1(yr, c, F32) * gam(c) - c1 - n * c2, sr ? load1(sr, c, F32) : 0.0f);
    if constexpr (F32)
      reinterpret_cast<float*>(dr)[c] = o;
    else
      reinterpret_cast<uint16_t*>(dr)[c] = f32_to_bf16(o);
  }
}

// ... and the weight gradients by columns, before dx may overwrite dy or x:
// block (b, strip) takes 256 columns and every gridDim.y-th row.
template <bool F32>
__global__ __launch_bounds__(256) void layer_norm_wgrad_long_kernel(NormBwd p) {
  constexpr int ES = F32 ? 4 : 2;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (c >= p.cols) return;
  float dga = 0.0f, dbe = 0.0f;
  for (int64_t r = blockIdx.y; r < p.rows; r += gridDim.y) {
    const float dy = load1(static_cast<const char*>(p.dy) + r * p.lddy * ES, c, F32);
    const float x = load1(static_cast<const char*>(p.x) + r * p.ldx * ES, c, F32);
    dga = __builtin_fmaf(dy, (x - p.mean[r]) * p.rstd[r], dga);
    dbe += dy;
  }
  float* out = p.partial + static_cast<int64_t>(blockIdx.y) * 2 * p.cols;
  out[c] = dga;
  out[p.cols + c] = dbe;
}

// out[c] = sum over r < n of partial[r][c]: 64 columns per block, each of 16
// waves sums a 16th of the rows, 8 loads in flight; joined in order (256 rows of
// 14336 columns in 4.8 us, from L2).
constexpr int kSumWaves = 16;
__global__ __launch_bounds__(64 * kSumWaves) void sum_partials_kernel(const float* __restrict__ partial, int64_t n,
                                                                      int64_t cols, int64_t split,
                                                                      float* __restrict__ out0,
                                                                      float* __restrict__ out1) {
  __shared__ float s_sum[kSumWaves][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 64 + lane;
  float acc = 0.0f;
  if (c < cols) {
    const int64_t per = (n + kSumWaves - 1) / kSumWaves, r1 = min(n, (w + 1) * per);
    int64_t r = w * per;
    for (; r + 8 <= r1; r += 8) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = partial[(r + i) * cols + c];
#pragma unroll
      for (int i = 0; i < 8; ++i) acc += v[i];
    }
    for (; r < r1; ++r) acc += partial[r * cols + c];
  }
  s_sum[w][lane] = acc;
  __syncthreads();
  if (w == 0 && c < cols) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kSumWaves; ++i) s += s_sum[i][lane];
    (c < split ? out0[c] : out1[c - split]) = s;
  }
}

hipError_t sum_partials(const float* partial, int64_t n, int64_t cols, int64_t split, float* o0, float* o1,
                        hipStream_t s) {
  sum_partials_kernel<<<static_cast<uint32_t>((cols + 63) / 64), 64 * kSumWaves, 0, s>>>(partial, n, cols, split, o0,
                                                                                       o1);
  return hipGetLastError();
}

// threads per row of the backward (two slots each; 512 threads also four); 0:
// the long-row kernels
int bwd_nt(int64_t cols) {
  for (int nt = 64; nt <= kBwdThreads; nt *= 2)
    if (cols <= nt * 16) return nt;
  return cols <= kBwdThreads * 32 ? kBwdThreads : 0;
}
int64_t bwd_partial_rows(int64_t rows, int64_t cols) {
  const int nt = bwd_nt(cols);
  if (nt == 0) return rows < 64 ? rows : 64;
  const int64_t rg = kBwdThreads / nt, blocks = (rows + rg - 1) / rg;
  return blocks < kBwdBlocks ? blocks : kBwdBlocks;
}

template <bool F32>
hipError_t launch_bwd(const NormBwd& p, hipStream_t s) {
  const uint32_t grid = static_cast<uint32_t>(bwd_partial_rows(p.rows, p.cols));
  switch (bwd_nt(p.cols)) {
#define DSMOE_LNB(NT, PER) layer_norm_bwd_kernel<F32, NT, PER><<<grid, kBwdThreads, 0, s>>>(p)
    case 64: DSMOE_LNB(64, 2); break;
    case 128: DSMOE_LNB(128, 2); break;
    case 256: DSMOE_LNB(256, 2); break;
    case 512:
      if (p.cols <= 512 * 16)
        DSMOE_LNB(512, 2);
      else
        DSMOE_LNB(512, 4);
      break;
#undef DSMOE_LNB
    default:
      if (p.partial) {
        const dim3 g(static_cast<uint32_t>((p.cols + 255) / 256), grid);
        layer_norm_wgrad_long_kernel<F32><<<g, 256, 0, s>>>(p);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
      }
      return by_row_ranges(p.rows, kLongThreads, [&](int64_t r0, int64_t n) {
        layer_norm_bwd_long_kernel<F32><<<static_cast<uint32_t>(n), kLongThreads, 0, s>>>(p, r0);
      });
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_layer_norm(const NormFwd& p, hipStream_t s) {
  return p.x_f32 ? launch_fwd<true>(p, s) : launch_fwd<false>(p, s);
}

size_t layer_norm_backward_partial_floats(int64_t rows, int64_t cols) {
  return static_cast<size_t>(bwd_partial_rows(rows, cols)) * 2 * cols;
}

hipError_t launch_layer_norm_backward(const NormBwd& p, hipStream_t s) {
  if (p.rows > 0) {
    const hipError_t e = p.x_f32 ? launch_bwd<true>(p, s) : launch_bwd<false>(p, s);
    if (e != hipSuccess) return e;
  }
  if (!p.dgamma) return hipSuccess;
  return sum_partials(p.partial, bwd_partial_rows(p.rows, p.cols), 2 * p.cols, p.cols, p.dgamma, p.dbeta, s);
}

hipError_t launch_sum_partials(const float* partial, int64_t n, int64_t cols, float* out, hipStream_t s) {
  return sum_partials(partial, n, cols, cols, out, out, s);
}

}  // namespace dsmoe
