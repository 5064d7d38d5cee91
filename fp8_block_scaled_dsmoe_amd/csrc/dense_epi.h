// Epilogues of the dense products for one result, shared by the kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "act.h"
#include "common.h"
#include "dense.h"

namespace dsmoe {

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

}  // namespace dsmoe
