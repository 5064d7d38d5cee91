// Activations of the dense feed-forward operators and their derivatives, in
// float32.
#pragma once

#include <hip/hip_runtime.h>

#include "dsmoe_dense.h"

namespace dsmoe {

// 1 / (1 + e^-z): e^-z overflows to infinity for z < -88, where the
// reciprocal gives the correct 0
__device__ __forceinline__ float sigmoid_f32(float z) { return __builtin_amdgcn_rcpf(1.0f + expf(-z)); }

// ReLU keeps NaN, as z * (z > 0) does
__device__ __forceinline__ float act_f32(int act, float z) {
  switch (act) {
    case DSMOE_ACT_SILU: return z * sigmoid_f32(z);
    case DSMOE_ACT_GELU: return 0.5f * z * (1.0f + erff(z * 0.70710678118654752f));
    case DSMOE_ACT_RELU: return z > 0.0f || z != z ? z : 0.0f;
    default: return z;
  }
}

// act(z) and act'(z)
__device__ __forceinline__ void act_and_grad_f32(int act, float z, float& f, float& d) {
  switch (act) {
    case DSMOE_ACT_SILU: {
      const float p = sigmoid_f32(z);
      f = z * p;
      d = p * (1.0f + z * (1.0f - p));
      break;
    }
    case DSMOE_ACT_GELU: {
      const float phi = 0.5f * (1.0f + erff(z * 0.70710678118654752f));
      f = z * phi;
      d = phi + z * 0.39894228040143268f * expf(-0.5f * z * z);
      break;
    }
    case DSMOE_ACT_RELU:
      f = z > 0.0f || z != z ? z : 0.0f;
      d = z > 0.0f ? 1.0f : 0.0f;
      break;
    default:
      f = z;
      d = 1.0f;
  }
}

}  // namespace dsmoe
