// Activations of the dense feed-forward operators and their derivatives, in
// float32.
#pragma once

#include <hip/hip_runtime.h>

#include "dsmoe_dense.h"

namespace dsmoe {

// 1 / (1 + e^-z) in p and 1 / (1 + e^z) in q.  Both come from e^-|z|, which
// does not overflow, so p keeps its digits where it is small: a reciprocal of
// 1 + e^-z would be 0 from z = -87.4 on, where float32 still has z p.  The
// reciprocal is the approximate one, within an ulp, of a value in [1, 2].
__device__ __forceinline__ void sigmoid_f32(float z, float& p, float& q) {
  const float t = expf(-__builtin_fabsf(z)), r = __builtin_amdgcn_rcpf(1.0f + t);
  p = z < 0.0f ? t * r : r;
  q = z < 0.0f ? r : t * r;
}

// P(-t) and e = exp(-t^2 / 2) for t = min(|z|, 16), P the normal distribution
// (at 16 both are 0 in float32).  P(-t) = e g(t), where g is smooth and falls
// like 1 / t: a polynomial in u = 1 / (1 + 0.26 t) for g / u, the least relative
// error of degree 8 on [0, 16] (2^-24.6; 2^-21.2 as evaluated here).  So P keeps
// its digits down to the smallest normal float, which 1 + erf does not: it has
// lost half of them at z = -3.5 and all at -5.5.  The square's rounding, up to
// 2^-17 of e, goes back into e.  No slower than with erff: linear 4096 x 7168 x
// 2048 with GELU and z 140 us (141).
__device__ __forceinline__ float normal_tail_f32(float z, float& e) {
  const float t = __builtin_fminf(__builtin_fabsf(z), 16.0f);
  const float s = t * t, s_lo = __builtin_fmaf(t, t, -s);
  e = expf(-0.5f * s);
  e = __builtin_fmaf(e, -0.5f * s_lo, e);
  const float u = __builtin_amdgcn_rcpf(__builtin_fmaf(0.26f, t, 1.0f));
  float g = 0.0294357352f;
  g = __builtin_fmaf(g, u, -0.147665113f);
  g = __builtin_fmaf(g, u, 0.240893915f);
  g = __builtin_fmaf(g, u, -0.138908073f);
  g = __builtin_fmaf(g, u, 0.152684376f);
  g = __builtin_fmaf(g, u, 0.0545265861f);
  g = __builtin_fmaf(g, u, 0.102139667f);
  g = __builtin_fmaf(g, u, 0.103141099f);
  g = __builtin_fmaf(g, u, 0.103751771f);
  return g * u * e;
}

// ReLU keeps NaN, as z * (z > 0) does
__device__ __forceinline__ float act_f32(int act, float z) {
  switch (act) {
    case DSMOE_ACT_SILU: {
      float p, q;
      sigmoid_f32(z, p, q);
      return z * p;
    }
    case DSMOE_ACT_GELU: {
      float e;
      const float p = normal_tail_f32(z, e);
      return z * (z < 0.0f ? p : 1.0f - p);
    }
    case DSMOE_ACT_RELU: return z > 0.0f || z != z ? z : 0.0f;
    default: return z;
  }
}

// act(z) and act'(z)
__device__ __forceinline__ void act_and_grad_f32(int act, float z, float& f, float& d) {
  switch (act) {
    case DSMOE_ACT_SILU: {
      float p, q;
      sigmoid_f32(z, p, q);
      f = z * p;
      d = p * (1.0f + z * q);
      break;
    }
    case DSMOE_ACT_GELU: {
      float e;
      const float p = normal_tail_f32(z, e), phi = z < 0.0f ? p : 1.0f - p;
      f = z * phi;
      d = phi + z * 0.39894228040143268f * e;
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
