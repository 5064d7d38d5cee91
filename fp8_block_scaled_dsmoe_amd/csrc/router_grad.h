// The router logits' gradient of one token, for the calls that have the gates'.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dsmoe {

// Lane j's value, j the same in all lanes.
__device__ __forceinline__ int32_t lane_value(int32_t v, int j) { return __builtin_amdgcn_readlane(v, j); }
__device__ __forceinline__ float lane_value(float v, int j) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), j));
}
__device__ __forceinline__ double lane_value(double v, int j) {
  return __hiloint2double(__builtin_amdgcn_readlane(__double2hiint(v), j), __builtin_amdgcn_readlane(__double2loint(v), j));
}

// With s = sigmoid(z) and S the sum of the chosen s, gate_k = s_k / S gives
//   dz_k = (dgate_k - sum_j dgate_j gate_j) gate_k (1 - s_k).
// A whole wave: lane k < K has the k-th chosen expert e, e's logit z and its gate's
// gradient d; in: it counts (lanes past K do not).  The wave writes the token's row
// of dlogits, 0 at the other experts; an expert chosen twice has both values.  All in double, rounded once: 1 - s is sigmoid(-z),
// since from s in float32 it has lost half its digits at z = 8 and all at 17.4; the
// bracket is the sum of (dgate_k - dgate_j) gate_j, which cancels nothing where one
// gate is near 1; and s_k / S is formed first, which stays in range where S does not
// (its reciprocal leaves float32 where every z is below -88).
__device__ __forceinline__ void write_router_grad(int32_t e, float z, float d, bool in, int K, int32_t E,
                                                  float* __restrict__ dlogits) {
  const double t = exp(-fabs(static_cast<double>(z))), r = 1.0 / (1.0 + t);
  const double s = !in ? 0.0 : z < 0.0f ? t * r : r, q = z < 0.0f ? r : t * r;
  double total = 0.0;
  for (int j = 0; j < K; ++j) total += lane_value(s, j);
  const double gate = in ? s / total : 0.0;
  double apart = 0.0;
  for (int j = 0; j < K; ++j) apart += (static_cast<double>(d) - static_cast<double>(lane_value(d, j))) * lane_value(gate, j);
  const float v = static_cast<float>(apart * gate * q);
  for (int32_t c = threadIdx.x & 63; c < E; c += 64) {
    float o = 0.0f;
    for (int k = 0; k < K; ++k)
      if (lane_value(e, k) == c) o += lane_value(v, k);
    dlogits[c] = o;
  }
}

}  // namespace dsmoe
