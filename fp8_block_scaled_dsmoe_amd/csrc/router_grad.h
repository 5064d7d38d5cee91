// The router logits' gradient of one token, for the calls that have the gates'.
#pragma once

#include <hip/hip_runtime.h>

namespace dsmoe {

// With s = sigmoid(z) and S the sum of the chosen s, gate_k = s_k / S gives
//   dz_k = (dgate_k - sum_j dgate_j gate_j) gate_k (1 - s_k).
// A wave's lane k < K has the k-th chosen logit z and its gate's gradient d; in: it
// counts (lanes past K do not).  All in double, rounded once: 1 - s is sigmoid(-z),
// since from s in float32 it has lost half its digits at z = 8 and all at 17.4; the
// bracket is the sum of (dgate_k - dgate_j) gate_j, which cancels nothing where one
// gate is near 1; and s_k / S is formed first, which stays in range where S does not
// (its reciprocal leaves float32 where every z is below -88).
__device__ __forceinline__ float router_logit_grad(float z, float d, bool in, int K) {
  const double zd = static_cast<double>(z), dd = static_cast<double>(d);
  const double s = in ? 1.0 / (1.0 + exp(-zd)) : 0.0;
  double total = 0.0;
  for (int j = 0; j < K; ++j) total += __shfl(s, j, 64);
  const double gate = in ? s / total : 0.0;
  double apart = 0.0;
  for (int j = 0; j < K; ++j) {
    const double dj = __shfl(dd, j, 64), gj = __shfl(gate, j, 64);
    apart += (dd - dj) * gj;
  }
  return static_cast<float>(apart * gate / (1.0 + exp(zd)));
}

}  // namespace dsmoe
