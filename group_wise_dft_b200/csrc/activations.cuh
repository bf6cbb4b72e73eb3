// Pointwise activations in the regular domain (where the group permutes slots,
// so any pointwise map commutes with it), fp32 in and out.
#pragma once

#include <math.h>

#include "eqlin.h"

namespace eqlin {

// SiLU: z s, s = 1 / (1 + e^-z); slope s (1 + z (1 - s)).
// GELU: z Phi(z), Phi(z) = (1 + erf(z / sqrt 2)) / 2; slope Phi(z) + z phi(z).
// The exponential and the quotient are the fast forms (relative error below
// 1e-6 over the range where the result is not negligible): with the IEEE
// forms the activation, not memory, would pace a kernel that applies it to
// every value it moves.  erff is CUDA's, so that fp32 results keep 1e-6.
__device__ __forceinline__ float sigmoid_fast(float z) { return __fdividef(1.0f, 1.0f + __expf(-z)); }

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
  if (ACT == EQLIN_ACT_SILU) return z * sigmoid_fast(z);
  if (ACT == EQLIN_ACT_GELU) return 0.5f * z * (1.0f + erff(z * 0.70710678118654752f));
  return z;
}

// value and slope together
template <int ACT>
__device__ __forceinline__ float act_slope(float z, float &value) {
  if (ACT == EQLIN_ACT_SILU) {
    const float s = sigmoid_fast(z);
    value = z * s;
    return s * fmaf(z, 1.0f - s, 1.0f);
  }
  if (ACT == EQLIN_ACT_GELU) {
    const float phi = 0.5f * (1.0f + erff(z * 0.70710678118654752f));
    value = z * phi;
    return fmaf(z * 0.39894228040143268f, __expf(-0.5f * z * z), phi);
  }
  value = z;
  return 1.0f;
}

// The activation as a launch argument (one uniform branch).
__device__ __forceinline__ float act_any(int act, float z) {
  return act == EQLIN_ACT_SILU ? act_value<EQLIN_ACT_SILU>(z)
         : act == EQLIN_ACT_GELU ? act_value<EQLIN_ACT_GELU>(z) : z;
}
__device__ __forceinline__ float slope_any(int act, float z, float &value) {
  if (act == EQLIN_ACT_SILU) return act_slope<EQLIN_ACT_SILU>(z, value);
  if (act == EQLIN_ACT_GELU) return act_slope<EQLIN_ACT_GELU>(z, value);
  value = z;
  return 1.0f;
}

}  // namespace eqlin
