// mass.cuh -- the two scalar rules of the accumulated attention weight, shared by its kernels.
#pragma once

#include <math.h>

namespace ispa {

// log-sum-exp of a query row over both branches; +inf for a row without any key (both -inf), so that
// exp(s - L) gives every key 0 from it.  NaN in either branch stays NaN: fmaxf drops it, the difference does not.
__device__ __forceinline__ float mass_row_lse(float lse_loc, float lse_hist) {
  const float d = lse_loc == lse_hist ? 0.f : fabsf(lse_loc - lse_hist);
  const float l = fmaxf(lse_loc, lse_hist) + log1pf(expf(-d));
  return l == -INFINITY ? INFINITY : l;
}

// The same in 64 bits.  L is one number for all keys of a query, so with few queries its rounding does not
// average out of the weights: at L = 20 half a unit of fp32 is already 1e-6 of every weight.
__device__ __forceinline__ double mass_row_lse64(float lse_loc, float lse_hist) {
  const double d = lse_loc == lse_hist ? 0.0 : fabs(static_cast<double>(lse_loc) - static_cast<double>(lse_hist));
  const double l = static_cast<double>(fmaxf(lse_loc, lse_hist)) + log1p(exp(-d));
  return l == -INFINITY ? INFINITY : l;
}

// A key's bias is common to all its terms, so it multiplies the sum.  The terms stay finite for the
// biases the attention admits where L covers the key itself, so that s - L <= -b <= 64.  An excluded key (bias
// -inf, or so low that its factor is 0) is in no row's L, and its sum may be anything: it gets 0
// whatever the sum is.
__device__ __forceinline__ float mass_apply_bias(float sum, float bias) {
  const float f = expf(bias);
  return f == 0.f ? 0.f : sum * f;
}

}  // namespace ispa
