// activation.cuh -- the activations of the experts' products.
#pragma once

#include "kernels.h"

namespace moeperm {

// v / (1 + e^-v), to about 2 + 1.2 |v| ulp; below about -87, where e^-v leaves the range
// of the quotient, it is 0 (the value is above -1.5e-36).
__device__ __forceinline__ float silu(float v) { return __fdividef(v, 1.0f + __expf(-v)); }
// v * (the normal distribution function): no cancellation for negative v
__device__ __forceinline__ float gelu(float v) { return v * normcdff(v); }

template <int N>
__device__ __forceinline__ void activate(float (&v)[N], int act) {
  if (act == kActRelu) {
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = v[j] <= 0.0f ? 0.0f : v[j];  // NaN stays NaN
  } else if (act == kActSilu) {
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = silu(v[j]);
  } else if (act == kActGelu) {
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = gelu(v[j]);
  }
}

}  // namespace moeperm
