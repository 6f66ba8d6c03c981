// gelu.cuh -- the GELU's erf form, for the kernels that apply it.
#pragma once

namespace i8 {

// GELU in erf form, x * Phi(x) with Phi the standard normal CDF.  With
// t = erfc(|x| / sqrt 2): Phi(x) = 1 - t / 2 for x >= 0 and t / 2 for x < 0.
// One erfc per element, the same call on every lane (no divergent branch),
// and no cancellation: the naive 1 + erf(x / sqrt 2) is 6e-7 at x = -5,
// where fp32 resolves only 6e-8 near 1.
__device__ __forceinline__ float gelu_erf(float x) {
  constexpr float kRsqrt2 = 0.70710678118654752f;
  const float t = erfcf(fabsf(x) * kRsqrt2);
  const float phi = x >= 0.0f ? 1.0f - 0.5f * t : 0.5f * t;
  return x * phi;
}

}  // namespace i8
