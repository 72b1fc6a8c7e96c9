// zq_math.cuh -- device math shared by the quantizers: GeLU in its exact form.
#pragma once
#include <cuda_runtime.h>

namespace zq {

// erfc(a) for a >= 0 in fp32: the Chebyshev approximation of Press, Teukolsky,
// Vetterling and Flannery, "Numerical Recipes", Sec. 6.2 (erfc with
// fractional error below 1.2e-7 everywhere), as
//   erfc(a) ~ t * exp(-a^2 + P(t)),  t = 1 / (1 + a/2),
// P a degree-9 polynomial, with the hardware exp2.  Fractional (not absolute)
// accuracy matters here: for negative v, GeLU is v times a tiny erfc.
__device__ __forceinline__ float erfc_nonneg(float a) {
  const float t = __frcp_rn(__fmaf_rn(0.5f, a, 1.0f));
  float p = 0.17087277f;
  p = __fmaf_rn(p, t, -0.82215223f);
  p = __fmaf_rn(p, t, 1.48851587f);
  p = __fmaf_rn(p, t, -1.13520398f);
  p = __fmaf_rn(p, t, 0.27886807f);
  p = __fmaf_rn(p, t, -0.18628806f);
  p = __fmaf_rn(p, t, 0.09678418f);
  p = __fmaf_rn(p, t, 0.37409196f);
  p = __fmaf_rn(p, t, 1.00002368f);
  p = __fmaf_rn(p, t, -1.26551223f);
  return t * __expf(__fmaf_rn(-a, a, p));
}

// GeLU, exact form: v * Phi(v) with Phi(v) = 0.5 erfc(-v / sqrt 2), i.e.
// 0.5 erfc(|v|/sqrt 2) for v <= 0 and 1 - 0.5 erfc(v/sqrt 2) for v > 0 (no
// cancellation for negative v).  The result stays well within an fp16 ulp of
// the correctly rounded value; the tests hold it to one fp16 ulp.
__device__ __forceinline__ float gelu_erf(float v) {
  const float h = 0.5f * erfc_nonneg(fabsf(v) * 0.70710678118654752f);
  return v * (v > 0.0f ? 1.0f - h : h);
}

}  // namespace zq
