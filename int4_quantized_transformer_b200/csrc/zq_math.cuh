// zq_math.cuh -- device math shared by the quantizers: GeLU in its exact form.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

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

// Two values of GeLU for kernels that are bound by instructions (37 per value
// as two calls of gelu_erf, 14 here): with a = |v| / sqrt 2 and
// t = 1 / (1 + 0.6 a), the tail beyond |v| is
//   h = 0.5 erfc(a) = t * 2^(P(t) - v^2 log2(e) / 2)
// and gelu(v) = max(v, 0) - |v| h for either sign.  P is the polynomial of
// degree 10 that comes nearest (Remez) to log2(exp(a^2) erfc(a) / (2 t)) for
// a <= 9.4, up to which h counts; its fractional error in h is 2.1e-8, the
// rounding of its coefficients included.  The 0.6 and the degree gave the least
// error with the rounding of the sums: in the mean 5.6e-8 of the result over
// normal values, where 0.5 v erfc(-v / sqrt 2) in fp32 has 5.5e-8, and the
// nine-degree polynomial above with its t had 6.9e-8 in this form.  (A Newton
// step on the reciprocal: 5.5e-8, for one instruction per value more.)
// It is evaluated in t / 4, with 2 in the constant: the power of two is then
// flushed to 0 only where the result is below 7e-39.  The reciprocal and the
// power of two are the hardware's approximations.  Relative error below 1e-6 +
// 1.5 * 2^-24 v^2 (the rounding of the exponent, which counts where h is tiny).
__device__ __forceinline__ float2 gelu_pair(float vx, float vy) {
  auto pack = [](float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
  };
  auto fma2 = [](uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
  };
  constexpr float kLog2e = 1.4426950408889634f;
  constexpr float kSlope = 1.697056275f;  // 4 * 0.6 / sqrt 2
  const float cs[11] = {-1.846338750e+05f, 2.199093750e+05f,  -8.859329688e+04f, 4.672667480e+03f,
                        6.626160645e+03f,  -1.754363037e+03f, 8.786123657e+01f,  -1.347990036e+01f,
                        7.825717926e+00f,  5.761138916e+00f,  -5.626241565e-01f};
  float tx, ty;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(tx) : "f"(fmaf(fabsf(vx), kSlope, 4.0f)));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(ty) : "f"(fmaf(fabsf(vy), kSlope, 4.0f)));
  const uint64_t t = pack(tx, ty), v = pack(vx, vy);
  uint64_t p = pack(cs[0], cs[0]);
#pragma unroll
  for (int i = 1; i < 11; ++i) p = fma2(p, t, pack(cs[i], cs[i]));
  uint64_t vv;
  asm("mul.rn.f32x2 %0, %1, %1;" : "=l"(vv) : "l"(v));
  p = fma2(vv, pack(-0.5f * kLog2e, -0.5f * kLog2e), p);
  float px, py, ex, ey;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(px), "=f"(py) : "l"(p));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(ex) : "f"(px));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(ey) : "f"(py));
  // (+Inf: |v| h is Inf * 0 but for the bound; -Inf and NaN give NaN)
  constexpr float kLargest = 0x1.fffffep127f;
  return make_float2(fmaf(-fabsf(fminf(vx, kLargest)), tx * ex, fmaxf(vx, 0.0f)),
                     fmaf(-fabsf(fminf(vy, kLargest)), ty * ey, fmaxf(vy, 0.0f)));
}

}  // namespace zq
