// zq_fp8.cuh -- 16-bit activations (fp16 or bf16) in and out of fp32, and the
// e4m3 block quantization step shared by the row and the weight quantizer.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "zq_internal.h"

namespace zq {

constexpr int kFp8Block = 128;        // k values (and weight rows) that share one scale
constexpr float kE4m3Max = 448.0f;    // largest finite e4m3 magnitude
constexpr float kAmaxFloor = 0x1p-110f;  // smallest block maximum that is told apart (448/amax stays finite)

// One 32-bit word of two 16-bit values to fp32 (exact) and back (round to nearest even).
template <typename E>
__device__ __forceinline__ float2 unpack2(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
template <typename E>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <typename E>
__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = unpack2<E>(w[i]);
    f[2 * i] = p.x;
    f[2 * i + 1] = p.y;
  }
}
template <typename E>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack2<E>(f[0], f[1]), pack2<E>(f[2], f[3]), pack2<E>(f[4], f[5]),
                    pack2<E>(f[6], f[7]));
}

// max(a, b), NaN if either is: a NaN in a block has to reach its scale.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// max(a, |b|, |c|) for a >= 0, NaN if any is.
__device__ __forceinline__ float max_nan_abs(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Two fp32 values in one 64-bit register: one instruction for both.
__device__ __forceinline__ uint64_t pack_f32x2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpack_f32x2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
// The two 16-bit values of a word as a pair of fp32.
template <typename E>
__device__ __forceinline__ uint64_t widen2(uint32_t w) {
  const float2 f = unpack2<E>(w);
  return pack_f32x2(f.x, f.y);
}

template <typename E>
__device__ __forceinline__ void widen8(const uint4& v, uint64_t (&y)[4]) {
  y[0] = widen2<E>(v.x);
  y[1] = widen2<E>(v.y);
  y[2] = widen2<E>(v.z);
  y[3] = widen2<E>(v.w);
}

// Largest magnitudes of two words of 16-bit values, half by half (NaN if any
// is; magnitudes of 16-bit values need no widening to be compared).
template <typename E>
__device__ __forceinline__ uint32_t max_abs2(uint32_t m, uint32_t w);
template <>
__device__ __forceinline__ uint32_t max_abs2<__half>(uint32_t m, uint32_t w) {
  const __half2 r = __hmax2_nan(*reinterpret_cast<const __half2*>(&m),
                                __habs2(*reinterpret_cast<const __half2*>(&w)));
  return *reinterpret_cast<const uint32_t*>(&r);
}
template <>
__device__ __forceinline__ uint32_t max_abs2<__nv_bfloat16>(uint32_t m, uint32_t w) {
  const __nv_bfloat162 r = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&m),
                                       __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w)));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// The factors that turn the values of one block into codes.  With
// a = max(amax, 2^-110), the code of y is the e4m3 value nearest to
// y * (448 / a).  448 / a is held as hi + lo (lo the remainder of the
// division), so that y * hi + y * lo has one rounding of relative size 2^-24
// and a quotient that lies exactly between two codes stays there.  Among
// normal weights 0.07% (fp16) and 0.65% (bf16) of the values are such ties,
// and a single rounded factor would send a ninth of them, 0.0075% and 0.074% of
// all codes, to the other neighbour.
// An all-zero block has scale 0 and codes 0; one that holds Inf or NaN has
// scale Inf or NaN and NaN codes.
struct BlockScale {
  uint64_t hi, lo;  // twice each
  float scale;
};
__device__ __forceinline__ BlockScale block_scale(float amax) {
  BlockScale r;
  if (amax == 0.0f) {
    r.hi = r.lo = 0ull;
    r.scale = 0.0f;
    return r;
  }
  // 1 / a from the hardware's approximation and a Newton step; each quotient
  // is then corrected by its exact remainder (Markstein's method)
  const float a = max_nan(amax, kAmaxFloor);
  float rcp;
  asm("rcp.approx.f32 %0, %1;" : "=f"(rcp) : "f"(a));
  rcp = __fmaf_rn(__fmaf_rn(-a, rcp, 1.0f), rcp, rcp);
  const float hi = kE4m3Max * rcp;
  const float lo = __fmaf_rn(-hi, a, kE4m3Max) * rcp;
  r.hi = pack_f32x2(hi, hi);
  r.lo = pack_f32x2(lo, lo);
  constexpr float kInv = 1.0f / kE4m3Max;
  const float s = a * kInv;
  r.scale = __fmaf_rn(__fmaf_rn(-kE4m3Max, s, a), kInv, s);
  return r;
}

// Two codes, the first in the low byte (rounded to nearest even; finite
// values never pass 448, NaN stays NaN).
__device__ __forceinline__ uint32_t e4m3x2(uint64_t v) {
  const float2 f = unpack_f32x2(v);
  uint16_t c;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(f.y), "f"(f.x));
  return c;
}
// Eight codes of four pairs.
__device__ __forceinline__ uint2 encode8(const uint64_t* y, const BlockScale& s) {
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = e4m3x2(fma_f32x2(y[i], s.hi, mul_f32x2(y[i], s.lo)));
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// Four pairs to eight 16-bit values.
template <typename E>
__device__ __forceinline__ uint4 narrow8(const uint64_t* y) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack_f32x2(y[i]);
    w[i] = pack2<E>(f.x, f.y);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Largest magnitude of N pairs and m (NaN if any is).
template <int N>
__device__ __forceinline__ float amax_pairs(const uint64_t (&y)[N], float m) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float2 f = unpack_f32x2(y[i]);
    m = max_nan_abs(m, f.x, f.y);
  }
  return m;
}

// Calls f with a value of the C++ type that `dtype` names.
template <typename F>
auto with_dtype(int dtype, F&& f) {
  return dtype == ZQ_F16 ? f(__half{}) : f(__nv_bfloat16{});
}

}  // namespace zq
