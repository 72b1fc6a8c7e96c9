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

// The factors that turn the values of one block into codes.  With
// a = max(amax, 2^-110), the code of y is the e4m3 value nearest to
// y * (448 / a).  448 / a is held as hi + lo (lo the remainder of the
// division), so that y * hi + y * lo has one rounding of relative size 2^-24
// and a quotient that lies exactly between two codes stays there: with fp16
// and bf16 inputs such ties are common, and a single rounded factor would
// send about 1% of the codes of a weight matrix to the other neighbour.
// An all-zero block has scale 0 and codes 0; one that holds Inf or NaN has
// scale Inf or NaN and NaN codes.
struct BlockScale {
  float hi, lo, scale;
};
__device__ __forceinline__ BlockScale block_scale(float amax) {
  BlockScale r;
  if (amax == 0.0f) {
    r.hi = r.lo = r.scale = 0.0f;
    return r;
  }
  const float a = max_nan(amax, kAmaxFloor);
  r.hi = __fdiv_rn(kE4m3Max, a);
  r.lo = __fmaf_rn(-r.hi, a, kE4m3Max) * (r.hi * (1.0f / kE4m3Max));
  r.scale = __fdiv_rn(a, kE4m3Max);
  return r;
}

// Four codes in one word, the first in the lowest byte (rounded to nearest
// even; finite values never pass 448, NaN stays NaN).
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}
__device__ __forceinline__ uint2 encode8(const float (&y)[8], const BlockScale& s) {
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __fmaf_rn(y[i], s.hi, __fmul_rn(y[i], s.lo));
  return make_uint2(e4m3x4(v[0], v[1], v[2], v[3]), e4m3x4(v[4], v[5], v[6], v[7]));
}

// Largest magnitude of eight values (NaN if any is).
__device__ __forceinline__ float amax8(const float (&y)[8]) {
  float m = fabsf(y[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) m = max_nan(m, fabsf(y[i]));
  return m;
}

// Calls f with a value of the C++ type that `dtype` names.
template <typename F>
auto with_dtype(int dtype, F&& f) {
  return dtype == ZQ_F16 ? f(__half{}) : f(__nv_bfloat16{});
}

}  // namespace zq
