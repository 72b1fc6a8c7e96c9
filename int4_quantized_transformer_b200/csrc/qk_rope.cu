// qk_rope.cu -- norm of each query and key head and its rotation by the
// token's position, in one pass over the heads (a QKV projection's output in
// place, or into tensors of its own), and the rotation's frequencies.
//
// For a head x of D values, x' = norm(x) * weight + bias (RMS or LayerNorm
// over the D values, or x itself), and each pair (a, b) of the first R
// values, whose frequency is f, becomes
//     (a cos t - b sin t, b cos t + a sin t) * scale,   t = position * f.
// The pass reads and writes each value once: HBM traffic bounds it at many
// tokens, launch latency at a few.
#include <math.h>

#include <algorithm>

#include "zq_fp8.cuh"
#include "zq_internal.h"
#include "zq_ptx.cuh"

namespace zq {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxHeadDim = 256;

struct Heads {  // one of queries, keys
  const void* in;
  void* out;
  const void* weight;
  const void* bias;
  long long in_token, in_head, out_token, out_head;  // strides in elements
  int n;
};

struct RopeParams {
  Heads q, k;
  const int32_t* positions;
  const float* inv_freq;
  int T, D, R, norm;
  int units;      // pairs of vectors that make up a head
  int chunks;     // CTAs per token
  int per_chunk;  // heads of a CTA
  int copy_rest;  // values behind R are written too (other output, or a norm)
  float scale, eps;
};

template <int BYTES>
struct VecOf;
template <>
struct VecOf<16> {
  using type = uint4;
};
template <>
struct VecOf<8> {
  using type = uint2;
};
template <>
struct VecOf<4> {
  using type = uint32_t;
};

template <typename E, int VEC>
__device__ __forceinline__ void load_vec(const E* p, float (&f)[VEC]) {
  union {
    typename VecOf<2 * VEC>::type v;
    uint32_t w[VEC / 2];
  } u;
  u.v = *reinterpret_cast<const decltype(u.v)*>(p);
#pragma unroll
  for (int i = 0; i < VEC / 2; ++i) {
    const float2 t = unpack2<E>(u.w[i]);
    f[2 * i] = t.x;
    f[2 * i + 1] = t.y;
  }
}
template <typename E, int VEC>
__device__ __forceinline__ void store_vec(E* p, const float (&f)[VEC]) {
  union {
    typename VecOf<2 * VEC>::type v;
    uint32_t w[VEC / 2];
  } u;
#pragma unroll
  for (int i = 0; i < VEC / 2; ++i) u.w[i] = pack2<E>(f[2 * i], f[2 * i + 1]);
  *reinterpret_cast<decltype(u.v)*>(p) = u.v;
}

// A head is cut into units of two vectors of VEC values, so that a lane has
// both values of every pair it rotates.  Halves layout: unit u < R / 2 / VEC
// holds values u VEC.. and R / 2 + u VEC..; neighbours layout: 2 u VEC.. and
// the vector after it.  Units behind the rotated ones hold two neighbouring
// vectors.  A group of 2^k lanes has a head, NU units to a lane.
template <typename E, int VEC, int NU, bool HALF, bool NORM>
__global__ void __launch_bounds__(kThreads) qk_rope_kernel(const RopeParams p, int lanes) {
  __shared__ float cs[kMaxHeadDim / 2], sn[kMaxHeadDim / 2];
  grid_dependency_wait();
  grid_launch_dependents();
  const unsigned token = blockIdx.x / p.chunks;
  const int chunk = static_cast<int>(blockIdx.x - token * p.chunks);
  const int pos = __ldg(p.positions + token);
  if (pos < 0) return;  // a row behind the last sequence: left as it is
  // The angle in turns, reduced to half a turn on either side in 64 bits (the
  // product of a position and an fp32 frequency is exact there), so that far
  // positions lose nothing before the fp32 sine and cosine.
  for (int i = threadIdx.x; i < p.R / 2; i += kThreads) {
    const double turns = static_cast<double>(pos) * static_cast<double>(__ldg(p.inv_freq + i)) *
                         0.15915494309189533577;  // 1 / (2 pi)
    float s, c;
    sincospif(static_cast<float>(2.0 * (turns - rint(turns))), &s, &c);
    cs[i] = c * p.scale;
    sn[i] = s * p.scale;
  }
  __syncthreads();
  const int lane = threadIdx.x & (lanes - 1);
  const int groups = kThreads / lanes;
  const int half = p.R / 2;
  const int rot_units = HALF ? half / VEC : (p.R / VEC + 1) / 2;
  const int h1 = min(p.q.n + p.k.n, (chunk + 1) * p.per_chunk);
  // all lanes of a warp make the same number of turns: the group reductions need them
  for (int h0 = chunk * p.per_chunk; h0 < h1; h0 += groups) {
    const int h = h0 + static_cast<int>(threadIdx.x) / lanes;
    const bool live = h < h1;
    const bool is_k = h >= p.q.n;
    const Heads& hd = is_k ? p.k : p.q;
    const int hh = live ? (is_k ? h - p.q.n : h) : 0;
    const E* src = static_cast<const E*>(hd.in) + token * hd.in_token + hh * hd.in_head;
    E* dst = static_cast<E*>(hd.out) + token * hd.out_token + hh * hd.out_head;
    float a[NU][VEC], b[NU][VEC];
    int oa[NU], ob[NU];  // value offsets of the unit's vectors, -1 = none
#pragma unroll
    for (int n = 0; n < NU; ++n) {
      const int u = lane + n * lanes;
      oa[n] = ob[n] = -1;
      if (live && u < p.units) {
        if (HALF && u < rot_units) {
          oa[n] = u * VEC;
          ob[n] = half + u * VEC;
        } else {
          oa[n] = HALF ? p.R + 2 * (u - rot_units) * VEC : 2 * u * VEC;
          ob[n] = oa[n] + VEC;
          if (!p.copy_rest && oa[n] >= p.R) oa[n] = -1;  // nothing to change there
          if (ob[n] >= p.D || (!p.copy_rest && ob[n] >= p.R)) ob[n] = -1;
        }
      }
#pragma unroll
      for (int i = 0; i < VEC; ++i) a[n][i] = b[n][i] = 0.0f;
      if (oa[n] >= 0) load_vec<E, VEC>(src + oa[n], a[n]);
      if (ob[n] >= 0) load_vec<E, VEC>(src + ob[n], b[n]);
    }
    if (NORM) {
      auto group_sum = [&](float v) {
        for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        return v;
      };
      const float inv_d = __fdiv_rn(1.0f, static_cast<float>(p.D));
      if (p.norm == ZQ_NORM_LAYER) {
        float s = 0.0f;
#pragma unroll
        for (int n = 0; n < NU; ++n)
#pragma unroll
          for (int i = 0; i < VEC; ++i) s += a[n][i] + b[n][i];
        const float mean = group_sum(s) * inv_d;
#pragma unroll
        for (int n = 0; n < NU; ++n)
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            if (oa[n] >= 0) a[n][i] -= mean;
            if (ob[n] >= 0) b[n][i] -= mean;
          }
      }
      float q = 0.0f;
#pragma unroll
      for (int n = 0; n < NU; ++n)
#pragma unroll
        for (int i = 0; i < VEC; ++i) q = fmaf(a[n][i], a[n][i], fmaf(b[n][i], b[n][i], q));
      const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(fmaf(group_sum(q), inv_d, p.eps)));
      const E* w = static_cast<const E*>(hd.weight);
      const E* bs = static_cast<const E*>(hd.bias);
      auto affine = [&](float (&v)[VEC], int off) {
        if (off < 0) return;
        float wv[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) wv[i] = 1.0f;
        if (w) load_vec<E, VEC>(w + off, wv);
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = v[i] * rstd * wv[i];
        if (bs) {
          load_vec<E, VEC>(bs + off, wv);
#pragma unroll
          for (int i = 0; i < VEC; ++i) v[i] += wv[i];
        }
      };
#pragma unroll
      for (int n = 0; n < NU; ++n) {
        affine(a[n], oa[n]);
        affine(b[n], ob[n]);
      }
    }
#pragma unroll
    for (int n = 0; n < NU; ++n) {
      if (HALF) {
        if (oa[n] >= 0 && oa[n] < half) {
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            const float c = cs[oa[n] + i], s = sn[oa[n] + i], t = a[n][i];
            a[n][i] = t * c - b[n][i] * s;
            b[n][i] = b[n][i] * c + t * s;
          }
        }
      } else {
        auto turn = [&](float (&v)[VEC], int off) {
          if (off < 0 || off >= p.R) return;
#pragma unroll
          for (int i = 0; i < VEC; i += 2) {
            const float c = cs[(off + i) / 2], s = sn[(off + i) / 2], t = v[i];
            v[i] = t * c - v[i + 1] * s;
            v[i + 1] = v[i + 1] * c + t * s;
          }
        };
        turn(a[n], oa[n]);
        turn(b[n], ob[n]);
      }
      if (oa[n] >= 0) store_vec<E, VEC>(dst + oa[n], a[n]);
      if (ob[n] >= 0) store_vec<E, VEC>(dst + ob[n], b[n]);
    }
  }
}

// The widest vector that cuts both the rotated values (each half of them, in
// the halves layout) and the rest into whole vectors.
int vector_width(int layout, int D, int R) {
  const int part = layout == ZQ_ROPE_HALF ? R / 2 : R;
  for (int v = 8; v > 2; v /= 2)
    if (part % v == 0 && (D - R) % v == 0) return v;
  return 2;
}

template <typename E, bool HALF, bool NORM>
cudaError_t launch_rope(const RopeParams& p0, int vec, cudaStream_t st) {
  RopeParams p = p0;
  p.units = (p.D / vec + 1) / 2;
  int lanes = 1;
  while (lanes < p.units && lanes < 32) lanes *= 2;
  const int heads = p.q.n + p.k.n, groups = kThreads / lanes;
  // With enough tokens one CTA has all heads of a token (the sines are then
  // computed once per token); with fewer, the heads are spread over CTAs
  // until the SMs are busy.
  const int turns = (heads + groups - 1) / groups;
  int chunks = 1;
  while (chunks < turns && static_cast<long long>(p.T) * chunks < 4ll * num_sms()) chunks *= 2;
  p.per_chunk = (turns + chunks - 1) / chunks * groups;
  p.chunks = (heads + p.per_chunk - 1) / p.per_chunk;
  const long long ctas = static_cast<long long>(p.T) * p.chunks;
  if (ctas > 0x7fffffffll) return cudaErrorInvalidValue;
  auto go = [&](auto* kernel) {
    return launch_pdl(kernel, dim3(static_cast<unsigned>(ctas)), dim3(kThreads), 0, st, p, lanes);
  };
  switch (vec) {
    case 8: return go(qk_rope_kernel<E, 8, 1, HALF, NORM>);
    case 4: return go(qk_rope_kernel<E, 4, 1, HALF, NORM>);
    default: return go(qk_rope_kernel<E, 2, 2, HALF, NORM>);
  }
}

// The checks of one of the two head sets; *out is only filled when it is fine.
zq_status check_heads(const zq_heads* h, int T, int D, Heads* out) {
  if (h->heads < 0 || h->heads > (1 << 20)) return ZQ_ERR_SHAPE;
  if (h->heads == 0 || T == 0) {
    *out = Heads{};
    return ZQ_OK;
  }
  if (!h->in || !h->out) return ZQ_ERR_NULL;
  const long long strides[4] = {h->in_token_stride, h->in_head_stride, h->out_token_stride,
                                h->out_head_stride};
  for (long long s : strides)
    if (s < 0 || s % 8 != 0) return ZQ_ERR_ALIGN;
  // written heads must not overlap: all heads of a token before the next
  // token, or all tokens of a head before the next head
  const __int128 hs = h->out_head_stride, ts = h->out_token_stride;
  const bool head_ok = h->heads == 1 || hs >= D, token_ok = T == 1 || ts >= D;
  if (!head_ok || !token_ok ||
      (h->heads > 1 && T > 1 && ts < (h->heads - 1) * hs + D && hs < (T - 1) * ts + D))
    return ZQ_ERR_SHAPE;
  if (!aligned16(h->in) || !aligned16(h->out) || (h->weight && !aligned16(h->weight)) ||
      (h->bias && !aligned16(h->bias)))
    return ZQ_ERR_ALIGN;
  // in place means the same layout on both sides
  if (h->in == h->out && ((h->heads > 1 && h->in_head_stride != h->out_head_stride) ||
                          (T > 1 && h->in_token_stride != h->out_token_stride)))
    return ZQ_ERR_SHAPE;
  *out = Heads{h->in, h->out, h->weight, h->bias, h->in_token_stride, h->in_head_stride,
               h->out_token_stride, h->out_head_stride, h->heads};
  return ZQ_OK;
}

}  // namespace
}  // namespace zq

using namespace zq;

extern "C" zq_status zq_qk_norm_rope(const zq_heads* q, const zq_heads* k, int dtype, int T, int D,
                                     int norm, float eps, const int32_t* positions,
                                     const float* inv_freq, int R, int layout, float scale,
                                     zq_stream_t stream) {
  if (dtype != ZQ_F16 && dtype != ZQ_BF16) return ZQ_ERR_UNSUPPORTED;
  if (norm != ZQ_NORM_NONE && norm != ZQ_NORM_RMS && norm != ZQ_NORM_LAYER)
    return ZQ_ERR_UNSUPPORTED;
  if (layout != ZQ_ROPE_HALF && layout != ZQ_ROPE_INTERLEAVED) return ZQ_ERR_UNSUPPORTED;
  if (T < 0 || D < 8 || D > kMaxHeadDim || D % 8 != 0 || R < 0 || R > D || R % 2 != 0)
    return ZQ_ERR_SHAPE;
  if (layout == ZQ_ROPE_HALF && R % 4 != 0) return ZQ_ERR_SHAPE;
  if (!q) return ZQ_ERR_NULL;
  RopeParams p{};
  zq_status rc = check_heads(q, T, D, &p.q);
  if (rc == ZQ_OK && k) rc = check_heads(k, T, D, &p.k);
  if (rc != ZQ_OK || T == 0 || p.q.n + p.k.n == 0) return rc;
  if (!positions || (R > 0 && !inv_freq)) return ZQ_ERR_NULL;
  if (reinterpret_cast<uintptr_t>(positions) % 4 || reinterpret_cast<uintptr_t>(inv_freq) % 4)
    return ZQ_ERR_ALIGN;
  p.positions = positions;
  p.inv_freq = inv_freq;
  p.T = T;
  p.D = D;
  p.R = R;
  p.norm = norm;
  p.scale = scale;
  p.eps = eps;
  // in place and without a norm, the values behind R stay as they are
  p.copy_rest = norm != ZQ_NORM_NONE || (p.q.n && p.q.in != p.q.out) || (p.k.n && p.k.in != p.k.out);
  if (!p.copy_rest && R == 0) return ZQ_OK;
  const int vec = vector_width(layout, D, R);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = with_dtype(dtype, [&](auto tag) {
    using E = decltype(tag);
    if (layout == ZQ_ROPE_HALF)
      return norm == ZQ_NORM_NONE ? launch_rope<E, true, false>(p, vec, st)
                                  : launch_rope<E, true, true>(p, vec, st);
    return norm == ZQ_NORM_NONE ? launch_rope<E, false, false>(p, vec, st)
                                : launch_rope<E, false, true>(p, vec, st);
  });
  return e == cudaSuccess ? ZQ_OK : ZQ_ERR_CUDA;
}

extern "C" zq_status zq_rope_frequencies(int R, double base, int scaling, double factor,
                                         double low, double high, int trained_len, float* inv_freq,
                                         float* scale) {
  if (R < 2 || R > kMaxHeadDim || R % 2 != 0) return ZQ_ERR_SHAPE;
  if (scaling < ZQ_ROPE_PLAIN || scaling > ZQ_ROPE_YARN) return ZQ_ERR_UNSUPPORTED;
  if (!inv_freq || !scale) return ZQ_ERR_NULL;
  if (!(base > 1.0) || !isfinite(base)) return ZQ_ERR_SHAPE;
  if (scaling != ZQ_ROPE_PLAIN && (!(factor >= 1.0) || !isfinite(factor))) return ZQ_ERR_SHAPE;
  const bool ranged = scaling == ZQ_ROPE_BANDS || scaling == ZQ_ROPE_YARN;
  // low < high turns over the trained length
  if (ranged && (trained_len < 1 || !(low > 0.0) || !(high > low) || !isfinite(high)))
    return ZQ_ERR_SHAPE;
  if (scaling == ZQ_ROPE_NTK && R == 2) return ZQ_ERR_SHAPE;  // R / (R - 2)
  const double two_pi = 6.283185307179586476925;
  *scale = 1.0f;
  if (scaling == ZQ_ROPE_NTK) base *= pow(factor, static_cast<double>(R) / (R - 2));
  // YaRN: the ramp runs over the dimension index at which a frequency makes
  // `high` (keep) and `low` (divide) turns over the trained length
  auto index_of = [&](double turns) {
    return R * log(trained_len / (turns * two_pi)) / (2.0 * log(base));
  };
  double first = 0.0, last = 0.0;
  if (scaling == ZQ_ROPE_YARN) {
    first = std::max(floor(index_of(high)), 0.0);
    last = std::min(ceil(index_of(low)), R - 1.0);
    *scale = static_cast<float>(factor <= 1.0 ? 1.0 : 0.1 * log(factor) + 1.0);
  }
  for (int i = 0; i < R / 2; ++i) {
    const double f = pow(base, -2.0 * i / R);
    double g = f;
    if (scaling == ZQ_ROPE_LINEAR) {
      g = f / factor;
    } else if (scaling == ZQ_ROPE_BANDS) {
      const double turns = trained_len * f / two_pi;
      const double keep = std::min(std::max((turns - low) / (high - low), 0.0), 1.0);
      g = keep * f + (1.0 - keep) * f / factor;
    } else if (scaling == ZQ_ROPE_YARN) {
      const double ramp =
          std::min(std::max((i - first) / std::max(last - first, 0.001), 0.0), 1.0);
      g = f * (1.0 - ramp) + f / factor * ramp;
    }
    inv_freq[i] = static_cast<float>(g);
  }
  return ZQ_OK;
}
