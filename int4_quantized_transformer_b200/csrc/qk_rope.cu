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
#include <type_traits>

#include "zq_fp8.cuh"
#include "zq_internal.h"
#include "zq_ptx.cuh"

namespace zq {
namespace {

constexpr int kThreads = 256;  // of a CTA without a norm
constexpr int kNormWarps = 12;  // most of a CTA with one
constexpr int kSmNormWarps = 24;  // of an SM: 80 registers per thread
constexpr int kMaxHeadDim = 256;
constexpr int kMaxTokens = 16;    // of a CTA
constexpr int kMaxAngles = 1024;  // sines (and cosines) of a CTA, padded

struct Heads {  // one of queries, keys
  const void* in;
  void* out;
  const void* weight;
  const void* bias;
  long long in_token, in_head, out_token, out_head;  // strides in elements
  int n;
};

struct RopeParams {
  Heads set[2];  // queries, keys
  const int32_t* positions;
  const float* inv_freq;
  int T, D, R, norm;
  int tokens;     // per CTA
  int columns;    // CTAs per token tile
  int copy_rest;  // values behind R are written too (other output, or a norm)
  float scale, eps;
};

// Both values of a rotated pair have to meet in one thread.  Halves layout: a
// unit is VEC values u VEC.. and the VEC values R / 2 behind them, VEC the
// widest vector that divides R / 2.  Neighbours: a unit is eight values.
enum Cut { kHalf8, kHalf4, kHalf2, kNeighbours };
template <int CUT>
struct CutOf {
  static constexpr bool HALF = CUT != kNeighbours;
  static constexpr int VEC = CUT == kHalf4 ? 4 : (CUT == kHalf2 ? 2 : 8);
  static constexpr int ANGLES = HALF ? VEC : 4;       // of a unit
  static constexpr int TAIL = CUT == kHalf2 ? 4 : 8;  // widest aligned vector of the rest
  __host__ __device__ static int rotated_units(int R) { return HALF ? R / 2 / VEC : (R + 7) / 8; }
  // first value that no unit has
  __host__ __device__ static int rest(int R) { return HALF ? R : (R + 7) / 8 * 8; }
  __host__ __device__ static int tail_units(int D, int R) { return (D - rest(R)) / TAIL; }
};

// Vectors of 2, 4 or 8 16-bit values in up to four words.
template <int N>
__device__ __forceinline__ void load_words(const void* p, uint32_t* w) {
  if constexpr (N == 8) {
    const uint4 v = *static_cast<const uint4*>(p);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  } else if constexpr (N == 4) {
    const uint2 v = *static_cast<const uint2*>(p);
    w[0] = v.x, w[1] = v.y;
  } else {
    w[0] = *static_cast<const uint32_t*>(p);
  }
}
template <int N>
__device__ __forceinline__ void store_words(void* p, const uint32_t* w) {
  if constexpr (N == 8)
    *static_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  else if constexpr (N == 4)
    *static_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  else
    *static_cast<uint32_t*>(p) = w[0];
}
template <typename E, int N>
__device__ __forceinline__ void widen(const uint32_t* w, float* f) {
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    const float2 t = unpack2<E>(w[i]);
    f[2 * i] = t.x;
    f[2 * i + 1] = t.y;
  }
}
template <typename E, int N>
__device__ __forceinline__ void narrow(const float* f, uint32_t* w) {
#pragma unroll
  for (int i = 0; i < N / 2; ++i) w[i] = pack2<E>(f[2 * i], f[2 * i + 1]);
}
// N floats of shared memory, aligned to their size (16 bytes at most).
template <int N>
__device__ __forceinline__ void load_floats(const float* p, float* f) {
  if constexpr (N >= 4) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 v = *reinterpret_cast<const float4*>(p + i);
      f[i] = v.x, f[i + 1] = v.y, f[i + 2] = v.z, f[i + 3] = v.w;
    }
  } else {
    const float2 v = *reinterpret_cast<const float2*>(p);
    f[0] = v.x, f[1] = v.y;
  }
}
// Rotates the pairs (x[i], y[i]), or the first `pairs` of four neighbours in x
// (the ones behind belong to values that do not rotate; a rotation by nothing
// would not leave them alone: 0 times an infinity next door is NaN).
template <int N>
__device__ __forceinline__ void rotate_halves(float* x, float* y, const float* c, const float* s) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float v = x[i];
    x[i] = v * c[i] - y[i] * s[i];
    y[i] = y[i] * c[i] + v * s[i];
  }
}
__device__ __forceinline__ void rotate_neighbours(float* x, const float* c, const float* s,
                                                  int pairs) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = x[2 * i], b = x[2 * i + 1];
    x[2 * i] = i < pairs ? a * c[i] - b * s[i] : a;
    x[2 * i + 1] = i < pairs ? b * c[i] + a * s[i] : b;
  }
}

// A CTA has a tile of tokens and one column of threads over the heads: a
// thread keeps its place in its head and goes through the tile's tokens, so
// that its addresses move by one addition.  The tile's sines and cosines are
// computed first, with all threads.
struct Tile {
  int column, tokens, row;  // row: angles of a token, padded to vectors of four
  long long token0;
};
__device__ __forceinline__ Tile tile_of(const RopeParams& p) {
  const unsigned tile = blockIdx.x / p.columns;
  Tile t;
  t.column = static_cast<int>(blockIdx.x - tile * p.columns);
  t.token0 = static_cast<long long>(tile) * p.tokens;
  t.tokens = static_cast<int>(min(static_cast<long long>(p.tokens), p.T - t.token0));
  t.row = (p.R / 2 + 3) & ~3;
  return t;
}
__device__ __forceinline__ void tile_angles(const RopeParams& p, const Tile& t, float* cs, float* sn,
                                            int* pos) {
  const int half = p.R / 2;
  // The angle in turns, reduced to half a turn on either side in 64 bits, before
  // the fp32 sine and cosine.  The product of position and frequency (exact for
  // positions up to 2^29), 1 / (2 pi) and their product are off by at most 2.8 *
  // 2^-53 of the angle: below half a step of fp32 up to 2^27 radians, 2^-20.5
  // radians at 2^31.
  for (int i = threadIdx.x; i < t.tokens * t.row; i += blockDim.x) {
    const int k = i / t.row, f = i - k * t.row;
    float s = 0.0f, c = 1.0f;
    if (f < half) {
      const double turns = static_cast<double>(__ldg(p.positions + t.token0 + k)) *
                           static_cast<double>(__ldg(p.inv_freq + f)) *
                           0.15915494309189533577;  // 1 / (2 pi)
      sincospif(static_cast<float>(2.0 * (turns - rint(turns))), &s, &c);
      s *= p.scale;
      c *= p.scale;
    }
    cs[i] = c;
    sn[i] = s;
  }
  if (threadIdx.x < t.tokens) pos[threadIdx.x] = __ldg(p.positions + t.token0 + threadIdx.x);
  __syncthreads();
}

// Without a norm; bound by HBM: 4096 tokens of 2 x 64 heads of 96, 24 rotated,
// to another output in 37.6 us (5.4 TB/s, 0.82 of a copy).  (Loads that bypass
// L1 took 8 us longer.)  Threads of rotated units come first, then (to another
// output) threads that copy the rest; each has the loads of AHEAD tokens in
// flight, the first ones during the sines: without that 8192 tokens of 40 heads
// of 128 took 32.6 us, not 27.3, 1000 of 72 heads 13.5, not 10.3.  Four tokens
// pay only where a unit is two values wide: 8192 tokens of 2 x 16 heads of 80
// in 17.9 us, with two 21.2; 1000 tokens of 72 heads of 128 in 12.3.  A token whose position is negative is passed over.
template <typename E, int CUT>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeParams p) {
  using C = CutOf<CUT>;
  constexpr int VEC = C::VEC, TAIL = C::TAIL, ANG = C::ANGLES, AHEAD = CUT == kHalf2 ? 4 : 2;
  __shared__ __align__(16) float cs[kMaxAngles], sn[kMaxAngles];
  __shared__ int pos[kMaxTokens];
  grid_dependency_wait();
  grid_launch_dependents();
  const Tile tl = tile_of(p);
  const int heads = p.set[0].n + p.set[1].n, half = p.R / 2;
  const int ru = C::rotated_units(p.R), tu = p.copy_rest ? C::tail_units(p.D, p.R) : 0;
  int c = tl.column * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x);
  const bool rotates = c < heads * ru;
  if (!rotates) c -= heads * ru;
  const int per_head = rotates ? ru : tu;
  const bool live = per_head > 0 && c < heads * per_head;
  int head = live ? c / per_head : 0;
  const int u = live ? c - head * per_head : 0;
  const int which = head >= p.set[0].n;
  if (which) head -= p.set[0].n;
  const Heads& hd = p.set[which];
  const int at = rotates ? u * VEC : C::rest(p.R) + u * TAIL;
  const E* in = static_cast<const E*>(hd.in) + tl.token0 * hd.in_token + head * hd.in_head + at;
  E* out = static_cast<E*>(hd.out) + tl.token0 * hd.out_token + head * hd.out_head + at;
  const long long di = hd.in_token, od = hd.out_token;
  uint32_t a[AHEAD][4], b[AHEAD][4];
  auto fetch = [&](int t0, auto rotated) {
#pragma unroll
    for (int k = 0; k < AHEAD; ++k)
      if (t0 + k < tl.tokens) {
        load_words<decltype(rotated)::value ? VEC : TAIL>(in + k * di, a[k]);
        if constexpr (decltype(rotated)::value && C::HALF)
          load_words<VEC>(in + k * di + half, b[k]);
      }
    in += AHEAD * di;
  };
  // the first loads are on their way during the sines
  if (live && rotates) fetch(0, std::true_type{});
  if (live && !rotates) fetch(0, std::false_type{});
  tile_angles(p, tl, cs, sn, pos);
  if (!live) return;
  if (rotates) {
    for (int t0 = 0; t0 < tl.tokens; t0 += AHEAD) {
      if (t0) fetch(t0, std::true_type{});
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
        if (t0 + k < tl.tokens && pos[t0 + k] >= 0) {
          float x[VEC], co[ANG], si[ANG];
          load_floats<ANG>(cs + (t0 + k) * tl.row + u * ANG, co);
          load_floats<ANG>(sn + (t0 + k) * tl.row + u * ANG, si);
          widen<E, VEC>(a[k], x);
          if constexpr (C::HALF) {
            float y[VEC];
            widen<E, VEC>(b[k], y);
            rotate_halves<VEC>(x, y, co, si);
            narrow<E, VEC>(y, b[k]);
            store_words<VEC>(out + half, b[k]);
            narrow<E, VEC>(x, a[k]);
          } else {  // a pair is a word: the ones behind R stay as they came
            const int pairs = half - ANG * u;
            rotate_neighbours(x, co, si, pairs);
            uint32_t turned[VEC / 2];
            narrow<E, VEC>(x, turned);
#pragma unroll
            for (int i = 0; i < VEC / 2; ++i)
              if (i < pairs) a[k][i] = turned[i];
          }
          store_words<VEC>(out, a[k]);
        }
        out += od;
      }
    }
  } else {
    for (int t0 = 0; t0 < tl.tokens; t0 += AHEAD) {
      if (t0) fetch(t0, std::false_type{});
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
        if (t0 + k < tl.tokens && pos[t0 + k] >= 0) store_words<TAIL>(out, a[k]);
        out += od;
      }
    }
  }
}

// With a norm; bound by the latency of a token's one chain from the load to the
// store (16 instructions per value, two reductions with a LayerNorm) at 24 warps
// per SM, whose issue slots are 62% taken: 3.7 to 4.9 TB/s at many tokens.  (On pairs
// of fp32 it was slower: 17.6 us instead of 15.1 for 2048 tokens of 32 heads of
// 256.)  2^k lanes have a head, NU units to a lane.  Units behind the
// rotated ones have 2 TAIL neighbouring values of the rest (in the neighbours
// layout all units are two vectors of eight neighbouring values), so that
// every lane has two vectors a and b.
template <int CUT>
struct NormCut {
  using C = CutOf<CUT>;
  static constexpr int VEC = C::VEC, TAIL = VEC == 8 ? 8 : 4, WIDE = TAIL > VEC ? TAIL : VEC;
  static constexpr int NU = CUT == kHalf2 ? 2 : 1;
  __host__ __device__ static int rotated(int R) { return C::HALF ? R / 2 / VEC : 0; }
  __host__ __device__ static int units(int D, int R) {
    return rotated(R) + ((C::HALF ? D - R : D) + 2 * TAIL - 1) / (2 * TAIL);
  }
};

template <typename E, int CUT>
__global__ void __launch_bounds__(32 * kNormWarps, kSmNormWarps / kNormWarps)
    norm_rope_kernel(const RopeParams p, int lanes) {
  using C = NormCut<CUT>;
  constexpr bool HALF = CutOf<CUT>::HALF;
  constexpr int NU = C::NU, VEC = C::VEC, TAIL = C::TAIL, WIDE = C::WIDE;
  __shared__ __align__(16) float cs[kMaxAngles], sn[kMaxAngles];
  __shared__ int pos[kMaxTokens];
  grid_dependency_wait();
  grid_launch_dependents();
  const Tile tl = tile_of(p);
  const int lane = threadIdx.x & (lanes - 1);
  int head = (tl.column * blockDim.x + static_cast<int>(threadIdx.x)) / lanes;
  // lanes past the last head go along for the group sums, with nothing to read
  const bool live = head < p.set[0].n + p.set[1].n;
  const int which = live && head >= p.set[0].n;
  if (which) head -= p.set[0].n;
  if (!live) head = 0;
  const Heads& hd = p.set[which];
  // value offsets of this lane's vectors (-1 = none), and whether they rotate
  int oa[NU], ob[NU];
  bool rot[NU];
#pragma unroll
  for (int n = 0; n < NU; ++n) {
    const int u = lane + n * lanes, ru = C::rotated(p.R);
    rot[n] = HALF && u < ru;
    oa[n] = rot[n] ? u * VEC : (HALF ? p.R : 0) + 2 * (u - ru) * TAIL;
    ob[n] = rot[n] ? p.R / 2 + u * VEC : oa[n] + TAIL;
    if (!live || oa[n] >= p.D) oa[n] = -1;
    if (!live || ob[n] >= p.D) ob[n] = -1;
  }
  auto load = [&](const E* src, int n, uint32_t* a, uint32_t* b) {
    if (VEC != TAIL && rot[n]) {
      if (oa[n] >= 0) load_words<VEC>(src + oa[n], a);
      if (ob[n] >= 0) load_words<VEC>(src + ob[n], b);
    } else {
      if (oa[n] >= 0) load_words<TAIL>(src + oa[n], a);
      if (ob[n] >= 0) load_words<TAIL>(src + ob[n], b);
    }
  };
  // the norm's weight and bias at this lane's values, for all tokens
  constexpr uint32_t kOnes = std::is_same<E, __half>::value ? 0x3C003C00u : 0x3F803F80u;
  uint32_t wa[NU][WIDE / 2], wb[NU][WIDE / 2], ba[NU][WIDE / 2], bb[NU][WIDE / 2];
#pragma unroll
  for (int n = 0; n < NU; ++n) {
#pragma unroll
    for (int i = 0; i < WIDE / 2; ++i) wa[n][i] = wb[n][i] = kOnes, ba[n][i] = bb[n][i] = 0;
    if (hd.weight) load(static_cast<const E*>(hd.weight), n, wa[n], wb[n]);
    if (hd.bias) load(static_cast<const E*>(hd.bias), n, ba[n], bb[n]);
  }
  const E* in = static_cast<const E*>(hd.in) + tl.token0 * hd.in_token + head * hd.in_head;
  E* out = static_cast<E*>(hd.out) + tl.token0 * hd.out_token + head * hd.out_head;
  const float inv_d = __fdiv_rn(1.0f, static_cast<float>(p.D));
  auto group_sum = [&](float v) {
    for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  };
  uint32_t ra[NU][WIDE / 2], rb[NU][WIDE / 2];
  auto fetch = [&] {
#pragma unroll
    for (int n = 0; n < NU; ++n) {
#pragma unroll
      for (int i = 0; i < WIDE / 2; ++i) ra[n][i] = rb[n][i] = 0;
      load(in, n, ra[n], rb[n]);
    }
    in += hd.in_token;
  };
  fetch();  // on its way during the sines
  tile_angles(p, tl, cs, sn, pos);
  for (int t = 0; t < tl.tokens; ++t) {
    float a[NU][WIDE], b[NU][WIDE];
#pragma unroll
    for (int n = 0; n < NU; ++n) {
      widen<E, WIDE>(ra[n], a[n]);
      widen<E, WIDE>(rb[n], b[n]);
    }
    if (t + 1 < tl.tokens) fetch();  // the next token's, ahead of this one's sums
    // (vectors that are not there, and the unused end of a short one, are 0)
    if (p.norm == ZQ_NORM_LAYER) {
      float sum = 0.0f;
#pragma unroll
      for (int n = 0; n < NU; ++n)
#pragma unroll
        for (int i = 0; i < WIDE; ++i) sum += a[n][i] + b[n][i];
      const float mean = group_sum(sum) * inv_d;
#pragma unroll
      for (int n = 0; n < NU; ++n) {
        const float ma = oa[n] >= 0 ? mean : 0.0f, mb = ob[n] >= 0 ? mean : 0.0f;
#pragma unroll
        for (int i = 0; i < WIDE; ++i) {
          const bool there = VEC == WIDE || i < VEC || !rot[n];
          a[n][i] -= there ? ma : 0.0f;
          b[n][i] -= there ? mb : 0.0f;
        }
      }
    }
    float q = 0.0f;
#pragma unroll
    for (int n = 0; n < NU; ++n)
#pragma unroll
      for (int i = 0; i < WIDE; ++i) q = fmaf(a[n][i], a[n][i], fmaf(b[n][i], b[n][i], q));
    const float rstd = rsqrtf(fmaf(group_sum(q), inv_d, p.eps));  // within two units of 2^-24
    if (live && pos[t] >= 0) {
      const float* ct = cs + t * tl.row;
      const float* st = sn + t * tl.row;
#pragma unroll
      for (int n = 0; n < NU; ++n) {
        float wf[WIDE], bf[WIDE];
        widen<E, WIDE>(wa[n], wf);
        widen<E, WIDE>(ba[n], bf);
#pragma unroll
        for (int i = 0; i < WIDE; ++i) a[n][i] = fmaf(a[n][i] * rstd, wf[i], bf[i]);
        widen<E, WIDE>(wb[n], wf);
        widen<E, WIDE>(bb[n], bf);
#pragma unroll
        for (int i = 0; i < WIDE; ++i) b[n][i] = fmaf(b[n][i] * rstd, wf[i], bf[i]);
        if constexpr (HALF) {
          if (rot[n]) {
            float co[VEC], si[VEC];
            load_floats<VEC>(ct + oa[n], co);
            load_floats<VEC>(st + oa[n], si);
            rotate_halves<VEC>(a[n], b[n], co, si);
          }
        } else {
          float co[4], si[4];
          if (oa[n] >= 0 && oa[n] < p.R) {
            load_floats<4>(ct + oa[n] / 2, co);
            load_floats<4>(st + oa[n] / 2, si);
            rotate_neighbours(a[n], co, si, (p.R - oa[n]) / 2);
          }
          if (ob[n] >= 0 && ob[n] < p.R) {
            load_floats<4>(ct + ob[n] / 2, co);
            load_floats<4>(st + ob[n] / 2, si);
            rotate_neighbours(b[n], co, si, (p.R - ob[n]) / 2);
          }
        }
        uint32_t va[WIDE / 2], vb[WIDE / 2];
        narrow<E, WIDE>(a[n], va);
        narrow<E, WIDE>(b[n], vb);
        if (VEC != TAIL && rot[n]) {
          store_words<VEC>(out + oa[n], va);
          store_words<VEC>(out + ob[n], vb);
        } else {
          if (oa[n] >= 0) store_words<TAIL>(out + oa[n], va);
          if (ob[n] >= 0) store_words<TAIL>(out + ob[n], vb);
        }
      }
    }
    out += hd.out_token;
  }
}

// Warps of a CTA with a norm, for heads that take `total` warps per token.
// Each column of CTAs computes the tokens' sines again, which costs a thread
// about as much per angle as 1/58 of a token; and columns that leave warps
// idle, or do not fill an SM's 24, cost in proportion.  Measured against 64
// threads for all: 2011 tokens of 40 heads of 128 (10 warps) in 11.1 us (13.0),
// 16384 of them in 68.5 (78.9), 8192 tokens of 20 heads of 256 in 35.4 (38.7).
// For 4096 tokens of 128 heads of 96, LayerNorm (32 warps; takes 8) 61.2 us,
// 11 warps 73, 2 warps 63.
long long norm_warps(long long T, long long total, int row) {
  if (T * total <= 4ll * num_sms()) return std::min(2ll, total);  // a few tokens: over the SMs
  int best = 1;
  double best_rate = 0.0;
  for (int w = 1; w <= kNormWarps; ++w) {
    const long long columns = (total + w - 1) / w;
    const double useful = static_cast<double>(total) / (columns * w) * (kSmNormWarps / w * w);
    const double rate = useful / (1.0 + row * (1.0 / 58) / w);
    if (rate >= best_rate) best = w, best_rate = rate;
  }
  return best;
}

template <typename E, int CUT, bool NORM>
cudaError_t launch_cut(const RopeParams& p0, cudaStream_t st) {
  using C = CutOf<CUT>;
  RopeParams p = p0;
  const long long heads = static_cast<long long>(p.set[0].n) + p.set[1].n;
  int lanes = 1;
  while (lanes < NormCut<CUT>::units(p.D, p.R) && lanes < 32) lanes *= 2;
  const long long threads =
      NORM ? heads * lanes
           : heads * (C::rotated_units(p.R) + (p.copy_rest ? C::tail_units(p.D, p.R) : 0));
  // tokens of a CTA at most: their sines have to fit
  const int row = std::max(4, (p.R / 2 + 3) & ~3), most = std::min(kMaxTokens, kMaxAngles / row);
  const long long warps = (threads + 31) / 32, rest_columns = (warps * 32 + kThreads - 1) / kThreads;
  const int cta = static_cast<int>(
      32 * (NORM ? norm_warps(p.T, warps, row) : (warps + rest_columns - 1) / rest_columns));
  const long long columns = (threads + cta - 1) / cta;
  if (NORM) {
    // whole waves of CTAs, the tokens spread over them evenly
    const long long tiles =
        std::max(1ll, static_cast<long long>(kSmNormWarps * 32 / cta) * num_sms() / columns);
    const long long waves = (p.T - 1) / (tiles * most) + 1;
    p.tokens = static_cast<int>((p.T - 1) / (waves * tiles) + 1);
  } else {
    // As many tokens as leave 20 CTAs of 256 threads for each SM, and two (the
    // loads in flight) from half of that; in CTAs that fit the heads (4096
    // tokens of 24 heads of 64, 96 threads each: 7.5 us, in CTAs of 256 15.1).
    // 10, 14 and 26 for the 20 made up to 10% of difference either way from 1000
    // to 16384 tokens; whole waves as above took up to 13% longer; 512 tokens of
    // 128 heads of 96 took 9.8 us one at a time and 7.3 by twos.
    const long long work = p.T * columns * cta / (static_cast<long long>(kThreads) * num_sms());
    p.tokens = static_cast<int>(std::min<long long>(std::max(work / 20, work < 20 ? 1ll : 2ll), most));
  }
  const long long ctas = (static_cast<long long>(p.T) + p.tokens - 1) / p.tokens * columns;
  if (ctas > 0x7fffffffll) return cudaErrorInvalidValue;
  p.columns = static_cast<int>(columns);
  const dim3 grid(static_cast<unsigned>(ctas));
  if (NORM) return launch_pdl(norm_rope_kernel<E, CUT>, grid, dim3(cta), 0, st, p, lanes);
  return launch_pdl(rope_kernel<E, CUT>, grid, dim3(cta), 0, st, p);
}

template <typename E, bool NORM>
cudaError_t launch_rope(const RopeParams& p, int layout, cudaStream_t st) {
  if (layout == ZQ_ROPE_INTERLEAVED) return launch_cut<E, kNeighbours, NORM>(p, st);
  if (p.R / 2 % 8 == 0) return launch_cut<E, kHalf8, NORM>(p, st);
  if (p.R / 2 % 4 == 0) return launch_cut<E, kHalf4, NORM>(p, st);
  return launch_cut<E, kHalf2, NORM>(p, st);
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
  zq_status rc = check_heads(q, T, D, &p.set[0]);
  if (rc == ZQ_OK && k) rc = check_heads(k, T, D, &p.set[1]);
  if (rc != ZQ_OK || T == 0 || p.set[0].n + p.set[1].n == 0) return rc;
  // what one set writes is not the other's to read or write
  if (p.set[0].n && p.set[1].n &&
      (p.set[0].out == p.set[1].out || p.set[0].out == p.set[1].in ||
       p.set[1].out == p.set[0].in))
    return ZQ_ERR_SHAPE;
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
  p.copy_rest = norm != ZQ_NORM_NONE;
  for (const Heads& h : p.set)
    if (h.n && h.in != h.out) p.copy_rest = 1;
  if (!p.copy_rest && R == 0) return ZQ_OK;  // nothing changes
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = with_dtype(dtype, [&](auto tag) {
    using E = decltype(tag);
    return norm == ZQ_NORM_NONE ? launch_rope<E, false>(p, layout, st)
                                : launch_rope<E, true>(p, layout, st);
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
