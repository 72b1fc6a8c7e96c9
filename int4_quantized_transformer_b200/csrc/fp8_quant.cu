// fp8_quant.cu -- e4m3 block quantization: activation rows with one fp32
// scale for each 128 consecutive values of a row (as they are, after a
// bias-add and GeLU, or after a LayerNorm in the same pass), and weights with
// one scale for each 128 x 128 block.
//
// All three read their fp16 or bf16 input once into registers, reduce the
// block maxima there, and write one byte per value and four per block, so
// HBM traffic (3 bytes per value) is what bounds them.
#include <algorithm>

#include "zq_fp8.cuh"
#include "zq_internal.h"
#include "zq_math.cuh"
#include "zq_ptx.cuh"

namespace zq {
namespace {

constexpr int kVec = 8;                           // values per 16-byte load
constexpr int kVecsPerBlock = kFp8Block / kVec;   // 16: a half warp holds one block

// Maximum over the 16 lanes of a half warp (NaN if any lane has it).
__device__ __forceinline__ float half_warp_max(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// ------------------------------------------------- rows without a LayerNorm

// One half warp per block of 128 values, UNROLL blocks with their loads in
// flight before the first is reduced.  Blocks are numbered row by row, so
// neighbouring half warps read neighbouring 256-byte pieces.  The last block
// of a row is short when K is no multiple of 128: its missing lanes hold 0.
template <typename E, int ACT, int UNROLL>
__global__ void __launch_bounds__(256)
    fp8_rows_kernel(const E* __restrict__ X, const E* __restrict__ bias, int K, unsigned kblocks,
                    unsigned long long items, uint8_t* __restrict__ Xq, float* __restrict__ s_blk,
                    E* __restrict__ Y) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & (kVecsPerBlock - 1);
  const unsigned long long first =
      blockIdx.x * 16ull * UNROLL + threadIdx.x / kVecsPerBlock;  // 16 half warps per CTA
  uint4 v[UNROLL];
  size_t at[UNROLL];
  int col[UNROLL];
#pragma unroll
  for (int u = 0; u < UNROLL; ++u) {
    const unsigned long long item = first + 16ull * u;
    unsigned long long row;
    unsigned blk;
    if (items <= 0xFFFFFFFFull) {  // 32-bit division whenever the numbers allow it
      const unsigned r = static_cast<unsigned>(item) / kblocks;
      row = r;
      blk = static_cast<unsigned>(item) - r * kblocks;
    } else {
      row = item / kblocks;
      blk = static_cast<unsigned>(item - row * kblocks);
    }
    col[u] = static_cast<int>(blk) * kFp8Block + lane * kVec;
    if (item >= items || col[u] >= K) col[u] = -1;
    at[u] = static_cast<size_t>(row) * K + (col[u] < 0 ? 0 : col[u]);
    v[u] = col[u] < 0 ? make_uint4(0, 0, 0, 0)
                      : __ldcs(reinterpret_cast<const uint4*>(X + at[u]));
  }
#pragma unroll
  for (int u = 0; u < UNROLL; ++u) {
    const unsigned long long item = first + 16ull * u;
    float y[8];
    unpack8<E>(v[u], y);
    if (bias && col[u] >= 0) {
      float b[8];
      unpack8<E>(__ldg(reinterpret_cast<const uint4*>(bias + col[u])), b);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = __fadd_rn(y[i], b[i]);
    }
    if (ACT == ZQ_ACT_GELU) {
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = gelu_erf(y[i]);
    }
    const BlockScale s = block_scale(half_warp_max(amax8(y)));
    if (item < items && lane == 0) s_blk[item] = s.scale;
    if (col[u] >= 0) {
      *reinterpret_cast<uint2*>(Xq + at[u]) = encode8(y, s);
      if (Y) *reinterpret_cast<uint4*>(Y + at[u]) = pack8<E>(y);
    }
  }
}

template <typename E, int ACT>
cudaError_t launch_rows(const void* X, const void* bias, int T, int K, void* Xq, float* s_blk,
                        void* Y, cudaStream_t st) {
  const unsigned kblocks = (K + kFp8Block - 1) / kFp8Block;
  const unsigned long long items = static_cast<unsigned long long>(T) * kblocks;
  auto go = [&](auto* kernel, int unroll) {
    const unsigned long long per_cta = 16ull * unroll;
    return launch_pdl(kernel, dim3(static_cast<unsigned>((items + per_cta - 1) / per_cta)),
                      dim3(256), 0, st, static_cast<const E*>(X), static_cast<const E*>(bias), K,
                      kblocks, items, static_cast<uint8_t*>(Xq), s_blk, static_cast<E*>(Y));
  };
  // one block per half warp while that leaves SMs without work
  if (items <= 16ull * 4 * 4 * num_sms()) return go(fp8_rows_kernel<E, ACT, 1>, 1);
  return go(fp8_rows_kernel<E, ACT, 4>, 4);
}

// ------------------------------------------------------ rows after a LayerNorm

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum over the W warps of a row; every thread gets it.  `red` is used once
// per barrier interval.
template <int W>
__device__ __forceinline__ float row_sum(float v, float* red) {
  v = warp_sum(v);
  if (W == 1) return v;
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.0f;
#pragma unroll
  for (int w = 0; w < W; ++w) s += red[w];
  return s;
}

// W warps per row (one row at a time per CTA; with W = 1 a CTA of four warps
// has four rows), VPT 16-byte vectors per thread: the row is read once, its
// mean and then its centred sum of squares are taken over the registers in
// fp32, and each half warp quantizes the blocks that it holds.  The CTAs stay
// for many rows: gamma and beta are kept in registers, and the next row's
// loads are issued before the current one is reduced.
template <typename E, int W, int VPT>
__global__ void __launch_bounds__(W == 1 ? 128 : 32 * W)
    fp8_ln_kernel(const E* __restrict__ X, const E* __restrict__ gamma, const E* __restrict__ beta,
                  int T, int K, float eps, uint8_t* __restrict__ Xq, float* __restrict__ s_blk,
                  E* __restrict__ Y) {
  constexpr int ROWS = W == 1 ? 4 : 1;
  constexpr int RT = 32 * W;  // threads of a row
  __shared__ float red[2][2][W];
  grid_dependency_wait();
  grid_launch_dependents();
  const int tid = W == 1 ? (threadIdx.x & 31) : threadIdx.x;
  const int kvecs = K / kVec, kblocks = (K + kFp8Block - 1) / kFp8Block;
  const float inv_k = __fdiv_rn(1.0f, static_cast<float>(K));
  uint4 g[VPT], b[VPT], x[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = i * RT + tid;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    g[i] = v < kvecs ? __ldg(reinterpret_cast<const uint4*>(gamma) + v) : zero;
    b[i] = v < kvecs && beta ? __ldg(reinterpret_cast<const uint4*>(beta) + v) : zero;
    x[i] = zero;
  }
  const int stride = gridDim.x * ROWS;
  int row = blockIdx.x * ROWS + (W == 1 ? threadIdx.x >> 5 : 0);
  auto fetch = [&](int r) {
    if (r >= T) return;
    const uint4* src = reinterpret_cast<const uint4*>(X + static_cast<size_t>(r) * K);
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      if (i * RT + tid < kvecs) x[i] = __ldcs(src + i * RT + tid);
  };
  fetch(row);
  for (int turn = 0; row < T; turn ^= 1) {
    float y[VPT][8];
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      unpack8<E>(x[i], y[i]);
      sum += ((y[i][0] + y[i][1]) + (y[i][2] + y[i][3])) +
             ((y[i][4] + y[i][5]) + (y[i][6] + y[i][7]));
    }
    const int next = static_cast<int>(min(static_cast<long long>(row) + stride, 0x7fffffffll));
    fetch(next);
    const float mean = row_sum<W>(sum, red[turn][0]) * inv_k;
    float sq = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      if (i * RT + tid < kvecs) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          y[i][e] -= mean;
          sq = fmaf(y[i][e], y[i][e], sq);
        }
      }
    }
    const float var = row_sum<W>(sq, red[turn][1]) * inv_k;
    const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(var + eps));
    uint8_t* qrow = Xq + static_cast<size_t>(row) * K;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = i * RT + tid;
      float gf[8], bf[8];
      unpack8<E>(g[i], gf);
      unpack8<E>(b[i], bf);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[i][e] = fmaf(y[i][e] * rstd, gf[e], bf[e]);  // 0 past K
      const BlockScale s = block_scale(half_warp_max(amax8(y[i])));
      if (v < kvecs) {
        reinterpret_cast<uint2*>(qrow)[v] = encode8(y[i], s);
        if (Y) reinterpret_cast<uint4*>(Y + static_cast<size_t>(row) * K)[v] = pack8<E>(y[i]);
        if ((v & (kVecsPerBlock - 1)) == 0)
          s_blk[static_cast<size_t>(row) * kblocks + v / kVecsPerBlock] = s.scale;
      }
    }
    row = next;
  }
}

template <typename E, int W, int VPT>
cudaError_t launch_ln_one(const void* X, const void* gamma, const void* beta, int T, int K,
                          float eps, void* Xq, float* s_blk, void* Y, cudaStream_t st) {
  constexpr int ROWS = W == 1 ? 4 : 1;
  constexpr int THREADS = W == 1 ? 128 : 32 * W;
  const int ctas = (T - 1) / ROWS + 1;
  const int resident = num_sms() * std::max(1, 1024 / THREADS);
  return launch_pdl(fp8_ln_kernel<E, W, VPT>, dim3(std::min(ctas, resident)), dim3(THREADS), 0, st,
                    static_cast<const E*>(X), static_cast<const E*>(gamma),
                    static_cast<const E*>(beta), T, K, eps, static_cast<uint8_t*>(Xq), s_blk,
                    static_cast<E*>(Y));
}

template <typename E, int W>
cudaError_t launch_ln_w(int vpt, const void* X, const void* gamma, const void* beta, int T, int K,
                        float eps, void* Xq, float* s_blk, void* Y, cudaStream_t st) {
  switch (vpt) {
    case 1: return launch_ln_one<E, W, 1>(X, gamma, beta, T, K, eps, Xq, s_blk, Y, st);
    case 2: return launch_ln_one<E, W, 2>(X, gamma, beta, T, K, eps, Xq, s_blk, Y, st);
    case 3: return launch_ln_one<E, W, 3>(X, gamma, beta, T, K, eps, Xq, s_blk, Y, st);
    default: return launch_ln_one<E, W, 4>(X, gamma, beta, T, K, eps, Xq, s_blk, Y, st);
  }
}

template <typename E>
cudaError_t launch_ln(const void* X, const void* gamma, const void* beta, int T, int K, float eps,
                      void* Xq, float* s_blk, void* Y, cudaStream_t st) {
  const int warps1 = (K / kVec + 31) / 32;  // warps of a row with one vector per thread
  int W = 1;
  while (W * 4 < warps1) W *= 2;
  const int vpt = (warps1 + W - 1) / W;
  switch (W) {
    case 1: return launch_ln_w<E, 1>(vpt, X, gamma, beta, T, K, eps, Xq, s_blk, Y, st);
    case 2: return launch_ln_w<E, 2>(vpt, X, gamma, beta, T, K, eps, Xq, s_blk, Y, st);
    case 4: return launch_ln_w<E, 4>(vpt, X, gamma, beta, T, K, eps, Xq, s_blk, Y, st);
    case 8: return launch_ln_w<E, 8>(vpt, X, gamma, beta, T, K, eps, Xq, s_blk, Y, st);
    case 16: return launch_ln_w<E, 16>(vpt, X, gamma, beta, T, K, eps, Xq, s_blk, Y, st);
    default: return launch_ln_w<E, 32>(vpt, X, gamma, beta, T, K, eps, Xq, s_blk, Y, st);
  }
}

// -------------------------------------------------------------------- weights

// One CTA per 128 x 128 block, held in registers (eight 16-byte vectors per
// thread, all loads in flight at once) between the maximum and the codes.
template <typename E>
__global__ void __launch_bounds__(256)
    fp8_weights_kernel(const E* __restrict__ W, int N, int K, unsigned kblocks,
                       uint8_t* __restrict__ Wq, float* __restrict__ s_blk) {
  __shared__ float red[8];
  grid_dependency_wait();
  grid_launch_dependents();
  const unsigned nb = blockIdx.x / kblocks, kb = blockIdx.x - nb * kblocks;
  const int col = static_cast<int>(kb) * kFp8Block + (threadIdx.x & 15) * kVec;
  const int row0 = static_cast<int>(nb) * kFp8Block + (threadIdx.x >> 4);
  uint4 v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = row0 + 16 * i;
    v[i] = (r < N && col < K)
               ? __ldcs(reinterpret_cast<const uint4*>(W + static_cast<size_t>(r) * K + col))
               : make_uint4(0, 0, 0, 0);
  }
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float y[8];
    unpack8<E>(v[i], y);
    m = max_nan(m, amax8(y));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) m = max_nan(m, red[w]);
  const BlockScale s = block_scale(m);
  if (threadIdx.x == 0) s_blk[blockIdx.x] = s.scale;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = row0 + 16 * i;
    if (r < N && col < K) {
      float y[8];
      unpack8<E>(v[i], y);
      *reinterpret_cast<uint2*>(Wq + static_cast<size_t>(r) * K + col) = encode8(y, s);
    }
  }
}

bool known_dtype(int dtype) { return dtype == ZQ_F16 || dtype == ZQ_BF16; }

zq_status check_rows(const void* X, int dtype, const void* a, const void* b, int T, int K,
                     const void* Xq, const float* s_blk, const void* Y) {
  if (!known_dtype(dtype)) return ZQ_ERR_UNSUPPORTED;
  if (T < 0 || K < 16 || K > 32768 || K % 16 != 0) return ZQ_ERR_SHAPE;
  if (T == 0) return ZQ_OK;
  if (!X || !Xq || !s_blk) return ZQ_ERR_NULL;
  if (!aligned16(X) || !aligned16(Xq) || (a && !aligned16(a)) || (b && !aligned16(b)) ||
      (Y && !aligned16(Y)) || reinterpret_cast<uintptr_t>(s_blk) % 4 != 0)
    return ZQ_ERR_ALIGN;
  return ZQ_OK;
}

}  // namespace
}  // namespace zq

using namespace zq;

extern "C" zq_status zq_bias_act_quant_fp8(const void* X, int dtype, const void* bias, int T, int K,
                                           int act, void* Xq, float* s_blk, void* Y_act,
                                           zq_stream_t stream) {
  if (act != ZQ_ACT_NONE && act != ZQ_ACT_GELU) return ZQ_ERR_UNSUPPORTED;
  const zq_status rc = check_rows(X, dtype, bias, nullptr, T, K, Xq, s_blk, Y_act);
  if (rc != ZQ_OK || T == 0) return rc;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = with_dtype(dtype, [&](auto tag) {
    using E = decltype(tag);
    return act == ZQ_ACT_GELU
               ? launch_rows<E, ZQ_ACT_GELU>(X, bias, T, K, Xq, s_blk, Y_act, st)
               : launch_rows<E, ZQ_ACT_NONE>(X, bias, T, K, Xq, s_blk, Y_act, st);
  });
  return e == cudaSuccess ? ZQ_OK : ZQ_ERR_CUDA;
}

extern "C" zq_status zq_ln_quant_fp8(const void* X, int dtype, const void* gamma, const void* beta,
                                     int T, int K, float eps, void* Xq, float* s_blk, void* Y_ln,
                                     zq_stream_t stream) {
  if (!gamma)  // quant-only, as zq_ln_quant
    return zq_bias_act_quant_fp8(X, dtype, nullptr, T, K, ZQ_ACT_NONE, Xq, s_blk, Y_ln, stream);
  const zq_status rc = check_rows(X, dtype, gamma, beta, T, K, Xq, s_blk, Y_ln);
  if (rc != ZQ_OK || T == 0) return rc;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = with_dtype(dtype, [&](auto tag) {
    return launch_ln<decltype(tag)>(X, gamma, beta, T, K, eps, Xq, s_blk, Y_ln, st);
  });
  return e == cudaSuccess ? ZQ_OK : ZQ_ERR_CUDA;
}

extern "C" zq_status zq_quantize_weights_fp8(const void* W, int dtype, int N, int K, void* Wq,
                                             float* s_blk, zq_stream_t stream) {
  if (!known_dtype(dtype)) return ZQ_ERR_UNSUPPORTED;
  if (N < 1 || K < 16 || K % 16 != 0) return ZQ_ERR_SHAPE;
  const long long kblocks = (static_cast<long long>(K) + kFp8Block - 1) / kFp8Block;
  const long long blocks = (static_cast<long long>(N) + kFp8Block - 1) / kFp8Block * kblocks;
  if (blocks > 0x7fffffffll) return ZQ_ERR_SHAPE;
  if (!W || !Wq || !s_blk) return ZQ_ERR_NULL;
  if (!aligned16(W) || !aligned16(Wq) || reinterpret_cast<uintptr_t>(s_blk) % 4 != 0)
    return ZQ_ERR_ALIGN;
  const cudaError_t e = with_dtype(dtype, [&](auto tag) {
    using E = decltype(tag);
    return launch_pdl(fp8_weights_kernel<E>, dim3(static_cast<unsigned>(blocks)), dim3(256), 0,
                      reinterpret_cast<cudaStream_t>(stream), static_cast<const E*>(W), N, K,
                      static_cast<unsigned>(kblocks), static_cast<uint8_t*>(Wq), s_blk);
  });
  return e == cudaSuccess ? ZQ_OK : ZQ_ERR_CUDA;
}
