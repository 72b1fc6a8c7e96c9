// fp8_quant.cu -- e4m3 block quantization: activation rows with one fp32
// scale for each 128 consecutive values of a row (as they are, after a
// bias-add and GeLU, or after a LayerNorm in the same pass), and weights with
// one scale for each 128 x 128 block.
//
// All three read their fp16 or bf16 input once into registers, reduce the
// block maxima there, and write one byte per value and four per block: HBM
// traffic (3 bytes per value) bounds the weights and the rows as they are,
// instructions the LayerNorm and the GeLU.
#include <algorithm>

#include "zq_fp8.cuh"
#include "zq_internal.h"
#include "zq_math.cuh"
#include "zq_ptx.cuh"

namespace zq {
namespace {

// Four lanes hold a block of 128 values: 16-byte vectors l, l + 4, l + 8 and
// l + 12 of the block in lane l (64 consecutive bytes per load of the four).
// With 32 values per lane the block's maximum costs two shuffles, and its two
// divisions are spread over 32 values; with one vector per lane they were
// half of all instructions (20.4 us for 4096 x 6144 instead of the copy's 12).
constexpr int kLanes = 4;
constexpr int kVecs = kFp8Block / 8 / kLanes;  // vectors per lane
constexpr int kWarpBlocks = 32 / kLanes;       // blocks per warp

__device__ __forceinline__ float quad_max(float v) {
  v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, 1));
  return max_nan(v, __shfl_xor_sync(0xffffffffu, v, 2));
}

// Quantizes a lane's part of a block.  `col` is the block's first column, q
// and y16 (may be null) its first value's place in the outputs.
template <typename E, bool FULL = false>
__device__ __forceinline__ void finish_block(const uint64_t (&y)[4 * kVecs], int lane, int col,
                                             int K, uint8_t* q, E* y16, float* s_out) {
  const BlockScale s = block_scale(quad_max(amax_pairs(y, 0.0f)));
  if (lane == 0 && (FULL || col < K)) *s_out = s.scale;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int at = 8 * (lane + kLanes * i);
    if (FULL || col + at < K) {
      *reinterpret_cast<uint2*>(q + at) = encode8(y + 4 * i, s);
      if (y16) *reinterpret_cast<uint4*>(y16 + at) = narrow8<E>(y + 4 * i);
    }
  }
}

// ------------------------------------------------- rows without a LayerNorm

constexpr int kRowsCtas = 4;  // CTAs per SM: 64 registers per thread

// Blocks are numbered row by row, so neighbouring lanes read neighbouring
// pieces.  The last block of a row is short when K is no multiple of 128: its
// missing lanes hold 0.  As they are, 4096 x 6144 take 13.9 us (5.4 TB/s, 0.83 of
// a copy); with a GeLU 1531 x 16384 take 24.5, bound by 23 instructions per
// value (issue slots 73% taken, the special-function unit half).
template <typename E, int ACT>
__global__ void __launch_bounds__(256, kRowsCtas)
    fp8_rows_kernel(const E* __restrict__ X, const E* __restrict__ bias, int K, unsigned kblocks,
                    unsigned long long items, uint8_t* __restrict__ Xq, float* __restrict__ s_blk,
                    E* __restrict__ Y) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & (kLanes - 1);
  const unsigned long long item =
      static_cast<unsigned long long>(blockIdx.x) * (blockDim.x / kLanes) + threadIdx.x / kLanes;
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
  // lanes past the last block take part in the shuffles with nothing to read
  const int col = item < items ? static_cast<int>(blk) * kFp8Block : K;
  const size_t at = static_cast<size_t>(row) * K + col;
  uint4 v[kVecs], b[kVecs];
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int o = 8 * (lane + kLanes * i);
    v[i] = b[i] = make_uint4(0, 0, 0, 0);
    if (col + o < K) {
      v[i] = __ldcs(reinterpret_cast<const uint4*>(X + at + o));
      if (bias) b[i] = __ldg(reinterpret_cast<const uint4*>(bias + col + o));
    }
  }
  uint64_t y[4 * kVecs];
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w}, c[4] = {b[i].x, b[i].y, b[i].z, b[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint64_t p = widen2<E>(w[j]);
      if (bias) p = add_f32x2(p, widen2<E>(c[j]));
      if (ACT == ZQ_ACT_GELU) {
        const float2 f = unpack_f32x2(p), e = gelu_pair(f.x, f.y);
        p = pack_f32x2(e.x, e.y);
      }
      y[4 * i + j] = p;
    }
  }
  finish_block<E>(y, lane, col, K, Xq + at, Y ? Y + at : nullptr, s_blk + item);
}

template <typename E, int ACT>
cudaError_t launch_rows(const void* X, const void* bias, int T, int K, void* Xq, float* s_blk,
                        void* Y, cudaStream_t st) {
  const unsigned kblocks = (K + kFp8Block - 1) / kFp8Block;
  const unsigned long long items = static_cast<unsigned long long>(T) * kblocks;
  // small CTAs while there are too few blocks to give every SM a large one
  const unsigned threads = items * kLanes <= 256ull * num_sms() ? 64 : 256;
  const unsigned long long per_cta = threads / kLanes;
  const unsigned long long ctas = (items + per_cta - 1) / per_cta;
  if (ctas > 0x7fffffffull) return cudaErrorInvalidValue;
  return launch_pdl(fp8_rows_kernel<E, ACT>, dim3(static_cast<unsigned>(ctas)), dim3(threads), 0,
                    st, static_cast<const E*>(X), static_cast<const E*>(bias), K, kblocks, items,
                    static_cast<uint8_t*>(Xq), s_blk, static_cast<E*>(Y));
}

// ------------------------------------------------------ rows after a LayerNorm

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum over the `warps` warps of a row (the CTA); every thread gets it.  `red`
// is written once between two uses of the other buffers; n is the power of two
// from `warps` up.
__device__ __forceinline__ float row_sum(float v, float* red, int warps, int n) {
  v = warp_sum(v);
  if (warps == 1) return v;
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  const int at = threadIdx.x & (n - 1);
  v = at < warps ? red[at] : 0.0f;
  for (int o = n >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// 1 / sqrt(v) for v >= 0: the library's, corrected by a Newton step unless it
// is 0 or infinite.
__device__ __forceinline__ float inv_sqrt(float v) {
  const float r = rsqrtf(v);
  const float c = __fmaf_rn(0.5f * r, __fmaf_rn(-v * r, r, 1.0f), r);
  return r > 0.0f && r < INFINITY ? c : r;
}

// A warp has 1024 consecutive values of a row, 32 per lane; the row is read
// once, its mean and then its centred sum of squares are taken over the
// registers in fp32.  Rows of up to 1024 values: one per warp (ROWS = 4 to a
// CTA), longer ones: one per CTA of at most THREADS.  The CTAs stay for many
// rows; with AHEAD the next row's loads are issued before the current row is
// reduced, for which 80 registers have to be left to a thread.  FULL: no lane
// of the CTA is past the row's end.  gamma and beta come from L1.
// 4096 x 6144 in 19.6 us, 3.9 TB/s, bound by the latency of a row's two sums
// and its block maxima at 24 warps per SM (issue slots 60% taken).  Without
// AHEAD, at 32 warps, 20.5; the next row copied into shared memory instead of
// registers 25.1; gamma and beta widened in shared memory 22.6; two rows at a
// time 20.2; one barrier per row instead of two, by joining the warps' means
// and squares, 19.9.
template <typename E, int ROWS, int THREADS, int REGS, bool AHEAD, bool FULL>
__global__ void __launch_bounds__(THREADS, 65536 / (REGS * THREADS))
    fp8_ln_kernel(const E* __restrict__ X, const E* __restrict__ gamma, const E* __restrict__ beta,
                  int T, int K, float eps, uint8_t* __restrict__ Xq, float* __restrict__ s_blk,
                  E* __restrict__ Y) {
  __shared__ float red[2][2][32];
  const int warps = ROWS > 1 ? 1 : blockDim.x / 32;
  const int tid = ROWS > 1 ? (threadIdx.x & 31) : threadIdx.x;
  int n = 1;  // the power of two from `warps` up
  while (n < warps) n *= 2;
  const int lane = tid & (kLanes - 1), blk = tid / kLanes, col = blk * kFp8Block;
  const int kblocks = (K + kFp8Block - 1) / kFp8Block;
  const float inv_k = __fdiv_rn(1.0f, static_cast<float>(K));
  const uint4 zero = make_uint4(0, 0, 0, 0);
  auto offset = [&](int i) { return col + 8 * (lane + kLanes * i); };
  auto in = [&](int i) { return FULL || offset(i) < K; };
  const long long stride = static_cast<long long>(gridDim.x) * ROWS;
  long long row = static_cast<long long>(blockIdx.x) * ROWS + (ROWS > 1 ? threadIdx.x / 32 : 0);
  uint4 x[kVecs];
  auto fetch = [&](long long r) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
      x[i] = r < T && in(i) ? __ldcs(reinterpret_cast<const uint4*>(X + r * K + offset(i))) : zero;
  };
  grid_dependency_wait();
  grid_launch_dependents();
  if (AHEAD) fetch(row);
  for (int turn = 0; row < T; row += stride, turn ^= 1) {
    if (!AHEAD) fetch(row);
    uint64_t y[4 * kVecs];
    uint64_t sum2 = 0ull;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        y[4 * i + j] = widen2<E>(w[j]);
        sum2 = add_f32x2(sum2, y[4 * i + j]);
      }
    }
    if (AHEAD) fetch(row + stride);
    const float2 s2 = unpack_f32x2(sum2);
    const float mean = row_sum(s2.x + s2.y, red[turn][0], warps, n) * inv_k;
    const uint64_t minus = pack_f32x2(-mean, -mean);
    uint64_t sq2 = 0ull;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      if (in(i)) {
#pragma unroll
        for (int j = 4 * i; j < 4 * i + 4; ++j) {
          y[j] = add_f32x2(y[j], minus);
          sq2 = fma_f32x2(y[j], y[j], sq2);
        }
      }
    }
    const float2 q2 = unpack_f32x2(sq2);
    const float rstd = inv_sqrt(row_sum(q2.x + q2.y, red[turn][1], warps, n) * inv_k + eps);
    const uint64_t rstd2 = pack_f32x2(rstd, rstd);
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      uint4 gv = zero, bv = zero;  // 0 past K
      if (in(i)) {
        gv = __ldg(reinterpret_cast<const uint4*>(gamma + offset(i)));
        if (beta) bv = __ldg(reinterpret_cast<const uint4*>(beta + offset(i)));
      }
      uint64_t g[4], b[4];
      widen8<E>(gv, g);
      widen8<E>(bv, b);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        y[4 * i + j] = fma_f32x2(mul_f32x2(y[4 * i + j], rstd2), g[j], b[j]);
    }
    const size_t at = static_cast<size_t>(row) * K + col;
    finish_block<E, FULL>(y, lane, col, K, Xq + at, Y ? Y + at : nullptr,
                          s_blk + static_cast<size_t>(row) * kblocks + blk);
  }
}

template <typename E, int ROWS, int THREADS>
cudaError_t launch_ln_one(int threads, const void* X, const void* gamma, const void* beta, int T,
                          int K, float eps, void* Xq, float* s_blk, void* Y, cudaStream_t st) {
  constexpr bool kAhead = THREADS <= 768;
  constexpr int kRegs = kAhead ? 80 : 64;
  // CTAs of an SM: 6 warps of 80 registers, or 8 of 64, fit each of its four schedulers
  const int ctas = (T - 1) / ROWS + 1, per_sm = (kAhead ? 24 : 32) * 32 / threads;
  auto go = [&](auto* kernel) {
    return launch_pdl(kernel, dim3(std::min(ctas, num_sms() * per_sm)), dim3(threads), 0, st,
                      static_cast<const E*>(X), static_cast<const E*>(gamma),
                      static_cast<const E*>(beta), T, K, eps, static_cast<uint8_t*>(Xq), s_blk,
                      static_cast<E*>(Y));
  };
  return K % 1024 == 0 ? go(fp8_ln_kernel<E, ROWS, THREADS, kRegs, kAhead, true>)
                       : go(fp8_ln_kernel<E, ROWS, THREADS, kRegs, kAhead, false>);
}

template <typename E>
cudaError_t launch_ln(const void* X, const void* gamma, const void* beta, int T, int K, float eps,
                      void* Xq, float* s_blk, void* Y, cudaStream_t st) {
  const int warps = (K + 1023) / 1024;
  if (warps == 1) return launch_ln_one<E, 4, 128>(128, X, gamma, beta, T, K, eps, Xq, s_blk, Y, st);
  if (warps <= 24)  // 768 threads of 80 registers still fit
    return launch_ln_one<E, 1, 768>(32 * warps, X, gamma, beta, T, K, eps, Xq, s_blk, Y, st);
  return launch_ln_one<E, 1, 1024>(32 * warps, X, gamma, beta, T, K, eps, Xq, s_blk, Y, st);
}

// -------------------------------------------------------------------- weights

constexpr int kWeightCtas = 4;  // CTAs per SM: 64 registers per thread

// One CTA per 128 x 128 block, held in registers (eight 16-byte vectors per
// thread, all loads in flight at once) between the maximum and the codes.
// The maximum is taken over 16-bit pairs as they came.  24576 x 6144 in 67.7
// us, 6.7 TB/s of the copy's 6.56; with the values widened first 87 us, at 48
// registers (five CTAs) 95, its maximum's registers being spilled.
template <typename E>
__global__ void __launch_bounds__(256, kWeightCtas)
    fp8_weights_kernel(const E* __restrict__ W, int N, int K, unsigned kblocks,
                       uint8_t* __restrict__ Wq, float* __restrict__ s_blk) {
  __shared__ float red[8];
  grid_dependency_wait();
  grid_launch_dependents();
  const unsigned nb = blockIdx.x / kblocks, kb = blockIdx.x - nb * kblocks;
  const int col = static_cast<int>(kb) * kFp8Block + (threadIdx.x & 15) * 8;
  const int row0 = static_cast<int>(nb) * kFp8Block + (threadIdx.x >> 4);
  uint4 v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = row0 + 16 * i;
    v[i] = (r < N && col < K)
               ? __ldcs(reinterpret_cast<const uint4*>(W + static_cast<size_t>(r) * K + col))
               : make_uint4(0, 0, 0, 0);
  }
  uint32_t m2 = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    m2 = max_abs2<E>(max_abs2<E>(max_abs2<E>(max_abs2<E>(m2, v[i].x), v[i].y), v[i].z), v[i].w);
  float m = max_nan(unpack2<E>(m2).x, unpack2<E>(m2).y);
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
      uint64_t y[4];
      widen8<E>(v[i], y);
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
