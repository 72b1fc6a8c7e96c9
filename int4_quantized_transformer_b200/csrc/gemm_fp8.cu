// gemm_fp8.cu -- the quantized linear layer on e4m3 codes with a scale for
// each block of 128: activations [T][K] with scales [T][KB], weights [N][K]
// with scales [NB][KB].
//
//   Y[t][o] = sum_b (s_x[t][b] * s_w[o/128][b]) * (x8[t, b] . w8[o, b]) + bias[o]
//
// The tensor cores sum the 128 products of a block; each block's sums are
// then scaled and added in fp32 registers.
#include <algorithm>

#include "zq_fp8.cuh"
#include "zq_internal.h"
#include "zq_ptx.cuh"

namespace zq {
namespace {

struct Fp8Params {
  const uint8_t* Xq;
  const float* s_x;
  const uint8_t* Wq;
  const float* s_w;
  const void* bias;
  void* Y;
  int T, N, K, kblocks;
};

// --------------------------------------------------------- weight streaming
//
// A few tokens: the weights' bytes bound the call, and each is used once, so
// they go from global memory straight into the registers that mma.sync reads
// as its 16 x 32 A operand (8 tokens are the B operand).  The sum over k does
// not care about the order of k, so a lane takes 16 consecutive bytes of its
// row where the instruction's layout names four pieces of four, and the same
// bytes of the token rows.  The warps of a CTA share 16 weight rows and take
// every eighth block of 128 k each; their sums are added in warp order.
constexpr int kStreamWarps = 8;
constexpr int kStreamRows = 16;

__device__ __forceinline__ void mma_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <typename E, int NT>
__global__ void __launch_bounds__(32 * kStreamWarps) fp8_stream_kernel(const Fp8Params p) {
  __shared__ float part[kStreamWarps][8 * NT][kStreamRows];
  grid_dependency_wait();
  grid_launch_dependents();
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const int g = lane >> 2, q = lane & 3;
  const int o0 = blockIdx.x * kStreamRows, t0 = blockIdx.y * 8 * NT;
  const uint8_t* wlo = p.Wq + static_cast<size_t>(o0 + g) * p.K;
  const uint8_t* whi = wlo + static_cast<size_t>(8) * p.K;
  const bool lo_ok = o0 + g < p.N, hi_ok = o0 + g + 8 < p.N;
  const float* sw = p.s_w + static_cast<size_t>(o0 / kFp8Block) * p.kblocks;
  const uint4 zero = make_uint4(0, 0, 0, 0);

  struct Block {
    uint4 lo[2], hi[2], x[NT][2];
    float sx[NT][2], sw;
  };
  auto fetch = [&](int kb, Block& f) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = kb * kFp8Block + h * 64 + q * 16;
      const bool in = k < p.K;
      f.lo[h] = lo_ok && in ? __ldcs(reinterpret_cast<const uint4*>(wlo + k)) : zero;
      f.hi[h] = hi_ok && in ? __ldcs(reinterpret_cast<const uint4*>(whi + k)) : zero;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int t = t0 + 8 * n + g;
        f.x[n][h] = t < p.T && in ? __ldg(reinterpret_cast<const uint4*>(
                                        p.Xq + static_cast<size_t>(t) * p.K + k))
                                  : zero;
      }
    }
    f.sw = __ldg(sw + kb);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int t = t0 + 8 * n + 2 * q + j;
        f.sx[n][j] = t < p.T ? __ldg(p.s_x + static_cast<size_t>(t) * p.kblocks + kb) : 0.0f;
      }
  };
  float acc[NT][4] = {};
  Block cur;
  if (warp < p.kblocks) fetch(warp, cur);
  for (int kb = warp; kb < p.kblocks; kb += kStreamWarps) {
    Block next;
    if (kb + kStreamWarps < p.kblocks) fetch(kb + kStreamWarps, next);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float d[4] = {};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        mma_e4m3(d, cur.lo[h].x, cur.hi[h].x, cur.lo[h].y, cur.hi[h].y, cur.x[n][h].x,
                 cur.x[n][h].y);
        mma_e4m3(d, cur.lo[h].z, cur.hi[h].z, cur.lo[h].w, cur.hi[h].w, cur.x[n][h].z,
                 cur.x[n][h].w);
      }
      const float s0 = cur.sx[n][0] * cur.sw, s1 = cur.sx[n][1] * cur.sw;
      acc[n][0] = fmaf(d[0], s0, acc[n][0]);  // row g, tokens 2q and 2q + 1
      acc[n][1] = fmaf(d[1], s1, acc[n][1]);
      acc[n][2] = fmaf(d[2], s0, acc[n][2]);  // row g + 8
      acc[n][3] = fmaf(d[3], s1, acc[n][3]);
    }
    cur = next;
  }
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    part[warp][8 * n + 2 * q][g] = acc[n][0];
    part[warp][8 * n + 2 * q + 1][g] = acc[n][1];
    part[warp][8 * n + 2 * q][g + 8] = acc[n][2];
    part[warp][8 * n + 2 * q + 1][g + 8] = acc[n][3];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 8 * NT * kStreamRows; i += 32 * kStreamWarps) {
    const int c = i / kStreamRows, r = i % kStreamRows;
    const int t = t0 + c, o = o0 + r;
    if (t >= p.T || o >= p.N) continue;
    float v = part[0][c][r];
#pragma unroll
    for (int w = 1; w < kStreamWarps; ++w) v += part[w][c][r];
    if (p.bias) v += static_cast<float>(static_cast<const E*>(p.bias)[o]);
    static_cast<E*>(p.Y)[static_cast<size_t>(t) * p.N + o] = static_cast<E>(v);
  }
}

template <typename E>
cudaError_t launch_stream(const Fp8Params& p, cudaStream_t st) {
  auto go = [&](auto* kernel, int nt) {
    const dim3 grid((p.N + kStreamRows - 1) / kStreamRows, (p.T + 8 * nt - 1) / (8 * nt));
    return launch_pdl(kernel, grid, dim3(32 * kStreamWarps), 0, st, p);
  };
  if (p.T <= 8) return go(fp8_stream_kernel<E, 1>, 1);
  if (p.T <= 16) return go(fp8_stream_kernel<E, 2>, 2);
  return go(fp8_stream_kernel<E, 4>, 4);
}

}  // namespace
}  // namespace zq

using namespace zq;

extern "C" zq_status zq_gemm_fp8(const void* Xq, const float* s_x, const void* Wq, const float* s_w,
                                 const void* bias, int T, int N, int K, int dtype, void* Y,
                                 zq_stream_t stream) {
  if (dtype != ZQ_F16 && dtype != ZQ_BF16) return ZQ_ERR_UNSUPPORTED;
  if (T < 0 || N < 8 || N % 8 != 0 || K < 16 || K > (1 << 20) || K % 16 != 0) return ZQ_ERR_SHAPE;
  const int path = option(ZQ_OPT_GEMM_PATH);
  if (path > 2) return ZQ_ERR_UNSUPPORTED;
  if (T == 0) return ZQ_OK;
  if (!Xq || !s_x || !Wq || !s_w || !Y) return ZQ_ERR_NULL;
  if (!aligned16(Xq) || !aligned16(Wq) || !aligned16(Y) || (bias && !aligned16(bias)) ||
      reinterpret_cast<uintptr_t>(s_x) % 4 || reinterpret_cast<uintptr_t>(s_w) % 4)
    return ZQ_ERR_ALIGN;
  Fp8Params p{};
  p.Xq = static_cast<const uint8_t*>(Xq);
  p.s_x = s_x;
  p.Wq = static_cast<const uint8_t*>(Wq);
  p.s_w = s_w;
  p.bias = bias;
  p.Y = Y;
  p.T = T;
  p.N = N;
  p.K = K;
  p.kblocks = (K + kFp8Block - 1) / kFp8Block;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e =
      with_dtype(dtype, [&](auto tag) { return launch_stream<decltype(tag)>(p, st); });
  return e == cudaSuccess ? ZQ_OK : ZQ_ERR_CUDA;
}
