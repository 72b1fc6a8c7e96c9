// gemm_fp8.cu -- the quantized linear layer on e4m3 codes with a scale for
// each block of 128: activations [T][K] with scales [T][KB], weights [N][K]
// with scales [NB][KB].
//
//   Y[t][o] = sum_b (s_x[t][b] * s_w[o/128][b]) * (x8[t, b] . w8[o, b]) + bias[o]
//
// The tensor cores sum the 128 products of a block; each block's sums are
// then scaled and added in fp32 registers.
#include <algorithm>
#include <atomic>
#include <type_traits>

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

// Every lane waits (bounded); true when all of them saw the phase complete.
__device__ __forceinline__ bool wait_all(uint64_t* bar, uint32_t parity, volatile int* abort,
                                         int* status, int site) {
  const bool ok = mbar_wait(bar, parity, abort, status, site);
  return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ void fma_f32x2(uint64_t& acc, uint32_t lo, uint32_t hi, uint64_t s) {
  asm("{\n\t.reg .b64 d;\n\tmov.b64 d, {%1, %2};\n\tfma.rn.f32x2 %0, d, %3, %0;\n\t}"
      : "+l"(acc)
      : "r"(lo), "r"(hi), "l"(s));
}

__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ void st_cluster_v4(uint32_t addr, float4 v) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(v.x), "f"(v.y),
               "f"(v.z), "f"(v.w)
               : "memory");
}

// Raises a kernel's dynamic shared-memory limit once per device.
template <typename K>
cudaError_t allow_smem(K* kernel, int bytes, std::atomic<uint64_t>& ready) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && (ready.load() >> dev & 1)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < 64) ready.fetch_or(1ull << dev);
  return e;
}

// Clusters of S CTAs of a kernel that the current device runs at once, as far
// as the occupancy query knows: it counts one CTA of a kernel that allocates
// tensor memory per SM.  Asked once per kernel, size and device (`known`).
template <typename K>
cudaError_t clusters_at_once(K* kernel, int threads, int smem, int S,
                             std::atomic<int> (&known)[64][9], int* out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int n = dev < 64 ? known[dev][S].load(std::memory_order_relaxed) : 0;
  if (n == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(S * 64);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = S;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
    if (e != cudaSuccess) return e;
    n = std::max(n, 1);
    if (dev < 64) known[dev][S].store(n, std::memory_order_relaxed);
  }
  *out = n;
  return cudaSuccess;
}

// ------------------------------------------------------------ weight rows
//
// Up to 64 tokens: the weights' bytes bound the call, so they have to flow
// without a pause.  A CTA has R weight rows (the 128-row operand of its
// MMAs; rows past R are never looked at) and TN token
// columns, streamed through a deep ring of 128-k slices by TMA.  The MMAs of
// a block write their own columns of an accumulator buffer in tensor memory;
// eight warps take BATCH blocks at a time from there and add them up in fp32
// registers, a lane per weight row and a factor per column:
// acc[c] += d[c] * (s_x[t(c)][b] * s_w[nb][b]).  (One block at a time, the
// waits and tensor-memory loads of a block took 650 cycles: more than its
// copy where R is small.)
//
// R is chosen so that one wave of CTAs covers the weights.  Where that would
// leave a CTA few rows (and so little to copy per block), the CTAs of a
// cluster share rows along K and exchange their sums through distributed
// shared memory: rank r ends with every token c with c mod S == r, added in
// rank order.
// At 48 tokens, weight rows against tiles (us): 24576 x 6144 33.9 / 35.0, 6144 x
// 24576 37.9 / 42.5, 6144 x 6144 15.6 / 15.6, 12288 x 4096 17.8 / 16.4, 4096 x 4096
// 11.7 / 9.9; from 65 on only tiles can.
constexpr int kRowsMaxTokens = 64;
constexpr int kRowsAccWarps = 8;
constexpr int kRowsThreads = 32 * (4 + kRowsAccWarps);  // copies, MMAs, scales (two warps)
constexpr int kRowsMaxStages = 16;
// Two CTAs fit an SM: their waits and ends overlap, and the next call's
// set-up and first copies to L2 overlap the end of this one.  A third must not
// fit: two have all of tensor memory, and CTAs of a cluster that wait for one
// another must not wait for its allocation in a circle.
constexpr int kRowsSmem = 112 * 1024, kRowsMinSmem = 77 * 1024;

template <int TN_>
struct RowsCfg {
  static constexpr int TN = TN_;        // token columns
  static constexpr int COLS = TN / 2;   // of an accumulating warp
  static constexpr int CHUNK = COLS < 32 ? COLS : 32;  // columns of one TMEM load
  // scale blocks per accumulator buffer: as many as a warp has 32 columns for
  static constexpr int BATCH = COLS >= 32 ? 1 : 32 / COLS;
  static constexpr int BUF_COLS = BATCH * TN;
  static constexpr int NBUF = 512 / BUF_COLS > 4 ? 4 : 512 / BUF_COLS;
  static constexpr int TMEM_COLS = BUF_COLS * NBUF;
  static_assert(2 * TMEM_COLS <= 512, "tensor memory of two CTAs");
  static_assert(TMEM_COLS >= 32 && (TMEM_COLS & (TMEM_COLS - 1)) == 0, "tensor memory allocation");
  // blocks whose scales travel together, and floats of such a slot: the
  // tokens' [block][token], then the weights' [row block][block]
  static constexpr int G = TN <= 32 ? 32 : 16;
  static constexpr int SX_ROW = TN + 4;
  static constexpr int W_BLOCKS = 2;  // weight blocks that R rows can touch
  static constexpr int SLOT = G * SX_ROW + W_BLOCKS * G;
};

struct RowsParams {
  const float* s_x;
  const float* s_w;
  const void* bias;
  void* Y;
  int* status;
  int T, N, kblocks;
  int rows, stages, stage_bytes;
  int off_slots, off_xchg;  // shared memory, from the aligned base
};

template <typename E, class C>
__global__ void __launch_bounds__(kRowsThreads, 2)
    fp8_rows_gemm_kernel(const __grid_constant__ CUtensorMap map_x,
                         const __grid_constant__ CUtensorMap map_w, const RowsParams p) {
  constexpr int NBUF = C::NBUF, COLS = C::COLS, CHUNK = C::CHUNK, G = C::G;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full_bar[kRowsMaxStages], empty_bar[kRowsMaxStages], tfull_bar[NBUF],
      tempty_bar[NBUF], sfull_bar[2], sempty_bar[2], drain_bar;
  __shared__ uint32_t tmem_holder;
  __shared__ int abort_word;
  volatile int* abort_flag = &abort_word;
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const int S = static_cast<int>(cluster_nctarank()), rank = static_cast<int>(cluster_ctarank());
  const int o_cta = static_cast<int>(blockIdx.x) / S * p.rows;
  const int kb0 = static_cast<int>(static_cast<long long>(p.kblocks) * rank / S);
  const int kb1 = static_cast<int>(static_cast<long long>(p.kblocks) * (rank + 1) / S);
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    for (int b = 0; b < NBUF; ++b) {
      mbar_init(&tfull_bar[b], 1);
      mbar_init(&tempty_bar[b], kRowsAccWarps);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sfull_bar[b], 2);
      mbar_init(&sempty_bar[b], kRowsAccWarps);
    }
    mbar_init(&drain_bar, 1);
    abort_word = 0;
    fence_mbar_init();
    // The first weight slices may go on their way to L2 before the previous
    // kernel of the stream has finished: only L2 is touched, which that
    // kernel's writes reach coherently.
    for (int kb = kb0; kb < min(kb1, kb0 + p.stages); ++kb)
      tma_prefetch_l2_2d(&map_w, kb * kFp8Block, o_cta);
  }
  if (warp == 1) {
    tmem_alloc(&tmem_holder, C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  if (S > 1) cluster_sync_all();  // all CTAs of the cluster are there before any remote use
  tc_fence_after();
  const uint32_t tmem_base = tmem_holder;
  grid_dependency_wait();
  grid_launch_dependents();

  if (warp == 0) {
    // ------------------------------------------------------ TMA producer
    if (lane == 0) {
      const uint64_t pol_w = l2_policy_evict_first(), pol_x = l2_policy_evict_last();
      int stage = 0, issued = 0;
      uint32_t phase = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait(&empty_bar[stage], phase ^ 1, abort_flag, p.status, 51)) break;
        uint8_t* dst = smem + stage * p.stage_bytes;
        mbar_arrive_expect_tx(&full_bar[stage], p.stage_bytes);
        tma_load_2d(dst, &map_w, &full_bar[stage], kb * kFp8Block, o_cta, pol_w);
        tma_load_2d(dst + p.rows * kFp8Block, &map_x, &full_bar[stage], kb * kFp8Block, 0, pol_x);
        ++issued;
        if (++stage == p.stages) {
          stage = 0;
          phase ^= 1;
        }
      }
      // every copy issued has landed before the CTA goes on
      int no_abort = 0;
      for (int s = 0; s < min(p.stages, issued); ++s)
        mbar_wait(&full_bar[s], ((issued - 1 - s) / p.stages) & 1, &no_abort, p.status, 52);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------ MMA issuer
    constexpr uint32_t idesc = make_idesc_e4m3(128, C::TN);
    const bool leader = elect_one();
    const uint64_t desc0 = make_sw128_desc(smem_u32(smem));
    int stage = 0, buf = 0;
    uint32_t phase = 0, tphase = 0;
    for (int kb = kb0; kb < kb1; ++kb) {
      const int b = (kb - kb0) % C::BATCH;
      const bool last = b == C::BATCH - 1 || kb + 1 == kb1;  // of the buffer
      if (!wait_all(&full_bar[stage], phase, abort_flag, p.status, 53) ||
          (b == 0 && !wait_all(&tempty_bar[buf], tphase ^ 1, abort_flag, p.status, 54)))
        break;
      tc_fence_after();
      const uint64_t da = desc0 + static_cast<uint64_t>(stage * (p.stage_bytes >> 4));
      const uint64_t db = da + static_cast<uint64_t>(p.rows * kFp8Block >> 4);
      if (leader) {
#pragma unroll
        for (int k = 0; k < kFp8Block / 32; ++k)  // 32 bytes further in the swizzle row: +2
          mma_f8(tmem_base + static_cast<uint32_t>(buf * C::BUF_COLS + b * C::TN), da + 2 * k,
                 db + 2 * k, idesc, k > 0);
        mma_commit(&empty_bar[stage]);
        if (last) mma_commit(&tfull_bar[buf]);
      }
      __syncwarp();
      if (++stage == p.stages) {
        stage = 0;
        phase ^= 1;
      }
      if (last && ++buf == NBUF) {
        buf = 0;
        tphase ^= 1;
      }
    }
    // all MMAs of this thread are done before tensor memory is freed
    if (leader) {
      mma_commit(&drain_bar);
      int no_abort = 0;
      mbar_wait(&drain_bar, 0, &no_abort, p.status, 55);
    }
    __syncwarp();
  } else if (warp < 4) {
    // ------------------------------------------------------ scales
    // The two warps take half of the tokens each; a lane reads one of G
    // neighbouring scales of every (32 / G)th token, all in flight together.
    constexpr int PER_LANE = C::TN / 2 * G / 32;
    const int j = lane & (G - 1), half = warp - 2;
    const int t0 = half * (C::TN / 2) + lane / G;
    int slot = 0;
    uint32_t phase = 0;
    for (int k0 = kb0; k0 < kb1; k0 += G) {
      const int kb = min(k0 + j, kb1 - 1);  // past the end: any value, it is not used
      float v[PER_LANE];
#pragma unroll
      for (int i = 0; i < PER_LANE; ++i)
        v[i] = __ldg(p.s_x + static_cast<size_t>(min(t0 + i * (32 / G), p.T - 1)) * p.kblocks + kb);
      const int nb = min(o_cta / kFp8Block + half, (p.N - 1) / kFp8Block);
      const float w = __ldg(p.s_w + static_cast<size_t>(nb) * p.kblocks + kb);
      if (!wait_all(&sempty_bar[slot], phase ^ 1, abort_flag, p.status, 56)) break;
      float* g = reinterpret_cast<float*>(smem + p.off_slots) + slot * C::SLOT;
#pragma unroll
      for (int i = 0; i < PER_LANE; ++i) g[j * C::SX_ROW + t0 + i * (32 / G)] = v[i];
      if (lane < G) g[G * C::SX_ROW + half * G + j] = w;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sfull_bar[slot]);
      slot ^= 1;
      phase ^= slot == 0;
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------ accumulation
    // Two warps per TMEM lane quadrant, each with half of the columns.
    const int quad = warp & 3, part = (warp - 4) >> 2;
    const int row = quad * 32 + lane;
    const int col0 = part * COLS;
    const int wb = (o_cta + row) / kFp8Block - o_cta / kFp8Block;
    const uint32_t t_row =
        tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + static_cast<uint32_t>(part * COLS);
    uint64_t acc[COLS / 2];
#pragma unroll
    for (int i = 0; i < COLS / 2; ++i) acc[i] = 0ull;
    int buf = 0, slot = 0;
    uint32_t tphase = 0, sphase = 0;
    bool ok = true;
    const float* g = nullptr;
#pragma unroll 1
    for (int kb = kb0; kb < kb1; kb += C::BATCH) {
      const int j = (kb - kb0) & (G - 1);  // G is a multiple of BATCH
      if (j == 0) {
        g = reinterpret_cast<const float*>(smem + p.off_slots) + slot * C::SLOT;
        ok = wait_all(&sfull_bar[slot], sphase, abort_flag, p.status, 57);
      }
      ok = ok && wait_all(&tfull_bar[buf], tphase, abort_flag, p.status, 58);
      if (!ok) break;
      tc_fence_after();
      const uint32_t d = t_row + static_cast<uint32_t>(buf * C::BUF_COLS);
#pragma unroll
      for (int c = 0; c < COLS; c += CHUNK) {
        uint32_t r[C::BATCH][CHUNK];
#pragma unroll
        for (int b = 0; b < C::BATCH; ++b)
          tmem_ld_32x32b(d + static_cast<uint32_t>(b * C::TN + c), r[b]);
#pragma unroll
        for (int b = 0; b < C::BATCH; ++b) tmem_ld_wait_for(r[b]);
        if (c + CHUNK == COLS) {  // the buffer has been read
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&tempty_bar[buf]);
        }
#pragma unroll
        for (int b = 0; b < C::BATCH; ++b) {
          if (kb + b >= kb1) break;  // (the columns of blocks past the end hold anything)
          // rows past R: any of the slot's numbers
          const float w = g[G * C::SX_ROW + min(wb, C::W_BLOCKS - 1) * G + j + b];
          const uint64_t w2 = pack_f32x2(w, w);
          const float4* sx = reinterpret_cast<const float4*>(g + (j + b) * C::SX_ROW + col0 + c);
#pragma unroll
          for (int i = 0; i < CHUNK / 4; ++i) {
            const float4 x = sx[i];
            fma_f32x2(acc[c / 2 + 2 * i], r[b][4 * i], r[b][4 * i + 1],
                      mul_f32x2(pack_f32x2(x.x, x.y), w2));
            fma_f32x2(acc[c / 2 + 2 * i + 1], r[b][4 * i + 2], r[b][4 * i + 3],
                      mul_f32x2(pack_f32x2(x.z, x.w), w2));
          }
        }
      }
      if (++buf == NBUF) {
        buf = 0;
        tphase ^= 1;
      }
      if (j + C::BATCH == G) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&sempty_bar[slot]);
        slot ^= 1;
        sphase ^= slot == 0;
      }
    }
    const int o = o_cta + row;
    const bool mine = row < p.rows && o < p.N;
    const float bias =
        mine && p.bias ? static_cast<float>(static_cast<const E*>(p.bias)[o]) : 0.0f;
    E* y = static_cast<E*>(p.Y) + o;
    if (S == 1) {
      if (ok && mine) {
#pragma unroll
        for (int c = 0; c < COLS; c += 2) {
          const float2 v = unpack_f32x2(acc[c / 2]);
          const int t = col0 + c;
          if (t < p.T) y[static_cast<size_t>(t) * p.N] = static_cast<E>(v.x + bias);
          if (t + 1 < p.T) y[static_cast<size_t>(t + 1) * p.N] = static_cast<E>(v.y + bias);
        }
      }
    } else {
      // to the token's owner, [source][token / S][row]
      const int slots = (C::TN + S - 1) / S;
      const uint32_t xchg = smem_u32(smem + p.off_xchg);
      if (ok) {
#pragma unroll
        for (int c = 0; c < COLS; ++c) {
          const float2 v = unpack_f32x2(acc[c / 2]);
          const int t = col0 + c;
          if (t < p.T)
            st_cluster_f32(mapa_shared(xchg + (((rank * slots + t / S) * 128 + row) << 2), t % S),
                           c & 1 ? v.y : v.x);
        }
      }
      __syncwarp();
      cluster_sync_all();  // all sums have arrived (the other warps: below)
      const float* in = reinterpret_cast<const float*>(smem + p.off_xchg);
      if (ok && mine) {
        // the two warps of a row take turns
        for (int i = part, t = rank + part * S; t < p.T; i += 2, t += 2 * S) {
          float v = 0.0f;
          for (int src = 0; src < S; ++src) v += in[(src * slots + i) * 128 + row];
          y[static_cast<size_t>(t) * p.N] = static_cast<E>(v + bias);
        }
      }
    }
  }
  if (S > 1 && warp < 4) {
    __syncwarp();
    cluster_sync_all();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, C::TMEM_COLS);
  }
}

template <typename E, class C>
cudaError_t launch_rows_gemm(const Fp8Params& p, int rows, int split, cudaStream_t st) {
  auto* kernel = fp8_rows_gemm_kernel<E, C>;
  static std::atomic<uint64_t> ready{0};
  int* status = device_status_ptr();
  if (!status) return cudaErrorUnknown;
  cudaError_t e = allow_smem(kernel, kRowsSmem, ready);
  if (e != cudaSuccess) return e;
  RowsParams rp{};
  rp.s_x = p.s_x;
  rp.s_w = p.s_w;
  rp.bias = p.bias;
  rp.Y = p.Y;
  rp.status = status;
  rp.T = p.T;
  rp.N = p.N;
  rp.kblocks = p.kblocks;
  rp.rows = rows;
  rp.stage_bytes = (rows + C::TN) * kFp8Block;
  // the MMAs read whole 128-row tiles, up to `over` bytes past the last stage
  const int over = std::max(0, (128 - rows - C::TN) * kFp8Block);
  const int slots = 2 * C::SLOT * 4;
  const int xchg = split > 1 ? split * ((C::TN + split - 1) / split) * 128 * 4 : 0;
  const int room = kRowsSmem - 1024 - over - slots - xchg - 16;
  rp.stages = std::min(std::min(kRowsMaxStages, room / rp.stage_bytes),
                       (p.kblocks + split - 1) / split);
  rp.off_slots = (rp.stages * rp.stage_bytes + over + 15) / 16 * 16;
  rp.off_xchg = rp.off_slots + (slots + 15) / 16 * 16;
  const int smem = std::max(rp.off_xchg + xchg + 1024, kRowsMinSmem);
  CUtensorMap mx, mw;
  if (!encode_tma_2d(&mx, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.Xq, p.K, p.T, p.K, kFp8Block, C::TN,
                     CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_tma_2d(&mw, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.Wq, p.K, p.N, p.K, kFp8Block, rows,
                     CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  const int grid = ((p.N - 1) / rows + 1) * split;
  return launch_pdl_cluster(kernel, dim3(grid), dim3(kRowsThreads), smem, st, split, mx, mw, rp);
}

// CTAs of the weight-row kernel in clusters of S that run at once, two to an
// SM.  Clusters of four and eight leave SMs over: 72 of four (288 CTAs) took a
// second wave, 70 did not, and the query says 66.
template <typename E>
cudaError_t rows_ctas_at_once(int S, long long* out) {
  auto* kernel = fp8_rows_gemm_kernel<E, RowsCfg<16>>;
  static std::atomic<int> known[64][9];
  static std::atomic<uint64_t> ready{0};
  int n = 0;
  cudaError_t e = allow_smem(kernel, kRowsSmem, ready);
  if (e == cudaSuccess) e = clusters_at_once(kernel, kRowsThreads, kRowsSmem, S, known, &n);
  *out = std::min(2ll * n * S, 2ll * num_sms());
  return e;
}

template <typename E>
cudaError_t launch_rows_any(const Fp8Params& p, cudaStream_t st) {
  const int forced = option(ZQ_OPT_SPLIT_K), cap = option(ZQ_OPT_MAX_CTAS);
  auto rows_for = [&](long long ctas) {  // rows of each, if there were so many (no fewer than 1)
    const long long eights = 8 * std::max(1ll, ctas);
    return static_cast<int>(std::min<long long>(128, (p.N + eights - 1) / eights * 8));
  };
  // One CTA per SM, or two where the weights are large; K is split until a CTA
  // has 64 rows (8 KB to copy per block) or little of K.  Measured, one against
  // two (us, N x K at T = 1, 16 and 40):
  //   4096 x 4096 (16 M weights)   8.0 / 10.1    8.3 / 11.5   11.4 / 16.5
  //   5120 x 5120, split           9.7 /  9.1   10.5 /  9.6   15.6 / 13.8
  //   6144 x 24576, split         32.4 / 26.2   33.3 / 26.9   49.2 / 37.4
  //   4096 x 8192, split further  10.7 / 11.3   11.4 / 11.7   16.6 / 17.4
  //   12288 x 4096, unsplit       13.2 / 11.9   13.2 / 12.6   17.9 / 19.0
  //   18432 x 6144, unsplit       21.4 / 20.3   21.6 / 20.4   26.0 / 33.7
  //   16384 x 2048, short K        9.2 /  9.4    9.3 / 10.6   11.0 / 14.8
  //   24576 x 6144, over 148 CTAs 25.6 / 24.8   25.7 / 24.7   34.0 / 33.5
  const int alone = rows_for(num_sms());  // rows of a CTA with one per SM and all of K
  const bool large =
      static_cast<long long>(p.N) * p.K >= (24ll << 20) &&
      (alone < 64 ? alone > 32
                  : p.K >= 4096 && (p.T <= 32 || p.N > 128ll * num_sms()));
  int split = 1;
  long long target = 0;  // CTAs of the launch
  auto plan = [&](int S) {
    split = S;
    target = cap ? cap : num_sms();
    return large && !cap ? rows_ctas_at_once<E>(S, &target) : cudaSuccess;
  };
  cudaError_t e = plan(forced ? forced : 1);
  while (e == cudaSuccess && !forced && split < 8 && 2 * split <= target &&
         rows_for(target / split) < 64 && p.kblocks >= 4 * split)
    e = plan(2 * split);
  if (e != cudaSuccess) return e;
  const int rows = rows_for(target / split);
  auto go = [&](auto tn) {
    return launch_rows_gemm<E, RowsCfg<decltype(tn)::value>>(p, rows, split, st);
  };
  if (p.T <= 16) return go(std::integral_constant<int, 16>{});
  if (p.T <= 32) return go(std::integral_constant<int, 32>{});
  return go(std::integral_constant<int, 64>{});
}

// ------------------------------------------------------------------ tiles
//
// Many tokens: tcgen05 tiles of 128 token rows x BN weight rows per CTA (a
// CTA pair: 256 x BN, each CTA holding 128 rows of A, BN/2 rows of B and its
// 128 rows of D).  A pipeline stage is one scale block, 128 k: four MMAs sum
// its products in one of NBUF accumulator buffers in tensor memory, and eight
// warps bring that buffer into fp32 registers with one packed FMA per two
// values, acc += d * (s_x[t][b] * s_w[nb][b]), while the tensor cores fill
// the next one.  A lane has one token row and the columns of one weight
// block, so the factor is one number per lane and stage.
//
// 4096 x 6144 x 18432 takes 412 us alone (2.25 PFLOP/s) and 490 to 505 in a row,
// where power lowers the clock: 628 thousand cycles, of which the MMAs alone
// are 383.  Copies of an earlier state that took 652, with parts left out: without
// the FMAs 543, without the output's stores 617, without both 470, without the scales'
// copies too 413.  A block's sums wait for their MMAs, are loaded, added, and handed
// back across the pair, with two buffers to cover that: the FMAs (256 cycles per
// block and scheduler at best, 512 the MMAs) lengthen it, the loads from tensor
// memory do not.  Three to six stages, 12 or 16 accumulating warps (192 columns
// or 16-column loads), 256-column MMAs, releasing a buffer earlier and one look
// at all barriers at once measured the same or slower; single CTAs of 128 x 256
// are 7% slower, tiles of 128 columns 40% and more.
//
// With too few tiles for the SMs, the CTAs of a cluster share a tile, each
// with its own part of the blocks; they exchange their partial sums through
// distributed shared memory (each ends with its share of the columns, added
// in rank order) and need no workspace and no second kernel.
constexpr int BM = 128;
constexpr int BK = kFp8Block;  // k of a stage: one 128-byte swizzle row
constexpr int kAuxWarp0 = 2;  // two warps that bring scales and bias into shared memory
constexpr int kAccWarp0 = 4;
constexpr int kAccWarps = 8;
constexpr int kAccPerQuad = kAccWarps / 4;  // accumulating warps per TMEM lane quadrant
constexpr int kChunk = 32;                  // columns of one TMEM load
constexpr int kTileThreads = 32 * (kAccWarp0 + kAccWarps);
// Registers per thread: 168 at launch (65536 / 384, rounded down to 8); the
// accumulating warps, with 128 sums and the columns on their way each, take
// what the first four warps give: 4 * 56 + 8 * 224 = 12 * 168.
constexpr int kRegsFirst = 56, kRegsAcc = 224;
constexpr int kTileSmem = 226 * 1024;
template <int BN_, bool PAIR_, bool SPLIT_>
struct TileCfg {
  static constexpr int BN = BN_;
  static constexpr bool PAIR = PAIR_;    // CTA pair on a 256 x BN tile
  static constexpr bool SPLIT = SPLIT_;  // the CTAs of a cluster share a tile along K
  static_assert(!(PAIR && SPLIT), "one kind of cluster");
  static constexpr int TILE_M = PAIR ? 2 * BM : BM;
  static constexpr int W_ROWS = PAIR ? BN / 2 : BN;
  static constexpr int COLS = BN / kAccPerQuad;  // columns of an accumulating warp
  static_assert(COLS <= kFp8Block && kFp8Block % COLS == 0, "a warp's columns lie in one weight block");
  static constexpr int NBUF = 512 / BN;
  // A 256-wide tile is two MMAs of 128 columns, each with an accumulator
  // buffer and four accumulating warps of its own: while the four warps of
  // one half read theirs, the other half's MMAs run.
  static constexpr int HALVES = BN / 128;
  static constexpr int MMA_N = BN / HALVES;
  static constexpr int WARPS_PER_BUF = kAccWarps / HALVES;
  static constexpr int ROWS_PER_HALF = W_ROWS / HALVES;  // weight rows of one MMA in this CTA
  static constexpr int A_BYTES = BM * BK, B_BYTES = W_ROWS * BK;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  // partial sums from all CTAs of a cluster: S * ceil(16 / S) float4 for each
  // accumulating thread, at most 21 (S = 7)
  static constexpr int PIECES = COLS / 4;
  static constexpr int XCHG_BYTES = SPLIT ? 21 * 32 * kAccWarps * 16 : 0;
  static_assert(!SPLIT || PIECES == 16, "room for the partial sums");
  // Scales travel in groups of blocks, [block][token row] (padded, so that a
  // warp that copies rows of scales writes each to another bank), followed by
  // the weight scales of the tile's two weight blocks: 32 blocks, a line of
  // 128 bytes of each row's (in groups of eight, 32 bytes of a row, their
  // requests to L2 held up the copies: tiles of 256 x 128 took 12% longer), and
  // eight where a CTA has a part of the blocks only.
  static constexpr int GROUP = SPLIT ? 8 : 32;
  static constexpr int GROUP_ROW = SPLIT ? BM + 4 : BM + 1;
  static constexpr int GROUP_BYTES = (GROUP * GROUP_ROW + 2 * GROUP) * 4;
  static constexpr int SLOTS = 2;  // groups on their way or in use
  // and the bias of as many units (one can take a single group)
  static constexpr int AUX_BYTES = SLOTS * (GROUP_BYTES + BN * 2);
  static constexpr int STAGES_RAW =
      (kTileSmem - 1536 - XCHG_BYTES - AUX_BYTES) / STAGE_BYTES;
  static constexpr int STAGES = STAGES_RAW > 8 ? 8 : STAGES_RAW;
  static_assert(STAGES >= 3, "pipeline depth");
  static constexpr int OFF_XCHG = STAGES * STAGE_BYTES;
  static constexpr int OFF_AUX = OFF_XCHG + XCHG_BYTES;
  static constexpr int OFF_BIAS = OFF_AUX + SLOTS * GROUP_BYTES;
  static constexpr int OFF_BAR = OFF_AUX + AUX_BYTES;
  static_assert(OFF_BIAS % 16 == 0 && OFF_BAR % 8 == 0, "alignment");
  static constexpr int NUM_BARS = 2 * STAGES + 2 * NBUF * HALVES + 2 * SLOTS + 1;
  static constexpr int SMEM_BYTES = OFF_BAR + NUM_BARS * 8 + 16 + 1024;  // + alignment slack
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");
};

struct TileParams {
  const float* s_x;
  const float* s_w;
  const void* bias;
  void* Y;
  int* status;
  int T, N, kblocks;
  int m_tiles, n_tiles, units;
  int group_m;  // token tiles that run through all weight tiles together
  int wide;     // 32-byte output stores are aligned
};

// Units run through the token tiles of a group first, then the weight tiles,
// then the groups: the CTAs that run at the same time share weight tiles, and
// a group's activations stay in L2.
__device__ __forceinline__ void tile_of(int u, const TileParams& p, int& m, int& n) {
  const int per_group = p.group_m * p.n_tiles;
  const int g = u / per_group, r = u - g * per_group;
  const int gm = min(p.group_m, p.m_tiles - g * p.group_m);
  n = r / gm;
  m = g * p.group_m + r - n * gm;
}

// Eight columns' bias, in 16-bit form, added to their sums.
template <typename E>
__device__ __forceinline__ void add_bias(float (&v)[8], const uint4& bias) {
  float b[8];
  unpack8<E>(bias, b);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] += b[i];
}

// A step of the transposition of 4 x 4 pieces (two words of 16 bytes each)
// among four lanes: pieces i and i ^ BIT change places with those of the lane
// BIT off, so that after both steps piece r of lane q is piece q of lane q ^ r.
template <int BIT>
__device__ __forceinline__ void swap_pieces(uint4 (&w)[8], bool upper) {
  uint32_t* v = reinterpret_cast<uint32_t*>(w);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (i & BIT) continue;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      uint32_t &lo = v[8 * i + k], &hi = v[8 * (i + BIT) + k];
      const uint32_t keep = upper ? hi : lo;
      hi = __shfl_xor_sync(0xffffffffu, upper ? lo : hi, BIT);
      lo = keep;
    }
  }
}

template <typename E, class C>
__global__ void __launch_bounds__(kTileThreads, 1)
    fp8_tile_kernel(const __grid_constant__ CUtensorMap map_x,
                    const __grid_constant__ CUtensorMap map_w, const TileParams p) {
  constexpr int STAGES = C::STAGES, NBUF = C::NBUF, HALVES = C::HALVES, COLS = C::COLS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* empty_bar = full_bar + STAGES;
  uint64_t* tfull_bar = empty_bar + STAGES;
  uint64_t* tempty_bar = tfull_bar + NBUF * HALVES;
  uint64_t* sfull_bar = tempty_bar + NBUF * HALVES;  // [SLOTS] a group of scales is there
  uint64_t* sempty_bar = sfull_bar + C::SLOTS;       // [SLOTS]
  uint64_t* drain_bar = sempty_bar + C::SLOTS;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain_bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  uint32_t rank = 0, csize = 1;  // of the cluster
  if constexpr (C::PAIR || C::SPLIT) {
    rank = cluster_ctarank();
    csize = C::PAIR ? 2u : cluster_nctarank();
  }
  const int unit0 = static_cast<int>(blockIdx.x / csize);
  const int ustep = static_cast<int>(gridDim.x / csize);
  // the blocks of this CTA (SPLIT: its part; every part has at least one)
  const int kb0 = C::SPLIT ? static_cast<int>(static_cast<long long>(p.kblocks) * rank / csize) : 0;
  const int kb1 = C::SPLIT ? static_cast<int>(static_cast<long long>(p.kblocks) * (rank + 1) / csize)
                           : p.kblocks;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    for (int b = 0; b < NBUF * HALVES; ++b) {
      mbar_init(&tfull_bar[b], 1);
      mbar_init(&tempty_bar[b], (C::PAIR ? 2 : 1) * C::WARPS_PER_BUF);
    }
    for (int b = 0; b < C::SLOTS; ++b) {
      mbar_init(&sfull_bar[b], 64);  // the lanes of two warps
      mbar_init(&sempty_bar[b], kAccWarps);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&map_x);
    tma_prefetch_desc(&map_w);
  }
  if (warp == 1) {
    if constexpr (C::PAIR) {
      tmem_alloc_pair(tmem_holder, 512);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_holder, 512);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  // all CTAs of the cluster are there before any remote use
  if constexpr (C::PAIR || C::SPLIT) cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  grid_dependency_wait();
  grid_launch_dependents();

  if (warp == 0) {
    // ------------------------------------------------------ TMA producer
    reg_give<kRegsFirst>();
    if (lane == 0) {
      const uint64_t pol = l2_policy_evict_normal();
      int stage = 0;
      uint32_t phase = 0, fills[STAGES];
      for (int s = 0; s < STAGES; ++s) fills[s] = 0;
      bool ok = true;
      for (int u = unit0; ok && u < p.units; u += ustep) {
        int m, n;
        tile_of(u, p, m, n);
        const int x_row = m * C::TILE_M + (C::PAIR ? static_cast<int>(rank) * BM : 0);
        // (a pair's halves take their weight rows from both CTAs in turn)
        const int w_row = n * C::BN + (C::PAIR ? static_cast<int>(rank) * C::ROWS_PER_HALF : 0);
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!mbar_wait(&empty_bar[stage], phase ^ 1, abort_flag, p.status, 31)) {
            ok = false;
            break;
          }
          uint8_t* a = smem + stage * C::STAGE_BYTES;
          if constexpr (C::PAIR) {  // both CTAs' bytes complete on the leader's barrier
            const uint32_t fb = mapa_shared(smem_u32(&full_bar[stage]), 0);
            if (rank == 0) mbar_arrive_expect_tx(&full_bar[stage], 2 * C::STAGE_BYTES);
            tma_load_2d_pair(a, &map_x, fb, kb * BK, x_row, pol);
#pragma unroll
            for (int h = 0; h < HALVES; ++h)
              tma_load_2d_pair(a + C::A_BYTES + h * C::ROWS_PER_HALF * BK, &map_w, fb, kb * BK,
                               w_row + 128 * h, pol);
          } else {
            mbar_arrive_expect_tx(&full_bar[stage], C::STAGE_BYTES);
            tma_load_2d(a, &map_x, &full_bar[stage], kb * BK, x_row, pol);
#pragma unroll
            for (int h = 0; h < HALVES; ++h)
              tma_load_2d(a + C::A_BYTES + h * C::ROWS_PER_HALF * BK, &map_w, &full_bar[stage],
                          kb * BK, w_row + 128 * h, pol);
          }
          ++fills[stage];
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      // every copy issued has landed before the CTA exits (a pair's follower
      // is held by the final cluster barrier)
      int no_abort = 0;
      if (!C::PAIR || rank == 0)
        for (int s = 0; s < STAGES; ++s)
          if (fills[s]) mbar_wait(&full_bar[s], (fills[s] - 1) & 1, &no_abort, p.status, 32);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------ MMA issuer
    reg_give<kRegsFirst>();
    // The whole warp runs the loop, one elected lane issues: the operands of
    // the MMAs are then uniform across the warp.
    if (!C::PAIR || rank == 0) {
      constexpr uint32_t idesc = make_idesc_e4m3(C::TILE_M, C::MMA_N);
      const bool leader = elect_one();
      const uint64_t desc0 = make_sw128_desc(smem_u32(smem));
      int stage = 0, buf = 0;
      uint32_t phase = 0, tphase = 0;
      bool ok = true;
      for (int u = unit0; ok && u < p.units; u += ustep) {
        for (int kb = kb0; kb < kb1; ++kb) {
          const uint64_t da = desc0 + static_cast<uint64_t>(stage * (C::STAGE_BYTES >> 4));
          ok = wait_all(&full_bar[stage], phase, abort_flag, p.status, 34);
#pragma unroll
          for (int h = 0; h < HALVES; ++h) {
            const int b = buf * HALVES + h;
            ok = ok && wait_all(&tempty_bar[b], tphase ^ 1, abort_flag, p.status, 33);
            if (!ok) break;
            tc_fence_after();
            const uint32_t d = tmem_base + static_cast<uint32_t>(b * C::MMA_N);
            const uint64_t db = da + static_cast<uint64_t>((C::A_BYTES + h * C::ROWS_PER_HALF * BK) >> 4);
            if (leader) {
#pragma unroll
              for (int k = 0; k < BK / 32; ++k) {  // 32 bytes further in the swizzle row: +2
                if constexpr (C::PAIR)
                  mma_f8_pair(d, da + 2 * k, db + 2 * k, idesc, k > 0);
                else
                  mma_f8(d, da + 2 * k, db + 2 * k, idesc, k > 0);
              }
              if constexpr (C::PAIR)
                mma_commit_pair_mc(&tfull_bar[b], 0x3);
              else
                mma_commit(&tfull_bar[b]);
            }
          }
          if (!ok) break;
          if (leader) {
            if constexpr (C::PAIR)
              mma_commit_pair_mc(&empty_bar[stage], 0x3);
            else
              mma_commit(&empty_bar[stage]);
          }
          __syncwarp();
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1;
          }
          if (++buf == NBUF) {
            buf = 0;
            tphase ^= 1;
          }
        }
      }
      // all MMAs of this thread are done before tensor memory is freed
      if (leader) {
        if constexpr (C::PAIR)
          mma_commit_pair_mc(drain_bar, 0x1);
        else
          mma_commit(drain_bar);
        int no_abort = 0;
        mbar_wait(drain_bar, 0, &no_abort, p.status, 35);
      }
      __syncwarp();
    }
  } else if (warp < kAccWarp0) {
    // ------------------------------------------------------ scales and bias
    // The two warps take 64 token rows each; neighbouring lanes copy the scales
    // of a row's neighbouring blocks, four bytes at a time (all that is known of
    // their alignment), asynchronously.  (Read by the accumulating warps
    // themselves, one scale per lane and block from 32 rows, the loads took as
    // much of the shared-memory bandwidth as the copies.)
    reg_give<kRegsFirst>();
    const int j = lane & (C::GROUP - 1), half = warp - kAuxWarp0;
    const int r0 = half * (BM / 2) + lane / C::GROUP;
    int slot = 0, bias_slot = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int u = unit0; ok && u < p.units; u += ustep, bias_slot = (bias_slot + 1) % C::SLOTS) {
      int m, n;
      tile_of(u, p, m, n);
      const int t0 = m * C::TILE_M + (C::PAIR ? static_cast<int>(rank) * BM : 0);
      const int nb = min(n * C::BN / kFp8Block + half, (p.N - 1) / kFp8Block);
      for (int k0 = kb0; k0 < kb1; k0 += C::GROUP) {
        const int kb = min(k0 + j, kb1 - 1);  // past the end: any value, it is not used
        ok = wait_all(&sempty_bar[slot], phase ^ 1, abort_flag, p.status, 37);
        if (!ok) break;
        float* g = reinterpret_cast<float*>(smem + C::OFF_AUX + slot * C::GROUP_BYTES);
#pragma unroll 4
        for (int r = r0; r < (half + 1) * (BM / 2); r += 32 / C::GROUP) {
          const int t = min(t0 + r, p.T - 1);
          copy_async_4(g + j * C::GROUP_ROW + r, p.s_x + static_cast<size_t>(t) * p.kblocks + kb);
        }
        if (lane < C::GROUP)
          copy_async_4(g + C::GROUP * C::GROUP_ROW + half * C::GROUP + j,
                       p.s_w + static_cast<size_t>(nb) * p.kblocks + kb);
        if (k0 == kb0 && p.bias && !C::SPLIT) {
          // the unit's bias, BN / 2 values from each warp (N % 8 == 0: the
          // 16-byte words are all in or all out)
          const int c = half * (C::BN / 2) + 8 * lane;
          if (lane < C::BN / 16 && n * C::BN + c < p.N)
            copy_async_16(smem + C::OFF_BIAS + (bias_slot * C::BN + c) * 2,
                          static_cast<const E*>(p.bias) + n * C::BN + c);
        }
        copy_async_arrive(&sfull_bar[slot]);
        if (++slot == C::SLOTS) {
          slot = 0;
          phase ^= 1;
        }
      }
    }
    copy_async_wait();  // none is on its way when the CTA ends
  } else {
    // ------------------------------------------------------ accumulation
    reg_take<kRegsAcc>();
    // Two warps per TMEM lane quadrant (a warp reads the 32 lanes of quadrant
    // warp % 4), each with half of the columns.
    const int quad = warp & 3, part = (warp - kAccWarp0) >> 2;
    const int row = quad * 32 + lane;
    const uint32_t t_row =
        tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + static_cast<uint32_t>(part * COLS);
    const int half = HALVES == 2 ? part : 0;  // the accumulator buffers this warp reads
    // the (pair's leader's) barriers that hand a buffer back
    const uint32_t release0 = C::PAIR ? mapa_shared(smem_u32(&tempty_bar[half]), 0)
                                      : smem_u32(&tempty_bar[half]);
    int buf = 0, slot = 0, bias_slot = 0;
    uint32_t tphase = 0, sphase = 0;
    bool ok = true;
    auto next_slot = [&] {
      if (++slot == C::SLOTS) {
        slot = 0;
        sphase ^= 1;
      }
    };
    for (int u = unit0; ok && u < p.units; u += ustep, bias_slot = (bias_slot + 1) % C::SLOTS) {
      int m, n;
      tile_of(u, p, m, n);
      const int t = m * C::TILE_M + (C::PAIR ? static_cast<int>(rank) * BM : 0) + row;
      const int o0 = n * C::BN + part * COLS;
      uint64_t acc[COLS / 2];
#pragma unroll
      for (int i = 0; i < COLS / 2; ++i) acc[i] = 0ull;
      // Shared memory is busy with the copies and the MMAs' operands, so every
      // access to it is slow (150 to 250 cycles): the next block's factors and
      // the state of its accumulator buffer are asked for ahead of their use.
      const float* scales;  // of the current group
      auto factor_at = [&](int j, float& x, float& w) {
        x = scales[j * C::GROUP_ROW + row];
        w = scales[C::GROUP * C::GROUP_ROW + part * COLS / kFp8Block * C::GROUP + j];
      };
      auto next_group = [&] {
        scales = reinterpret_cast<const float*>(smem + C::OFF_AUX + slot * C::GROUP_BYTES);
        return wait_all(&sfull_bar[slot], sphase, abort_flag, p.status, 38);
      };
      if (!next_group()) break;
      float fx, fw;
      factor_at(0, fx, fw);
      // The loads from tensor memory never pause: while a chunk of columns is
      // added the next one is on its way, across blocks too.  (A wait that gave
      // up ends the tile behind its last block; the waits until then give up at
      // once.  With an exit from the loop the sums took 1.3% longer.)
      static_assert(COLS / kChunk % 2 == 0, "the chunk buffers alternate across blocks");
      uint32_t r[2][kChunk];
      if (!wait_all(&tfull_bar[buf * HALVES + half], tphase, abort_flag, p.status, 36)) break;
      tc_fence_after();
      tmem_ld_32x32b_x32(t_row + static_cast<uint32_t>(buf * C::BN), r[0]);
#pragma unroll 1
      for (int kb = kb0; kb < kb1; ++kb) {
        const bool more = kb + 1 < kb1;
        // rows and columns past the end are zero fill: any factor will do
        const float s = fx * fw;
        const uint64_t s2 = pack_f32x2(s, s);
        const int next_buf = buf + 1 == NBUF ? 0 : buf + 1;
        const uint32_t next_phase = tphase ^ (next_buf == 0);
        bool probe = false;
#pragma unroll
        for (int c = 0; c < COLS / kChunk; ++c) {
          tmem_ld_wait_for(r[c & 1]);
          if (c + 1 < COLS / kChunk) {
            tmem_ld_32x32b_x32(t_row + static_cast<uint32_t>(buf * C::BN + kChunk * (c + 1)),
                               r[(c + 1) & 1]);
          } else {  // the buffer has been read: release it, go on to the next
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              const uint32_t bar = release0 + static_cast<uint32_t>(buf * HALVES * 8);
              if constexpr (C::PAIR)
                mbar_arrive_cluster_tmem(bar);
              else
                mbar_arrive_addr(bar);
            }
            buf = next_buf;
            tphase = next_phase;
            if (more) {
              if (!__all_sync(0xffffffffu, probe))
                ok &= wait_all(&tfull_bar[buf * HALVES + half], tphase, abort_flag, p.status, 36);
              tc_fence_after();
              tmem_ld_32x32b_x32(t_row + static_cast<uint32_t>(buf * C::BN), r[0]);
            }
          }
          if (c == 0 && more) {
            probe = mbar_test_wait(&tfull_bar[next_buf * HALVES + half], next_phase);
            const int j = (kb + 1 - kb0) & (C::GROUP - 1);
            if (j == 0) {  // the last block of a group: hand it back, take the next
              __syncwarp();
              if (lane == 0) mbar_arrive(&sempty_bar[slot]);
              next_slot();
              ok &= next_group();
            }
            factor_at(j, fx, fw);
          }
#pragma unroll
          for (int i = 0; i < kChunk / 2; ++i)
            fma_f32x2(acc[kChunk / 2 * c + i], r[c & 1][2 * i], r[c & 1][2 * i + 1], s2);
        }
      }
      tmem_ld_wait();
      if (!ok) break;
      if constexpr (!C::SPLIT) {
        // Bias and rounding; then groups of four lanes exchange their rows'
        // pieces of 16 columns, so that each stores the same piece of four
        // rows: a store of the warp is eight lines of 128 bytes, not 32 pieces
        // of them, and needs no staging in shared memory.
        const uint8_t* bias = smem + C::OFF_BIAS + (bias_slot * C::BN + part * COLS) * 2;
        const int piece = lane & 3, first_t = t - piece;
        E* y = static_cast<E*>(p.Y) + o0 + 16 * piece;
#pragma unroll
        for (int c0 = 0; c0 < COLS; c0 += 64) {
          uint4 bv[8] = {};  // ahead of their use, all in flight together
          if (p.bias) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              bv[i] = *reinterpret_cast<const uint4*>(bias + (c0 + 8 * i) * 2);
          }
          uint4 w[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float v[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 f = unpack_f32x2(acc[c0 / 2 + 4 * i + k]);
              v[2 * k] = f.x;
              v[2 * k + 1] = f.y;
            }
            if (p.bias) add_bias<E>(v, bv[i]);
            w[i] = pack8<E>(v);
          }
          swap_pieces<1>(w, piece & 1);
          swap_pieces<2>(w, piece & 2);
#pragma unroll
          for (int r = 0; r < 4; ++r) {  // the row r lanes off in the group
            const int row_t = first_t + (piece ^ r), o = o0 + c0 + 16 * piece;
            if (row_t < p.T) {  // N % 8 == 0: eight columns are all in or all out
              E* to = y + static_cast<size_t>(row_t) * p.N + c0;
              if (p.wide && o + 8 < p.N) {
                st_global_32(to, w[2 * r], w[2 * r + 1]);
              } else {
                if (o < p.N) *reinterpret_cast<uint4*>(to) = w[2 * r];
                if (o + 8 < p.N) *reinterpret_cast<uint4*>(to + 8) = w[2 * r + 1];
              }
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sempty_bar[slot]);
        next_slot();
      } else {
        // Four columns at a time, in turn to the CTAs of the cluster, as float4
        // [source][turn][thread]: neighbouring lanes, neighbouring words.
        const int tid = threadIdx.x - 32 * kAccWarp0, S = static_cast<int>(csize);
        const int turns = (C::PIECES + S - 1) / S;
        const uint32_t xchg = smem_u32(smem + C::OFF_XCHG);
        int to = 0, turn = 0;
#pragma unroll
        for (int i = 0; i < C::PIECES; ++i) {
          const float2 a = unpack_f32x2(acc[2 * i]), b = unpack_f32x2(acc[2 * i + 1]);
          const int at = (static_cast<int>(rank) * turns + turn) * (32 * kAccWarps) + tid;
          st_cluster_v4(mapa_shared(xchg + (static_cast<uint32_t>(at) << 4), to),
                        make_float4(a.x, a.y, b.x, b.y));
          if (++to == S) {
            to = 0;
            ++turn;
          }
        }
      }
    }
  }

  if constexpr (C::SPLIT) {
    __syncwarp();
    cluster_sync_all();  // all partial sums have arrived
    if (warp >= kAccWarp0) {
      const int quad = warp & 3, part = (warp - kAccWarp0) >> 2;
      const int tid = threadIdx.x - 32 * kAccWarp0, S = static_cast<int>(csize);
      const int turns = (C::PIECES + S - 1) / S;
      int m, n;
      tile_of(unit0, p, m, n);
      const int t = m * BM + quad * 32 + lane;
      const int o0 = n * C::BN + part * COLS;
      const float4* in = reinterpret_cast<const float4*>(smem + C::OFF_XCHG) + tid;
      E* y = static_cast<E*>(p.Y) + static_cast<size_t>(t) * p.N + o0;
      const E* bias = static_cast<const E*>(p.bias);
      for (int turn = 0; turn < turns; ++turn) {
        const int c = 4 * (turn * S + static_cast<int>(rank));
        if (c >= COLS || t >= p.T || o0 + c >= p.N) break;
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int src = 0; src < S; ++src) {
          const float4 a = in[(src * turns + turn) * (32 * kAccWarps)];
          v.x += a.x, v.y += a.y, v.z += a.z, v.w += a.w;
        }
        if (bias) {
          const uint2 b = __ldg(reinterpret_cast<const uint2*>(bias + o0 + c));
          const float2 b0 = unpack2<E>(b.x), b1 = unpack2<E>(b.y);
          v.x += b0.x, v.y += b0.y, v.z += b1.x, v.w += b1.y;
        }
        *reinterpret_cast<uint2*>(y + c) = make_uint2(pack2<E>(v.x, v.y), pack2<E>(v.z, v.w));
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (C::PAIR) cluster_sync_all();  // no CTA leaves while its pair may still signal it
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    if constexpr (C::PAIR)
      tmem_dealloc_pair(tmem_base, 512);
    else
      tmem_dealloc(tmem_base, 512);
  }
}

template <typename E, class C>
cudaError_t launch_tile(const Fp8Params& p, int split, int* status, cudaStream_t st) {
  auto* kernel = fp8_tile_kernel<E, C>;
  static std::atomic<uint64_t> ready{0};
  const cudaError_t e = allow_smem(kernel, C::SMEM_BYTES, ready);
  if (e != cudaSuccess) return e;
  CUtensorMap mx, mw;
  if (!encode_tma_2d(&mx, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.Xq, p.K, p.T, p.K, BK, BM,
                     CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_tma_2d(&mw, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.Wq, p.K, p.N, p.K, BK,
                     C::ROWS_PER_HALF,
                     CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  TileParams tp{};
  tp.s_x = p.s_x;
  tp.s_w = p.s_w;
  tp.bias = p.bias;
  tp.Y = p.Y;
  tp.status = status;
  tp.T = p.T;
  tp.N = p.N;
  tp.kblocks = p.kblocks;
  tp.m_tiles = (p.T - 1) / C::TILE_M + 1;
  tp.n_tiles = (p.N - 1) / C::BN + 1;
  const long long units = static_cast<long long>(tp.m_tiles) * tp.n_tiles;
  if (units > (1ll << 30)) return cudaErrorInvalidValue;
  tp.units = static_cast<int>(units);
  // a group's activations take at most about a third of L2
  const long long tile_bytes = static_cast<long long>(C::TILE_M) * p.K;
  tp.group_m = static_cast<int>(
      std::min<long long>(tp.m_tiles, std::max<long long>(1, (40ll << 20) / tile_bytes)));
  tp.wide = p.N % 16 == 0 && reinterpret_cast<uintptr_t>(p.Y) % 32 == 0;
  const int sms = num_sms();
  int grid;
  if (C::SPLIT) {
    grid = tp.units * split;  // one unit per cluster
    return launch_pdl_cluster(kernel, dim3(grid), dim3(kTileThreads), C::SMEM_BYTES, st, split, mx,
                              mw, tp);
  }
  if (C::PAIR) {
    grid = 2 * std::min(tp.units, sms / 2);
    return launch_pdl_cluster(kernel, dim3(grid), dim3(kTileThreads), C::SMEM_BYTES, st, 2, mx, mw,
                              tp);
  }
  grid = std::min(tp.units, sms);
  return launch_pdl(kernel, dim3(grid), dim3(kTileThreads), C::SMEM_BYTES, st, mx, mw, tp);
}

// Clusters of S CTAs of the split tile that fit the current device at once.
template <typename E>
cudaError_t split_clusters(int S, int* out) {
  using C = TileCfg<128, false, true>;
  auto* kernel = fp8_tile_kernel<E, C>;
  static std::atomic<int> known[64][9];
  static std::atomic<uint64_t> ready{0};
  const cudaError_t e = allow_smem(kernel, C::SMEM_BYTES, ready);
  return e == cudaSuccess ? clusters_at_once(kernel, kTileThreads, C::SMEM_BYTES, S, known, out) : e;
}

// The tiling for many tokens: the least of these estimates (us), fitted to 40
// shapes of 65 to 4096 tokens.  A tile costs so much per scale block (bound
// by the copies into an SM, which a row pitch that is no multiple of 128
// bytes doubles in lines) and for its output; a split tile some more for the
// exchange.
template <typename E>
cudaError_t launch_tiles(const Fp8Params& p, cudaStream_t st) {
  int* status = device_status_ptr();
  if (!status) return cudaErrorUnknown;
  const int sms = num_sms();
  const int fbn = option(ZQ_OPT_GEMM_BN), fpair = option(ZQ_OPT_CTA_PAIR),
            fsplit = option(ZQ_OPT_SPLIT_K);
  auto tiles = [&](int tm, int tn) {
    return static_cast<long long>((p.T - 1) / tm + 1) * ((p.N - 1) / tn + 1);
  };
  const bool aligned = p.K % kFp8Block == 0;
  struct Option {
    int bn, pair;
    double per_block, per_tile;  // (per block with one wave: at most 0.46)
  };
  const Option options[4] = {{128, 0, aligned ? 0.39 : 0.52, 1.6},
                             {128, 1, 0.50, 2.0},
                             {256, 0, aligned ? 0.60 : 0.85, 2.2},
                             {256, 1, 0.56, 2.1}};
  double best = 1e30;
  const Option* pick = nullptr;
  for (const Option& o : options) {
    if ((fbn && o.bn != fbn) || (fpair ? o.pair != fpair - 1 : o.pair && p.T <= BM)) continue;
    const long long at_once = o.pair ? sms / 2 : sms;
    const long long waves = (tiles(o.pair ? 2 * BM : BM, o.bn) + at_once - 1) / at_once;
    const double per_block = waves == 1 ? std::min(o.per_block, o.bn == 128 ? 0.46 : 1.0) : o.per_block;
    const double cost = static_cast<double>(waves) * (p.kblocks * per_block + o.per_tile);
    if (cost < best) best = cost, pick = &o;
  }
  // few tiles: share each along K, at least three blocks to a CTA
  int split = 1;
  const long long small = tiles(BM, 128);
  if (fsplit > 1) {
    split = fsplit;
  } else if (fsplit == 0 && !fbn && !fpair && small * 2 <= sms) {
    for (int S = 2; S <= 8 && p.kblocks >= 3 * S; ++S) {
      int clusters = 0;
      const cudaError_t e = split_clusters<E>(S, &clusters);
      if (e != cudaSuccess) return e;
      if (small > clusters) continue;
      const double cost =
          (p.kblocks + S - 1) / S * (aligned ? 0.40 : 0.46) + 1.6 + 4.0;
      if (cost < best) best = cost, split = S;
    }
  }
  if (split > 1) return launch_tile<E, TileCfg<128, false, true>>(p, split, status, st);
  if (pick->bn == 256)
    return pick->pair ? launch_tile<E, TileCfg<256, true, false>>(p, 1, status, st)
                      : launch_tile<E, TileCfg<256, false, false>>(p, 1, status, st);
  return pick->pair ? launch_tile<E, TileCfg<128, true, false>>(p, 1, status, st)
                    : launch_tile<E, TileCfg<128, false, false>>(p, 1, status, st);
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
  const int split = option(ZQ_OPT_SPLIT_K), bn = option(ZQ_OPT_GEMM_BN);
  if (path > 2 || (path == 2 && T > kRowsMaxTokens) || split > 8 ||
      split > (K + kFp8Block - 1) / kFp8Block || (bn && bn != 128 && bn != 256))
    return ZQ_ERR_UNSUPPORTED;
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
  const bool rows = path == 2 || (path == 0 && T <= kRowsMaxTokens);
  const cudaError_t e = with_dtype(dtype, [&](auto tag) {
    using E = decltype(tag);
    return rows ? launch_rows_any<E>(p, st) : launch_tiles<E>(p, st);
  });
  return e == cudaSuccess ? ZQ_OK : ZQ_ERR_CUDA;
}
