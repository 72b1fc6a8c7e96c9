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
constexpr int kStreamMaxTokens = 32;

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
// Scales travel in groups of eight blocks, [block][token row] with four words
// of padding (so that a warp that reads rows of eight scales writes each to
// another bank), followed by the weight scales of the tile's weight blocks.
constexpr int kGroup = 8;
constexpr int kGroupRow = BM + 4;
constexpr int kGroupBytes = (kGroup * kGroupRow + 2 * kGroup) * 4;

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
  static constexpr int XCHG_BYTES = SPLIT ? BM * BN * 4 : 0;  // partial sums of the other CTAs
  static constexpr int AUX_BYTES = 2 * kGroupBytes + 2 * BN * 2;  // two scale groups, two units' bias
  static constexpr int STAGES_RAW =
      (kTileSmem - 1536 - XCHG_BYTES - AUX_BYTES) / STAGE_BYTES;
  static constexpr int STAGES = STAGES_RAW > 8 ? 8 : STAGES_RAW;
  static_assert(STAGES >= 3, "pipeline depth");
  static constexpr int OFF_XCHG = STAGES * STAGE_BYTES;
  static constexpr int OFF_AUX = OFF_XCHG + XCHG_BYTES;
  static constexpr int OFF_BIAS = OFF_AUX + 2 * kGroupBytes;
  static constexpr int OFF_BAR = OFF_AUX + AUX_BYTES;
  static_assert(OFF_BIAS % 16 == 0 && OFF_BAR % 8 == 0, "alignment");
  static constexpr int NUM_BARS = 2 * STAGES + 2 * NBUF * HALVES + 4 + 1;
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

// Every lane waits (bounded); true when all of them saw the phase complete.
__device__ __forceinline__ bool wait_all(uint64_t* bar, uint32_t parity, volatile int* abort,
                                         int* status, int site) {
  const bool ok = mbar_wait(bar, parity, abort, status, site);
  return __all_sync(0xffffffffu, ok);
}

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
__device__ __forceinline__ void fma_f32x2(uint64_t& acc, uint32_t lo, uint32_t hi, uint64_t s) {
  asm("{\n\t.reg .b64 d;\n\tmov.b64 d, {%1, %2};\n\tfma.rn.f32x2 %0, d, %3, %0;\n\t}"
      : "+l"(acc)
      : "r"(lo), "r"(hi), "l"(s));
}

__device__ __forceinline__ void st_cluster_v4(uint32_t addr, float4 v) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(v.x), "f"(v.y),
               "f"(v.z), "f"(v.w)
               : "memory");
}

// Eight columns' bias, in 16-bit form, added to their sums.
template <typename E>
__device__ __forceinline__ void add_bias(float (&v)[8], const uint4& bias) {
  float b[8];
  unpack8<E>(bias, b);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] += b[i];
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
  uint64_t* sfull_bar = tempty_bar + NBUF * HALVES;  // [2] a group of scales is there
  uint64_t* sempty_bar = sfull_bar + 2;     // [2]
  uint64_t* drain_bar = sempty_bar + 2;
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
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sfull_bar[b], 2);
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
    // The two warps take 64 token rows each; a lane reads one of eight
    // neighbouring scales of every fourth row.  (Read by the accumulating
    // warps themselves, one scale per lane and block from 32 rows, the loads
    // took as much of the shared-memory bandwidth as the copies.)
    reg_give<kRegsFirst>();
    const int j = lane & (kGroup - 1), half = warp - kAuxWarp0;
    const int r0 = half * (BM / 2) + lane / kGroup;
    int slot = 0, parity = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int u = unit0; ok && u < p.units; u += ustep, parity ^= 1) {
      int m, n;
      tile_of(u, p, m, n);
      const int t0 = m * C::TILE_M + (C::PAIR ? static_cast<int>(rank) * BM : 0);
      for (int k0 = kb0; k0 < kb1; k0 += kGroup) {
        const int kb = min(k0 + j, kb1 - 1);  // past the end: any value, it is not used
        const int nb = min(n * C::BN / kFp8Block + half, (p.N - 1) / kFp8Block);
        const float w = __ldg(p.s_w + static_cast<size_t>(nb) * p.kblocks + kb);
        float* g = reinterpret_cast<float*>(smem + C::OFF_AUX + slot * kGroupBytes);
#pragma unroll 1
        for (int i0 = 0; ok && i0 < BM / 8; i0 += 8) {
          float v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int t = min(t0 + r0 + 4 * (i0 + i), p.T - 1);
            v[i] = __ldg(p.s_x + static_cast<size_t>(t) * p.kblocks + kb);
          }
          if (i0 == 0) ok = wait_all(&sempty_bar[slot], phase ^ 1, abort_flag, p.status, 37);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (ok) g[j * kGroupRow + r0 + 4 * (i0 + i)] = v[i];
        }
        if (!ok) break;
        if (lane < kGroup) g[kGroup * kGroupRow + half * kGroup + j] = w;
        if (k0 == kb0 && p.bias && !C::SPLIT) {
          // the unit's bias, BN / 2 values from each warp (N % 8 == 0: the
          // 16-byte words are all in or all out)
          const int c = half * (C::BN / 2) + 8 * lane;
          if (lane < C::BN / 16 && n * C::BN + c < p.N)
            *reinterpret_cast<uint4*>(smem + C::OFF_BIAS + (parity * C::BN + c) * 2) =
                __ldg(reinterpret_cast<const uint4*>(static_cast<const E*>(p.bias) + n * C::BN + c));
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sfull_bar[slot]);
        slot ^= 1;
        phase ^= slot == 0;
      }
    }
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
    int buf = 0, slot = 0, parity = 0;
    uint32_t tphase = 0, sphase = 0;
    bool ok = true;
    for (int u = unit0; ok && u < p.units; u += ustep, parity ^= 1) {
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
        x = scales[j * kGroupRow + row];
        w = scales[kGroup * kGroupRow + part * COLS / kFp8Block * kGroup + j];
      };
      auto next_group = [&] {
        scales = reinterpret_cast<const float*>(smem + C::OFF_AUX + slot * kGroupBytes);
        return wait_all(&sfull_bar[slot], sphase, abort_flag, p.status, 38);
      };
      if (!next_group()) break;
      float fx, fw;
      factor_at(0, fx, fw);
      // The loads from tensor memory never pause: while a chunk of columns is
      // added the next one is on its way, across blocks too.
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
                ok = wait_all(&tfull_bar[buf * HALVES + half], tphase, abort_flag, p.status, 36);
              tc_fence_after();
              tmem_ld_32x32b_x32(t_row + static_cast<uint32_t>(buf * C::BN), r[0]);
            }
          }
          if (c == 0 && more) {
            probe = mbar_test_wait(&tfull_bar[next_buf * HALVES + half], next_phase);
            const int j = (kb + 1 - kb0) & (kGroup - 1);
            if (j == 0) {  // the last block of a group: hand it back, take the next
              __syncwarp();
              if (lane == 0) mbar_arrive(&sempty_bar[slot]);
              slot ^= 1;
              sphase ^= slot == 0;
              ok = next_group();
            }
            factor_at(j, fx, fw);
          }
#pragma unroll
          for (int i = 0; i < kChunk / 2; ++i)
            fma_f32x2(acc[kChunk / 2 * c + i], r[c & 1][2 * i], r[c & 1][2 * i + 1], s2);
        }
        if (!ok) {
          tmem_ld_wait();
          break;
        }
      }
      if (!ok) break;
      if constexpr (!C::SPLIT) {
        // Bias, rounding, and 32 bytes of a row per store: whole sectors, and
        // half of the shared-memory traffic that staging for a copy would take.
        const uint8_t* bias = smem + C::OFF_BIAS + (parity * C::BN + part * COLS) * 2;
        E* y = static_cast<E*>(p.Y) + static_cast<size_t>(t) * p.N + o0;
#pragma unroll
        for (int c0 = 0; c0 < COLS; c0 += 64) {
          uint4 bv[8] = {};  // ahead of the stores, all in flight together
          if (p.bias) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              bv[i] = *reinterpret_cast<const uint4*>(bias + (c0 + 8 * i) * 2);
          }
#pragma unroll
          for (int c = c0; c < c0 + 64; c += 16) {
            uint4 w[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float v[8];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float2 f = unpack_f32x2(acc[c / 2 + 4 * h + i]);
                v[2 * i] = f.x;
                v[2 * i + 1] = f.y;
              }
              if (p.bias) add_bias<E>(v, bv[(c - c0) / 8 + h]);
              w[h] = pack8<E>(v);
            }
            if (t < p.T) {  // N % 8 == 0: eight columns are all in or all out
              if (p.wide && o0 + c + 8 < p.N) {
                st_global_32(y + c, w[0], w[1]);
              } else {
                if (o0 + c < p.N) *reinterpret_cast<uint4*>(y + c) = w[0];
                if (o0 + c + 8 < p.N) *reinterpret_cast<uint4*>(y + c + 8) = w[1];
              }
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sempty_bar[slot]);
        slot ^= 1;
        sphase ^= slot == 0;
      } else {
        // Column chunk j (COLS / csize columns of each warp) goes to CTA j,
        // as float4 [source][piece][thread]: neighbouring lanes, neighbouring
        // 16-byte words.
        const int tid = threadIdx.x - 32 * kAccWarp0;
        const int pieces = COLS / 4 / static_cast<int>(csize);
        const uint32_t xchg = smem_u32(smem + C::OFF_XCHG);
#pragma unroll
        for (int i = 0; i < COLS / 4; ++i) {
          const int to = i / pieces, piece = i - to * pieces;
          const float2 a = unpack_f32x2(acc[2 * i]), b = unpack_f32x2(acc[2 * i + 1]);
          st_cluster_v4(
              mapa_shared(xchg + (((static_cast<int>(rank) * pieces + piece) * (32 * kAccWarps) + tid) << 4), to),
              make_float4(a.x, a.y, b.x, b.y));
        }
      }
    }
  }

  if constexpr (C::SPLIT) {
    __syncwarp();
    cluster_sync_all();  // all partial sums have arrived
    if (warp >= kAccWarp0) {
      const int quad = warp & 3, part = (warp - kAccWarp0) >> 2;
      const int tid = threadIdx.x - 32 * kAccWarp0;
      const int cols = COLS / static_cast<int>(csize), pieces = cols / 4;
      int m, n;
      tile_of(unit0, p, m, n);
      const int t = m * BM + quad * 32 + lane;
      const int o0 = n * C::BN + part * COLS + static_cast<int>(rank) * cols;
      const float4* in = reinterpret_cast<const float4*>(smem + C::OFF_XCHG);
      E* y = static_cast<E*>(p.Y) + static_cast<size_t>(t) * p.N + o0;
      const E* bias = static_cast<const E*>(p.bias);
      for (int c = 0; c < cols; c += 8) {
        if (t >= p.T || o0 + c >= p.N) break;
        float v[8] = {};
        for (uint32_t src = 0; src < csize; ++src) {
          const float4 a = in[(src * pieces + c / 4) * (32 * kAccWarps) + tid];
          const float4 b = in[(src * pieces + c / 4 + 1) * (32 * kAccWarps) + tid];
          v[0] += a.x; v[1] += a.y; v[2] += a.z; v[3] += a.w;
          v[4] += b.x; v[5] += b.y; v[6] += b.z; v[7] += b.w;
        }
        if (bias) add_bias<E>(v, __ldg(reinterpret_cast<const uint4*>(bias + o0 + c)));
        *reinterpret_cast<uint4*>(y + c) = pack8<E>(v);
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
  static std::atomic<uint64_t> ready{0};  // devices whose shared-memory limit is raised
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev > 63 || !(ready.load() >> dev & 1)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    if (dev <= 63) ready.fetch_or(1ull << dev);
  }
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

// The tile for many tokens, from the number of waves that each tiling needs.
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
  const long long small = tiles(BM, 128);
  // few tiles: share each along K, at least four blocks to a CTA
  int split = 1;
  while (split < 8 && small * split * 2 <= sms && p.kblocks >= split * 2 * 4) split *= 2;
  if (fsplit) split = fsplit;
  if (split > 1 && !fpair && !fbn) {
    if (split != 2 && split != 4 && split != 8) return cudaErrorInvalidValue;
    if (p.kblocks < split) return cudaErrorInvalidValue;
    return launch_tile<E, TileCfg<128, false, true>>(p, split, status, st);
  }
  // cost of a tiling: waves x columns per CTA
  const long long c128 = (small + sms - 1) / sms * 128;
  const long long c256 = (tiles(BM, 256) + sms - 1) / sms * 256;
  const long long cpair = (tiles(2 * BM, 256) + sms / 2 - 1) / (sms / 2) * 256;
  int pair = fpair ? fpair - 1 : cpair <= std::min(c128, c256);
  int bn = fbn ? fbn : (pair ? 256 : (c256 <= c128 ? 256 : 128));
  if (pair && bn == 256) return launch_tile<E, TileCfg<256, true, false>>(p, 1, status, st);
  if (pair) return launch_tile<E, TileCfg<128, true, false>>(p, 1, status, st);
  if (bn == 256) return launch_tile<E, TileCfg<256, false, false>>(p, 1, status, st);
  return launch_tile<E, TileCfg<128, false, false>>(p, 1, status, st);
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
  const bool tiles = path == 1 || (path == 0 && T > kStreamMaxTokens);
  const cudaError_t e = with_dtype(dtype, [&](auto tag) {
    using E = decltype(tag);
    return tiles ? launch_tiles<E>(p, st) : launch_stream<E>(p, st);
  });
  return e == cudaSuccess ? ZQ_OK : ZQ_ERR_CUDA;
}
