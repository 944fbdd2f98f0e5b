// Projection on e4m3 codes with a scale per block of 128:
//   y[t][n] = sum_b x_scale[t][b] * w_scale[n / 128][b] * sum_{k in b} x[t][k] w[n][k]
//
// The tensor core applies no fp32 scale, so each block of 128 input dims gets an
// accumulator of its own: four tcgen05.mma (K = 32 each) into one slot of a TMEM
// ring, from which warps add it, times the two scales, to fp32 sums in registers
// while the tensor core works on the next block.  Two kernels: 128 x 256 tiles for
// many rows, bound by that chain (2.2 PFLOP/s at 4,096 x 2,048 x 32,768), and one for
// few rows, bound by the weights' bytes (8 x 2,048 x 32,768: 12.7 us, 5.3 TB/s) or, where
// they are few, by latency (8 x 7,168 x 512: 4.6 us).
#include <cuda_bf16.h>
#include <string.h>

#include "csa2_device.cuh"
#include "csa2_e4m3.cuh"
#include "csa2_internal.h"
#include "csa2_rope.cuh"

namespace csa2 {
namespace {

constexpr int kTileM = 128;   // rows of x a tile
constexpr int kBlockK = 128;  // input dims of a scale block: one swizzled 128-B row of codes
constexpr int kAccWarps = 8;
constexpr int kThreads = (kAccWarps + 4) * 32;  // 168 registers a thread, which 128 sums just fit

struct LinearParams {
  const float* x_scale;
  const float* w_scale;
  const int* row_pos;
  void* out;
  float* out_scale;
  long long ld_xs, ld_ws, ld_out, ld_os;
  int T, N, K;
  int rope_head;
  int vec;         // output rows are 16-B aligned
  int vec_scales;  // scale rows are 16-B aligned
  int w_ready;
  uint32_t* err;
  uint64_t turn[32];  // RoPE turn rates of the 32 pairs
};

// ---------------------------------------------------------------- many rows
// A CTA walks output tiles of 128 rows x 256 columns (persistent grid, the tiles of
// one column block behind each other so that its weights stay in L2).  Warps 0..7
// add and write (a lane is a row, four warps a column half), 8 is the TMA producer,
// 9 and 10 issue the products of one accumulator each, 11 brings the scales.  N =
// 256 because an instruction costs 137 cycles there and 92 at N = 128.  A block
// takes about 830 cycles: product and commit 566, sums 480, joined by four waits,
// with two accumulators to overlap them.
template <int BN>
struct WideCfg {
  static constexpr int kStages = 4;
  static constexpr int kStageBytes = (kTileM + BN) * kBlockK;
  static constexpr int kAccs = 512 / BN;          // TMEM ring: 512 columns
  static constexpr int kCols = BN / 2;            // columns of a tile an accumulation warp holds
  static constexpr int kOffOut = kStages * kStageBytes;  // 32 rows x 64 B of output per accumulation warp
  static constexpr int kScaleSlots = 4;                  // ring of the scales of four blocks: 128 rows, 2 column halves
  static constexpr int kScaleBytes = 4 * (kTileM + 2) * 4;  // per block: the rows', the halves'
  static constexpr int kOffScales = kOffOut + kAccWarps * 2048;
  static constexpr int kOffBars = kOffScales + kScaleSlots * kScaleBytes;
  static constexpr int kSmem = 1024 + kOffBars + 256;
};

// mbar_wait with the first look in line: half the time (46 against 92 cycles) where
// the phase is complete.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  return mbar_try_wait(bar, parity) || mbar_wait(bar, parity, abort);
}
__device__ __forceinline__ float ld_shared_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr));
  return v;
}

// Four consecutive scales of a row, of which n (<= 0: none) exist; 0 for the others.
__device__ __forceinline__ float4 load_scales(const float* s, int n, bool vec) {
  if (vec && n >= 4) return __ldg(reinterpret_cast<const float4*>(s));
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (n > 0) v.x = __ldg(s);
  if (n > 1) v.y = __ldg(s + 1);
  if (n > 2) v.z = __ldg(s + 2);
  if (n > 3) v.w = __ldg(s + 3);
  return v;
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// The 16-byte piece i of a row's output values y (f: the factor to e4m3 codes).
template <int OUT, int C>
__device__ __forceinline__ uint4 out_piece(const float (&y)[C], int i, float f) {
  if (OUT == CSA2_OUT_F32)
    return make_uint4(__float_as_uint(y[4 * i]), __float_as_uint(y[4 * i + 1]), __float_as_uint(y[4 * i + 2]),
                      __float_as_uint(y[4 * i + 3]));
  if (OUT == CSA2_OUT_BF16)
    return make_uint4(bf16x2(y[8 * i], y[8 * i + 1]), bf16x2(y[8 * i + 2], y[8 * i + 3]),
                      bf16x2(y[8 * i + 4], y[8 * i + 5]), bf16x2(y[8 * i + 6], y[8 * i + 7]));
  return make_uint4(e4m3x4(y[16 * i] * f, y[16 * i + 1] * f, y[16 * i + 2] * f, y[16 * i + 3] * f),
                    e4m3x4(y[16 * i + 4] * f, y[16 * i + 5] * f, y[16 * i + 6] * f, y[16 * i + 7] * f),
                    e4m3x4(y[16 * i + 8] * f, y[16 * i + 9] * f, y[16 * i + 10] * f, y[16 * i + 11] * f),
                    e4m3x4(y[16 * i + 12] * f, y[16 * i + 13] * f, y[16 * i + 14] * f, y[16 * i + 15] * f));
}
__host__ __device__ constexpr int out_size(int format) {
  return format == CSA2_OUT_F32 ? 4 : (format == CSA2_OUT_BF16 ? 2 : 1);
}

// A CTA's share of the work: tiles first, first + step, .. and of each the blocks
// [b0, b0 + blocks).  SPLIT: a cluster of two CTAs has one tile and halves its
// blocks (the first share a multiple of 4, as scales come in fours).
template <int BN, bool SPLIT>
struct Share {
  int m_tiles, b0, blocks;
  long long tiles, first, step;
  __device__ __forceinline__ explicit Share(const LinearParams& p) {
    m_tiles = (p.T + kTileM - 1) / kTileM;
    tiles = static_cast<long long>(m_tiles) * ((p.N + BN - 1) / BN);
    const int all = (p.K + kBlockK - 1) / kBlockK;
    if (SPLIT) {
      const int half = ((all + 1) / 2 + 3) & ~3;
      b0 = (blockIdx.x & 1) ? half : 0;
      blocks = (blockIdx.x & 1) ? all - half : half;
      first = blockIdx.x >> 1;
      step = tiles;
    } else {
      b0 = 0;
      blocks = all;
      first = blockIdx.x;
      step = gridDim.x;
    }
  }
  __device__ __forceinline__ int row(long long tile) const { return static_cast<int>(tile % m_tiles) * kTileM; }
  __device__ __forceinline__ int column(long long tile) const { return static_cast<int>(tile / m_tiles) * BN; }
};

// The accumulation warps' part: sums each tile in registers and writes it.
// False when a wait gave up (the same in a warp's lanes).
template <int BN, int OUT, bool SPLIT>
__device__ __forceinline__ bool accumulate_and_store(const CUtensorMap& map_out, const LinearParams& p, uint8_t* smem,
                                                     uint32_t tmem, uint64_t* tfull, uint64_t* tempty, uint64_t* empty,
                                                     uint64_t* sfull, uint64_t* sempty, volatile int* s_abort) {
  using Cfg = WideCfg<BN>;
  constexpr int S = Cfg::kStages, NA = Cfg::kAccs, C = Cfg::kCols, SS = Cfg::kScaleSlots;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int half = warp >> 2;            // columns half * C .. of the tile
  const int r = (warp & 3) * 32 + lane;  // row of the tile: TMEM lane
  const uint32_t taddr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + half * C;
  uint8_t* s_out = smem + Cfg::kOffOut + warp * 2048;
  const Share<BN, SPLIT> mine(p);
  const int blocks = mine.blocks;
  const uint32_t row_scales = smem_u32(smem) + Cfg::kOffScales + r * 4;
  const uint32_t half_scales = smem_u32(smem) + Cfg::kOffScales + (kTileM + half) * 4;
  uint32_t it = 0, g = 0;  // blocks and groups of four blocks so far
  for (long long tile = mine.first; tile < mine.tiles; tile += mine.step) {
    const int n0 = mine.column(tile) + half * C, t0 = mine.row(tile);
    const int row = t0 + r;
    float y[C];  // this row's sums
#pragma unroll
    for (int i = 0; i < C; ++i) y[i] = 0.f;
#pragma unroll 1
    for (int b = 0; b < blocks; ++b, ++it) {
      if ((b & 3) == 0 && !__all_sync(0xffffffffu, wait(&sfull[g % SS], (g / SS) & 1, s_abort))) return false;
      const uint32_t at = (g % SS) * Cfg::kScaleBytes + (b & 3) * (kTileM + 2) * 4;
      const float sx = ld_shared_f32(row_scales + at), sw = ld_shared_f32(half_scales + at);
      if (!__all_sync(0xffffffffu, wait(&tfull[it % NA], (it / NA) & 1, s_abort))) return false;
      tc_fence_after();
      // the products have read the stage: one commit a block serves both rings
      // (a second one costs the tensor pipe some 60 cycles)
      if (warp == 0 && lane == 0) mbar_arrive(&empty[it % S]);
      const uint64_t s2 = pack_f32x2(sx * sw, sx * sw);
      const uint32_t ta = taddr + (it % NA) * BN;
#pragma unroll
      for (int c = 0; c < C / 16; ++c) {
        uint32_t v[16];
        tmem_ld32x16_async(ta + c * 16, v);
        tmem_wait_ld16(v);
        if (c + 1 == C / 16) {  // all of it is in registers: the next product may have the accumulator
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&tempty[it % NA]);
            if ((b & 3) == 3 || b + 1 == blocks) mbar_arrive(&sempty[g % SS]);
          }
        }
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          const float2 sum = unpack_f32x2(fma_f32x2(pack_f32x2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), s2,
                                                    pack_f32x2(y[c * 16 + i], y[c * 16 + i + 1])));
          y[c * 16 + i] = sum.x;
          y[c * 16 + i + 1] = sum.y;
        }
      }
      if ((b & 3) == 3 || b + 1 == blocks) ++g;
    }
    if (SPLIT) {
      // Rank 0 finishes the left half of the columns, rank 1 the right one: the
      // other half's sums go to the peer through the stages, which are done with
      // (every product of this CTA is complete, and the peer reads its own).
      const int rank = static_cast<int>(blockIdx.x & 1);
      float* part = reinterpret_cast<float*>(smem) + r;
      if (half != rank) {
#pragma unroll
        for (int i = 0; i < C; ++i) part[i * kTileM] = y[i];
      }
      cluster_sync();
      if (half == rank) {
        const uint32_t at = map_rank(smem_u32(part), static_cast<uint32_t>(rank ^ 1));
#pragma unroll
        for (int i = 0; i < C; ++i) y[i] += ld_cluster_f32(at + i * kTileM * 4);
      }
      cluster_sync();  // no CTA leaves while its sums may still be read
      if (half != rank) break;
    }
    if (n0 >= p.N || t0 + (warp & 3) * 32 >= p.T) continue;
    if (p.rope_head && (n0 + C) % p.rope_head == 0) {  // the 64 columns below a head's end
      const int pos = __ldg(p.row_pos + min(row, p.T - 1));
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        float sn, cs;
        // fp32 output: as the few rows' kernel, so that a row's turn does not depend on
        // how many rows there are (4,096 x 2,048 x 4,096: 51.1 us, 46.4 with the fast
        // functions); the other types' rounding hides the fast functions' error
        if (OUT == CSA2_OUT_F32) rope_angle_turns(pos, p.turn[i], &sn, &cs);
        else rope_angle_fast(pos, p.turn[i], &sn, &cs);
        rope_pair(y[C - 64 + 2 * i], y[C - 63 + 2 * i], sn, cs);
      }
    }
    float f = 0.f;
    if (OUT == CSA2_OUT_FP8) {
      float m = 0.f;
#pragma unroll
      for (int i = 0; i < C; ++i) {
        y[i] = finite_or_nan(y[i]);
        m = fmaxf(m, fabsf(y[i]));
      }
      const float sc = e4m3_block(m, &f);
      if (row < p.T) p.out_scale[static_cast<long long>(row) * p.ld_os + (n0 >> 7)] = sc;
    }
    constexpr int kSize = out_size(OUT), kPieces = C * kSize / 16;
    // 32 rows x 64 B at a time through shared memory (swizzled, so that the lanes'
    // 16-byte stores do not collide) and out by a tensor store; rows that are not
    // 16-byte aligned (never e4m3) element by element, 64 B of a row side by side
#pragma unroll
    for (int c = 0; c < kPieces; c += 4) {
      if (lane == 0) bulk_wait_read();
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<uint4*>(s_out + lane * 64 + ((i ^ ((lane >> 1) & 3)) * 16)) = out_piece<OUT, C>(y, c + i, f);
      const int x = n0 * kSize + c * 16;  // byte of the output row
      if (p.vec) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && x < p.N * kSize) {
          tma_store_2d(&map_out, s_out, x, t0 + (warp & 3) * 32);
          bulk_commit();
        }
      } else if (OUT != CSA2_OUT_FP8) {
        __syncwarp();
        constexpr int kEl = 64 / kSize;  // elements of a row here
        const int e = lane % kEl, n = x / kSize + e;
#pragma unroll 4
        for (int q = lane / kEl; q < 32; q += 32 / kEl) {
          const uint8_t* src = s_out + q * 64 + (((e * kSize / 16) ^ ((q >> 1) & 3)) * 16) + e * kSize % 16;
          const long long at = static_cast<long long>(t0 + (warp & 3) * 32 + q) * p.ld_out + n;
          if (t0 + (warp & 3) * 32 + q < p.T && n < p.N) {
            if (OUT == CSA2_OUT_F32) static_cast<float*>(p.out)[at] = *reinterpret_cast<const float*>(src);
            else static_cast<uint16_t*>(p.out)[at] = *reinterpret_cast<const uint16_t*>(src);
          }
        }
      }
    }
  }
  if (lane == 0) bulk_wait_all();
  return true;
}

template <int BN, int OUT, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
    fp8_linear_wide_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                           const __grid_constant__ CUtensorMap map_out, const __grid_constant__ LinearParams p) {
  using Cfg = WideCfg<BN>;
  constexpr int S = Cfg::kStages, NA = Cfg::kAccs, C = Cfg::kCols, SS = Cfg::kScaleSlots;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + Cfg::kOffBars);
  uint64_t* empty = full + S;
  uint64_t* tfull = empty + S;
  uint64_t* tempty = tfull + NA;
  uint64_t* sfull = tempty + NA;
  uint64_t* sempty = sfull + SS;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(sempty + SS);
  volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    *s_abort = 0;
    for (int i = 0; i < S; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < NA; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], kAccWarps);
    }
    for (int i = 0; i < SS; ++i) {
      mbar_init(&sfull[i], 1);
      mbar_init(&sempty[i], kAccWarps);
    }
    fence_mbar_init();
    prefetch_tmap(&map_x);
    prefetch_tmap(&map_w);
  }
  if (warp == kAccWarps + 1) {
    tmem_alloc(s_tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_wait();
  pdl_trigger();  // every CTA holds its TMEM
  const uint32_t tmem = *s_tmem;
  const Share<BN, SPLIT> mine(p);
  const int blocks = mine.blocks;

  if (warp == kAccWarps) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      const uint64_t keep = l2_policy_evict_last();
      long long it = 0;
      bool ok = true;
      for (long long tile = mine.first; tile < mine.tiles && ok; tile += mine.step) {
        const int n0 = mine.column(tile), t0 = mine.row(tile);
        for (int b = 0; b < blocks; ++b, ++it) {
          const int s = static_cast<int>(it % S);
          if (!(ok = mbar_wait(&empty[s], static_cast<uint32_t>((it / S) & 1) ^ 1u, s_abort))) break;
          uint8_t* dst = smem + s * Cfg::kStageBytes;
          mbar_arrive_expect_tx(&full[s], Cfg::kStageBytes);
          tma_load_2d(dst, &map_x, (mine.b0 + b) * kBlockK, t0, &full[s], keep);
          tma_load_2d(dst + kTileM * kBlockK, &map_w, (mine.b0 + b) * kBlockK, n0, &full[s], keep);
        }
      }
      if (!ok) {
        *s_abort = 1;
        set_error(p.err, kErrTimeout);
      }
      // the copies of the last stages must land before the CTA may exit
      for (long long i = (it > S ? it - S : 0); i < it; ++i)
        mbar_wait(&full[i % S], static_cast<uint32_t>((i / S) & 1), nullptr);
    }
  } else if (warp > kAccWarps && warp <= kAccWarps + NA) {
    // ------------------------------------------------------------ MMA issuers
    // One warp for each accumulator: the products of a block are queued while the
    // other warp still waits for its accumulator.
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_e4m3_f32(kTileM, BN);
      constexpr uint64_t kStageDesc = Cfg::kStageBytes >> 4;
      const uint64_t x_desc = smem_desc_sw128(smem), w_desc = smem_desc_sw128(smem + kTileM * kBlockK);
      const long long all = (mine.tiles - mine.first + mine.step - 1) / mine.step * blocks;  // blocks of this CTA's tiles
      const int a = warp - kAccWarps - 1;
      const uint32_t d = tmem + a * BN;
      uint32_t s = a, phase = 0, a_phase = 1;
      bool ok = true;
      for (long long i = a; i < all; i += NA) {
        if (!(ok = wait(&full[s], phase, s_abort))) break;
        const uint64_t ad = x_desc + s * kStageDesc, bd = w_desc + s * kStageDesc;
        if (!(ok = wait(&tempty[a], a_phase, s_abort))) break;
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < 4; ++k)  // 32 B of the swizzled rows a step
          mma_e4m3(d, ad + 2 * k, bd + 2 * k, idesc, k > 0 ? 1u : 0u);
        mma_commit(&tfull[a]);
        a_phase ^= 1;
        s += NA;
        if (s >= S) {
          s -= S;
          phase ^= 1;
        }
      }
      if (!ok) {
        *s_abort = 1;
        set_error(p.err, kErrTimeout);
        // the last product of this accumulator still reads its stage and writes TMEM
        mbar_wait(&tfull[a], a_phase, nullptr);
      }
    }
  } else if (warp > kAccWarps + NA) {
    // ------------------------------------------------------------ scales
    // Four blocks' at a time into shared memory: a load of an accumulation warp would
    // be waited for at its next barrier arrival.
    long long g = 0;
    bool ok = true;
    for (long long tile = mine.first; tile < mine.tiles && ok; tile += mine.step) {
      const int n0 = mine.column(tile), t0 = mine.row(tile);
      const float* xs[4];  // of rows lane, lane + 32, ..
#pragma unroll
      for (int i = 0; i < 4; ++i)
        xs[i] = p.x_scale + static_cast<long long>(min(t0 + i * 32 + lane, p.T - 1)) * p.ld_xs + mine.b0;
      // lanes 0 and 1: the weight scales of a column half
      const float* ws = p.w_scale + static_cast<long long>(min(n0 + (lane & 1) * C, p.N - 1) >> 7) * p.ld_ws + mine.b0;
      for (int b = 0; b < blocks; b += 4, ++g) {
        const int s = static_cast<int>(g % SS);
        ok = __all_sync(0xffffffffu, mbar_wait(&sempty[s], static_cast<uint32_t>((g / SS) & 1) ^ 1u, s_abort));
        if (!ok) break;
        float* dst = reinterpret_cast<float*>(smem + Cfg::kOffScales + s * Cfg::kScaleBytes);
        auto put = [&](int i, const float4& v) {
          dst[i] = v.x;
          dst[i + kTileM + 2] = v.y;
          dst[i + 2 * (kTileM + 2)] = v.z;
          dst[i + 3 * (kTileM + 2)] = v.w;
        };
        float4 v[4], vw;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = load_scales(xs[i] + b, blocks - b, p.vec_scales);
        if (lane < 2) vw = load_scales(ws + b, blocks - b, p.vec_scales);
#pragma unroll
        for (int i = 0; i < 4; ++i) put(i * 32 + lane, v[i]);
        if (lane < 2) put(kTileM + lane, vw);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sfull[s]);
      }
    }
    if (!ok) {
      *s_abort = 1;
      set_error(p.err, kErrTimeout);
    }
  } else {
    if (!accumulate_and_store<BN, OUT, SPLIT>(map_out, p, smem, tmem, tfull, tempty, empty, sfull, sempty, s_abort)) {
      *s_abort = 1;
      set_error(p.err, kErrTimeout);
      if (lane == 0) bulk_wait_all();  // the last tile's output still leaves shared memory
      __syncwarp();
      if (SPLIT) {  // the waits that gave up came before the cluster's two barriers
        cluster_sync();
        cluster_sync();
      }
    }
  }
  if (SPLIT && warp >= kAccWarps) {
    __syncwarp();
    cluster_sync();
    cluster_sync();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kAccWarps + 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int BN>
long long wide_tiles(const csa2_fp8_linear_args& a) {
  return ((static_cast<long long>(a.T) + kTileM - 1) / kTileM) * ((static_cast<long long>(a.N) + BN - 1) / BN);
}

template <int BN, int OUT, bool SPLIT>
cudaError_t launch_wide(const csa2_fp8_linear_args& a, const LinearParams& p, const DeviceCtx& ctx, cudaStream_t st,
                        const char** why) {
  CUtensorMap map_x, map_w, map_out = {};
  if (encode_tmap_2d_u8(&map_x, a.x, a.K, a.T, a.ld_x, kBlockK, kTileM) != CUDA_SUCCESS ||
      encode_tmap_2d_u8(&map_w, a.w, a.K, a.N, a.ld_w, kBlockK, BN) != CUDA_SUCCESS ||
      (p.vec && encode_tmap_2d_u8(&map_out, a.out, static_cast<uint64_t>(a.N) * out_size(OUT), a.T,
                                  a.ld_out * out_size(OUT), 64, 32, CU_TENSOR_MAP_SWIZZLE_64B) != CUDA_SUCCESS)) {
    *why = "csa2_fp8_linear: a tensor map could not be encoded";
    return cudaErrorInvalidValue;
  }
  auto kern = fp8_linear_wide_kernel<BN, OUT, SPLIT>;
  cudaError_t e = prefer_max_smem_once<fp8_linear_wide_kernel<BN, OUT, SPLIT>>(ctx.device, WideCfg<BN>::kSmem);
  if (e != cudaSuccess) return e;
  const long long tiles = wide_tiles<BN>(a);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(SPLIT ? 2 * tiles : (tiles < ctx.num_sms ? tiles : ctx.num_sms)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = WideCfg<BN>::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = SPLIT ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, map_x, map_w, map_out, p);
}

// ---------------------------------------------------------------- few rows
// Up to a few hundred rows the weights are what is read, so they take the M side
// of the product: a CTA has 128 output columns (one block of weight scales) by
// NT rows of x, and a cluster of CTAs splits the input dims and adds its parts
// through distributed shared memory, in rank order.  Warps: 0 TMA producer, 1
// MMA issuer, 2..9 accumulation (a lane is an output column; two groups of four
// take the blocks in turn), all of them the output (a warp is a row of x).
constexpr int kNarrowThreads = 320;
constexpr int kScaleSeg = 16;  // blocks whose scales are staged at a time (even)

template <int NT>
struct NarrowCfg {
  static constexpr int kStages = 4;
  static constexpr int kStageBytes = (128 + NT) * kBlockK;
  static constexpr int kAccs = 4;
  static constexpr int kCols = kAccs * NT < 32 ? 32 : kAccs * NT;
  static constexpr int kOffScales = kStages * kStageBytes;  // the parts [NT][128] reuse the stages
  static constexpr int kOffBars = kOffScales + kScaleSeg * NT * 4;
  static constexpr int kSmem = 1024 + kOffBars + 256;
  static_assert(NT * 128 * 4 <= kOffScales, "the parts fit the stages");
};

template <int NT, int OUT>
__global__ void __launch_bounds__(kNarrowThreads, NT == 64 ? 1 : 2)
    fp8_linear_narrow_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                             const __grid_constant__ LinearParams p) {
  using Cfg = NarrowCfg<NT>;
  constexpr int S = Cfg::kStages, NA = Cfg::kAccs;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + Cfg::kOffBars);
  uint64_t* empty = full + S;
  uint64_t* tfull = empty + S;
  uint64_t* tempty = tfull + NA;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(tempty + NA);
  volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n0 = blockIdx.x * 128, t0 = blockIdx.y * NT;
  const int splits = gridDim.z, rank = blockIdx.z;
  const int all = (p.K + kBlockK - 1) / kBlockK;
  const int b0 = all * rank / splits, blocks = all * (rank + 1) / splits - b0;
  const uint64_t pol_w = l2_policy_evict_first(), pol_x = l2_policy_evict_last();

  if (threadIdx.x == 0) {
    *s_abort = 0;
    for (int i = 0; i < S; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < NA; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], 4);
    }
    fence_mbar_init();
    prefetch_tmap(&map_x);
    prefetch_tmap(&map_w);
    if (p.w_ready) {  // the first weights do not wait for the previous launch
      for (int b = 0; b < min(S, blocks); ++b) {
        mbar_arrive_expect_tx(&full[b], Cfg::kStageBytes);
        tma_load_2d(smem + b * Cfg::kStageBytes, &map_w, (b0 + b) * kBlockK, n0, &full[b], pol_w);
      }
    }
  }
  if (warp == 1) {
    tmem_alloc(s_tmem, Cfg::kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_wait();
  pdl_trigger();  // every CTA holds its TMEM
  const uint32_t tmem = *s_tmem;

  bool ok = true;
  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      int b = 0;
      for (; b < blocks; ++b) {
        const int s = b % S;
        if (b >= S && !(ok = mbar_wait(&empty[s], static_cast<uint32_t>(b / S - 1) & 1u, s_abort))) break;
        uint8_t* dst = smem + s * Cfg::kStageBytes;
        if (b >= S || !p.w_ready) {
          mbar_arrive_expect_tx(&full[s], Cfg::kStageBytes);
          tma_load_2d(dst, &map_w, (b0 + b) * kBlockK, n0, &full[s], pol_w);
        }
        tma_load_2d(dst + 128 * kBlockK, &map_x, (b0 + b) * kBlockK, t0, &full[s], pol_x);
      }
      if (!ok) {
        *s_abort = 1;
        set_error(p.err, kErrTimeout);
      }
      // the copies must land before shared memory is reused
      for (int i = (b > S ? b - S : 0); i < b; ++i) mbar_wait(&full[i % S], static_cast<uint32_t>(i / S) & 1u, nullptr);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_e4m3_f32(128, NT);
      int b = 0;
      for (; b < blocks; ++b) {
        const int s = b % S, a = b % NA;
        if (!(ok = mbar_wait(&full[s], static_cast<uint32_t>(b / S) & 1u, s_abort))) break;
        if (b >= NA && !(ok = mbar_wait(&tempty[a], static_cast<uint32_t>(b / NA - 1) & 1u, s_abort))) break;
        tc_fence_after();
        const uint64_t wd = smem_desc_sw128(smem + s * Cfg::kStageBytes);
        const uint64_t xd = smem_desc_sw128(smem + s * Cfg::kStageBytes + 128 * kBlockK);
#pragma unroll
        for (int k = 0; k < 4; ++k) mma_e4m3(tmem + a * NT, wd + 2 * k, xd + 2 * k, idesc, k > 0 ? 1u : 0u);
        mma_commit(&tfull[a]);
      }
      if (!ok) {
        *s_abort = 1;
        set_error(p.err, kErrTimeout);
        // the last products still read their stages and write TMEM
        for (int i = (b > NA ? b - NA : 0); i < b; ++i)
          mbar_wait(&tfull[i % NA], static_cast<uint32_t>(i / NA) & 1u, nullptr);
      }
    }
  } else {
    // ------------------------------------------------------------ accumulation
    const int quad = warp & 3, group = (warp - 2) >> 2;
    const uint32_t taddr = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    float* s_scale = reinterpret_cast<float*>(smem + Cfg::kOffScales);  // [block][NT]: both scales
    const float* ws = p.w_scale + static_cast<long long>(n0 >> 7) * p.ld_ws + b0;
    const int tid = threadIdx.x - 64;
    uint64_t acc[NT / 2];
#pragma unroll
    for (int i = 0; i < NT / 2; ++i) acc[i] = 0;
    for (int seg = 0; seg < blocks; seg += kScaleSeg) {
      const int n = min(kScaleSeg, blocks - seg);
      if (seg > 0) named_bar_sync(1, 256);  // the last segment has been used
      for (int i = tid; i < n * NT; i += 256) {
        const int t = i / n, b = i - t * n;
        const float* xs = p.x_scale + (t0 + t) * p.ld_xs + b0 + seg;
        s_scale[b * NT + t] = t0 + t < p.T ? __ldg(xs + b) * __ldg(ws + seg + b) : 0.f;
      }
      named_bar_sync(1, 256);
      for (int j = group; j < n && ok; j += 2) {  // kScaleSeg is even: a group keeps its blocks' parity
        const int b = seg + j, a = b % NA;
        ok = __all_sync(0xffffffffu, mbar_wait(&tfull[a], static_cast<uint32_t>(b / NA) & 1u, s_abort));
        if (!ok) break;
        tc_fence_after();
        if (quad == 0 && lane == 0) mbar_arrive(&empty[b % S]);  // the products have read the stage
        const ulonglong2* sc = reinterpret_cast<const ulonglong2*>(s_scale + j * NT);
#pragma unroll
        for (int c = 0; c < NT / 16; ++c) {
          uint32_t v[16];
          tmem_ld32x16_async(taddr + a * NT + c * 16, v);
          tmem_wait_ld16(v);
          if (c + 1 == NT / 16) {  // all of it is in registers
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&tempty[a]);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const ulonglong2 m = sc[c * 4 + i];
            uint64_t* s2 = acc + c * 8 + i * 2;
            s2[0] = fma_f32x2(pack_f32x2(__uint_as_float(v[4 * i]), __uint_as_float(v[4 * i + 1])), m.x, s2[0]);
            s2[1] = fma_f32x2(pack_f32x2(__uint_as_float(v[4 * i + 2]), __uint_as_float(v[4 * i + 3])), m.y, s2[1]);
          }
        }
      }
    }
    if (!ok) {
      *s_abort = 1;
      set_error(p.err, kErrTimeout);
    }
    // every product is complete (or given up), so the stages hold the parts now
    float* part = reinterpret_cast<float*>(smem) + quad * 32 + lane;
    named_bar_sync(1, 256);
    if (ok && group == 0) {
#pragma unroll
      for (int i = 0; i < NT / 2; ++i) {
        const float2 f = unpack_f32x2(acc[i]);
        part[(2 * i) * 128] = f.x;
        part[(2 * i + 1) * 128] = f.y;
      }
    }
    named_bar_sync(1, 256);
    if (ok && group == 1) {
#pragma unroll
      for (int i = 0; i < NT / 2; ++i) {
        const float2 f = unpack_f32x2(acc[i]);
        part[(2 * i) * 128] += f.x;
        part[(2 * i + 1) * 128] += f.y;
      }
    }
  }
  __syncthreads();
  if (splits > 1) cluster_sync();
  // ------------------------------------------------------------ output: a warp takes a row
  if (!*s_abort) {
    for (int t = rank + splits * warp; t < NT && t0 + t < p.T; t += splits * (kNarrowThreads / 32)) {
      const uint32_t at = smem_u32(reinterpret_cast<float*>(smem) + t * 128 + lane * 4);
      float y[4] = {0.f, 0.f, 0.f, 0.f};
      for (int r = 0; r < splits; ++r) {
        float4 v;
        if (splits > 1) {
          asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                       : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                       : "r"(map_rank(at, static_cast<uint32_t>(r))));
        } else {
          v = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(smem) + t * 128 + lane * 4);
        }
        y[0] += v.x;
        y[1] += v.y;
        y[2] += v.z;
        y[3] += v.w;
      }
      const long long row = t0 + t;
      if (p.rope_head && (n0 + 128) % p.rope_head == 0 && lane >= 16) {
        const int pos = __ldg(p.row_pos + row);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float sn, cs;
          if (OUT == CSA2_OUT_F32) rope_angle_turns(pos, p.turn[(lane - 16) * 2 + h], &sn, &cs);
          else rope_angle(pos, p.turn[(lane - 16) * 2 + h], &sn, &cs);
          rope_pair(y[2 * h], y[2 * h + 1], sn, cs);
        }
      }
      const int n = n0 + lane * 4;
      if (OUT == CSA2_OUT_FP8) {
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          y[i] = finite_or_nan(y[i]);
          m = fmaxf(m, fabsf(y[i]));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        float f;
        const float sc = e4m3_block(m, &f);
        *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.out) + row * p.ld_out + n) =
            e4m3x4(y[0] * f, y[1] * f, y[2] * f, y[3] * f);
        if (lane == 0) p.out_scale[row * p.ld_os + (n0 >> 7)] = sc;
      } else if (OUT == CSA2_OUT_F32) {
        float* o = static_cast<float*>(p.out) + row * p.ld_out + n;
        if (p.vec && n + 4 <= p.N) {
          *reinterpret_cast<float4*>(o) = make_float4(y[0], y[1], y[2], y[3]);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (n + i < p.N) o[i] = y[i];
        }
      } else {
        __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.out) + row * p.ld_out + n;
        if (p.vec && n + 4 <= p.N) {
          *reinterpret_cast<uint2*>(o) = make_uint2(bf16x2(y[0], y[1]), bf16x2(y[2], y[3]));
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (n + i < p.N) o[i] = __float2bfloat16_rn(y[i]);
        }
      }
    }
  }
  if (splits > 1) cluster_sync();  // no CTA leaves while its part may still be read
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, Cfg::kCols);
  }
}

// Clusters of `splits` CTAs that run at once on the device, by the runtime's count (an
// SM holds one CTA of NT = 64, by its registers, and two of the others), which is asked
// for once a device, kernel and size.
template <int NT, int OUT>
int narrow_clusters(const cudaLaunchConfig_t& cfg, int splits, int device) {
  constexpr auto kern = fp8_linear_narrow_kernel<NT, OUT>;
  static std::atomic<int> known[64][5];
  int i = 0;
  while ((1 << i) < splits) ++i;
  int n = known[device][i].load(std::memory_order_acquire);
  if (n == 0) {
    // clusters above 8 CTAs have to be allowed, once, before the first is asked for
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
      (void)cudaGetLastError();
      n = 0;
    }
    if (n < 1) n = -1;
    known[device][i].store(n, std::memory_order_release);
  }
  return n;
}

// Time of the wide kernel's launch, in the time of one block's products of one
// tile (about 0.43 us): rounds of tiles with their output, or half the blocks and
// the exchange, and what a launch takes before its first and after its last block.
bool wide_splits(const csa2_fp8_linear_args& a, const DeviceCtx& ctx) {
  return 2 * wide_tiles<256>(a) <= ctx.num_sms && (a.K + 127) / 128 >= 16;
}
long long wide_time(const csa2_fp8_linear_args& a, const DeviceCtx& ctx) {
  const int blocks = (a.K + 127) / 128;
  if (wide_splits(a, ctx)) return blocks / 2 + 14;
  return (wide_tiles<256>(a) + ctx.num_sms - 1) / ctx.num_sms * (blocks + 4) + 8;
}

// Launches the few-rows kernel, or sets *taken to false where 128 x 256 tiles take
// less time.  Up to 32 rows the weights' bytes decide, and this kernel reads them
// once; with more it has to run at once (one CTA an SM, by its registers) and be the quicker by
// wide_time's measure, a CTA's blocks and 7 (K = 7168, N = 512: 12.3 us here, 20 us
// there for 512 rows, 32 and 20 us for 2,048).
template <int NT, int OUT>
cudaError_t launch_narrow(const csa2_fp8_linear_args& a, const LinearParams& p, const DeviceCtx& ctx, cudaStream_t st,
                          const char** why, bool* taken) {
  auto kern = fp8_linear_narrow_kernel<NT, OUT>;
  const long long n_tiles = (static_cast<long long>(a.N) + 127) / 128;
  const int t_tiles = (a.T + NT - 1) / NT, blocks = (a.K + 127) / 128;
  *taken = NT < 64 || n_tiles * t_tiles <= ctx.num_sms;
  if (!*taken) return cudaSuccess;
  cudaError_t e = prefer_max_smem_once<fp8_linear_narrow_kernel<NT, OUT>>(ctx.device, NarrowCfg<NT>::kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kNarrowThreads);
  cfg.dynamicSmemBytes = NarrowCfg<NT>::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 1;
  attr[1].val.clusterDim.y = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  // The largest split whose CTAs keep two blocks each and run at once: up to 32 rows
  // two CTAs an SM (8 rows, K = 4,096, N = 7,168: 8.6 us split by 4, 10.2 by 2; K = 7,168,
  // N = 4,096: 8.2 by 8, 9.9 by 4), above one; clusters of 16, and all above 32 rows, by
  // the runtime's count, as clusters do not fill every SM.
  const long long tiles = n_tiles * t_tiles;
  int splits = 16;
  for (; splits > 1; splits >>= 1) {
    cfg.gridDim = dim3(static_cast<unsigned>(n_tiles), t_tiles, splits);
    attr[1].val.clusterDim.z = splits;
    if (2 * splits <= blocks && (NT < 64 && splits <= 8 ? tiles * splits <= 2 * ctx.num_sms
                                                        : tiles <= narrow_clusters<NT, OUT>(cfg, splits, ctx.device)))
      break;
  }
  *taken = NT < 64 || (blocks + splits - 1) / splits + 7 <= wide_time(a, ctx);
  if (!*taken) return cudaSuccess;
  cfg.gridDim = dim3(static_cast<unsigned>(n_tiles), t_tiles, splits);
  attr[1].val.clusterDim.z = splits;
  CUtensorMap map_x, map_w;
  if (encode_tmap_2d_u8(&map_x, a.x, a.K, a.T, a.ld_x, kBlockK, NT) != CUDA_SUCCESS ||
      encode_tmap_2d_u8(&map_w, a.w, a.K, a.N, a.ld_w, kBlockK, 128) != CUDA_SUCCESS) {
    *why = "csa2_fp8_linear: a tensor map could not be encoded";
    return cudaErrorInvalidValue;
  }
  return cudaLaunchKernelEx(&cfg, kern, map_x, map_w, p);
}

template <int OUT>
cudaError_t launch_out(const csa2_fp8_linear_args& a, const LinearParams& p, const DeviceCtx& ctx, cudaStream_t st,
                       const char** why) {
  bool taken = false;
  cudaError_t e = a.T <= 16   ? launch_narrow<16, OUT>(a, p, ctx, st, why, &taken)
                  : a.T <= 32 ? launch_narrow<32, OUT>(a, p, ctx, st, why, &taken)
                              : launch_narrow<64, OUT>(a, p, ctx, st, why, &taken);
  if (e != cudaSuccess || taken) return e;
  // Tiles for less than half the SMs share their blocks between two CTAs (4,096 x
  // 7,168 x 512: 28.9 -> 19.9 us).
  return wide_splits(a, ctx) ? launch_wide<256, OUT, true>(a, p, ctx, st, why)
                             : launch_wide<256, OUT, false>(a, p, ctx, st, why);
}

}  // namespace

cudaError_t launch_fp8_linear(const csa2_fp8_linear_args& a, const DeviceCtx& ctx, cudaStream_t st, const char** why) {
  LinearParams p;
  p.x_scale = a.x_scale;
  p.w_scale = a.w_scale;
  p.row_pos = a.row_pos;
  p.out = a.out;
  p.out_scale = a.out_scale;
  p.ld_xs = a.ld_x_scale;
  p.ld_ws = a.ld_w_scale;
  p.ld_out = a.ld_out;
  p.ld_os = a.ld_out_scale;
  p.T = a.T;
  p.N = a.N;
  p.K = a.K;
  p.rope_head = a.rope_head;
  p.vec = (a.ld_out * out_size(a.out_format)) % 16 == 0;
  p.vec_scales = (reinterpret_cast<uintptr_t>(a.x_scale) | reinterpret_cast<uintptr_t>(a.w_scale)) % 16 == 0 &&
                 a.ld_x_scale % 4 == 0 && a.ld_w_scale % 4 == 0;
  p.w_ready = a.w_ready;
  p.err = ctx.err;
  if (a.rope_head) {
    // the 32 powers take longer than the launch: the thread keeps the last theta's
    static thread_local double known = 0.0;
    static thread_local uint64_t turn[32];
    const double theta = a.rope_theta > 0.f ? a.rope_theta : 10000.0;
    if (theta != known) {
      for (int i = 0; i < 32; ++i) turn[i] = rope_turn_rate(theta, i);
      known = theta;
    }
    memcpy(p.turn, turn, sizeof(turn));
  }
  switch (a.out_format) {
    case CSA2_OUT_F32: return launch_out<CSA2_OUT_F32>(a, p, ctx, st, why);
    case CSA2_OUT_BF16: return launch_out<CSA2_OUT_BF16>(a, p, ctx, st, why);
    default: return launch_out<CSA2_OUT_FP8>(a, p, ctx, st, why);
  }
}

}  // namespace csa2
