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
//
// LORA: each adapter that a tile's rows use (lora.cu lists them) brings one more block for
// every 64 or 32 ranks, whichever fit a stage: bf16 products of the parts of the rows' v with
// the adapter's b, summed like the others but only to the rows that have the adapter.  The
// projection's own blocks come first, and only what lora.cu wrote waits for it.  4,096 x
// 2,048 x 32,768 with 4 adapters of rank 64: 292 us, 236 without adapters (an adapter takes two
// blocks there); 64 rows with 16 of rank 32: 25.7 us, 16.1 without adapters, and b's bytes are 5 more.
#include <cuda_bf16.h>
#include <string.h>

#include <type_traits>

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

// What LORA adds to a launch: nothing without it.
template <bool LORA>
struct LoraParams {};
template <>
struct LoraParams<true> {
  // Inner products [planes T, pitch] and b [adapters N, rank], as boxes of a block's row by
  // a tile's rows or columns: of the runs of `run` ranks, and of the last one if it is shorter.
  CUtensorMap map_v, map_b, map_v_last, map_b_last;
  const int* row_adapter;
  const int* lists;  // of tiles of 128 rows, kLoraListWords each; a tile of fewer makes its own
  int n_adapters, rank;
  int run;     // ranks of a block
  int pieces;  // blocks of an adapter
  int planes;  // of v
  int v_rows;  // of a plane of v in a stage
};
// Bytes of a row of v or b of some ranks in shared memory.  The least that hold them: a box
// whose rows end far past the matrix's costs time (64 x 2,048 x 32,768 with 16 adapters of
// rank 8: 43 us with 128, 26 with 32), though less than plain copies of the rows (50 us).
__host__ __device__ __forceinline__ int lora_row_bytes(int ranks) { return ranks <= 16 ? 32 : ranks <= 32 ? 64 : 128; }
// Block i of a tile's adapters: the adapter, where its ranks start and how many there are.
// In a stage the planes of v come first, whose products with b, behind them, are one sum.
struct LoraBlock {
  int adapter, rank0, ranks, row;
  __device__ __forceinline__ LoraBlock(const LoraParams<true>& lo, const int* list, int i) {
    const int j = i / lo.pieces, k = i - j * lo.pieces;
    adapter = list[4 + j];
    rank0 = k * lo.run;
    ranks = min(lo.run, lo.rank - rank0);
    row = lora_row_bytes(ranks);
  }
  __device__ __forceinline__ void expect(const LoraParams<true>& lo, uint64_t* full, int b_rows) const {
    mbar_arrive_expect_tx(full, (lo.planes * lo.v_rows + b_rows) * row);
  }
  // Behind b's columns, and in the columns of 8 ranks without a partner, are zeros.
  __device__ __forceinline__ void copy_b(const LoraParams<true>& lo, uint8_t* stage, uint64_t* full, int n0, int N,
                                         uint64_t policy) const {
    tma_load_2d(stage + lo.planes * lo.v_rows * row, ranks < lo.run ? &lo.map_b_last : &lo.map_b, rank0 * 2, adapter * N + n0,
                full, policy);
  }
  __device__ __forceinline__ void copy_v(const LoraParams<true>& lo, uint8_t* stage, uint64_t* full, int t0, int T,
                                         uint64_t policy) const {
    for (int i = 0; i < lo.planes; ++i)
      tma_load_2d(stage + i * lo.v_rows * row, ranks < lo.run ? &lo.map_v_last : &lo.map_v, rank0 * 2, i * T + t0, full, policy);
  }
  // The block's products; V_FIRST: v is the first operand, of whose 128 rows those from v_rows on
  // are whatever follows in the stage: rows that the output does not have.
  template <bool V_FIRST>
  __device__ __forceinline__ void products(const LoraParams<true>& lo, uint32_t d, const uint8_t* stage, uint32_t idesc) const {
    const uint64_t bd = smem_desc_rows(stage + lo.planes * lo.v_rows * row, row);
    const int steps = (ranks + 15) >> 4;  // of 16 ranks
    for (int i = 0; i < lo.planes; ++i) {
      const uint64_t vd = smem_desc_rows(stage + i * lo.v_rows * row, row);
      for (int k = 0; k < steps; ++k)
        umma_bf16(d, (V_FIRST ? vd : bd) + 2 * k, (V_FIRST ? bd : vd) + 2 * k, idesc, i + k > 0 ? 1u : 0u);
    }
  }
};
// The adapters among a tile's NT rows, each once, in the order of their first rows, and the
// rows' own, by a warp: list[0] how many, list[4 ..] which; own: -1 for none or no row.
template <int NT>
__device__ __forceinline__ void tile_adapters(const LoraParams<true>& lo, int t0, int T, int* list, int* own) {
  const int lane = threadIdx.x & 31;
  int count = 0;
#pragma unroll
  for (int h = 0; h < (NT + 31) / 32; ++h) {
    const int row = h * 32 + lane;
    int id = row < NT && t0 + row < T ? __ldg(lo.row_adapter + t0 + row) : -1;
    if (id < 0 || id >= lo.n_adapters) id = -1;
    if (row < NT) own[row] = id;
    const uint32_t same = __match_any_sync(0xffffffffu, id);  // all lanes take part
    bool first = id >= 0 && __ffs(same) - 1 == lane;
    for (int j = 0; j < h * 32; j += 4) {
      const int4 v = *reinterpret_cast<const int4*>(own + j);
      first = first & (v.x != id) & (v.y != id) & (v.z != id) & (v.w != id);
    }
    const uint32_t mask = __ballot_sync(0xffffffffu, first);
    if (first) list[4 + count + __popc(mask & ((1u << lane) - 1))] = id;
    count += __popc(mask);
    __syncwarp();
  }
  if (lane == 0) list[0] = count;
  __syncwarp();
}

// What a launch has to know of its adapters on the host.
struct NoLora {
  static constexpr bool kOn = false;
};
struct WithLora {
  static constexpr bool kOn = true;
  const csa2_lora_linear_args* args;
  void* workspace;
};
// ---------------------------------------------------------------- many rows
// A CTA walks output tiles of 128 rows x 256 columns (persistent grid, the tiles of
// one column block behind each other so that its weights stay in L2).  Warps 0..7
// add and write (a lane is a row, four warps a column half), 8 is the TMA producer,
// 9 and 10 issue the products of one accumulator each, 11 brings the scales.  N =
// 256 because an instruction costs 137 cycles there and 92 at N = 128.  A block
// takes about 830 cycles: product and commit 566, sums 480, joined by four waits,
// with two accumulators to overlap them.
template <int BN, bool LORA>
struct WideCfg {
  static constexpr int kStages = 4;
  static constexpr int kStageBytes = (kTileM + BN) * kBlockK;
  static constexpr int kAccs = 512 / BN;          // TMEM ring: 512 columns
  // an issuer waits for every phase of the stages that it waits for at all
  static_assert(kStages % kAccs == 0, "a stage's blocks are all of one accumulator");
  static constexpr int kCols = BN / 2;            // columns of a tile an accumulation warp holds
  static constexpr int kOffOut = kStages * kStageBytes;  // 32 rows x 64 B of output per accumulation warp
  static constexpr int kScaleSlots = 4;                  // ring of the scales of four blocks: 128 rows, 2 column halves
  static constexpr int kScaleBytes = 4 * (kTileM + 2) * 4;  // per block: the rows', the halves'
  static constexpr int kOffScales = kOffOut + kAccWarps * 2048;
  static constexpr int kOffBars = kOffScales + kScaleSlots * kScaleBytes;
  // LORA: of two tiles, how many blocks their adapters have, the adapters, the rows' own
  static constexpr int kOffLists = kOffBars + 256;
  static constexpr int kListWords = 4 + 2 * kTileM;
  static constexpr int kSmem = 1024 + kOffLists + (LORA ? 2 * kListWords * 4 : 0);
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
  // The adapters' blocks of a shared tile are the second CTA's, which has the fewer others.
  __device__ __forceinline__ bool adapters_too() const { return !SPLIT || (blockIdx.x & 1); }
  __device__ __forceinline__ int row(long long tile) const { return static_cast<int>(tile % m_tiles) * kTileM; }
  __device__ __forceinline__ int column(long long tile) const { return static_cast<int>(tile / m_tiles) * BN; }
};

// The adapters' blocks of a tile.  The lists are there when the previous launch is done,
// which is waited for behind the first tile's other blocks; later tiles' counts are asked
// for ahead of theirs.
template <bool SPLIT>
struct TileAdapters {
  const LoraParams<true>& lo;
  const Share<256, SPLIT>& mine;
  const int* list;
  int count;
  __device__ __forceinline__ TileAdapters(const LoraParams<true>& lo, const Share<256, SPLIT>& mine) : lo(lo), mine(mine) {}
  __device__ __forceinline__ void look(long long tile) {
    list = lo.lists + static_cast<long long>(mine.row(tile) / kTileM) * kLoraListWords;
    if (tile != mine.first) count = list[0];
  }
  __device__ __forceinline__ int blocks(long long tile) {
    if (tile == mine.first) {
      pdl_wait();
      count = list[0];
    }
    return mine.adapters_too() ? count * lo.pieces : 0;
  }
  __device__ __forceinline__ LoraBlock at(int i) const { return LoraBlock(lo, list, i); }
};

// The accumulation warps' part: sums each tile in registers and writes it.
// False when a wait gave up (the same in a warp's lanes).
template <int BN, int OUT, bool SPLIT, bool LORA>
__device__ __forceinline__ bool accumulate_and_store(const CUtensorMap& map_out, const LinearParams& p,
                                                     const LoraParams<LORA>& lo, uint8_t* smem,
                                                     uint32_t tmem, uint64_t* tfull, uint64_t* tempty, uint64_t* empty,
                                                     uint64_t* sfull, uint64_t* sempty, uint64_t* lfull, uint64_t* lempty,
                                                     volatile int* s_abort) {
  using Cfg = WideCfg<BN, LORA>;
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
  uint32_t n_tile = 0;     // tiles so far, LORA only
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
    if constexpr (LORA) {
      // from shared memory: what is held through the loop above costs it its registers
      // (4,096 x 2,048 x 32,768 without an adapter: 290 us, 246 so)
      const int* list = reinterpret_cast<const int*>(smem + Cfg::kOffLists) + (n_tile & 1) * Cfg::kListWords;
      if (!__all_sync(0xffffffffu, wait(&lfull[n_tile & 1], (n_tile >> 1) & 1, s_abort))) return false;
      const int extra = list[0], own = list[4 + kTileM + r];
#pragma unroll 1
      for (int i = 0, j = 0, k = 0; i < extra; ++i, ++it) {
        const bool add = list[4 + j] == own;
        const uint32_t adds = __ballot_sync(0xffffffffu, add);
        if (++k == lo.pieces) {
          k = 0;
          ++j;
        }
        if (!__all_sync(0xffffffffu, wait(&tfull[it % NA], (it / NA) & 1, s_abort))) return false;
        tc_fence_after();
        if (warp == 0 && lane == 0) mbar_arrive(&empty[it % S]);
        const uint32_t ta = taddr + (it % NA) * BN;
        if (adds == 0) {  // none of the warp's rows
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&tempty[it % NA]);
          continue;
        }
#pragma unroll
        for (int c = 0; c < C / 16; ++c) {
          uint32_t v[16];
          tmem_ld32x16_async(ta + c * 16, v);
          tmem_wait_ld16(v);
          if (c + 1 == C / 16) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&tempty[it % NA]);
          }
          if (add) {  // another row's products are left alone, whatever they are
#pragma unroll
            for (int k = 0; k < 16; k += 2) {
              const float2 sum = unpack_f32x2(add_f32x2(pack_f32x2(__uint_as_float(v[k]), __uint_as_float(v[k + 1])),
                                                        pack_f32x2(y[c * 16 + k], y[c * 16 + k + 1])));
              y[c * 16 + k] = sum.x;
              y[c * 16 + k + 1] = sum.y;
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&lempty[n_tile & 1]);
      ++n_tile;
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

template <int BN, int OUT, bool SPLIT, bool LORA>
__global__ void __launch_bounds__(kThreads, 1)
    fp8_linear_wide_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                           const __grid_constant__ CUtensorMap map_out, const __grid_constant__ LinearParams p,
                           const __grid_constant__ LoraParams<LORA> lo) {
  using Cfg = WideCfg<BN, LORA>;
  constexpr int S = Cfg::kStages, NA = Cfg::kAccs, C = Cfg::kCols, SS = Cfg::kScaleSlots;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + Cfg::kOffBars);
  uint64_t* empty = full + S;
  uint64_t* tfull = empty + S;
  uint64_t* tempty = tfull + NA;
  uint64_t* sfull = tempty + NA;
  uint64_t* sempty = sfull + SS;
  uint64_t* lfull = sempty + SS;  // LORA: the lists of two tiles
  uint64_t* lempty = lfull + 2;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(lempty + 2);
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
    for (int i = 0; i < (LORA ? 2 : 0); ++i) {
      mbar_init(&lfull[i], 1);
      mbar_init(&lempty[i], kAccWarps);
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
  if constexpr (!LORA) {  // else the previous launch is lora.cu's, behind the launch that wrote x
    pdl_wait();
    pdl_trigger();  // every CTA holds its TMEM
  }
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
        if constexpr (LORA) {  // the adapters' blocks
          if (!ok) break;
          TileAdapters<SPLIT> adapters(lo, mine);
          adapters.look(tile);
          const int extra = adapters.blocks(tile);
          for (int i = 0; i < extra; ++i, ++it) {
            const LoraBlock at = adapters.at(i);
            const int s = static_cast<int>(it % S);
            if (!(ok = mbar_wait(&empty[s], static_cast<uint32_t>((it / S) & 1) ^ 1u, s_abort))) break;
            uint8_t* dst = smem + s * Cfg::kStageBytes;
            at.expect(lo, &full[s], BN);
            at.copy_v(lo, dst, &full[s], t0, p.T, keep);
            at.copy_b(lo, dst, &full[s], n0, p.N, keep);
          }
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
      // this accumulator's next product: `issue` makes it
      auto block = [&](auto&& issue) {
        if (!wait(&full[s], phase, s_abort)) return false;
        const uint64_t ad = x_desc + s * kStageDesc, bd = w_desc + s * kStageDesc;
        if (!wait(&tempty[a], a_phase, s_abort)) return false;
        tc_fence_after();
        issue(ad, bd);
        mma_commit(&tfull[a]);
        a_phase ^= 1;
        s += NA;
        if (s >= S) {
          s -= S;
          phase ^= 1;
        }
        return true;
      };
      auto codes = [&](uint64_t ad, uint64_t bd) {
#pragma unroll
        for (int k = 0; k < 4; ++k)  // 32 B of the swizzled rows a step
          mma_e4m3(d, ad + 2 * k, bd + 2 * k, idesc, k > 0 ? 1u : 0u);
      };
      if constexpr (LORA) {
        constexpr uint32_t idesc_b = idesc_bf16_f32(kTileM, BN, 0, 0);
        int next = a;  // blocks until this accumulator's next one
        TileAdapters<SPLIT> adapters(lo, mine);
        for (long long tile = mine.first; tile < mine.tiles && ok; tile += mine.step) {
          adapters.look(tile);
          for (; next < blocks && ok; next += NA) ok = block(codes);
          next -= blocks;
          const int extra = adapters.blocks(tile);
          for (; next < extra && ok; next += NA) {
            const LoraBlock at = adapters.at(next);
            ok = block([&](uint64_t, uint64_t) {
              at.products<true>(lo, d, smem + s * Cfg::kStageBytes, idesc_b);
            });
          }
          next -= extra;
        }
      } else {
        for (long long i = a; i < all && ok; i += NA) ok = block(codes);
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
    uint32_t n_tile = 0;
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
      if constexpr (LORA) {  // the tile's adapters and its rows', behind its last scales
        if (!ok) break;
        if (tile == mine.first) {
          pdl_wait();
          pdl_trigger();  // every CTA holds its TMEM
        }
        const int slot = static_cast<int>(n_tile & 1);
        ok = __all_sync(0xffffffffu, mbar_wait(&lempty[slot], static_cast<uint32_t>((n_tile >> 1) & 1) ^ 1u, s_abort));
        if (!ok) break;
        ++n_tile;
        int* dst = reinterpret_cast<int*>(smem + Cfg::kOffLists) + slot * Cfg::kListWords;
        const int* src = lo.lists + static_cast<long long>(t0 / kTileM) * kLoraListWords;
        const int count = mine.adapters_too() ? src[0] : 0;
        if (lane == 0) dst[0] = count * lo.pieces;
#pragma unroll
        for (int i = lane; i < kTileM; i += 32) {
          if (i < count) dst[4 + i] = src[4 + i];
          // a row without an adapter has none of the list's
          dst[4 + kTileM + i] = t0 + i < p.T ? __ldg(lo.row_adapter + t0 + i) : -1;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&lfull[slot]);
      }
    }
    if (!ok) {
      *s_abort = 1;
      set_error(p.err, kErrTimeout);
    }
  } else {
    if (!accumulate_and_store<BN, OUT, SPLIT, LORA>(map_out, p, lo, smem, tmem, tfull, tempty, empty, sfull, sempty,
                                                    lfull, lempty, s_abort)) {
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

// With adapters: their inner products, and the lists of tiles of 128 rows, are launched
// first and described to the projection with tiles of `rows` rows and `columns` columns and
// stages of `stage` bytes.  Nothing without.
cudaError_t prepare_lora(const NoLora&, LoraParams<false>*, int, int, int, long long, const DeviceCtx&, cudaStream_t, const char**) {
  return cudaSuccess;
}
cudaError_t prepare_lora(const WithLora& l, LoraParams<true>* lo, int rows, int columns, int stage, long long ctas,
                         const DeviceCtx& ctx, cudaStream_t st, const char** why) {
  const csa2_lora_linear_args& a = *l.args;
  const LoraInner to = lora_inner_at(a, l.workspace, rows == kTileM);
  lo->n_adapters = a.n_adapters;
  lo->rank = a.rank;
  lo->row_adapter = a.row_adapter;
  lo->lists = to.lists;
  lo->planes = lora_planes(a.base.out_format);
  // The ranks of a block are 64 where b and all planes of v fit a stage, else 32 (they do with 3 x
  // 128 rows).  Up to 64 rows take as many of a tile of 128 (64 x 2,048 x 32,768 with 16 adapters of
  // rank 64: 31.6 us, 45.6 with 128 and so 32 ranks; rank 32: 25.6 and 27.2).
  lo->v_rows = a.base.T <= 64 && rows > 64 ? 64 : rows;
  lo->run = (lo->planes * lo->v_rows + columns) * 128 <= stage ? 64 : 32;
  lo->pieces = (a.rank + lo->run - 1) / lo->run;
  const uint64_t row = 2 * static_cast<uint64_t>(a.rank);
  const uint64_t v_row = 2 * static_cast<uint64_t>(lora_pitch(a.rank));
  const uint64_t v_all = lo->planes * static_cast<uint64_t>(a.base.T), b_rows = static_cast<uint64_t>(a.n_adapters) * a.base.N;
  auto encode = [&](int bytes, CUtensorMap* v, CUtensorMap* b) {
    const CUtensorMapSwizzle swizzle = bytes == 32   ? CU_TENSOR_MAP_SWIZZLE_32B
                                       : bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                                     : CU_TENSOR_MAP_SWIZZLE_128B;
    return encode_tmap_2d_u8(v, to.v, v_row, v_all, v_row, bytes, lo->v_rows, swizzle) == CUDA_SUCCESS &&
           encode_tmap_2d_u8(b, a.b, row, b_rows, row, bytes, columns, swizzle) == CUDA_SUCCESS;
  };
  const int last = a.rank % lo->run;
  if ((a.rank >= lo->run && !encode(2 * lo->run, &lo->map_v, &lo->map_b)) ||
      (last && !encode(lora_row_bytes(last), &lo->map_v_last, &lo->map_b_last))) {
    *why = "csa2_lora_linear: a tensor map could not be encoded";
    return cudaErrorInvalidValue;
  }
  return launch_lora_inner(a, to, static_cast<int>(ctas < ctx.num_sms ? ctas : ctx.num_sms), ctx, st, why);
}

template <int BN, int OUT, bool SPLIT, class L>
cudaError_t launch_wide(const csa2_fp8_linear_args& a, const LinearParams& p, const L& lora, const DeviceCtx& ctx,
                        cudaStream_t st, const char** why) {
  CUtensorMap map_x, map_w, map_out = {};
  if (encode_tmap_2d_u8(&map_x, a.x, a.K, a.T, a.ld_x, kBlockK, kTileM) != CUDA_SUCCESS ||
      encode_tmap_2d_u8(&map_w, a.w, a.K, a.N, a.ld_w, kBlockK, BN) != CUDA_SUCCESS ||
      (p.vec && encode_tmap_2d_u8(&map_out, a.out, static_cast<uint64_t>(a.N) * out_size(OUT), a.T,
                                  a.ld_out * out_size(OUT), 64, 32, CU_TENSOR_MAP_SWIZZLE_64B) != CUDA_SUCCESS)) {
    *why = "csa2_fp8_linear: a tensor map could not be encoded";
    return cudaErrorInvalidValue;
  }
  auto kern = fp8_linear_wide_kernel<BN, OUT, SPLIT, L::kOn>;
  cudaError_t e = prefer_max_smem_once<fp8_linear_wide_kernel<BN, OUT, SPLIT, L::kOn>>(ctx.device, WideCfg<BN, L::kOn>::kSmem);
  if (e != cudaSuccess) return e;
  LoraParams<L::kOn> lo{};
  e = prepare_lora(lora, &lo, kTileM, BN, WideCfg<BN, L::kOn>::kStageBytes, SPLIT ? 2 * wide_tiles<BN>(a) : wide_tiles<BN>(a), ctx, st, why);
  if (e != cudaSuccess) return e;
  const long long tiles = wide_tiles<BN>(a);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(SPLIT ? 2 * tiles : (tiles < ctx.num_sms ? tiles : ctx.num_sms)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = WideCfg<BN, L::kOn>::kSmem;
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
  return cudaLaunchKernelEx(&cfg, kern, map_x, map_w, map_out, p, lo);
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

// Of n blocks, those that a cluster's CTA `rank` takes: rank, rank + splits, ..
__device__ __forceinline__ int shares_of(int n, int rank, int splits) { return n > rank ? (n - rank - 1) / splits + 1 : 0; }

template <int NT, int OUT, bool LORA>
struct NarrowCfg {
  static constexpr int kStages = 4;
  static constexpr int kBlockBytes = (128 + NT) * kBlockK;
  // room for a block of 64 ranks in two planes (16 x 2,048 x 32,768 with 16 adapters of rank 64:
  // 26.4 us, 32.1 with blocks of 32 ranks in stages of kBlockBytes; 32 rows: 32.7 and 41.2)
  static constexpr int kStageBytes = LORA && lora_planes(OUT) == 2 ? (128 + 2 * NT) * 128 : kBlockBytes;
  static constexpr int kAccs = 4;
  static constexpr int kCols = kAccs * NT < 32 ? 32 : kAccs * NT;
  static constexpr int kOffScales = kStages * kStageBytes;  // the parts [NT][128] reuse the stages
  static constexpr int kOffBars = kOffScales + kScaleSeg * NT * 4;
  // LORA: the tile's adapters and its rows' own
  static constexpr int kOffLists = kOffBars + 256;
  static constexpr int kSmem = 1024 + kOffLists + (LORA ? (4 + 2 * NT) * 4 : 0);
  static_assert(NT * 128 * 4 <= kOffScales, "the parts fit the stages");
};

template <int NT, int OUT, bool LORA>
__global__ void __launch_bounds__(kNarrowThreads, NT == 64 ? 1 : 2)
    fp8_linear_narrow_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                             const __grid_constant__ LinearParams p, const __grid_constant__ LoraParams<LORA> lo) {
  using Cfg = NarrowCfg<NT, OUT, LORA>;
  constexpr int S = Cfg::kStages, NA = Cfg::kAccs;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + Cfg::kOffBars);
  uint64_t* empty = full + S;
  uint64_t* tfull = empty + S;
  uint64_t* tempty = tfull + NA;
  uint64_t* lready = tempty + NA;  // LORA: the tile's adapters
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(lready + 1);
  volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
  int* s_list = reinterpret_cast<int*>(smem + Cfg::kOffLists);  // [4 + NT], then [NT], LORA only
  int* s_own = s_list + 4 + NT;
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
    if (LORA) mbar_init(lready, 1);
    fence_mbar_init();
    prefetch_tmap(&map_x);
    prefetch_tmap(&map_w);
    if (LORA || p.w_ready) {  // the first weights do not wait for the previous launch
      for (int b = 0; b < min(S, blocks); ++b) {
        mbar_arrive_expect_tx(&full[b], Cfg::kBlockBytes);
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
  if constexpr (!LORA) {  // else the previous launch is lora.cu's, behind the launch that wrote x
    pdl_wait();
    pdl_trigger();  // every CTA holds its TMEM
  }
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
        if (b >= S || !(LORA || p.w_ready)) {
          mbar_arrive_expect_tx(&full[s], Cfg::kBlockBytes);
          tma_load_2d(dst, &map_w, (b0 + b) * kBlockK, n0, &full[s], pol_w);
        }
        tma_load_2d(dst + 128 * kBlockK, &map_x, (b0 + b) * kBlockK, t0, &full[s], pol_x);
      }
      if constexpr (LORA) {  // the adapters' blocks: only v waits for the previous launch
        ok = ok && mbar_wait(lready, 0u, s_abort);
        const int extra = ok ? shares_of(s_list[0] * lo.pieces, rank, splits) : 0;
        const int ahead = min(extra, S);
        for (int i = 0; i < ahead; ++i, ++b) {
          const int s = b % S;
          if (b >= S && !(ok = mbar_wait(&empty[s], static_cast<uint32_t>(b / S - 1) & 1u, s_abort))) break;
          const LoraBlock at(lo, s_list, rank + i * splits);
          at.expect(lo, &full[s], 128);
          at.copy_b(lo, smem + s * Cfg::kStageBytes, &full[s], n0, p.N, pol_x);
        }
        if (b > blocks) pdl_wait();
        for (int i = 0; blocks + i < b; ++i) {
          const int s = (blocks + i) % S;
          LoraBlock(lo, s_list, rank + i * splits).copy_v(lo, smem + s * Cfg::kStageBytes, &full[s], t0, p.T, pol_x);
        }
        for (int i = ahead; ok && i < extra; ++i, ++b) {
          const int s = b % S;
          if (!(ok = mbar_wait(&empty[s], static_cast<uint32_t>(b / S - 1) & 1u, s_abort))) break;
          const LoraBlock at(lo, s_list, rank + i * splits);
          at.expect(lo, &full[s], 128);
          at.copy_b(lo, smem + s * Cfg::kStageBytes, &full[s], n0, p.N, pol_x);
          at.copy_v(lo, smem + s * Cfg::kStageBytes, &full[s], t0, p.T, pol_x);
        }
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
      auto block = [&](auto&& issue) {  // block b's products: `issue` makes them
        const int s = b % S, a = b % NA;
        if (!mbar_wait(&full[s], static_cast<uint32_t>(b / S) & 1u, s_abort)) return false;
        if (b >= NA && !mbar_wait(&tempty[a], static_cast<uint32_t>(b / NA - 1) & 1u, s_abort)) return false;
        tc_fence_after();
        issue(tmem + a * NT, smem_desc_sw128(smem + s * Cfg::kStageBytes),
              smem_desc_sw128(smem + s * Cfg::kStageBytes + 128 * kBlockK));
        mma_commit(&tfull[a]);
        ++b;
        return true;
      };
      while (b < blocks && ok)
        ok = block([&](uint32_t d, uint64_t wd, uint64_t xd) {
#pragma unroll
          for (int k = 0; k < 4; ++k) mma_e4m3(d, wd + 2 * k, xd + 2 * k, idesc, k > 0 ? 1u : 0u);
        });
      if constexpr (LORA) {
        constexpr uint32_t idesc_b = idesc_bf16_f32(128, NT, 0, 0);
        ok = ok && mbar_wait(lready, 0u, s_abort);
        const int extra = ok ? shares_of(s_list[0] * lo.pieces, rank, splits) : 0;
        for (int i = 0; ok && i < extra; ++i) {
          const LoraBlock at(lo, s_list, rank + i * splits);
          ok = block([&](uint32_t d, uint64_t, uint64_t) {
            at.products<false>(lo, d, smem + (b % S) * Cfg::kStageBytes, idesc_b);
          });
        }
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
    if constexpr (LORA) {
      if (warp == 2) {
        tile_adapters<NT>(lo, t0, p.T, s_list, s_own);
        if (lane == 0) mbar_arrive(lready);
      }
    }
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
    if constexpr (LORA) {
      pdl_wait();
      pdl_trigger();  // every CTA holds its TMEM
      ok = __all_sync(0xffffffffu, ok && mbar_wait(lready, 0u, s_abort));
      const int extra = ok ? shares_of(s_list[0] * lo.pieces, rank, splits) : 0;
      for (int i = (blocks + group) & 1; i < extra && ok; i += 2) {  // the block's parity is the group, as above
        const int b = blocks + i, a = b % NA;
        const int adapter = s_list[4 + (rank + i * splits) / lo.pieces];
        uint32_t rows[(NT + 31) / 32];  // a bit for each row that has the adapter
#pragma unroll
        for (int h = 0; h < (NT + 31) / 32; ++h)
          rows[h] = __ballot_sync(0xffffffffu, h * 32 + lane < NT && s_own[h * 32 + lane] == adapter);
        ok = __all_sync(0xffffffffu, mbar_wait(&tfull[a], static_cast<uint32_t>(b / NA) & 1u, s_abort));
        if (!ok) break;
        tc_fence_after();
        if (quad == 0 && lane == 0) mbar_arrive(&empty[b % S]);
#pragma unroll
        for (int c = 0; c < NT / 16; ++c) {
          const uint32_t mine = rows[c / 2] >> (c % 2 * 16);
          if (!(mine & 0xFFFFu)) continue;
          uint32_t v[16];
          tmem_ld32x16_async(taddr + a * NT + c * 16, v);
          tmem_wait_ld16(v);
#pragma unroll
          for (int k = 0; k < 16; k += 2) {  // another row's products are left alone, whatever they are
            float2 f = unpack_f32x2(acc[c * 8 + k / 2]);
            if (mine >> k & 1u) f.x += __uint_as_float(v[k]);
            if (mine >> (k + 1) & 1u) f.y += __uint_as_float(v[k + 1]);
            acc[c * 8 + k / 2] = pack_f32x2(f.x, f.y);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tempty[a]);
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
template <int NT, int OUT, bool LORA>
int narrow_clusters(const cudaLaunchConfig_t& cfg, int splits, int device) {
  constexpr auto kern = fp8_linear_narrow_kernel<NT, OUT, LORA>;
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
template <int NT, int OUT, class L>
cudaError_t launch_narrow(const csa2_fp8_linear_args& a, const LinearParams& p, const L& lora, const DeviceCtx& ctx,
                          cudaStream_t st, const char** why, bool* taken) {
  constexpr int kSmem = NarrowCfg<NT, OUT, L::kOn>::kSmem;
  auto kern = fp8_linear_narrow_kernel<NT, OUT, L::kOn>;
  const long long n_tiles = (static_cast<long long>(a.N) + 127) / 128;
  const int t_tiles = (a.T + NT - 1) / NT, blocks = (a.K + 127) / 128;
  *taken = NT < 64 || n_tiles * t_tiles <= ctx.num_sms;
  if (!*taken) return cudaSuccess;
  cudaError_t e = prefer_max_smem_once<fp8_linear_narrow_kernel<NT, OUT, L::kOn>>(ctx.device, kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kNarrowThreads);
  cfg.dynamicSmemBytes = kSmem;
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
                                                        : tiles <= narrow_clusters<NT, OUT, L::kOn>(cfg, splits, ctx.device)))
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
  LoraParams<L::kOn> lo{};
  e = prepare_lora(lora, &lo, NT, 128, NarrowCfg<NT, OUT, L::kOn>::kStageBytes, tiles * splits, ctx, st, why);
  if (e != cudaSuccess) return e;
  return cudaLaunchKernelEx(&cfg, kern, map_x, map_w, p, lo);
}

template <int OUT, class L>
cudaError_t launch_out(const csa2_fp8_linear_args& a, const LinearParams& p, const L& lora, const DeviceCtx& ctx,
                       cudaStream_t st, const char** why) {
  bool taken = false;
  cudaError_t e = a.T <= 16   ? launch_narrow<16, OUT>(a, p, lora, ctx, st, why, &taken)
                  : a.T <= 32 ? launch_narrow<32, OUT>(a, p, lora, ctx, st, why, &taken)
                              : launch_narrow<64, OUT>(a, p, lora, ctx, st, why, &taken);
  if (e != cudaSuccess || taken) return e;
  // Tiles for less than half the SMs share their blocks between two CTAs (4,096 x
  // 7,168 x 512: 28.9 -> 19.9 us).
  return wide_splits(a, ctx) ? launch_wide<256, OUT, true>(a, p, lora, ctx, st, why)
                             : launch_wide<256, OUT, false>(a, p, lora, ctx, st, why);
}

template <class L>
cudaError_t launch_linear(const csa2_fp8_linear_args& a, const L& lora, const DeviceCtx& ctx, cudaStream_t st,
                          const char** why) {
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
    case CSA2_OUT_F32: return launch_out<CSA2_OUT_F32>(a, p, lora, ctx, st, why);
    case CSA2_OUT_BF16: return launch_out<CSA2_OUT_BF16>(a, p, lora, ctx, st, why);
    default: return launch_out<CSA2_OUT_FP8>(a, p, lora, ctx, st, why);
  }
}

}  // namespace

cudaError_t launch_fp8_linear(const csa2_fp8_linear_args& a, const DeviceCtx& ctx, cudaStream_t st, const char** why) {
  return launch_linear(a, NoLora{}, ctx, st, why);
}
cudaError_t launch_lora_linear(const csa2_lora_linear_args& a, void* ws, const DeviceCtx& ctx, cudaStream_t st,
                               const char** why) {
  return launch_linear(a.base, WithLora{&a, ws}, ctx, st, why);
}

}  // namespace csa2
