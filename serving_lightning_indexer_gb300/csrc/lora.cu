// Inner products of low-rank adapters with the rows that use them,
//   v[t][r] = s[i] * sum_b x_scale[t][b] * sum_{k in b} x[t][k] a[i][r][k],  i = row_adapter[t],
// and the list of adapters that each 128 rows of the projection need.  The
// projection (fp8_linear.cu) adds v[t] b[i]^T to its sums before RoPE and rounding.
//
// The codes are exact in bf16 and a is bf16, so a block's 128 products are summed by
// the tensor core in fp32 and the block's scale is applied to the sum.  The result is
// written as the bf16 nearest to it, the bf16 nearest to what that leaves (at most 2^-17 of it is
// left, for bf16 output next to nothing) and, but for bf16 output, what that leaves: two would leave
// fp32 output 2^-17 of v off, and e4m3 output, where a code on the other side of its border is
// 2^-3 off however near the border was, three times the codes there that fp32's own roundings do.
//
// Two kernels, both bound by latency: launch, ids, operands, products, sums.  For few rows
// a CTA takes 16 of them, one of their adapters and 8 of its ranks, its 8 to 32 warps the
// blocks of 128 input dims in turn, added in warp order: 8 x 7,168 x 512 with 8 adapters
// takes 8.4 us with its projection, 4.7 without adapters.  For many a CTA takes 128 rows,
// 64 ranks and a share of the input dims, and goes through the tile's adapters with a in a
// ring in shared memory; a cluster adds the shares in rank order: about 12 us of the 292 of
// 4,096 x 2,048 x 32,768 at rank 64.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "csa2_device.cuh"
#include "csa2_internal.h"

namespace csa2 {
namespace {

struct InnerParams {
  const uint8_t* x;
  const float* x_scale;
  const uint16_t* a;
  const float* adapter_scale;
  const int* row_adapter;
  uint16_t* v;  // [planes][T][pitch]: the bf16 values, what they leave, and what that leaves
  int* lists;  // NULL: the projection's tiles are smaller and make their own
  long long ld_x, ld_xs;
  int T, K, rank, pitch, n_adapters;
  int planes;  // 2 or 3
  int ready;   // a and row_adapter may be read before the previous launch completes
  uint32_t* err;
};

// Two e4m3 codes (the low half of c) as bf16, exactly; a NaN code is NaN.
__device__ __forceinline__ uint32_t bf16_of_e4m3x2(uint32_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(c)));
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
  return *reinterpret_cast<const uint32_t*>(&b);
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The adapters among 128 rows, each once, in the order of their first rows: list[0] how
// many, list[4 ..] which.  All threads, 128 or more.
__device__ __forceinline__ void write_list(const InnerParams& p, long long t0, int* list, int* s_id, int* s_base) {
  constexpr int n = 128;
  const int i = threadIdx.x, lane = i & 31;
  int id = -1;
  if (i < n && t0 + i < p.T) {
    id = __ldg(p.row_adapter + t0 + i);
    if (id < -1 || id >= p.n_adapters) {
      set_error(p.err, kErrBounds);
      id = -1;
    }
  }
  if (i < n) s_id[i] = id;
  __syncthreads();
  // the first of its warp with this adapter, and none of an earlier warp has it
  const uint32_t same = __match_any_sync(0xffffffffu, id);
  bool first = id >= 0 && __ffs(same) - 1 == lane;
  const int before = min(i & ~31, n);
#pragma unroll 8
  for (int j = 0; j < before; j += 4) {
    const int4 v = *reinterpret_cast<const int4*>(s_id + j);
    first = first & (v.x != id) & (v.y != id) & (v.z != id) & (v.w != id);
  }
  const uint32_t mask = __ballot_sync(0xffffffffu, first);
  if (lane == 0) s_base[i >> 5] = __popc(mask);
  __syncthreads();
  int at = 0;
  for (int w = 0; w < (i >> 5); ++w) at += s_base[w];
  if (first) list[4 + at + __popc(mask & ((1u << lane) - 1))] = id;
  if (i == static_cast<int>(blockDim.x) - 1) list[0] = at + __popc(mask);
  __syncthreads();
}

// Writes v of a row and N ranks from `rank` on, in as many bf16 as there are planes.  An
// infinite or NaN value is all in the first; a finite one past bf16's range keeps bf16's largest
// there, where rounding to nearest would make it an infinity.
template <int N>
__device__ __forceinline__ void store_v(const InnerParams& p, long long row, int rank, float (&v)[N]) {
  uint16_t* to = p.v + row * p.pitch + rank;
  for (int plane = 0; plane < p.planes; ++plane, to += static_cast<long long>(p.T) * p.pitch) {
    alignas(8) uint16_t h[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
      __nv_bfloat16 b = __float2bfloat16_rn(v[k]);
      if (__hisinf(b)) b = __float2bfloat16_rz(v[k]);  // of an infinity, itself
      const float rest = v[k] - __bfloat162float(b);
      v[k] = isfinite(rest) ? rest : 0.f;
      h[k] = *reinterpret_cast<const uint16_t*>(&b);
    }
    if constexpr (N == 4) *reinterpret_cast<uint2*>(to) = *reinterpret_cast<const uint2*>(h);
    else to[0] = h[0];
  }
}

// W warps: 8, 16 or 32.
template <int W>
__global__ void __launch_bounds__(W * 32) lora_inner_kernel(const __grid_constant__ InnerParams p) {
  __shared__ float part[W][16][8];
  __shared__ __align__(16) int s_id[128];
  __shared__ int s_base[W];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (!p.ready) pdl_wait();
  const int t0 = blockIdx.x * 16;
  // the blockIdx.z-th adapter among the 16 rows
  int id = -1;
  if (lane < 16 && t0 + lane < p.T) id = __ldg(p.row_adapter + t0 + lane);
  if (id < -1 || id >= p.n_adapters) {
    if (blockIdx.y == 0 && blockIdx.z == 0) set_error(p.err, kErrBounds);
    id = -1;
  }
  const uint32_t same = __match_any_sync(0xffffffffu, id);
  uint32_t firsts = __ballot_sync(0xffffffffu, id >= 0 && __ffs(same) - 1 == lane);
  for (int j = blockIdx.z; j > 0; --j) firsts &= firsts - 1;
  const int adapter = __shfl_sync(0xffffffffu, id, firsts ? __ffs(firsts) - 1 : 0);
  if (!p.ready) pdl_trigger();
  if (p.lists && blockIdx.y == 0 && blockIdx.z == 0 && t0 % 128 == 0) {
    if (p.ready) {  // the last call's projection may still read its lists
      pdl_wait();
      pdl_trigger();
    }
    write_list(p, t0, p.lists + static_cast<long long>(t0 / 128) * kLoraListWords, s_id, s_base);
  }
  if (!firsts) {
    if (p.ready) {
      pdl_wait();
      pdl_trigger();
    }
    return;
  }

  const int g = lane >> 2, q = lane & 3, r0 = blockIdx.y * 8;
  const int blocks = r0 < p.rank ? (p.K + 127) / 128 : 0;
  const uint16_t* a = p.a + (static_cast<long long>(adapter) * p.rank + r0 + g) * p.K + q * 8;
  const int ra = min(t0 + g, p.T - 1), rb = min(t0 + g + 8, p.T - 1);
  const uint8_t* xa = p.x + ra * p.ld_x + q * 8;
  const uint8_t* xb = p.x + rb * p.ld_x + q * 8;
  float sum[4] = {0.f, 0.f, 0.f, 0.f};
  // The order of the products of a block is free: a lane holds 8 dims in a row of each
  // 32, which the fragments of two steps take as their four pairs.
  uint4 av[4];
  auto load_a = [&](int b) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int k = b * 128 + c * 32;
      av[c] = k + q * 8 < p.K ? __ldg(reinterpret_cast<const uint4*>(a + k)) : make_uint4(0, 0, 0, 0);
    }
  };
  if (p.ready) {  // the first block of a does not wait for the previous launch
    if (warp < blocks) load_a(warp);
    pdl_wait();
    pdl_trigger();
  }
  for (int b = warp; b < blocks; b += W) {
    if (!p.ready || b != warp) load_a(b);
    uint2 xv[4], yv[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int k = b * 128 + c * 32;
      const bool in = k + q * 8 < p.K;
      xv[c] = in ? __ldg(reinterpret_cast<const uint2*>(xa + k)) : make_uint2(0, 0);
      yv[c] = in ? __ldg(reinterpret_cast<const uint2*>(xb + k)) : make_uint2(0, 0);
    }
    const float sa = __ldg(p.x_scale + ra * p.ld_xs + b), sb = __ldg(p.x_scale + rb * p.ld_xs + b);
    float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      mma_bf16(d, bf16_of_e4m3x2(xv[c].x), bf16_of_e4m3x2(yv[c].x), bf16_of_e4m3x2(xv[c].x >> 16),
               bf16_of_e4m3x2(yv[c].x >> 16), av[c].x, av[c].y);
      mma_bf16(d, bf16_of_e4m3x2(xv[c].y), bf16_of_e4m3x2(yv[c].y), bf16_of_e4m3x2(xv[c].y >> 16),
               bf16_of_e4m3x2(yv[c].y >> 16), av[c].z, av[c].w);
    }
    sum[0] = fmaf(sa, d[0], sum[0]);
    sum[1] = fmaf(sa, d[1], sum[1]);
    sum[2] = fmaf(sb, d[2], sum[2]);
    sum[3] = fmaf(sb, d[3], sum[3]);
  }
  part[warp][g][2 * q] = sum[0];
  part[warp][g][2 * q + 1] = sum[1];
  part[warp][g + 8][2 * q] = sum[2];
  part[warp][g + 8][2 * q + 1] = sum[3];
  __syncthreads();
  if (tid < 128) {
    const int i = tid >> 3, r = tid & 7;
    if (t0 + i < p.T && __ldg(p.row_adapter + t0 + i) == adapter) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) v += part[w][i][r];
      if (p.adapter_scale) v *= __ldg(p.adapter_scale + adapter);
      float one[1] = {v};
      store_v(p, t0 + i, r0 + r, one);
    }
  }
}

// ---------------------------------------------------------------- many rows
// Products on tcgen05: with many adapters in a tile each of them is a product with all 128
// rows, several times what the rows need.  Each block of 128 input dims of the CTA's rows becomes bf16
// in a ring in shared memory; each adapter's block of a comes by tensor copies; each of
// these pairs is a product of its own, which eight warps (a lane is a row, four warps
// half the ranks) add, times the row's scale, to the sums of the rows that have the
// adapter.  So a row's sums stay in registers throughout.
constexpr int kTileRows = 128, kTileRanks = 64, kTileStages = 4, kTileXStages = 3, kTileRaw = 4, kTileAccs = 4;
constexpr int kSumWarps = 8, kConvertWarps = 8, kCopyWarp = kSumWarps + kConvertWarps, kIssueWarp = kCopyWarp + 1;
constexpr int kTileWarps = kIssueWarp + 1;
constexpr int kTileXBytes = kTileRows * 256;  // a block of x: two halves of 64 dims, rows of 128 bytes
constexpr int kTileOffRaw = kTileXStages * kTileXBytes;  // blocks of codes, a lane's own words side by side; then the sums
static_assert(kTileRows * kTileRanks * 4 <= kTileRaw * kTileRows * 128, "the sums fit where the codes were");
constexpr int kTileOffA = kTileOffRaw + kTileRaw * kTileRows * 128;
constexpr int kTileABytes = 3 * kTileRanks * 256;  // the ring of blocks of a: three of 64 ranks, four of 48
// Rows' scales, of the blocks between the farthest copied one and the first that a sum warp may
// still have to read.  A converting warp asks for block b + kTileRaw - 1 when it has seen the
// products of block b - 1 - kTileXStages complete; these were issued when every sum warp was
// done with the product kTileAccs before them, so with one product a block the slowest warp may be
// at block b - kTileXStages - kTileAccs: kTileRaw + kTileXStages + kTileAccs blocks in all.
constexpr int kTileScales = 16, kTileOffScales = kTileOffA + kTileABytes;
static_assert(kTileRaw + kTileXStages + kTileAccs <= kTileScales, "a scale stays until it is used");
constexpr int kTileSmem = 1024 + kTileOffScales + kTileScales * kTileRows * 4;

// Grid: row tiles, shares of the input dims (a cluster), runs of 64 ranks times slots;
// slot z takes the tile's adapters z, z + slots, ..  map_a: a as rows of K, boxes of 64
// dims by `box` ranks (a run's, in sixteens).  G adapters of 16 or 32 ranks share a
// product, 64 columns wide, as its columns have nothing to do with each other (1,024 x
// 7,168 x 512 with 16 adapters of rank 16, all in each tile: 83 us with one, 43 with four).
__global__ void __launch_bounds__(kTileWarps * 32, 1)
    lora_tile_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ InnerParams p, int slots, int box,
                     int stages) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* part = reinterpret_cast<float*>(smem + kTileOffRaw);  // [rows][ranks]: a row's own adapter's sums
  uint8_t* x_ring = smem;
  uint8_t* a_ring = smem + kTileOffA;
  const int G = box <= 32 ? kTileRanks / box : 1, a_bytes = G * box * 256;
  __shared__ __align__(16) int s_id[kTileRows], s_list[kTileRows + 4];
  __shared__ int s_place[kTileRows];  // a row's adapter's place in the list, or -1
  __shared__ int s_base[kTileWarps];
  __shared__ uint64_t s_full[kTileStages], s_empty[kTileStages], s_xfull[kTileXStages], s_xempty[kTileXStages];
  __shared__ uint64_t s_tfull[kTileAccs], s_tempty[kTileAccs];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const long long t0 = static_cast<long long>(blockIdx.x) * kTileRows;
  const int splits = gridDim.y, rank = blockIdx.y;
  if (tid == 0) {
    s_abort = 0;
    for (int i = 0; i < stages; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], 1);
    }
    for (int i = 0; i < kTileXStages; ++i) {
      mbar_init(&s_xfull[i], kConvertWarps);
      mbar_init(&s_xempty[i], 1);
    }
    for (int i = 0; i < kTileAccs; ++i) {
      mbar_init(&s_tfull[i], 1);
      mbar_init(&s_tempty[i], kSumWarps);
    }
    fence_mbar_init();
    prefetch_tmap(&map_a);
  }
  if (warp == kIssueWarp) {
    tmem_alloc(&s_tmem, kTileAccs * kTileRanks);
    tmem_relinquish();
  }
  if (tid < kTileRows) s_list[4 + tid] = -1;
  if (!p.ready) pdl_wait();
  const int slot = blockIdx.z % slots, r0 = blockIdx.z / slots * kTileRanks;
  const int ranks = min(kTileRanks, p.rank - r0), columns = (ranks + 15) & ~15;
  const int all = (p.K + 127) / 128;
  const int b0 = all * rank / splits, nb = all * (rank + 1) / splits - b0;
  tc_fence_before();
  write_list(p, t0, s_list, s_id, s_base);
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  const int n = s_list[0];
  if (tid < kTileRows) {
    const int id = s_id[tid];
    int at = -1;
#pragma unroll 1
    for (int j = 0; j < n; j += 4) {  // -1 behind the list's end
      const int4 v = *reinterpret_cast<const int4*>(s_list + 4 + j);
      at = v.x == id ? j : v.y == id ? j + 1 : v.z == id ? j + 2 : v.w == id ? j + 3 : at;
    }
    s_place[tid] = id >= 0 ? at : -1;
  }
  const int mine = n > slot ? (n - slot - 1) / slots + 1 : 0;  // adapters of this slot
  const int groups = (mine + G - 1) / G;
  __syncthreads();                                             // s_place
  // a is asked for first; what else is read waits for the previous launch
  if (warp != kCopyWarp) {
    if (p.ready) pdl_wait();
    pdl_trigger();  // every CTA holds its TMEM
  }
  bool ok = true;
  if (mine == 0) {
  } else if (warp == kCopyWarp) {
    // ------------------------------------------------------------ a
    if (lane == 0) {
      const uint64_t keep = l2_policy_evict_last();
      int s = 0, sent = 0;
      uint32_t phase = 0;
      for (int b = 0; b < nb && ok; ++b)
        for (int j = 0; j < groups; ++j, ++sent) {
          if (sent >= stages && !(ok = mbar_wait(&s_empty[s], phase ^ 1u, &s_abort))) break;
          const int members = min(G, mine - j * G);
          mbar_arrive_expect_tx(&s_full[s], members * box * 256);
          for (int g = 0; g < members; ++g) {
            const int y = s_list[4 + slot + (j * G + g) * slots] * p.rank + r0;
#pragma unroll
            for (int h = 0; h < 2; ++h)
              tma_load_2d(a_ring + s * a_bytes + h * (a_bytes / 2) + g * box * 128, &map_a, ((b0 + b) * 128 + h * 64) * 2, y,
                          &s_full[s], keep);
          }
          if (++s == stages) {
            s = 0;
            phase ^= 1u;
          }
        }
      if (!ok) {
        s_abort = 1;
        set_error(p.err, kErrTimeout);
      }
      // copies in flight must land before the CTA may exit
      for (int i = 0; i < min(stages, sent); ++i) {
        if (--s < 0) {
          s = stages - 1;
          phase ^= 1u;
        }
        mbar_wait(&s_full[s], phase, nullptr);
      }
    }
  } else if (warp == kIssueWarp) {
    // ------------------------------------------------------------ products
    if (lane == 0) {
      const uint32_t idesc = idesc_bf16_f32(kTileRows, G > 1 ? kTileRanks : columns, 0, 0);
      const uint64_t xd = smem_desc_sw128(x_ring), ad = smem_desc_sw128(a_ring);
      int s = 0;
      uint32_t phase = 0, at = 0;
      for (int b = 0; b < nb && ok; ++b) {
        const int xs = b % kTileXStages;
        if (!(ok = mbar_wait(&s_xfull[xs], static_cast<uint32_t>(b / kTileXStages) & 1u, &s_abort))) break;
        for (int j = 0; j < groups; ++j, ++at) {
          const int acc = static_cast<int>(at % kTileAccs);
          if (!(ok = mbar_wait(&s_full[s], phase, &s_abort))) break;
          if (at >= kTileAccs && !(ok = mbar_wait(&s_tempty[acc], (at / kTileAccs - 1) & 1u, &s_abort))) break;
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < 8; ++k)  // 16 dims each: four to a half
            umma_bf16(tmem + acc * kTileRanks, xd + ((xs * kTileXBytes + (k >> 2) * (kTileXBytes / 2)) >> 4) + (k & 3) * 2,
                      ad + ((s * a_bytes + (k >> 2) * (a_bytes / 2)) >> 4) + (k & 3) * 2, idesc, k > 0 ? 1u : 0u);
          mma_commit(&s_tfull[acc]);
          if (++s == stages) {
            s = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok) {
        s_abort = 1;
        set_error(p.err, kErrTimeout);
        // the last products still read shared memory and write TMEM
        for (uint32_t i = at > kTileAccs ? at - kTileAccs : 0; i < at; ++i)
          mbar_wait(&s_tfull[i % kTileAccs], (i / kTileAccs) & 1u, nullptr);
      }
    }
  } else if (warp >= kSumWarps) {
    // ------------------------------------------------------------ x
    // A lane's 16 codes are two words of the swizzled rows; eight lanes have a row's
    // block, a warp four rows of it at a time.  Codes are copied kTileRaw - 1 blocks ahead
    // to places of the lane's own.  Loops stay rolled: a launch runs this code once, and
    // fetching it takes longer than running it.
    constexpr int kSteps = kTileRows / kConvertWarps / 4;
    const int q = lane & 7, first = (warp - kSumWarps) * (kSteps * 4) + (lane >> 3);
    uint8_t* raw = smem + kTileOffRaw + ((warp - kSumWarps) * 32 + lane) * 16;
    const uint8_t* x = p.x + (t0 + first) * p.ld_x + q * 16;
    auto fetch = [&](int b) {
      const int k = (b0 + b) * 128;
      // nothing, not even zeros, behind the last block: the sums go where the codes were
#pragma unroll 1
      for (int j = 0; b < nb && j < kSteps; ++j) {
        const bool in = t0 + first + j * 4 < p.T && k + q * 16 < p.K;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                         smem_u32(raw + ((b % kTileRaw) * kSteps + j) * kConvertWarps * 512)),
                     "l"(in ? x + j * 4 * p.ld_x + k : p.x), "r"(in ? 16 : 0)
                     : "memory");
      }
      const int r = (warp - kSumWarps) * (kSteps * 4) + lane;
      if (lane < kSteps * 4 && b < nb && t0 + r < p.T)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(
                         smem_u32(smem + kTileOffScales + ((b % kTileScales) * kTileRows + r) * 4)),
                     "l"(p.x_scale + (t0 + r) * p.ld_xs + b0 + b)
                     : "memory");
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll 1
    for (int b = 0; b < kTileRaw - 1; ++b) fetch(b);
#pragma unroll 1
    for (int b = 0; b < nb; ++b) {
      const int xs = b % kTileXStages;
      fetch(b + kTileRaw - 1);
      asm volatile("cp.async.wait_group %0;" ::"n"(kTileRaw - 1) : "memory");
      if (b >= kTileXStages) {
        ok = __all_sync(0xffffffffu, mbar_wait(&s_xempty[xs], static_cast<uint32_t>(b / kTileXStages - 1) & 1u, &s_abort));
        if (!ok) break;
      }
      uint8_t* dst = x_ring + xs * kTileXBytes + (q >> 2) * (kTileXBytes / 2);
#pragma unroll
      for (int j = 0; j < kSteps; ++j) {
        const int r = first + j * 4;
        const uint4 v = *reinterpret_cast<const uint4*>(raw + ((b % kTileRaw) * kSteps + j) * kConvertWarps * 512);
        *reinterpret_cast<uint4*>(dst + r * 128 + (((2 * (q & 3)) ^ (r & 7)) * 16)) =
            make_uint4(bf16_of_e4m3x2(v.x), bf16_of_e4m3x2(v.x >> 16), bf16_of_e4m3x2(v.y), bf16_of_e4m3x2(v.y >> 16));
        *reinterpret_cast<uint4*>(dst + r * 128 + (((2 * (q & 3) + 1) ^ (r & 7)) * 16)) =
            make_uint4(bf16_of_e4m3x2(v.z), bf16_of_e4m3x2(v.z >> 16), bf16_of_e4m3x2(v.w), bf16_of_e4m3x2(v.w >> 16));
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s_xfull[xs]);
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (!ok && lane == 0) {
      s_abort = 1;
      set_error(p.err, kErrTimeout);
    }
  } else {
    // ------------------------------------------------------------ sums
    const int quad = warp & 3, half = warp >> 2, row = quad * 32 + lane;
    const int place = s_place[row];
    const float* scales = reinterpret_cast<const float*>(smem + kTileOffScales) + row;
    const float factor = p.adapter_scale && place >= 0 ? __ldg(p.adapter_scale + s_id[row]) : 1.f;
    const uint32_t taddr = tmem + (static_cast<uint32_t>(quad * 32) << 16) + half * 32;
    // The row's adapter's product, and where its ranks start among this warp's 32 columns:
    // each warp has half of one adapter's, all of one's, or two's.
    const int index = place >= 0 && place % slots == slot ? place / slots : -1, member = index % G;
    const bool here = index >= 0 && (G == 1 ? half * 32 < columns : member * box >> 5 == half);
    const int own_group = here ? index / G : -1;
    const bool second = G == 4 && (member & 1);
    float y[32];
#pragma unroll
    for (int k = 0; k < 32; ++k) y[k] = 0.f;
    int s = 0;
    uint32_t at = 0;
    for (int b = 0; b < nb && ok; ++b) {
      for (int j = 0; j < groups; ++j, ++at) {
        const int acc = static_cast<int>(at % kTileAccs);
        const bool own = own_group == j;
        ok = __all_sync(0xffffffffu, mbar_wait(&s_tfull[acc], (at / kTileAccs) & 1u, &s_abort));
        if (!ok) break;
        tc_fence_after();
        if (warp == 0 && lane == 0) {  // the products have read the stages
          mbar_arrive(&s_empty[s]);
          if (j + 1 == groups) mbar_arrive(&s_xempty[b % kTileXStages]);
        }
        if (++s == stages) s = 0;
        if (__any_sync(0xffffffffu, own)) {
          uint32_t v[2][16];
          tmem_ld32x16_async(taddr + acc * kTileRanks, v[0]);
          tmem_ld32x16_async(taddr + acc * kTileRanks + 16, v[1]);
          tmem_wait_ld16(v[0]);
          tmem_wait_ld16(v[1]);
          if (own) {
            const float scale = scales[(b % kTileScales) * kTileRows];
#pragma unroll
            for (int k = 0; k < 32; ++k)
              y[k] = fmaf(scale, __uint_as_float(k < 16 && second ? v[1][k] : v[k >> 4][k & 15]), y[k]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_tempty[acc]);
      }
    }
    if (!ok && lane == 0) {
      s_abort = 1;
      set_error(p.err, kErrTimeout);
    }
    // every block has been converted: its products are done
    if (here) {  // the pieces of a row turned by its number: lanes do not collide
      float4* dst = reinterpret_cast<float4*>(part + row * kTileRanks);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        dst[((G == 1 ? half * 8 : 0) + k) ^ (row & 15)] = make_float4(y[4 * k] * factor, y[4 * k + 1] * factor, y[4 * k + 2] * factor,
                                                         y[4 * k + 3] * factor);
    }
  }
  if (warp == kCopyWarp) {
    __syncwarp();
    if (p.ready) pdl_wait();
    pdl_trigger();
    if (p.lists && rank == 0 && blockIdx.z == 0)
      for (int i = lane; i < 4 + n; i += 32) p.lists[t0 / kTileRows * kLoraListWords + i] = s_list[i];
  }
  tc_fence_before();
  __syncwarp();
  __syncthreads();
  if (warp == kIssueWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTileAccs * kTileRanks);
  }
  if (mine == 0) return;  // the same in a cluster's CTAs
  if (splits > 1) cluster_sync();
  // a share of the rows for each CTA: 16 threads a row, 4 ranks each
  const int row0 = kTileRows * rank / splits, row1 = kTileRows * (rank + 1) / splits;
#pragma unroll 1
  for (int i = row0 + (tid >> 4); s_abort == 0 && i < row1; i += kTileWarps * 2) {
    const int r = (tid & 15) * 4;
    if (s_place[i] < 0 || s_place[i] % slots != slot || r >= columns) continue;
    const uint32_t at = smem_u32(part + i * kTileRanks + (((tid & 15) ^ (i & 15)) * 4));
    float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int c = 0; c < splits; ++c) {  // in rank order
      float4 w;
      asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                   : "=f"(w.x), "=f"(w.y), "=f"(w.z), "=f"(w.w)
                   : "r"(splits > 1 ? map_rank(at, static_cast<uint32_t>(c)) : at));
      v[0] += w.x;
      v[1] += w.y;
      v[2] += w.z;
      v[3] += w.w;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = r + k < ranks ? v[k] : 0.f;
    store_v(p, t0 + i, r0 + r, v);
  }
  __syncwarp();
  if (splits > 1) cluster_sync();  // no CTA leaves while its part may still be read
}

}  // namespace

// The lists, kLoraListWords for each tile of 128 rows, in 80 bytes for each 16 rows (640 for 528):
// tiles of fewer rows, whose lists are in shared memory, would have room for theirs too.
static size_t lists_offset(int T, int rank) {
  return (2 * kLoraPlanes * static_cast<size_t>(T) * lora_pitch(rank) + 255) & ~static_cast<size_t>(255);
}
size_t lora_workspace_bytes(int T, int rank) {
  return lists_offset(T, rank) + (static_cast<size_t>(T) + 15) / 16 * 80 + 528;
}

LoraInner lora_inner_at(const csa2_lora_linear_args& a, void* ws, bool lists) {
  uint8_t* base = static_cast<uint8_t*>(ws);
  return LoraInner{reinterpret_cast<uint16_t*>(base),
                   lists ? reinterpret_cast<int*>(base + lists_offset(a.base.T, a.rank)) : nullptr};
}

cudaError_t launch_lora_inner(const csa2_lora_linear_args& a, const LoraInner& to, int ctas, const DeviceCtx& ctx,
                              cudaStream_t st, const char** why) {
  const csa2_fp8_linear_args& l = a.base;
  const InnerParams p{l.x, l.x_scale, a.a, a.adapter_scale, a.row_adapter, to.v, to.lists, l.ld_x, l.ld_x_scale, l.T, l.K,
                      a.rank, lora_pitch(a.rank), a.n_adapters, lora_planes(l.out_format), l.w_ready,
                      ctx.err};
  const int tiles = (l.T + kTileRows - 1) / kTileRows, runs = (a.rank + kTileRanks - 1) / kTileRanks, blocks = (l.K + 127) / 128;
  // The tiles' CTAs, one an SM: shares of the input dims, then of the adapters.  If the SMs
  // that the projection's CTAs leave hold those of a slot, not more than they: the two
  // launches run side by side (64 x 2,048 x 32,768 with 16 of rank 64: 32.1 us, 37.1 on all;
  // 200 x 7,168 x 512: 30.2 and 36.5).
  int splits = ctx.num_sms / (tiles * runs);
  splits = splits < 1 ? 1 : splits > 8 ? 8 : splits;
  if (splits > blocks) splits = blocks;
  const int left = ctx.num_sms - ctas, room = tiles * runs * splits <= left ? left : ctx.num_sms;
  const int box = a.rank > 48 ? kTileRanks : (a.rank + 15) & ~15, G = box <= 32 ? kTileRanks / box : 1;
  const int groups = ((a.n_adapters < kTileRows ? a.n_adapters : kTileRows) + G - 1) / G;  // of a tile, at most
  int slots = room / (tiles * runs * splits);
  if (slots > groups) slots = groups;
  slots = slots < 1 ? 1 : slots > 16 ? 16 : slots;
  // The small CTAs while they, by the most adapters that 16 rows can have, and their blocks
  // are few (the projection's time counted in): 333 x 1,360 x 1,001 with 5 of rank 24 take
  // 11.0 us, 13.2 with the tiles; 64 x 4,096 x 8,192 with 16 of rank 80: 40 and 57; 200 x
  // 2,048 x 4,096 with 16 of rank 64: 34.6 and 32.4; 96 x 7,168 x 512 with 16 of rank 48: 25.3
  // and 21.7 (but 200 rows with 16 of rank 16: 24.5 and 19.0).  But not where the tiles' take no
  // longer, at half a microsecond a product and 10 more, than the projection beside them (its
  // weights at 4.2 TB/s): 128 x 2,048 x 32,768 with 16 of rank 32 take 26.6 us with them and
  // 30.0; 64 rows of rank 128: 54 and 43.
  // 8 ranks without a partner get 8 zeros beside them: products are of 16.
  const dim3 grid((l.T + 15) / 16, (a.rank + 15) / 16 * 2, a.n_adapters < 16 ? a.n_adapters : 16);
  const long long small = static_cast<long long>(grid.x) * grid.y * grid.z;
  const int products = (blocks + splits - 1) / splits * ((groups + slots - 1) / slots);
  const bool beside = tiles * runs * splits <= left && 20 + products <= (static_cast<long long>(l.N) * l.K) >> 21;
  if (!beside && small * (blocks + 8) <= 190LL * ctx.num_sms) {
    // Up to 16 blocks, 8 warps where 16 would be more than an SM's two CTAs (333 x 1,360 x
    // 1,001: 11.0 and 11.6 us); above, 32 (8 x 7,168 x 512 with 8 of rank 16: 8.5 us, 10.5 with 16,
    // 14.1 with 8; 400 rows: 26.6, 24.4 and 34.4).
    if (blocks <= 16 && small > 2 * ctx.num_sms) return launch_pdl(lora_inner_kernel<8>, grid, dim3(256), 0, st, p);
    return blocks > 16 ? launch_pdl(lora_inner_kernel<32>, grid, dim3(1024), 0, st, p)
                       : launch_pdl(lora_inner_kernel<16>, grid, dim3(512), 0, st, p);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(tiles, splits, runs * slots);
  cfg.blockDim = dim3(kTileWarps * 32);
  cfg.dynamicSmemBytes = kTileSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 1;
  attr[1].val.clusterDim.y = splits;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = splits > 1 ? 2 : 1;
  CUtensorMap map_a;
  const uint64_t row = 2 * static_cast<uint64_t>(l.K);
  if (encode_tmap_2d_u8(&map_a, a.a, row, static_cast<uint64_t>(a.n_adapters) * a.rank, row, 128, box) != CUDA_SUCCESS) {
    *why = "csa2_lora_linear: a tensor map could not be encoded";
    return cudaErrorInvalidValue;
  }
  cudaError_t e = prefer_max_smem_once<lora_tile_kernel>(ctx.device, kTileSmem);
  if (e != cudaSuccess) return e;
  const int stages = kTileABytes / ((box <= 32 ? kTileRanks : box) * 256);
  return cudaLaunchKernelEx(&cfg, lora_tile_kernel, map_a, p, slots, box, stages);
}

}  // namespace csa2
