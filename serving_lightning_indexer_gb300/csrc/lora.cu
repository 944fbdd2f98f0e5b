// Inner products of low-rank adapters with the rows that use them,
//   v[t][r] = s[i] * sum_b x_scale[t][b] * sum_{k in b} x[t][k] a[i][r][k],  i = row_adapter[t],
// and the list of adapters that each of the projection's row tiles needs.  The
// projection (fp8_linear.cu) adds v[t] b[i]^T to its sums before RoPE and rounding.
//
// The codes are exact in bf16 and a is bf16, so a block's 128 products are summed by
// the tensor core (mma.sync, fp32) and the block's scale is applied to the sum.  The
// result is written as the bf16 nearest to it and, for outputs that can tell (fp32,
// and the fp32 scales of e4m3), the bf16 nearest to what that leaves: 2^-17 together.
//
// A CTA takes 16 rows, one of the adapters among them and 8 of its ranks; its 16
// warps take the blocks of 128 input dims in turn and are added in warp order.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "csa2_device.cuh"
#include "csa2_internal.h"

namespace csa2 {
namespace {

constexpr int kInnerWarps = 16;

struct InnerParams {
  const uint8_t* x;
  const float* x_scale;
  const uint16_t* a;
  const float* adapter_scale;
  const int* row_adapter;
  uint16_t* v;  // [2][T][rank]: the bf16 values, and what they leave
  int* lists;
  long long ld_x, ld_xs;
  int T, K, rank, n_adapters;
  int tile_rows;  // rows of the projection's tiles
  int low;        // the second plane is wanted
  int ready;      // a and row_adapter may be read before the previous launch completes
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

// The adapters among a tile's rows, each once, in the order of their first rows:
// list[0] how many, list[4 ..] which.  n <= 128 threads of whole warps, all of them.
__device__ __forceinline__ void write_list(const InnerParams& p, long long t0, int n, int* list, int* s_id, int* s_base) {
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
  bool first = id >= 0;
  for (int j = 0; j < i && j < n; ++j) first = first && s_id[j] != id;
  const uint32_t mask = __ballot_sync(0xffffffffu, first);
  if (lane == 0) s_base[i >> 5] = __popc(mask);
  __syncthreads();
  int at = 0;
  for (int w = 0; w < (i >> 5); ++w) at += s_base[w];
  if (first) list[4 + at + __popc(mask & ((1u << lane) - 1))] = id;
  if (i == static_cast<int>(blockDim.x) - 1) list[0] = at + __popc(mask);
  __syncthreads();
}

__global__ void __launch_bounds__(kInnerWarps * 32) lora_inner_kernel(const __grid_constant__ InnerParams p) {
  __shared__ float part[kInnerWarps][16][8];
  __shared__ int s_id[128], s_base[kInnerWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (!p.ready) pdl_wait();
  const int t0 = blockIdx.x * 16;
  // the blockIdx.z-th adapter among the 16 rows
  int id = -1;
  if (lane < 16 && t0 + lane < p.T) id = __ldg(p.row_adapter + t0 + lane);
  if (id >= p.n_adapters) id = -1;
  const uint32_t same = __match_any_sync(0xffffffffu, id);
  uint32_t firsts = __ballot_sync(0xffffffffu, id >= 0 && __ffs(same) - 1 == lane);
  for (int j = blockIdx.z; j > 0; --j) firsts &= firsts - 1;
  const int adapter = __shfl_sync(0xffffffffu, id, firsts ? __ffs(firsts) - 1 : 0);
  if (p.ready) pdl_wait();
  pdl_trigger();
  if (blockIdx.y == 0 && blockIdx.z == 0 && t0 % p.tile_rows == 0)
    write_list(p, t0, p.tile_rows, p.lists + static_cast<long long>(t0 / p.tile_rows) * (p.tile_rows + 4), s_id, s_base);
  if (!firsts) return;

  const int g = lane >> 2, q = lane & 3, r0 = blockIdx.y * 8;
  const int blocks = (p.K + 127) / 128;
  const uint16_t* a = p.a + (static_cast<long long>(adapter) * p.rank + r0 + g) * p.K + q * 8;
  const int ra = min(t0 + g, p.T - 1), rb = min(t0 + g + 8, p.T - 1);
  const uint8_t* xa = p.x + ra * p.ld_x + q * 8;
  const uint8_t* xb = p.x + rb * p.ld_x + q * 8;
  float sum[4] = {0.f, 0.f, 0.f, 0.f};
  for (int b = warp; b < blocks; b += kInnerWarps) {
    // The order of the products of a block is free: a lane holds 8 dims in a row of
    // each 32, which the fragments of two steps take as their four pairs.
    uint4 av[4];
    uint2 xv[4], yv[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int k = b * 128 + c * 32;
      const bool in = k + q * 8 < p.K;
      av[c] = in ? __ldg(reinterpret_cast<const uint4*>(a + k)) : make_uint4(0, 0, 0, 0);
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
      for (int w = 0; w < kInnerWarps; ++w) v += part[w][i][r];
      if (p.adapter_scale) v *= __ldg(p.adapter_scale + adapter);
      const __nv_bfloat16 hi = __float2bfloat16_rn(v);
      const long long at = static_cast<long long>(t0 + i) * p.rank + r0 + r;
      p.v[at] = *reinterpret_cast<const uint16_t*>(&hi);
      if (p.low) {
        // an infinite or NaN value is all in the first plane
        const float rest = v - __bfloat162float(hi);
        const __nv_bfloat16 lo = __float2bfloat16_rn(isfinite(rest) ? rest : 0.f);
        p.v[at + static_cast<long long>(p.T) * p.rank] = *reinterpret_cast<const uint16_t*>(&lo);
      }
    }
  }
}

}  // namespace

// The lists for any tile height: (rows + 4) words a tile of 16, 32, 64 or 128 rows.
static size_t lists_offset(int T, int rank) {
  return (4 * static_cast<size_t>(T) * rank + 255) & ~static_cast<size_t>(255);
}
size_t lora_workspace_bytes(int T, int rank) {
  return lists_offset(T, rank) + (static_cast<size_t>(T) + 15) / 16 * 80 + 528;
}

LoraInner lora_inner_at(const csa2_lora_linear_args& a, void* ws, int tile_rows) {
  uint8_t* base = static_cast<uint8_t*>(ws);
  return LoraInner{reinterpret_cast<uint16_t*>(base), reinterpret_cast<int*>(base + lists_offset(a.base.T, a.rank)), tile_rows};
}

cudaError_t launch_lora_inner(const csa2_lora_linear_args& a, const LoraInner& to, const DeviceCtx& ctx, cudaStream_t st) {
  const csa2_fp8_linear_args& l = a.base;
  const InnerParams p{l.x, l.x_scale, a.a, a.adapter_scale, a.row_adapter, to.v, to.lists, l.ld_x, l.ld_x_scale, l.T, l.K,
                      a.rank, a.n_adapters, to.tile_rows, l.out_format != CSA2_OUT_BF16, l.w_ready, ctx.err};
  const dim3 grid((l.T + 15) / 16, a.rank / 8, a.n_adapters < 16 ? a.n_adapters : 16);
  return launch_pdl(lora_inner_kernel, grid, dim3(kInnerWarps * 32), 0, st, p);
}

}  // namespace csa2
