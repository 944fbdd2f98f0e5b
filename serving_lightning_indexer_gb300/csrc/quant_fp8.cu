// e4m3 codes with one fp32 scale per block of 128 columns of a row (optionally
// of the row's RMSNorm), or per 128 x 128 tile.
//
// Bound: HBM (2 B read and 1 B + 4/128 B written per value): rows of 4,096 x 7,168
// take 14.7 us, 6.1 TB/s (a copy of as many bytes 14.3 us), tiles of 32,768 x 2,048
// 33.1 us, 6.1 TB/s.  A decode step's few rows are launch and load latency (8 x
// 7,168 with the norm: 2.4 us).
#include <cuda_bf16.h>

#include "csa2_device.cuh"
#include "csa2_e4m3.cuh"
#include "csa2_internal.h"

namespace csa2 {
namespace {

struct QuantParams {
  const __nv_bfloat16* x;
  long long ld_x;
  int T, K;
  const float* gamma;
  float eps;
  uint8_t* codes;
  long long ld_codes;
  float* scale;
  long long ld_scale;
};

// 16 consecutive bf16 values as fp32.
__device__ __forceinline__ void unpack16(const uint4 (&v)[2], float (&y)[16]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t w[4] = {v[h].x, v[h].y, v[h].z, v[h].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[h * 8 + 2 * i] = __uint_as_float(w[i] << 16);
      y[h * 8 + 2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
}
// Largest finite magnitude; infinities become NaN.
__device__ __forceinline__ float amax16(float (&y)[16]) {
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    y[i] = finite_or_nan(y[i]);
    a = fmaxf(a, fabsf(y[i]));
  }
  return a;
}
// The same with the finite case apart (a NaN is dropped by fmaxf and coded as
// such): 14.7 against 15.7 us for rows of 4,096 x 7,168.  The tiles' kernel keeps the
// one above, at the 80 registers that three CTAs an SM leave it (33.1 against 39.4 us
// for 32,768 x 2,048).
__device__ __forceinline__ float amax16_rows(float (&y)[16]) {
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) a = fmaxf(a, fabsf(y[i]));
  return a > kLargest ? amax16(y) : a;
}
__device__ __forceinline__ uint4 codes16(const float (&y)[16], float f) {
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = e4m3x4(y[4 * i] * f, y[4 * i + 1] * f, y[4 * i + 2] * f, y[4 * i + 3] * f);
  return make_uint4(r[0], r[1], r[2], r[3]);
}
// The exact quotients' codes of bf16 values.  PACKED: two values an instruction, for
// the rows (14.7 us for 4,096 x 7,168, 14.9 without); the tiles have not the registers
// (32,768 x 2,048: 33.1 us without, 37.5 packed).
template <bool PACKED>
__device__ __forceinline__ uint4 codes16_exact(const float (&y)[16], float f, float low) {
  float q[16];
#pragma unroll
  for (int i = 0; i < 16; i += 2) {
    if (PACKED) {
      const uint64_t y2 = pack_f32x2(y[i], y[i + 1]);
      const uint64_t rest = fma_f32x2(y2, pack_f32x2(low, low), pack_f32x2(-0.f, -0.f));
      const float2 v = unpack_f32x2(fma_f32x2(y2, pack_f32x2(f, f), rest));
      q[i] = v.x;
      q[i + 1] = v.y;
    } else {
      q[i] = fmaf(y[i], f, y[i] * low);
      q[i + 1] = fmaf(y[i + 1], f, y[i + 1] * low);
    }
  }
  return codes16(q, 1.f);
}
// Maximum over the 8 lanes that hold one block of 128 columns.
__device__ __forceinline__ float max8(float a) {
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
  return a;
}

// Rows without a norm: a warp takes U runs of 512 columns, a lane 16 of each (a
// block of 128 is 8 lanes, its maximum three shuffles); all of them are loaded
// before the first is used (U = 2: 14.7 us where U = 1 took 15.6).
template <int U>
__global__ void __launch_bounds__(256) quant_rows_kernel(const __grid_constant__ QuantParams p, int chunks) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const uint32_t item0 = (blockIdx.x * 8 + (threadIdx.x >> 5)) * U;
  uint4 v[U][2];
  int t[U], c[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    t[u] = static_cast<int>((item0 + u) / static_cast<uint32_t>(chunks));
    c[u] = static_cast<int>(item0 + u - static_cast<uint32_t>(t[u]) * chunks) * 512 + lane * 16;
    v[u][0] = v[u][1] = make_uint4(0, 0, 0, 0);
    if (t[u] < p.T && c[u] < p.K) {
      const uint4* src = reinterpret_cast<const uint4*>(p.x + t[u] * p.ld_x + c[u]);
      v[u][0] = __ldg(src);
      v[u][1] = __ldg(src + 1);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float y[16];
    unpack16(v[u], y);
    float f, low;
    const float s = e4m3_block_exact(max8(amax16_rows(y)), &f, &low);
    if (t[u] >= p.T || c[u] >= p.K) continue;
    *reinterpret_cast<uint4*>(p.codes + t[u] * p.ld_codes + c[u]) = codes16_exact<true>(y, f, low);
    if ((lane & 7) == 0) p.scale[t[u] * p.ld_scale + (c[u] >> 7)] = s;
  }
}

// Rows with RMSNorm: one CTA a row; the row stays in registers between the sum
// of squares and the codes.  V: runs of 16 columns a thread holds.
template <int V>
__global__ void __launch_bounds__(256) quant_norm_kernel(const __grid_constant__ QuantParams p) {
  __shared__ float part[8];
  pdl_wait();
  pdl_trigger();
  const long long t = blockIdx.x;
  const int tid = threadIdx.x;
  uint4 v[V][2];
  float ss = 0.f;
#pragma unroll
  for (int r = 0; r < V; ++r) {
    const int c = (r * 256 + tid) * 16;
    v[r][0] = v[r][1] = make_uint4(0, 0, 0, 0);
    if (c < p.K) {
      const uint4* src = reinterpret_cast<const uint4*>(p.x + t * p.ld_x + c);
      v[r][0] = __ldg(src);
      v[r][1] = __ldg(src + 1);
    }
  }
#pragma unroll
  for (int r = 0; r < V; ++r) {
    float y[16];
    unpack16(v[r], y);
#pragma unroll
    for (int i = 0; i < 16; ++i) ss = fmaf(y[i], y[i], ss);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  if ((tid & 31) == 0) part[tid >> 5] = ss;
  __syncthreads();
  ss = 0.f;
#pragma unroll
  for (int w = 0; w < 8; ++w) ss += part[w];
  const float inv = 1.0f / sqrtf(ss / static_cast<float>(p.K) + p.eps);
#pragma unroll
  for (int r = 0; r < V; ++r) {
    const int c = (r * 256 + tid) * 16;
    const bool in = c < p.K;
    float y[16];
    unpack16(v[r], y);
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const float4 g = in ? __ldg(reinterpret_cast<const float4*>(p.gamma + c + i)) : make_float4(0.f, 0.f, 0.f, 0.f);
      y[i] = y[i] * inv * g.x;
      y[i + 1] = y[i + 1] * inv * g.y;
      y[i + 2] = y[i + 2] * inv * g.z;
      y[i + 3] = y[i + 3] * inv * g.w;
    }
    if (!in) {
#pragma unroll
      for (int i = 0; i < 16; ++i) y[i] = 0.f;  // 0 * inv is NaN where inv is infinite
    }
    float f;
    const float s = e4m3_block(max8(amax16_rows(y)), &f);
    if (in) {
      *reinterpret_cast<uint4*>(p.codes + t * p.ld_codes + c) = codes16(y, f);
      if ((tid & 7) == 0) p.scale[t * p.ld_scale + (c >> 7)] = s;
    }
  }
}

// 128 x 128 tiles: one CTA a tile, a thread 16 columns of 4 rows.
__global__ void __launch_bounds__(256) quant_tiles_kernel(const __grid_constant__ QuantParams p, int col_tiles) {
  __shared__ float part[8];
  pdl_wait();
  pdl_trigger();
  const int rt = blockIdx.x / col_tiles, ct = blockIdx.x - rt * col_tiles;
  const int tid = threadIdx.x;
  const int c = ct * 128 + (tid & 7) * 16;
  uint4 v[4][2];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const long long row = static_cast<long long>(rt) * 128 + r * 32 + (tid >> 3);
    v[r][0] = v[r][1] = make_uint4(0, 0, 0, 0);
    if (row < p.T && c < p.K) {
      const uint4* src = reinterpret_cast<const uint4*>(p.x + row * p.ld_x + c);
      v[r][0] = __ldg(src);
      v[r][1] = __ldg(src + 1);
    }
  }
  float a = 0.f;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    float y[16];
    unpack16(v[r], y);
    a = fmaxf(a, amax16(y));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
  if ((tid & 31) == 0) part[tid >> 5] = a;
  __syncthreads();
  a = 0.f;
#pragma unroll
  for (int w = 0; w < 8; ++w) a = fmaxf(a, part[w]);
  float f, low;
  const float s = e4m3_block_exact(a, &f, &low);
  if (tid == 0) p.scale[rt * p.ld_scale + ct] = s;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const long long row = static_cast<long long>(rt) * 128 + r * 32 + (tid >> 3);
    if (row < p.T && c < p.K) {
      float y[16];
      unpack16(v[r], y);
#pragma unroll
      for (int i = 0; i < 16; ++i) y[i] = finite_or_nan(y[i]);
      *reinterpret_cast<uint4*>(p.codes + row * p.ld_codes + c) = codes16_exact<false>(y, f, low);
    }
  }
}

}  // namespace

cudaError_t launch_quant_fp8(const csa2_quant_fp8_args& a, cudaStream_t st) {
  const QuantParams p{reinterpret_cast<const __nv_bfloat16*>(a.x), a.ld_x, a.T, a.K, a.gamma, a.eps, a.codes,
                      a.ld_codes, a.scale, a.ld_scale};
  if (a.block_rows == 128) {
    const int ct = (a.K + 127) / 128;
    const long long tiles = static_cast<long long>((static_cast<long long>(a.T) + 127) / 128) * ct;
    return launch_pdl(quant_tiles_kernel, dim3(static_cast<unsigned>(tiles)), dim3(256), 0, st, p, ct);
  }
  if (a.gamma) {
    const dim3 grid(static_cast<unsigned>(a.T)), block(256);
    if (a.K <= 4096) return launch_pdl(quant_norm_kernel<1>, grid, block, 0, st, p);
    if (a.K <= 8192) return launch_pdl(quant_norm_kernel<2>, grid, block, 0, st, p);
    return launch_pdl(quant_norm_kernel<4>, grid, block, 0, st, p);
  }
  const int chunks = (a.K + 511) / 512;
  const long long items = static_cast<long long>(a.T) * chunks;
  return launch_pdl(quant_rows_kernel<2>, dim3(static_cast<unsigned>((items + 15) / 16)), dim3(256), 0, st, p, chunks);
}

}  // namespace csa2
