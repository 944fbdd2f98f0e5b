// Projection on e4m3 codes with a scale per block of 128:
//   y[t][n] = sum_b x_scale[t][b] * w_scale[n / 128][b] * sum_{k in b} x[t][k] w[n][k]
//
// The tensor core applies no fp32 scale, so each block of 128 input dims gets an
// accumulator of its own: four tcgen05.mma (K = 32 each) into one slot of a TMEM
// ring, from which the accumulation warps take it, times the two scales, into
// fp32 registers while the tensor core works on the next block.  Warp roles:
// eight accumulation warps, one TMA producer, one MMA issuer.  A CTA walks
// output tiles of 128 rows x BN columns (persistent grid).
#include <cuda_bf16.h>

#include "csa2_device.cuh"
#include "csa2_e4m3.cuh"
#include "csa2_internal.h"
#include "csa2_rope.cuh"

namespace csa2 {
namespace {

constexpr int kTileM = 128;   // rows of x a tile
constexpr int kBlockK = 128;  // input dims of a scale block: one swizzled 128-B row of codes
constexpr int kAccWarps = 8;
constexpr int kThreads = (kAccWarps + 2) * 32;

struct LinearParams {
  const float* x_scale;
  const float* w_scale;
  const int* row_pos;
  void* out;
  float* out_scale;
  long long ld_xs, ld_ws, ld_out, ld_os;
  int T, N, K;
  int rope_head;
  int vec;      // output rows are 16-B aligned
  int w_ready;
  uint32_t* err;
  uint64_t turn[32];  // RoPE turn rates of the 32 pairs
};

template <int BN>
struct WideCfg {
  static constexpr int kStages = BN == 256 ? 4 : 6;
  static constexpr int kStageBytes = (kTileM + BN) * kBlockK;
  static constexpr int kAccs = 512 / BN;          // TMEM ring: 512 columns
  static constexpr int kCols = BN / 2;            // columns of a tile an accumulation warp holds
  static constexpr int kOffBars = kStages * kStageBytes;
  static constexpr int kOffMax = kOffBars + 256;  // block maxima of the two column halves
  static constexpr int kSmem = 1024 + kOffMax + 2 * kTileM * 4;
};

// Writes NV consecutive values of one row from column c on; only columns < N.
template <int OUT, int NV>
__device__ __forceinline__ void store_row(const LinearParams& p, long long row, int c, const float (&y)[NV]) {
  if (OUT == CSA2_OUT_F32) {
    float* o = static_cast<float*>(p.out) + row * p.ld_out + c;
    if (p.vec && c + NV <= p.N) {
#pragma unroll
      for (int i = 0; i < NV; i += 4) *reinterpret_cast<float4*>(o + i) = make_float4(y[i], y[i + 1], y[i + 2], y[i + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (c + i < p.N) o[i] = y[i];
    }
  } else {
    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.out) + row * p.ld_out + c;
    if (p.vec && c + NV <= p.N) {
#pragma unroll
      for (int i = 0; i < NV; i += 8) {
        uint32_t r[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const __nv_bfloat162 h = __floats2bfloat162_rn(y[i + 2 * j], y[i + 2 * j + 1]);
          r[j] = *reinterpret_cast<const uint32_t*>(&h);
        }
        *reinterpret_cast<uint4*>(o + i) = make_uint4(r[0], r[1], r[2], r[3]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (c + i < p.N) o[i] = __float2bfloat16_rn(y[i]);
    }
  }
}

template <int BN, int OUT>
__global__ void __launch_bounds__(kThreads, 1)
    fp8_linear_wide_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                           const __grid_constant__ LinearParams p) {
  using Cfg = WideCfg<BN>;
  constexpr int S = Cfg::kStages, NA = Cfg::kAccs, C = Cfg::kCols;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + Cfg::kOffBars);
  uint64_t* empty = full + S;
  uint64_t* tfull = empty + S;
  uint64_t* tempty = tfull + NA;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(tempty + NA);
  volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
  float* s_max = reinterpret_cast<float*>(smem + Cfg::kOffMax);
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
    fence_mbar_init();
    prefetch_tmap(&map_x);
    prefetch_tmap(&map_w);
  }
  if (warp == kAccWarps + 1) {
    tmem_alloc(s_tmem, 512);
    tmem_relinquish();
  }
  pdl_wait();
  pdl_trigger();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  const int m_tiles = (p.T + kTileM - 1) / kTileM, n_tiles = (p.N + BN - 1) / BN;
  const int blocks = (p.K + kBlockK - 1) / kBlockK;
  const long long tiles = static_cast<long long>(m_tiles) * n_tiles;

  if (warp == kAccWarps) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      const uint64_t keep = l2_policy_evict_last();
      long long it = 0;
      bool ok = true;
      for (long long tile = blockIdx.x; tile < tiles && ok; tile += gridDim.x) {
        const int n0 = static_cast<int>(tile / m_tiles) * BN, t0 = static_cast<int>(tile % m_tiles) * kTileM;
        for (int b = 0; b < blocks; ++b, ++it) {
          const int s = static_cast<int>(it % S);
          if (!(ok = mbar_wait(&empty[s], static_cast<uint32_t>((it / S) & 1) ^ 1u, s_abort))) break;
          uint8_t* dst = smem + s * Cfg::kStageBytes;
          mbar_arrive_expect_tx(&full[s], Cfg::kStageBytes);
          tma_load_2d(dst, &map_x, b * kBlockK, t0, &full[s], keep);
          tma_load_2d(dst + kTileM * kBlockK, &map_w, b * kBlockK, n0, &full[s], keep);
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
  } else if (warp == kAccWarps + 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_e4m3_f32(kTileM, BN);
      long long it = 0;
      bool ok = true;
      for (long long tile = blockIdx.x; tile < tiles && ok; tile += gridDim.x) {
        for (int b = 0; b < blocks; ++b, ++it) {
          const int s = static_cast<int>(it % S), a = static_cast<int>(it % NA);
          if (!(ok = mbar_wait(&full[s], static_cast<uint32_t>((it / S) & 1), s_abort))) break;
          if (!(ok = mbar_wait(&tempty[a], static_cast<uint32_t>((it / NA) & 1) ^ 1u, s_abort))) break;
          tc_fence_after();
          const uint64_t ad = smem_desc_sw128(smem + s * Cfg::kStageBytes);
          const uint64_t bd = smem_desc_sw128(smem + s * Cfg::kStageBytes + kTileM * kBlockK);
#pragma unroll
          for (int k = 0; k < 4; ++k)  // 32 B of the swizzled rows a step
            mma_e4m3(tmem + a * BN, ad + 2 * k, bd + 2 * k, idesc, k > 0 ? 1u : 0u);
          mma_commit(&empty[s]);
          mma_commit(&tfull[a]);
        }
      }
      if (!ok) {
        *s_abort = 1;
        set_error(p.err, kErrTimeout);
      }
    }
  } else {
    // ------------------------------------------------------------ accumulation and output
    const int half = warp >> 2;                       // columns half * C .. of the tile
    const int r = (warp & 3) * 32 + lane;             // row of the tile: TMEM lane
    const uint32_t taddr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + half * C;
    long long it = 0;
    bool ok = true;  // the same in a warp's lanes; a warp that gave up still takes part in the barriers below
    for (long long tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
      const int n0 = static_cast<int>(tile / m_tiles) * BN + half * C, t0 = static_cast<int>(tile % m_tiles) * kTileM;
      const int row = t0 + r;
      const float* xs = p.x_scale + static_cast<long long>(min(row, p.T - 1)) * p.ld_xs;
      const float* ws = p.w_scale + static_cast<long long>(min(n0, p.N - 1) >> 7) * p.ld_ws;
      uint64_t acc[C / 2];
#pragma unroll
      for (int i = 0; i < C / 2; ++i) acc[i] = 0;
      float sx = __ldg(xs), sw = __ldg(ws);
      for (int b = 0; b < blocks && ok; ++b, ++it) {
        const float s = sx * sw;
        if (b + 1 < blocks) {  // the next block's scales, under this block's product
          sx = __ldg(xs + b + 1);
          sw = __ldg(ws + b + 1);
        }
        const uint64_t s2 = pack_f32x2(s, s);
        const int a = static_cast<int>(it % NA);
        ok = __all_sync(0xffffffffu, mbar_wait(&tfull[a], static_cast<uint32_t>((it / NA) & 1), s_abort));
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < C; c += 16) {
          uint32_t v[16];
          tmem_ld32x16_async(taddr + a * BN + c, v);
          tmem_wait_ld16(v);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            acc[c / 2 + i] = fma_f32x2(pack_f32x2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), s2, acc[c / 2 + i]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tempty[a]);
      }
      // RoPE: the 64 columns below a head's end
      float y[C];
#pragma unroll
      for (int i = 0; i < C / 2; ++i) {
        const float2 f = unpack_f32x2(acc[i]);
        y[2 * i] = f.x;
        y[2 * i + 1] = f.y;
      }
      if (p.rope_head && (n0 + C) % p.rope_head == 0 && n0 < p.N) {
        const int pos = __ldg(p.row_pos + min(row, p.T - 1));
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          float sn, cs;
          rope_angle(pos, p.turn[i], &sn, &cs);
          const float u = y[C - 64 + 2 * i], v = y[C - 63 + 2 * i];
          y[C - 64 + 2 * i] = u * cs - v * sn;
          y[C - 63 + 2 * i] = u * sn + v * cs;
        }
      }
      if (OUT == CSA2_OUT_FP8) {
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < C; ++i) {
          y[i] = finite_or_nan(y[i]);
          m = fmaxf(m, fabsf(y[i]));
        }
        if (C == 64) {  // a block's two halves are in two warps
          s_max[half * kTileM + r] = m;
          named_bar_sync(1, kAccWarps * 32);
          m = fmaxf(m, s_max[(half ^ 1) * kTileM + r]);
          named_bar_sync(1, kAccWarps * 32);  // read before the next tile writes
        }
        float f;
        const float sc = e4m3_block(m, &f);
        if (ok && row < p.T && n0 < p.N) {
          uint8_t* o = static_cast<uint8_t*>(p.out) + static_cast<long long>(row) * p.ld_out + n0;
#pragma unroll
          for (int i = 0; i < C; i += 16)
            *reinterpret_cast<uint4*>(o + i) =
                make_uint4(e4m3x4(y[i] * f, y[i + 1] * f, y[i + 2] * f, y[i + 3] * f),
                           e4m3x4(y[i + 4] * f, y[i + 5] * f, y[i + 6] * f, y[i + 7] * f),
                           e4m3x4(y[i + 8] * f, y[i + 9] * f, y[i + 10] * f, y[i + 11] * f),
                           e4m3x4(y[i + 12] * f, y[i + 13] * f, y[i + 14] * f, y[i + 15] * f));
          if (C == 128 || half == 0) p.out_scale[static_cast<long long>(row) * p.ld_os + (n0 >> 7)] = sc;
        }
      } else if (ok && row < p.T && n0 < p.N) {
        store_row<OUT, C>(p, row, n0, y);
      }
    }
    if (!ok) {
      *s_abort = 1;
      set_error(p.err, kErrTimeout);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kAccWarps + 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int BN, int OUT>
cudaError_t launch_wide(const csa2_fp8_linear_args& a, const LinearParams& p, const DeviceCtx& ctx, cudaStream_t st,
                        const char** why) {
  CUtensorMap map_x, map_w;
  if (encode_tmap_2d_u8(&map_x, a.x, a.K, a.T, a.ld_x, kBlockK, kTileM) != CUDA_SUCCESS ||
      encode_tmap_2d_u8(&map_w, a.w, a.K, a.N, a.ld_w, kBlockK, BN) != CUDA_SUCCESS) {
    *why = "csa2_fp8_linear: a tensor map could not be encoded";
    return cudaErrorInvalidValue;
  }
  auto kern = fp8_linear_wide_kernel<BN, OUT>;
  cudaError_t e = prefer_max_smem(kern, WideCfg<BN>::kSmem);
  if (e != cudaSuccess) return e;
  const long long tiles = ((static_cast<long long>(a.T) + kTileM - 1) / kTileM) * ((static_cast<long long>(a.N) + BN - 1) / BN);
  const unsigned grid = static_cast<unsigned>(tiles < ctx.num_sms ? tiles : ctx.num_sms);
  return launch_pdl(kern, dim3(grid), dim3(kThreads), WideCfg<BN>::kSmem, st, map_x, map_w, p);
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
  const int size = a.out_format == CSA2_OUT_F32 ? 4 : (a.out_format == CSA2_OUT_BF16 ? 2 : 1);
  p.vec = (a.ld_out * size) % 16 == 0;
  p.w_ready = a.w_ready;
  p.err = ctx.err;
  if (a.rope_head) {
    const double theta = a.rope_theta > 0.f ? a.rope_theta : 10000.0;
    for (int i = 0; i < 32; ++i) p.turn[i] = rope_turn_rate(theta, i);
  }
  switch (a.out_format) {
    case CSA2_OUT_F32: return launch_wide<128, CSA2_OUT_F32>(a, p, ctx, st, why);
    case CSA2_OUT_BF16: return launch_wide<128, CSA2_OUT_BF16>(a, p, ctx, st, why);
    default: return launch_wide<128, CSA2_OUT_FP8>(a, p, ctx, st, why);
  }
}

}  // namespace csa2
