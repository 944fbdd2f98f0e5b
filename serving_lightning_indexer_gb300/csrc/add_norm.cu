// The residual's addition, its RMSNorm, and the e4m3 codes of the result:
//   r = round(x + residual),  y = r / sqrt(mean(r^2) + eps) * gamma,  codes(y)
//
// Bound: HBM, each value read and written once: 7 B a value with a bf16 residual
// (2 + 2 read, 2 + 1 written), 11 with an fp32 one.  4,096 x 7,168 bf16: 40 us, 5.1 TB/s
// (a plain copy: 6.8).  A decode step's few rows are launch and load latency: 8 x 7,168 in
// 3.1 us.
#include <cuda_bf16.h>

#include "csa2_device.cuh"
#include "csa2_e4m3.cuh"
#include "csa2_internal.h"

namespace csa2 {
namespace {

struct AddNormParams {
  const __nv_bfloat16* x;
  const void* residual;
  void* residual_out;
  const float* gamma;
  uint8_t* codes;
  float* scale;
  __nv_bfloat16* y;
  long long ld_x, ld_res, ld_out, ld_codes, ld_scale, ld_y;
  int T, K;
  float eps;
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void pack16(const float (&y)[16], uint4 (&v)[2]) {
#pragma unroll
  for (int h = 0; h < 2; ++h)
    v[h] = make_uint4(pack_bf16(y[8 * h], y[8 * h + 1]), pack_bf16(y[8 * h + 2], y[8 * h + 3]),
                      pack_bf16(y[8 * h + 4], y[8 * h + 5]), pack_bf16(y[8 * h + 6], y[8 * h + 7]));
}

// Codes are of r * gamma * 448 / a, a the block's largest |r * gamma|, rounded once to fp32:
// the norm's factor has no part in them.  In fp32 alone that is off by at most five roundings
// (the product, a, 448 / a, what is less or more of it, and the last product).  Where values
// six roundings to either side have one code, that is the code; where not (some 9 of a
// million values), exact_codes decides.  With fp32's own roundings instead, 13 of 29.4 M codes
// of 4,096 x 7,168 are on the other side of a border, and it takes 38.1 us, 40.1 so.
// Of blocks with a smaller or no finite a, of the norm itself.
constexpr float kLeastTop = 8.271806125530277e-25f;  // 2^-80: its products' second parts are normal
constexpr float kNear = 3.5762786865234375e-7f;  // 6 x 2^-24

// A magnitude in two parts; the larger of two, without a NaN.
struct Pair {
  float hi, lo;
};
__device__ __forceinline__ Pair larger(Pair a, Pair b) {
  const bool take = b.hi > a.hi || (b.hi == a.hi && b.lo > a.lo);
  return Pair{take ? b.hi : a.hi, take ? b.lo : a.lo};
}
// The codes of a run from the stored r, the products and the largest of them in two parts
// (2^-45 off).  By whole warps and seldom, so with few registers where many are taken
// already (V above 1): unrolled, 4,096 x 7,168 takes 51 us in place of 40, and 1,003 x 2,064
// 7.4 in place of 8.0.
template <bool F32, int V>
__device__ __forceinline__ void exact_codes(const uint4* r, const float* gamma, bool in, bool usual, uint32_t (&q)[4]) {
  auto times = [&](int i, float (&hi)[4], float (&lo)[4]) {  // columns 4 i .. of the run
    float x[4];
    if constexpr (F32) {
      const uint4 v = r[i];
      x[0] = __uint_as_float(v.x), x[1] = __uint_as_float(v.y), x[2] = __uint_as_float(v.z), x[3] = __uint_as_float(v.w);
    } else {
      const uint2 v = reinterpret_cast<const uint2*>(r)[i];
      x[0] = __uint_as_float(v.x << 16), x[1] = __uint_as_float(v.x & 0xFFFF0000u);
      x[2] = __uint_as_float(v.y << 16), x[3] = __uint_as_float(v.y & 0xFFFF0000u);
    }
    const float4 g = __ldg(reinterpret_cast<const float4*>(gamma) + i);
    const float w[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      hi[k] = x[k] * w[k];
      lo[k] = fmaf(x[k], w[k], -hi[k]);
    }
  };
  constexpr int kUnroll = V == 1 ? 4 : 1;
  float hi[4], lo[4];
  Pair a = {0.f, 0.f};
#pragma unroll kUnroll
  for (int i = 0; i < 4; ++i) {
    if (!in) break;
    times(i, hi, lo);
#pragma unroll
    for (int k = 0; k < 4; ++k) a = larger(a, Pair{fabsf(hi[k]), hi[k] < 0.f ? -lo[k] : lo[k]});
  }
  __syncwarp();
#pragma unroll
  for (int o = 4; o > 0; o >>= 1)
    a = larger(a, Pair{__shfl_xor_sync(0xffffffffu, a.hi, o), __shfl_xor_sync(0xffffffffu, a.lo, o)});
  if (!in || !usual) return;
  // 448 / a as a factor, rounded down so that a zero keeps its sign, and what that lacks
  float f = kE4m3Max / a.hi;
  if (fmaf(-f, a.lo, fmaf(-f, a.hi, kE4m3Max)) < 0.f) f = __int_as_float(__float_as_int(f) - 1);
  const float low = fmaf(-f, a.lo, fmaf(-f, a.hi, kE4m3Max)) * (f * (1.f / kE4m3Max));
#pragma unroll kUnroll
  for (int i = 0; i < 4; ++i) {
    times(i, hi, lo);
#pragma unroll
    for (int k = 0; k < 4; ++k) hi[k] = fmaf(hi[k], f, fmaf(lo[k], f, hi[k] * low));
    const uint32_t v = e4m3x4(hi[0], hi[1], hi[2], hi[3]);
    q[0] = i == 0 ? v : q[0];  // a rolled loop cannot index registers
    q[1] = i == 1 ? v : q[1];
    q[2] = i == 2 ? v : q[2];
    q[3] = i == 3 ? v : q[3];
  }
}

// A run of r from its words.
template <bool F32>
__device__ __forceinline__ void values(const uint4 (&v)[F32 ? 4 : 2], float (&y)[16]) {
  if constexpr (F32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[4 * i] = __uint_as_float(v[i].x);
      y[4 * i + 1] = __uint_as_float(v[i].y);
      y[4 * i + 2] = __uint_as_float(v[i].z);
      y[4 * i + 3] = __uint_as_float(v[i].w);
    }
  } else {
    unpack16(v, y);
  }
}
// y = y * by * gamma
__device__ __forceinline__ void scaled(float (&y)[16], float by, const float* gamma) {
#pragma unroll
  for (int i = 0; i < 16; i += 4) {
    const float4 g = __ldg(reinterpret_cast<const float4*>(gamma + i));
    y[i] = y[i] * by * g.x;
    y[i + 1] = y[i + 1] * by * g.y;
    y[i + 2] = y[i + 2] * by * g.z;
    y[i + 3] = y[i + 3] * by * g.w;
  }
}

// A CTA takes a row and keeps it in registers between the sum of squares and the
// codes; V: runs of 16 columns a thread holds.  Rows on their way hide each other's
// latency: CTAs that stay and copy their next rows into shared memory meanwhile took 42 us
// for 4,096 x 7,168, since fewer of them fit.  The sum is normalised as it is
// stored, so that the result does not depend on whether a later launch reads the
// residual again.  A thread writes only columns that it has read, which is what
// allows residual_out to be residual.
template <int V, bool F32, int MOST>
__global__ void __launch_bounds__(MOST) add_norm_kernel(const __grid_constant__ AddNormParams p) {
  constexpr int kWords = F32 ? 4 : 2;  // 16-byte words of a run of the residual
  __shared__ float part[MOST / 32];
  pdl_wait();
  pdl_trigger();
  const long long t = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y;
  if (t >= p.T) return;  // a whole warp of a CTA that has no barrier
  const int tid = threadIdx.x, threads = blockDim.x;
  const __nv_bfloat16* x = p.x + t * p.ld_x;
  const uint4* res = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.residual) + t * p.ld_res * (F32 ? 4 : 2));
  uint4* out = reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.residual_out) + t * p.ld_out * (F32 ? 4 : 2));
  uint4 xv[V][2], rv[V][kWords];
#pragma unroll
  for (int r = 0; r < V; ++r) {
    const int c = (r * threads + tid) * 16;
    if (c < p.K) {
      const uint4* src = reinterpret_cast<const uint4*>(x + c);
#pragma unroll
      for (int i = 0; i < 2; ++i) xv[r][i] = src[i];
#pragma unroll
      for (int i = 0; i < kWords; ++i) rv[r][i] = res[c / 16 * kWords + i];
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) xv[r][i] = make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < kWords; ++i) rv[r][i] = make_uint4(0, 0, 0, 0);
    }
  }
  float ss = 0.f;
#pragma unroll
  for (int r = 0; r < V; ++r) {
    float a[16], b[16];
    unpack16(xv[r], a);
    if constexpr (F32) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        b[4 * i] = a[4 * i] + __uint_as_float(rv[r][i].x);
        b[4 * i + 1] = a[4 * i + 1] + __uint_as_float(rv[r][i].y);
        b[4 * i + 2] = a[4 * i + 2] + __uint_as_float(rv[r][i].z);
        b[4 * i + 3] = a[4 * i + 3] + __uint_as_float(rv[r][i].w);
        rv[r][i] = make_uint4(__float_as_uint(b[4 * i]), __float_as_uint(b[4 * i + 1]), __float_as_uint(b[4 * i + 2]),
                              __float_as_uint(b[4 * i + 3]));
      }
    } else {
      unpack16(rv[r], b);
#pragma unroll
      for (int i = 0; i < 16; ++i) b[i] += a[i];
      pack16(b, rv[r]);
      unpack16(rv[r], b);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) ss = fmaf(b[i], b[i], ss);
  }
#pragma unroll
  for (int r = 0; r < V; ++r) {
    const int c = (r * threads + tid) * 16;
    if (c < p.K) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) out[c / 16 * kWords + i] = rv[r][i];
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  if (threads > 32) {
    if ((tid & 31) == 0) part[tid >> 5] = ss;
    __syncthreads();
    ss = 0.f;
    for (int w = 0; w < threads >> 5; ++w) ss += part[w];
  }
  const float inv = 1.0f / sqrtf(ss / static_cast<float>(p.K) + p.eps);
#pragma unroll
  for (int r = 0; r < V; ++r) {
    const int c = (r * threads + tid) * 16;
    const bool in = c < p.K;
    float y[16];  // r * gamma
    values<F32>(rv[r], y);
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const float4 g = in ? __ldg(reinterpret_cast<const float4*>(p.gamma + c + i)) : make_float4(0.f, 0.f, 0.f, 0.f);
      y[i] *= g.x;
      y[i + 1] *= g.y;
      y[i + 2] *= g.z;
      y[i + 3] *= g.w;
    }
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) top = fmaxf(top, fabsf(y[i]));
    top = max8(top);
    const float a = top * inv;
    // The same in a block's lanes, but for those behind the last column, whose values are zeros
    // and have no part in the block: where the block is not usual they go along and write nothing.
    const bool usual = !in || (top >= kLeastTop && top <= kLargest && a >= kAmaxFloor && a <= kLargest);
    auto store_y = [&](float by) {
      float n[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) n[i] = y[i] * by;
      uint4 h[2];
      pack16(n, h);
      uint4* dst = reinterpret_cast<uint4*>(p.y + t * p.ld_y + c);
      dst[0] = h[0];
      dst[1] = h[1];
    };
    if (p.y && in && usual) store_y(inv);
    float s = a / kE4m3Max;
    uint32_t q[4], differ = 0;
    if (p.codes && usual) {
      const float f = kE4m3Max / top, less = f * (1.f - kNear), more = f * (1.f + kNear);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        q[i] = e4m3x4(y[4 * i] * less, y[4 * i + 1] * less, y[4 * i + 2] * less, y[4 * i + 3] * less);
        differ |= q[i] ^ e4m3x4(y[4 * i] * more, y[4 * i + 1] * more, y[4 * i + 2] * more, y[4 * i + 3] * more);
      }
    }
    if (__builtin_expect(!__all_sync(0xffffffffu, usual), 0)) {
      // a block's norm is zero or next to it, or it or r * gamma is not finite: from the stored r
#pragma unroll
      for (int i = 0; i < 16; ++i) y[i] = 0.f;
      if (in) {
        uint4 v[kWords];
#pragma unroll
        for (int i = 0; i < kWords; ++i) v[i] = out[c / 16 * kWords + i];
        values<F32>(v, y);
        scaled(y, inv, p.gamma + c);
      }
      if (p.y && in && !usual) store_y(1.f);
      __syncwarp();
      float f;
      const float scale = e4m3_block(max8(amax16(y)), &f);  // by all lanes
      if (!usual) {
        const uint4 w = codes16(y, f);
        q[0] = w.x, q[1] = w.y, q[2] = w.z, q[3] = w.w;
        s = scale;
      }
    }
    if (__builtin_expect(__any_sync(0xffffffffu, differ != 0), 0)) exact_codes<F32, V>(out + c / 16 * kWords, p.gamma + c, in, usual, q);
    if (p.codes && in) {
      *reinterpret_cast<uint4*>(p.codes + t * p.ld_codes + c) = make_uint4(q[0], q[1], q[2], q[3]);
      if ((tid & 7) == 0) p.scale[t * p.ld_scale + (c >> 7)] = s;
    }
  }
}

template <int V, int MOST>
cudaError_t launch_v(const csa2_add_norm_fp8_args& a, const AddNormParams& p, cudaStream_t st) {
  // whole warps, no more than the row's runs need
  const int threads = ((a.K + 16 * V - 1) / (16 * V) + 31) / 32 * 32;
  // Rows of one warp go two to a CTA: an SM holds 32 CTAs, which is half its warps (6,000 x
  // 512: 6.5 -> 5.1 us, 16,000 x 512: 16.6 -> 11.2 us, 600 x 512: 2.2 us either way).
  const int rows = threads == 32 ? 2 : 1;
  const dim3 grid(static_cast<unsigned>((a.T + rows - 1) / rows)), block(threads, rows);
  return a.residual_f32 ? launch_pdl(add_norm_kernel<V, true, MOST>, grid, block, 0, st, p)
                        : launch_pdl(add_norm_kernel<V, false, MOST>, grid, block, 0, st, p);
}

}  // namespace

cudaError_t launch_add_norm_fp8(const csa2_add_norm_fp8_args& a, const DeviceCtx& ctx, cudaStream_t st) {
  const AddNormParams p{reinterpret_cast<const __nv_bfloat16*>(a.x), a.residual, a.residual_out, a.gamma, a.codes, a.scale,
                        reinterpret_cast<__nv_bfloat16*>(a.y), a.ld_x, a.ld_residual, a.ld_residual_out, a.ld_codes,
                        a.ld_scale, a.ld_y, a.T, a.K, a.eps};
  // Runs a thread, and threads a CTA at most.  Up to two rows an SM want the shorter work a
  // thread (8 x 7,168: 3.1 us with one run, 3.7 with two; 304 rows: 4.5 and 5.1), more rows
  // the more CTAs an SM (456: 7.3 and 7.0; 4,096: 48.8 and 40.0); four runs hold registers for
  // too few warps (2,048 x 16,384: 53.9 us, 48.0 with two).
  if (a.K <= 4096) return launch_v<1, 256>(a, p, st);
  if (a.K > 8192) return launch_v<2, 512>(a, p, st);
  return a.T <= 2 * ctx.num_sms ? launch_v<1, 512>(a, p, st) : launch_v<2, 256>(a, p, st);
}

}  // namespace csa2
