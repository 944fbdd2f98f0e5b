// The e4m3 block rule shared by the quantisers and the projection's e4m3 output:
// one fp32 scale for 128 values.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

namespace csa2 {

constexpr float kE4m3Max = 448.f;
// Blocks of smaller values are scaled as if this were their maximum, so that
// 448 / a stays finite in fp32 (a = 448 * 2^-120).
constexpr float kAmaxFloor = 448.f * 7.52316384526264e-37f;

constexpr float kLargest = 3.402823466e38f;  // finite fp32
// An infinity or NaN as NaN, everything else unchanged.  fmaxf drops the NaN
// from a block's maximum and the conversion below codes it 0x7F.
__device__ __forceinline__ float finite_or_nan(float y) { return fabsf(y) <= kLargest ? y : __int_as_float(0x7FC00000); }
// Scale of a block with the largest magnitude amax >= 0, and the factor that
// takes its values to codes.
__device__ __forceinline__ float e4m3_block(float amax, float* to_code) {
  const float a = fmaxf(amax, kAmaxFloor);
  *to_code = kE4m3Max / a;
  return amax > 0.f ? a / kE4m3Max : 1.f;
}
// The same with what the factor lacks, to some six bits or more: fma(y, factor, y *
// low) is y * 448 / a rounded once.  A bf16 y and a bf16 a put y * 448 / a on a border
// between two codes, where the tie goes to the even one, or at least 2^-14 of itself
// away from every border; y times a rounded factor leaves a border to either side
// (one code in 2,400 to 3,700 of normal data was the odd one).  The factor is rounded
// down, so that low >= 0 and a zero keeps its sign.
__device__ __forceinline__ float e4m3_block_exact(float amax, float* to_code, float* low) {
  const float a = fmaxf(amax, kAmaxFloor);
  float f = kE4m3Max / a;
  if (fmaf(-f, a, kE4m3Max) < 0.f) f = __int_as_float(__float_as_int(f) - 1);
  *to_code = f;
  *low = fmaf(-f, a, kE4m3Max) * (f * (1.f / kE4m3Max));
  return amax > 0.f ? a / kE4m3Max : 1.f;
}
// e4m3 codes of (lo, hi), round-to-nearest-even, saturating; lo in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  return e4m3x2(a, b) | (e4m3x2(c, d) << 16);
}

// ---- runs of 16 columns, as the row kernels hold them (8 lanes a block of 128)
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
// Maximum over the 8 lanes that hold one block of 128 columns.
__device__ __forceinline__ float max8(float a) {
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
  return a;
}

}  // namespace csa2
