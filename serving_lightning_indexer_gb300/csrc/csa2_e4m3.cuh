// The e4m3 block rule shared by the quantiser and the projection's e4m3 output:
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

}  // namespace csa2
