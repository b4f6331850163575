// FP32 numbers as operands of TF32 products, and small arithmetic of the kernels that use
// them (tree decode, the state cache).
#pragma once

#include "kda_common.cuh"

namespace kda {

// TF32 products take the upper 19 bits of an operand.  A factor of 1 + 2^-11.5 ahead of
// that makes the cut a rounding: it adds 0.35 to 0.71 units in the last place of TF32, so
// that the error is 0.71 units at most and has no bias (rms 0.31 units, 0.29 for rounding
// to nearest), numbers that TF32 holds stay as they are, and so do infinities and NaN,
// which adding half a unit to the bits would lose.  The conversion instruction is too slow
// (tree decode of 512 x 32 heads x 16 places: 272 us with it, 236 with the product).
constexpr float kTf32 = 1.00034526698f, kLog2Tf32 = 4.98029e-4f;
__device__ __forceinline__ float to_tf32(float x) { return x * kTf32; }
// The same with the cut made, for values that are used outside the products, too.
__device__ __forceinline__ float cut_tf32(float x) {
  return __uint_as_float(__float_as_uint(x * kTf32) & 0xffffe000u);
}

__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// The larger of two numbers, NaN if one is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

}  // namespace kda
