// norm_math.cuh -- the reciprocal square root of the RMSNorm kernels (simt.cu, rope.cu).
#pragma once

namespace cpattn {

// 1/sqrt(a) for a > 0: the special-function unit's estimate refined by one Newton step on
// f(y) = 1/y^2 - a (y' = y * (3 - a y^2) / 2), which brings it to about an ulp of the
// float32 1/sqrt(a) for every positive finite a (subnormal a included).
__device__ __forceinline__ float rsqrt_refined(float a) {
  float y;
  asm("rsqrt.approx.f32 %0, %1;" : "=f"(y) : "f"(a));
  const float hy = 0.5f * y;
  return fmaf(hy, fmaf(-a * y, y, 1.0f), y);  // y + (y/2)(1 - a y^2)
}

// The factor of a row with a = mean(x^2) + eps.  An all-zero row with eps = 0 stays 0; a NaN or an
// infinity in a row, or squares past float32, make it NaN as a whole (any test that NaN fails, such as
// a > 0, would turn the rest of such a row into zeros).
__device__ __forceinline__ float row_factor(float a) { return a == 0.f ? 0.f : rsqrt_refined(a); }

}  // namespace cpattn
