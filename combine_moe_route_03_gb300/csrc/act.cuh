// The activations of dense products and their slopes, binary32.
#pragma once

#include "common.cuh"

namespace moe {
namespace {

// The normal distribution function, and e^(-z^2 / 2) that it needs on the way.  For x >= 0
//   Phi(-x) = e^(-x^2 / 2) t P(t),  t = 1 / (1 + 0.4 x),
// with P of degree 9 fitted for x up to 13.5 by weighted least squares whose weights rise where the
// relative error is large (Lawson's iteration), to 2^-26 of the value; on the right 1 - Phi(-z).
// The tail on the left is a product, so it keeps its relative error where the function is next to
// nothing: with the quotient and the exponential within 2^-22 of theirs, all of it is within
// 1.15 2^-20 (1 + z^2 / 8) of the value (the second term: the exponential's argument in binary32).
// (Slopes of 8192 x 4096 values: 46 us, of silu 44.  Abramowitz and Stegun 7.1.26, four
// multiplications fewer, took 45, but its absolute error passes a 16-bit rounding of the value
// left of z = -3.6; the library's erff takes two branches, of which a warp mostly runs both: 52.)
__device__ __forceinline__ float normal_cdf(float z, float &e) {
  const float x = fabsf(z), t = __fdividef(1.0f, fmaf(0.4f, x, 1.0f));
  float p = 0.0319654532f;
  p = fmaf(p, t, -0.175461844f);
  p = fmaf(p, t, 0.379125178f);
  p = fmaf(p, t, -0.36978963f);
  p = fmaf(p, t, 0.115964055f);
  p = fmaf(p, t, -0.0249578636f);
  p = fmaf(p, t, 0.090691641f);
  p = fmaf(p, t, 0.133274511f);
  p = fmaf(p, t, 0.159611866f);
  p = fmaf(p, t, 0.159576654f);
  e = __expf(-0.5f * x * x);
  const float q = p * t * e;
  return z < 0.0f ? q : 1.0f - q;
}

__device__ __forceinline__ float activate(float z, int act) {
  if (act == MOE_ACT_RELU) return z < 0.0f ? 0.0f : z;  // keeps NaN
  if (act == MOE_ACT_GELU) {
    float e;
    return z * normal_cdf(z, e);
  }
  // silu: below -87 the quotient's divisor passes binary32's range; the sigmoid is e^z there
  if (act == MOE_ACT_SILU) return z < -87.0f ? z * __expf(z) : __fdividef(z, 1.0f + __expf(-z));
  return z;
}

__device__ __forceinline__ float slope(float z, int act) {
  if (act == MOE_ACT_RELU) return z > 0.0f ? 1.0f : z != z ? z : 0.0f;
  if (act == MOE_ACT_GELU) {  // Phi(z) + z phi(z)
    float e;
    const float c = normal_cdf(z, e);
    return fmaf(z * 0.39894228040143268f, e, c);
  }
  if (act == MOE_ACT_SILU) {
    // s + z s (1 - s), as above
    if (z < -87.0f) return __expf(z) * (1.0f + z);
    const float s = __fdividef(1.0f, 1.0f + __expf(-z));
    return fmaf(z * s, 1.0f - s, s);
  }
  return 1.0f;
}

}  // namespace
}  // namespace moe
