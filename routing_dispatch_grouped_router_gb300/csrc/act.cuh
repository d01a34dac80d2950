// Activations of the dense product and their derivatives, in fp32.  silu and
// the tanh form of gelu are both z sigmoid(a(z)):
//   silu: a = z;  gelu: a = 2 sqrt(2/pi) (z + 0.044715 z^3)
//   (z sigmoid(a))' = sig + z sig (1 - sig) a'
// The sigmoid through the hardware exponential and reciprocal: __expf is within
// 2 + 1.17 |a| ulp, so that silu near -20 has some 25 ulp (of a value of -4e-8),
// and the sigmoid is 0 from 1 + exp(-a) = 2^126 on (a below -87).
#pragma once

#include "../../include/mok.h"

namespace mok {

constexpr float kGeluA = 1.5957691216057308f;  // 2 sqrt(2/pi)
constexpr float kGeluB = 0.044715f;

__device__ __forceinline__ float act_sigmoid(float a) {
  return __fdividef(1.0f, 1.0f + __expf(-a));
}

__device__ __forceinline__ float act_value(float z, int act) {
  if (act == MOK_ACT_NONE) return z;
  if (act == MOK_ACT_RELU) return z > 0.f ? z : (z <= 0.f ? 0.f : z);  // NaN stays
  const float a = act == MOK_ACT_SILU ? z : kGeluA * fmaf(kGeluB * z * z, z, z);
  const float s = act_sigmoid(a);
  return s == 0.f ? 0.f : z * s;  // the limit for z -> -inf, where z s is -inf 0
}

__device__ __forceinline__ float act_slope(float z, int act) {
  if (act == MOK_ACT_NONE) return 1.0f;
  if (act == MOK_ACT_RELU) return z > 0.f ? 1.0f : 0.0f;
  const bool silu = act == MOK_ACT_SILU;
  const float a = silu ? z : kGeluA * fmaf(kGeluB * z * z, z, z);
  const float da = silu ? 1.0f : kGeluA * fmaf(3.0f * kGeluB * z, z, 1.0f);
  const float s = act_sigmoid(a);
  const float u = s * (1.0f - s);
  return u == 0.f ? s : fmaf(z * u, da, s);  // (a' may be inf where the sigmoid is 0 or 1)
}

}  // namespace mok
