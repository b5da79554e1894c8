// The activations of the feed-forward block, in FP32, and their derivatives.
//
//   ReLU      z for z > 0, else 0                  SiLU  z s(z),  s(v) = 1 / (1 + e^-v)
//   GELU      z Phi(z), Phi(z) = erfc(-z / sqrt 2) / 2
//   GELU_TANH z (1 + tanh a) / 2 = z s(2 a),       a = sqrt(2 / pi) (z + 0.044715 z^3)
// The logistic function is formed from e^-|v|, which neither overflows nor
// cancels, so the left tails keep their relative precision (what
// 1 + erf or 1 + tanh would lose there).  Beyond |z| = 200 a tail is what it is
// at 200 (0, or z itself), so that an infinity gives the limit and not inf * 0.
// A NaN stays one.  e^v is 2^(v log2 e) with the hardware's 2^v: off by |v| 2^-24
// and 2^-22 of its value, so at most 3e-7 of anything that is formed with it
// (where |v| is large the value itself is small).
#pragma once

#include "device_common.hpp"

namespace fp8g {

constexpr int kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4;  // FP8G_ACT_*

__device__ __forceinline__ float exp_fast(float v) { return __builtin_amdgcn_exp2f(v * 1.44269504f); }

// s(v) and s(-v).
__device__ __forceinline__ void logistic(float v, float& p, float& q) {
  const float e = exp_fast(-fabsf(v)), r = __builtin_amdgcn_rcpf(1.f + e);
  p = v < 0.f ? e * r : r;
  q = v < 0.f ? r : e * r;
}

__device__ __forceinline__ float gelu_tanh_arg(float z) {  // 2 a
  return 1.59576912f * fmaf(0.044715f * z * z, z, z);
}

__device__ __forceinline__ float activate(int act, float z) {
  if (act == kActNone) return z;
  if (act == kActRelu) return z < 0.f ? 0.f : z;
  const float b = z < -200.f ? -200.f : z;
  if (act == kActGelu) return b * (0.5f * erfcf(b * -0.707106781f));
  const float v = act == kActSilu ? b : gelu_tanh_arg(b > 200.f ? 200.f : b);
  float p, q;
  logistic(v, p, q);
  return b * p;
}

__device__ __forceinline__ float activate_grad(int act, float z) {
  if (act == kActNone) return 1.f;
  if (act == kActRelu) return z > 0.f ? 1.f : z != z ? z : 0.f;
  const float b = z < -200.f ? -200.f : z > 200.f ? 200.f : z;
  if (act == kActGelu) return fmaf(b * 0.398942280f, exp_fast(-0.5f * b * b), 0.5f * erfcf(b * -0.707106781f));
  const float v = act == kActSilu ? b : gelu_tanh_arg(b);
  const float dv = act == kActSilu ? 1.f : 1.59576912f * fmaf(3.f * 0.044715f * b, b, 1.f);
  float p, q;
  logistic(v, p, q);
  return fmaf(b * dv * p, q, p);
}

}  // namespace fp8g
