// The activations of the feed-forward block, in FP32, and their derivatives.
//
//   ReLU      z for z > 0, else 0                  SiLU  z s(z),  s(v) = 1 / (1 + e^-v)
//   GELU      z Phi(z), Phi the normal distribution's function
//   GELU_TANH z (1 + tanh a) / 2 = z s(2 a),       a = sqrt(2 / pi) (z + 0.044715 z^3)
// Nothing here cancels, so the left tails keep their relative precision (what
// 1 + erf or 1 + tanh would lose there) down to values of 1e-36; what is smaller
// may come out as 0, since the logistic function is the reciprocal of 1 + e^-v as
// it stands and the hardware's reciprocal has no subnormal results.  Phi(-z) for z >= 0 is e^(-z^2 / 2) R(t), t = 1 /
// (1 + 0.3 z), R a polynomial fitted to e^(z^2 / 2) erfc(z / sqrt 2) / 2 for the
// least relative error (1.6e-7 on 0 <= z <= 14.5, 5e-7 as FP32 forms it).  An
// infinity gives the limit (0 or itself) because what is multiplied is cut off
// at -200, where every function is 0; a NaN stays one.  e^v is the hardware's
// 2^(v log2 e), off by |v| 2^-24 and 2^-22 of its value.
//
// A tile's epilogue runs while its matrix cores wait, so the instructions
// count: of the 64 a clock that a CU does, an element takes about 14 for the
// logistic forms (the exponential and the reciprocal as four each).
#pragma once

#include "device_common.hpp"

namespace fp8g {

constexpr int kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4;  // FP8G_ACT_*

// 1 / (1 + 2^v).
__device__ __forceinline__ float logistic2(float v) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(v));
}

// v with -200 in place of anything below it.
__device__ __forceinline__ float not_below(float v) { return v < -200.f ? -200.f : v; }

constexpr float kLog2e = 1.44269504f;
constexpr float kGeluTanh0 = -1.59576912f * kLog2e, kGeluTanh1 = 0.044715f * kGeluTanh0;  // of z and z^3: -2 a log2 e

// Phi(-|z|), and e^(-z^2 / 2).
__device__ __forceinline__ float normal_tail(float z, float& gauss) {
  const float t = __builtin_amdgcn_rcpf(fmaf(0.3f, fabsf(z), 1.f));
  gauss = __builtin_amdgcn_exp2f(z * z * (-0.5f * kLog2e));
  float r = 0.0354237121f;
  r = fmaf(r, t, -0.156158359f);
  r = fmaf(r, t, 0.204556645f);
  r = fmaf(r, t, -0.0520339007f);
  r = fmaf(r, t, 0.127691717f);
  r = fmaf(r, t, 0.100175962f);
  r = fmaf(r, t, 0.120712134f);
  r = fmaf(r, t, 0.119632007f);
  return r * t * gauss;
}

template <int ACT>
__device__ __forceinline__ float activate(float z) {
  if constexpr (ACT == kActRelu) return z < 0.f ? 0.f : z;
  if constexpr (ACT == kActSilu) return not_below(z) * logistic2(z * -kLog2e);
  if constexpr (ACT == kActGeluTanh) return not_below(z) * logistic2(z * fmaf(z * z, kGeluTanh1, kGeluTanh0));
  if constexpr (ACT == kActGelu) {
    float gauss;
    const float q = normal_tail(z, gauss);
    return not_below(z) * (z < 0.f ? q : 1.f - q);
  }
  return z;
}

template <int ACT>
__device__ __forceinline__ float activate_grad(float z) {
  if constexpr (ACT == kActNone) return 1.f;
  if constexpr (ACT == kActRelu) return z > 0.f ? 1.f : z != z ? z : 0.f;
  const float b = z < -200.f ? -200.f : z > 200.f ? 200.f : z;  // beyond, the derivative is 0 or 1
  if constexpr (ACT == kActGelu) {
    float gauss;
    const float q = normal_tail(b, gauss);
    return fmaf(b * 0.398942280f, gauss, z < 0.f ? q : 1.f - q);
  }
  // p + b v' p (1 - p), 1 - p as the logistic function of -v
  const float k = ACT == kActSilu ? b * -kLog2e : b * fmaf(b * b, kGeluTanh1, kGeluTanh0);
  const float e = __builtin_amdgcn_exp2f(-fabsf(k)), r = __builtin_amdgcn_rcpf(1.f + e), er = e * r;
  const float p = k > 0.f ? er : r;
  const float bdv = ACT == kActSilu ? b : b * fmaf(b * b, 3.f * 0.044715f * 1.59576912f, 1.59576912f);
  return fmaf(bdv * r, er, p);
}

// f(Int<act>{}) with the activation as a compile-time constant.
template <int N>
struct ActTag { static constexpr int value = N; };
template <typename F>
__device__ __forceinline__ void by_activation(int act, F&& f) {
  switch (act) {
    case kActRelu: f(ActTag<kActRelu>{}); break;
    case kActGelu: f(ActTag<kActGelu>{}); break;
    case kActGeluTanh: f(ActTag<kActGeluTanh>{}); break;
    case kActSilu: f(ActTag<kActSilu>{}); break;
    default: f(ActTag<kActNone>{}); break;
  }
}

__device__ __forceinline__ float activate(int act, float z) {
  float v = 0.f;
  by_activation(act, [&](auto tag) { v = activate<decltype(tag)::value>(z); });
  return v;
}

}  // namespace fp8g
