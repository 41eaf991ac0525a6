// The activations of the plain layers and their derivatives, in fp32.
//
// SiLU p h with h = 1 / (1 + e^-p), and GELU in its tanh form, which is p h
// with h = 1 / (1 + e^-2w), w = sqrt(2 / pi) (p + 0.044715 p^3). The hardware's
// exponential and reciprocal are within 1 ulp, the exponent's product within
// |p| 2^-24 of e^-p: some 10^-7 of the result where it is not negligible.
#pragma once

#include "common.h"
#include "../../include/ttt.h"

constexpr float kGelu0 = 0.7978845608028654f, kGelu1 = 0.044715f;

__device__ __forceinline__ float sigmoid_of(float p, int act) {
  const float e = act == TTT_ACT_SILU ? p : 2.f * kGelu0 * (p + kGelu1 * p * p * p);
  return __builtin_amdgcn_rcpf(1.0f + __expf(-e));
}

// The comparisons let a NaN through.
__device__ __forceinline__ float act_of(float p, int act) {
  if (act == TTT_ACT_NONE) return p;
  if (act == TTT_ACT_RELU) return p < 0.f ? 0.f : p;
  return p * sigmoid_of(p, act);
}

// Both, from one h. Beyond |p| = 120 the derivatives are 0 and 1 to fp32's
// last bit, and products such as p^2 h would leave its range, so p is held
// there.
__device__ __forceinline__ void act_grad_of(float p, int act, float &a, float &da) {
  if (act == TTT_ACT_NONE) {
    a = p;
    da = 1.f;
    return;
  }
  if (act == TTT_ACT_RELU) {
    a = p < 0.f ? 0.f : p;
    da = p != p ? p : p > 0.f ? 1.f : 0.f;
    return;
  }
  const float q = p > 120.f ? 120.f : p < -120.f ? -120.f : p;
  const float h = sigmoid_of(q, act);
  a = p * h;
  const float slope = act == TTT_ACT_SILU ? 1.f : 2.f * kGelu0 * (1.f + 3.f * kGelu1 * q * q);
  da = h + q * h * (1.f - h) * slope;
}
