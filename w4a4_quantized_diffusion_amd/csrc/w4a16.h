// Shared pieces of the weight-only (W4A16) operators: the gate activations of
// a gated feed-forward block and their derivatives.
#pragma once

#include "internal.h"

namespace svdq_dev {

constexpr float LOG2E = 1.44269504088896340736f;

// a = act(x) and d = act'(x), for the SiLU x s, s = 1 / (1 + exp(-x)), and the
// tanh form of GELU, 0.5 x (1 + tanh u) = x s with s = 1 / (1 + exp(-2u)),
// u = sqrt(2/pi) (x + 0.044715 x^3).  With t the sigmoid's argument
// (x or 2u), act' = s + x t' s (1 - s).  exp by exp2 and the reciprocal are
// the hardware's (1 ulp each).  Beyond |x| = 128, s (1 - s) is 0 in fp32 for
// both (s or 1 - s is), and the clamp keeps x t' finite there, so that a large
// |x| gives act' = 0 or 1 and never inf * 0.
template <int ACT>
__device__ __forceinline__ float gate_sigmoid(float x) {
  float t = x;
  if constexpr (ACT == SVDQ_GELU) t = 1.5957691216057308f * (x + 0.044715f * x * x * x);
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-t * LOG2E));
}

template <int ACT>
__device__ __forceinline__ float gate_act(float x) {
  return x * gate_sigmoid<ACT>(x);
}

template <int ACT>
__device__ __forceinline__ void gate_act_grad(float x, float& a, float& d) {
  const float s = gate_sigmoid<ACT>(x);
  const float c = fminf(fmaxf(x, -128.f), 128.f);
  float t1 = 1.f;
  if constexpr (ACT == SVDQ_GELU) t1 = 1.5957691216057308f * (1.f + 0.134145f * c * c);
  a = x * s;
  d = s + c * t1 * (s * (1.f - s));
}

}  // namespace svdq_dev
