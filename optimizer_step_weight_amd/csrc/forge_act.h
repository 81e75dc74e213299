// forge_act.h -- activations of a gated product and their derivatives, in fp32.
//
// The logistic function is 1 / (1 + 2^(-x log2 e)) by the hardware's exponential and reciprocal (one step
// of fp32 each); the rounded exponent adds |x| 2^-24 of its value, which the 2^-9 of a bf16 result does
// not show.  2^x runs into infinity and 1 / infinity is 0, so no |x| needs a branch.
#pragma once

#include "forge_ffn_internal.h"
#include "forge_rows.h"

namespace forge {

__device__ __forceinline__ float logistic(float x) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x * -1.4426950408889634f));
}

// value = act(g), slope = act'(g).
template <int ACT>
__device__ __forceinline__ void act_pair(float g, float& value, float& slope) {
  if constexpr (ACT == FORGE_ACT_K_SILU) {
    const float p = logistic(g);
    value = g * p;
    slope = p * __builtin_fmaf(g, 1.0f - p, 1.0f);
  } else if constexpr (ACT == FORGE_ACT_K_GELU_TANH) {
    // (1 + tanh z) / 2 is the logistic function of 2 z; past |g| = 64 it has its limit, and g^2 stays finite
    constexpr float c = 1.5957691216057308f;  // 2 sqrt(2 / pi)
    const float b = __builtin_fminf(__builtin_fmaxf(g, -64.0f), 64.0f), b2 = b * b;
    const float p = logistic(c * (b * __builtin_fmaf(0.044715f, b2, 1.0f)));
    value = g * p;
    slope = __builtin_fmaf(g * (p * (1.0f - p)), c * __builtin_fmaf(0.134145f, b2, 1.0f), p);
  } else if constexpr (ACT == FORGE_ACT_K_GELU) {
    const float p = 0.5f * erfcf(g * -0.70710678118654752f);
    value = g * p;
    slope = __builtin_fmaf(g * 0.3989422804014327f, __builtin_amdgcn_exp2f(g * (g * -0.72134752044448170f)), p);
  } else {
    value = g > 0.0f ? g : (g != g ? g : 0.0f);
    slope = g > 0.0f ? 1.0f : 0.0f;
  }
}

// f(activation) for the call's activation, the same in all lanes.
template <class F>
__device__ __forceinline__ void by_act(int act, F&& f) {
  using std::integral_constant;
  switch (act) {
    case FORGE_ACT_K_SILU: f(integral_constant<int, FORGE_ACT_K_SILU>{}); break;
    case FORGE_ACT_K_GELU: f(integral_constant<int, FORGE_ACT_K_GELU>{}); break;
    case FORGE_ACT_K_GELU_TANH: f(integral_constant<int, FORGE_ACT_K_GELU_TANH>{}); break;
    default: f(integral_constant<int, FORGE_ACT_K_RELU>{}); break;
  }
}

}  // namespace forge
