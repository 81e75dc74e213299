// forge_act.h -- activations of a gated product and their derivatives, in fp32.
//
// The logistic function is 1 / (1 + 2^(-x log2 e)) by the hardware's exponential and reciprocal (one step
// of fp32 each); the rounded exponent adds |x| 2^-24 of its value, which the 2^-9 of a bf16 result does
// not show.  2^x runs into infinity and 1 / infinity is 0, so no |x| needs a branch.  Neither instruction gives numbers
// below 2^-126: there exponentials and logistic functions are 0.
#pragma once

#include "forge_ffn_internal.h"
#include "forge_rows.h"

namespace forge {

// The logistic function of x = -e / log2 e.
__device__ __forceinline__ float logistic_exp2(float e) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(e));
}

// value = act(g), slope = act'(g).
template <int ACT>
__device__ __forceinline__ void act_pair(float g, float& value, float& slope) {
  if constexpr (ACT == FORGE_ACT_K_SILU) {
    const float p = logistic_exp2(g * -1.4426950408889634f);
    value = g * p;
    slope = p * __builtin_fmaf(g, 1.0f - p, 1.0f);
  } else if constexpr (ACT == FORGE_ACT_K_GELU_TANH) {
    // (1 + tanh z) / 2 is the logistic function of 2 z; past |g| = 64 it has its limit, and g^2 stays finite
    constexpr float c = 1.5957691216057308f, l = -2.3022081981443250f;  // 2 sqrt(2 / pi), -c log2 e
    const float b = __builtin_amdgcn_fmed3f(g, -64.0f, 64.0f), b2 = b * b;
    const float p = logistic_exp2(b * __builtin_fmaf(0.044715f * l, b2, l));
    value = g * p;
    slope = __builtin_fmaf(value * (1.0f - p), __builtin_fmaf(0.134145f * c, b2, c), p);
  } else if constexpr (ACT == FORGE_ACT_K_GELU) {
    // For a = |g|, q = erfc(a / sqrt 2) / 2 = e^(-a^2 / 2) t R(t) with t = 1 / (1 + 0.45 a / sqrt 2): e^(z^2) erfc(z) is
    // smooth in t from z = 0 to infinity, so one polynomial (fitted to its relative error, 3.2e-8) serves all a
    // without branches; q is off by (a^2 + 7) 2^-24 of itself.
    const float a = fabsf(g), e = __builtin_amdgcn_exp2f(g * (g * -0.72134752044448170f));
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.31819806f, a, 1.0f));
    float r = -0.020695472f;
    r = __builtin_fmaf(r, t, 0.09534358f);
    r = __builtin_fmaf(r, t, -0.15029059f);
    r = __builtin_fmaf(r, t, 0.07119987f);
    r = __builtin_fmaf(r, t, -0.011178632f);
    r = __builtin_fmaf(r, t, 0.05997511f);
    r = __builtin_fmaf(r, t, 0.087626085f);
    r = __builtin_fmaf(r, t, 0.11413582f);
    r = __builtin_fmaf(r, t, 0.12694158f);
    r = __builtin_fmaf(r, t, 0.12694266f);
    const float q = e * (t * r), p = g < 0.0f ? q : 1.0f - q;
    value = g * p;
    slope = __builtin_fmaf(g * 0.3989422804014327f, e, p);
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
