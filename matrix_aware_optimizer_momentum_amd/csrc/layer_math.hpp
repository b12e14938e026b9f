// The activations of the feed-forward layers and their derivatives, in
// float32, and what the products' epilogues make of them.
#pragma once

#include "layer_internal.hpp"

namespace sm {

// 1 / (1 + e^-z).  FINE (float32 layers): the compiler's exact division and
// expf.  Else (bf16 layers) the hardware's exp2 and reciprocal, off by a few
// 2^-23 and by |z| 2^-24 from the argument's rounding: far below bf16's half
// step of 2^-8 for every |z| that leaves a value above 1e-30.
template <bool FINE>
__device__ __forceinline__ float logistic(float z) {
  if constexpr (FINE) return 1.0f / (1.0f + expf(-z));
  else return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -1.44269504f));
}

// Phi(z) of the normal distribution, through the complement that keeps its
// relative precision at negative z.
__device__ __forceinline__ float normal_cdf(float z) { return 0.5f * erfcf(z * -0.70710678f); }

// 2u of gelu_tanh: its activation is z logistic(2u).
__device__ __forceinline__ float tanh_arg(float z) {
  return 1.59576912f * (z + 0.044715f * (z * z * z));
}

template <bool FINE>
__device__ __forceinline__ float act_value(int act, float z) {
  switch (act) {
    case SM_ACT_RELU: return z > 0.f ? z : (z == z ? 0.f : z);
    case SM_ACT_SILU: return z * logistic<FINE>(z);
    case SM_ACT_GELU: return z * normal_cdf(z);
    case SM_ACT_GELU_TANH: return z * logistic<FINE>(tanh_arg(z));
    default: return z;
  }
}

struct ActBoth {
  float value, slope;
};
template <bool FINE>
__device__ __forceinline__ ActBoth act_both(int act, float z) {
  switch (act) {
    case SM_ACT_RELU: return z > 0.f ? ActBoth{z, 1.f} : (z == z ? ActBoth{0.f, 0.f} : ActBoth{z, z});
    case SM_ACT_SILU: {
      const float p = logistic<FINE>(z);
      return {z * p, p * (1.f + z * (1.f - p))};
    }
    case SM_ACT_GELU: {
      const float p = normal_cdf(z);
      // phi(z) = e^(-z^2/2) / sqrt(2 pi)
      const float q = 0.39894228f * (FINE ? expf(-0.5f * z * z)
                                          : __builtin_amdgcn_exp2f(z * z * -0.72134752f));
      return {z * p, p + z * q};
    }
    case SM_ACT_GELU_TANH: {
      const float p = logistic<FINE>(tanh_arg(z));
      // (2u)' grows as z^2; beyond 16 p (1 - p) is 0, and stays so if z^2 overflows
      const float zc = fminf(fmaxf(z, -16.f), 16.f);
      const float du = 1.59576912f * (1.f + 0.134145f * (zc * zc));
      return {z * p, p + zc * p * (1.f - p) * du};
    }
    default: return {z, 1.f};
  }
}

}  // namespace sm
