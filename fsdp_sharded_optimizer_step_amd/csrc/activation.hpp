// Activations and their derivatives, binary32.
#pragma once

#include "tensor_place.hpp"

namespace zs {

constexpr float kSqrtHalf = 0.70710678118654752f, kInvSqrt2Pi = 0.39894228040143268f;
constexpr float kTanhScale = 1.59576912160573071f;  // 2 sqrt(2 / pi)

// 1 / (1 + exp(-x))
__device__ __forceinline__ float sigmoid(float x) { return 1.f / (1.f + expf(-x)); }
// the normal distribution's function; by erfc, which keeps its digits where
// the value is next to zero
__device__ __forceinline__ float normal_cdf(float x) { return 0.5f * erfcf(-x * kSqrtHalf); }

template <int ACT>
__device__ __forceinline__ float activate(float x) {
  if constexpr (ACT == ZERO_ACT_RELU) return x > 0.f ? x : (x != x ? x : 0.f);
  if constexpr (ACT == ZERO_ACT_GELU) return x * normal_cdf(x);
  if constexpr (ACT == ZERO_ACT_GELU_TANH)  // (1 + tanh(u)) / 2 = sigmoid(2u)
    return x * sigmoid(kTanhScale * (x + 0.044715f * x * x * x));
  if constexpr (ACT == ZERO_ACT_SILU) return x * sigmoid(x);
  return x;
}
template <int ACT>
__device__ __forceinline__ float slope(float x) {
  if constexpr (ACT == ZERO_ACT_RELU) return x > 0.f ? 1.f : 0.f;
  if constexpr (ACT == ZERO_ACT_GELU) return normal_cdf(x) + x * (kInvSqrt2Pi * expf(-0.5f * x * x));
  if constexpr (ACT == ZERO_ACT_GELU_TANH) {
    if (__builtin_fabsf(x) > 30.f) return x > 0.f ? 1.f : 0.f;  // before x*x overflows
    const float p = sigmoid(kTanhScale * (x + 0.044715f * x * x * x));
    return p + x * p * (1.f - p) * (kTanhScale * (1.f + 0.134145f * x * x));
  }
  if constexpr (ACT == ZERO_ACT_SILU) {
    const float p = sigmoid(x);
    return p + x * p * (1.f - p);
  }
  return 1.f;
}

// Four values; one branch for the wave.
template <int ACT, bool SLOPE>
__device__ __forceinline__ void apply4(f32x4& v) {
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = SLOPE ? slope<ACT>(v[j]) : activate<ACT>(v[j]);
}
template <bool SLOPE>
__device__ __forceinline__ f32x4 apply4(int act, f32x4 v) {
  switch (act) {
    case ZERO_ACT_RELU: apply4<ZERO_ACT_RELU, SLOPE>(v); break;
    case ZERO_ACT_GELU: apply4<ZERO_ACT_GELU, SLOPE>(v); break;
    case ZERO_ACT_GELU_TANH: apply4<ZERO_ACT_GELU_TANH, SLOPE>(v); break;
    case ZERO_ACT_SILU: apply4<ZERO_ACT_SILU, SLOPE>(v); break;
    default: apply4<ZERO_ACT_NONE, SLOPE>(v); break;
  }
  return v;
}

inline bool activation_ok(int32_t act) { return act >= ZERO_ACT_NONE && act <= ZERO_ACT_SILU; }

}  // namespace zs
