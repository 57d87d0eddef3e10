// Activations and their derivatives, binary32.
//
// One exponential and one reciprocal each, of the hardware's accuracy: below
// zero the relative error grows with the exponential's argument (at every bf16
// x below -5: gelu_tanh 111 * 2^-24 at most, silu 58 * 2^-24, at -87), far below
// what bf16 resolves, and factors below 2^-126 are 0.
#pragma once

#include "tensor_place.hpp"

namespace zs {

constexpr float kSqrtHalf = 0.70710678118654752f, kInvSqrt2Pi = 0.39894228040143268f;
constexpr float kTanhScale = 1.59576912160573071f;  // 2 sqrt(2 / pi)

// e^x by the exponential instruction (of 2, 1 unit of the last place off): its
// argument's rounding makes it |x| 2^-24 of itself off.  Results below 2^-126
// are 0.
__device__ __forceinline__ float exp_of(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504088896341f); }
// 1 / (1 + e^-x); the reciprocal is 1 unit of the last place off
__device__ __forceinline__ float sigmoid(float x) { return __builtin_amdgcn_rcpf(1.f + exp_of(-x)); }

// The normal distribution's function, by erfc(z) = t exp(-z^2 + Q(t)), t = 1 /
// (1 + 0.4 z), for z >= 0: next to zero, for x below it, it keeps its digits,
// which 1 + erf would not.  Q, of degree 8, is fitted to log(erfc(z) exp(z^2) /
// t) over z up to 10.5 for the smallest largest error, 9e-8 (least squares over
// Chebyshev polynomials, reweighted).  In binary32 the function is off by 5 *
// 2^-24 at most, and down to x = -5 by 44 * 2^-24 of itself.  Further down the
// error of z^2 and of the exponential's argument tells: 2^-24 * (44 + 3.5 x^2) of
// itself at most; x times it at every bf16 x: 84 * 2^-24 down to -8, 218 * 2^-24
// (1.3e-5) down to -13, where it becomes 0.
__device__ __forceinline__ float normal_cdf(float x) {
  const float z = __builtin_fabsf(x) * kSqrtHalf;
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.4f, z, 1.f));
  float q = -0.207837114f;
  q = __builtin_fmaf(q, t, 0.926345742f);
  q = __builtin_fmaf(q, t, -1.48961016f);
  q = __builtin_fmaf(q, t, 1.00340859f);
  q = __builtin_fmaf(q, t, -0.446484282f);
  q = __builtin_fmaf(q, t, 0.301732f);
  q = __builtin_fmaf(q, t, 0.399403593f);
  q = __builtin_fmaf(q, t, 1.00175667f);
  q = __builtin_fmaf(q, t, -1.48871513f);
  const float h = 0.5f * t * exp_of(__builtin_fmaf(-z, z, q));
  return x < 0.f ? h : 1.f - h;
}

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
  if constexpr (ACT == ZERO_ACT_GELU) return normal_cdf(x) + x * (kInvSqrt2Pi * exp_of(-0.5f * x * x));
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

template <bool SLOPE>
__device__ __forceinline__ float apply1(int act, float x) {
  switch (act) {
    case ZERO_ACT_RELU: return SLOPE ? slope<ZERO_ACT_RELU>(x) : activate<ZERO_ACT_RELU>(x);
    case ZERO_ACT_GELU: return SLOPE ? slope<ZERO_ACT_GELU>(x) : activate<ZERO_ACT_GELU>(x);
    case ZERO_ACT_GELU_TANH: return SLOPE ? slope<ZERO_ACT_GELU_TANH>(x) : activate<ZERO_ACT_GELU_TANH>(x);
    case ZERO_ACT_SILU: return SLOPE ? slope<ZERO_ACT_SILU>(x) : activate<ZERO_ACT_SILU>(x);
    default: return SLOPE ? 1.f : x;
  }
}
// Eight values; one branch for the wave.
template <int ACT, bool SLOPE>
__device__ __forceinline__ void apply8(float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = SLOPE ? slope<ACT>(v[j]) : activate<ACT>(v[j]);
}
template <bool SLOPE>
__device__ __forceinline__ void apply8(int act, float (&v)[8]) {
  switch (act) {
    case ZERO_ACT_RELU: apply8<ZERO_ACT_RELU, SLOPE>(v); break;
    case ZERO_ACT_GELU: apply8<ZERO_ACT_GELU, SLOPE>(v); break;
    case ZERO_ACT_GELU_TANH: apply8<ZERO_ACT_GELU_TANH, SLOPE>(v); break;
    case ZERO_ACT_SILU: apply8<ZERO_ACT_SILU, SLOPE>(v); break;
    default: apply8<ZERO_ACT_NONE, SLOPE>(v); break;
  }
}

// 8 bf16 values, as loaded, and back.
__device__ __forceinline__ void widen8(u32x4 w, float (&x)[8]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    x[2 * k] = bf16_lo(w[k]);
    x[2 * k + 1] = bf16_hi(w[k]);
  }
}
// To nearest, ties to even, subnormals kept, by the conversion instruction.
__device__ __forceinline__ uint32_t round2(float lo, float hi) {
  typedef float v2f __attribute__((ext_vector_type(2)));
  typedef __bf16 v2b __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((v2f{lo, hi}), v2b));
}
__device__ __forceinline__ u32x4 round8(const float (&x)[8]) {
  return u32x4{round2(x[0], x[1]), round2(x[2], x[3]), round2(x[4], x[5]), round2(x[6], x[7])};
}
// The first n of 8 neighbouring values, n below 8; the others are zeros.
__device__ __forceinline__ u32x4 load_some(const uint16_t* p, int n) {
  u32x4 w = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int k = 0; k < 7; ++k)
    if (k < n) w[k >> 1] |= (uint32_t)p[k] << (16 * (k & 1));
  return w;
}
__device__ __forceinline__ void store_some(uint16_t* p, u32x4 w, int n) {
#pragma unroll
  for (int k = 0; k < 7; ++k)
    if (k < n) p[k] = (uint16_t)(w[k >> 1] >> (16 * (k & 1)));
}

inline bool activation_ok(int32_t act) { return act >= ZERO_ACT_NONE && act <= ZERO_ACT_SILU; }

}  // namespace zs
