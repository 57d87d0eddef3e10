// The AdamW element update and its per-call scalars, shared by the steps with
// binary32 and with 8-bit moments.
//
// Page "Infra: Data Parallel" (pufanyi.com), section "Zero Redundancy
// Optimizer (ZeRO)": AdamW updates each element independently.
#pragma once

#include <cmath>

#include "device_common.hpp"
#include "zero_shard.h"

namespace zs {

struct Scalars {
  float s, rho, a_wd, B1, C1, B2, C2, E;
};

// The AdamW element update, binary32, one rounding per operation.
__device__ __forceinline__ void adamw(float g, float& th, float& m, float& v, const Scalars& k) {
  const float m1 = k.B1 * m + k.C1 * g;
  const float v1 = k.B2 * v + k.C2 * (g * g);
  const float d = __builtin_sqrtf(v1) * k.rho + k.E;
  th = k.a_wd * th - k.s * (m1 / d);
  m = m1;
  v = v1;
}

// -------------------------------------------------------------- host side
inline bool hp_ok(const zero_adamw& hp) {
  return std::isfinite(hp.lr) && std::isfinite(hp.eps) && std::isfinite(hp.weight_decay) &&
         std::isfinite(hp.beta1) && std::isfinite(hp.beta2) && hp.beta1 >= 0.0 &&
         hp.beta1 < 1.0 && hp.beta2 >= 0.0 && hp.beta2 < 1.0;
}

// Per-call scalars: binary64, each rounded once to binary32.
inline Scalars make_scalars(const zero_adamw& hp, int64_t t) {
  const double bc1 = 1.0 - std::pow(hp.beta1, (double)t);
  const double bc2 = 1.0 - std::pow(hp.beta2, (double)t);
  Scalars k;
  k.s = (float)(hp.lr / bc1);
  k.rho = (float)(1.0 / std::sqrt(bc2));
  k.a_wd = (float)(1.0 - hp.lr * hp.weight_decay);
  k.B1 = (float)hp.beta1;
  k.C1 = (float)(1.0 - hp.beta1);
  k.B2 = (float)hp.beta2;
  k.C2 = (float)(1.0 - hp.beta2);
  k.E = (float)hp.eps;
  return k;
}

}  // namespace zs
