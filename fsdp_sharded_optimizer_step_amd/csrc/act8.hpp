// The 8-bit activation format on the device.
//
// A row is cut into blocks of 128 columns (the last may be shorter).  A block
// holds e4m3 codes (OCP: four exponent bits, three fraction bits, largest
// value 448, a NaN, no infinities) and one byte e, the biased exponent of its
// scale 2^(e-127): the smallest power of two, e at least 10, that brings the
// block's largest finite magnitude to 448 at most.  A code is the rounding
// (to nearest, ties to even) of x / scale, which is exact before that one
// rounding because the scale is a power of two, and no finite value
// saturates.  Infinities and NaN become NaN codes and leave the other values
// of their block alone.  e >= 10 makes every value that a code stands for
// (2^-9 * 2^-117 at least) a normal bf16 number or zero, so reading back into
// bf16, and the bf16 product of the weight gradient, rounds nothing.
#pragma once

#include "tensor_place.hpp"

namespace zs {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

constexpr int kAct8Block = ZERO_ACT8_BLOCK;
constexpr int kAct8MinByte = 10;
constexpr int kAct8Lanes = kAct8Block / 8;  // lanes of a block, 8 columns each: one row of 16 lanes

// Magnitude bits that count for the scale: 0 for infinities and NaN.
__device__ __forceinline__ uint32_t finite_mag(float x) {
  const uint32_t b = __float_as_uint(x) & 0x7fffffffu;
  return b < 0x7f800000u ? b : 0u;
}

// Largest value over the 16 lanes of a DPP row, in every lane.
template <int ROR>
__device__ __forceinline__ uint32_t ror16(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + ROR, 0xf, 0xf, false);
}
__device__ __forceinline__ uint32_t max16(uint32_t v) {
  v = max(v, ror16<8>(v));
  v = max(v, ror16<4>(v));
  v = max(v, ror16<2>(v));
  return max(v, ror16<1>(v));
}

// The block's byte from its largest magnitude m*2^k, 1 <= m < 2:
// 448 = 1.75 * 2^8, so the scale is 2^(k-8), or 2^(k-7) where m > 1.75.
__device__ __forceinline__ uint32_t act8_byte(uint32_t amax) {
  const int e = (int)(amax >> 23) - 8 + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0);
  return (uint32_t)max(e, kAct8MinByte);
}
__device__ __forceinline__ float act8_scale(uint32_t e) { return __uint_as_float(e << 23); }
// 1 / scale = 2^(127-e), exact (e is 10 to 247)
__device__ __forceinline__ float act8_inv(uint32_t e) { return __uint_as_float((254u - e) << 23); }

// Codes of 4 values.  The conversion instruction rounds to nearest even; an
// infinity is made a NaN first (inf - inf), since it would saturate.
__device__ __forceinline__ float nan_if_inf(float x) {
  return (__float_as_uint(x) & 0x7fffffffu) == 0x7f800000u ? __uint_as_float(0x7fc00000u) : x;
}
__device__ __forceinline__ uint32_t act8_pack4(const float* x, float inv) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(nan_if_inf(x[0]) * inv, nan_if_inf(x[1]) * inv, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(nan_if_inf(x[2]) * inv, nan_if_inf(x[3]) * inv,
                                                   w, true);
}

// Two codes of a word (low or high half) as bf16 or binary32 values.
template <bool HI>
__device__ __forceinline__ uint32_t act8_bf16(uint32_t w, float scale) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)w, scale, HI));
}
template <bool HI>
__device__ __forceinline__ f32x2 act8_f32(uint32_t w, float scale) {
  return __builtin_amdgcn_cvt_scalef32_pk_f32_fp8((int)w, scale, HI);
}
__device__ __forceinline__ u32x2 act8_bf16x4(uint32_t w, float scale) {
  return u32x2{act8_bf16<false>(w, scale), act8_bf16<true>(w, scale)};
}

}  // namespace zs
