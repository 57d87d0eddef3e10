// Moments in 8 bits on the device.
//
// A bucket's slice of the shard is cut into blocks of 128 elements (the last
// may be shorter).  A block of a moment is a code an element and one byte e,
// the biased exponent of the block's scale 2^(e-127).
//
//   first moment   the e4m3 codes and the scale of the 8-bit activations
//   second moment  4 exponent and 4 fraction bits and no sign:
//                  c < 16: c * 2^-18,  else (1 + (c & 15) / 16) * 2^((c >> 4) - 15)
//                  times the scale; 255 is a NaN.  It is never negative, so the
//                  sign's bit buys a fraction bit; the exponent's range, 2^19 in
//                  the moment, is 2^9.5 in the gradients that it averages.
//
// A moment decays by (1 - beta) of itself a step, less than the distance of
// two codes where beta is near 1: the nearest code would be the old one for
// ever.  So the step rounds at random, up with the probability of the part
// that is cut off: the expected value is the moment itself.  But a second moment
// above zero keeps the smallest code at least, since one of zero would leave the
// first moment divided by eps: next to the smallest code, 2^-19 to 2^-18 of the
// block's largest value, it is biased upwards and stops decaying.
#pragma once

#include "act8.hpp"

namespace zs {

constexpr int kMomentBlock = ZERO_ACT8_BLOCK;
constexpr int kVMinByte = 19;   // its smallest code is 2^-126: every value is a normal number
constexpr int kVMaxByte = 253;  // 2^(127-253) is still a normal number

// Largest value over the 32 lanes of a block: two DPP rows.
__device__ __forceinline__ uint32_t max32(uint32_t v) {
  v = max16(v);
  const auto w = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  return max((uint32_t)w[0], (uint32_t)w[1]);
}

// The block's byte from its largest magnitude m*2^k, 1 <= m < 2: the largest
// code of scale 1 is 1.875.
__device__ __forceinline__ uint32_t v8_byte(uint32_t amax) {
  const int e = (int)(amax >> 23) + ((amax & 0x7fffffu) > 0x700000u ? 1 : 0);
  return (uint32_t)min(max(e, kVMinByte), kVMaxByte);
}

// A code is the upper part of the pattern of a binary32 value that has the
// code's own exponent field, small codes being subnormals.
constexpr float kToM = 0x1p-120f, kToV = 0x1p-112f, kFromV = 0x1p112f;

__device__ __forceinline__ float v8_value(uint32_t c, float scale) {
  const float x = __uint_as_float(c << 19) * kFromV * scale;
  return c == 255u ? __uint_as_float(0x7fc00000u) : x;
}

// What is added to a pattern before its lower bits are cut off: 16 random
// bits at the top of those (their middle, so that the sum of the parts above
// and below is even), or what rounds to the nearest, ties to even.
struct AtRandom {
  uint32_t h;  // 32 bits: the lower half for the first moment, the upper half for the second
  __device__ __forceinline__ uint32_t m(uint32_t) const { return ((h & 0xffffu) << 4) + 8u; }
  __device__ __forceinline__ uint32_t v(uint32_t) const { return ((h >> 16) << 3) + 4u; }
};
struct ToNearest {
  __device__ __forceinline__ uint32_t m(uint32_t b) const { return 0x7ffffu + ((b >> 20) & 1u); }
  __device__ __forceinline__ uint32_t v(uint32_t b) const { return 0x3ffffu + ((b >> 19) & 1u); }
};

// inv: 1 / scale
template <class R>
__device__ __forceinline__ uint32_t m8_code(float x, float inv, const R& r) {
  const uint32_t a = __float_as_uint(x) & 0x7fffffffu;
  const uint32_t b = __float_as_uint(__uint_as_float(a) * inv * kToM);
  uint32_t c = min((b + r.m(b)) >> 20, 126u);
  if (a >= 0x7f800000u) c = 127u;
  return c | ((__float_as_uint(x) >> 24) & 0x80u);
}
template <class R>
__device__ __forceinline__ uint32_t v8_code(float x, float inv, const R& r) {
  const uint32_t a = __float_as_uint(x) & 0x7fffffffu;
  const uint32_t b = __float_as_uint(__uint_as_float(a) * inv * kToV);
  uint32_t c = min((b + r.v(b)) >> 19, 254u);
  c = max(c, a != 0u ? 1u : 0u);
  return a >= 0x7f800000u ? 255u : c;
}

// 32 random bits for element i of the shard: products with odd numbers and
// shifts, keyed by the step's two words.  The numbers are four of the five
// prime constants of the published hash xxHash32; the steps are not its own.
struct Random {
  uint32_t k0, k1;
};
constexpr uint32_t kMulLow = 0x9E3779B1u, kMulHigh = 0x85EBCA77u;
__device__ __forceinline__ uint32_t random_seed(const Random& r, int64_t i) {
  return (uint32_t)i * kMulLow + (uint32_t)(i >> 32) * kMulHigh + r.k0;
}
__device__ __forceinline__ uint32_t random_bits(const Random& r, uint32_t seed) {
  uint32_t h = (seed ^ (seed >> 16)) * 0xC2B2AE3Du + r.k1;
  h = (h ^ (h >> 15)) * 0x27D4EB2Fu;
  return h ^ (h >> 16);
}

// The two words of step t, by a published mixer of 64 bits (degski's: two rounds
// of a shift by half the word and this product); t is spread by 2^64 over the
// golden ratio first.
inline Random random_of(uint64_t seed, int64_t t) {
  uint64_t x = seed ^ ((uint64_t)t * 0x9E3779B97F4A7C15ull);
  for (int k = 0; k < 2; ++k) {
    x ^= x >> 32;
    x *= 0xD6E8FEB86659FD93ull;
  }
  x ^= x >> 32;
  return Random{(uint32_t)x, (uint32_t)(x >> 32)};
}

}  // namespace zs
