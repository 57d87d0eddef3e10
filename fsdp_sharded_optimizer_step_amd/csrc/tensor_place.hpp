// A tensor's elements in the rank's flat buffers, and what a parameter
// gradient does with them: shared by the embedding, norm and weight-gradient
// kernels.
//
// Page "Infra: Data Parallel" (pufanyi.com), section "Fully Sharded Data
// Parallel (FSDP)", "FSDP1": the parameters are flattened and concatenated,
// so a tensor is a range of the flat buffer; bucket padding can fall inside
// that range.  Section "Naive Data Parallelism": micro-batch gradients are
// summed locally, each scaled by 1/n_micro.
#pragma once

#include <cstdint>

#include "device_common.hpp"
#include "layout.hpp"
#include "zero_shard.h"

namespace zs {

// Vectors at any element alignment: gfx950 loads and stores them whole.
typedef u32x2 u32x2_a1 __attribute__((aligned(1)));
typedef u32x2 u32x2_a2 __attribute__((aligned(2)));
typedef u32x4 u32x4_a1 __attribute__((aligned(1)));
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef f32x4 f32x4_a4 __attribute__((aligned(4)));

// Streamed once: non-temporal.
__device__ __forceinline__ f32x4 ld4_stream(const float* p) {
  return __builtin_nontemporal_load((const f32x4_a4*)p);
}
__device__ __forceinline__ void st4_stream(float* p, f32x4 v) {
  __builtin_nontemporal_store(v, (f32x4_a4*)p);
}

// Element i of the tensor lies at flat position x0 + i where no padding falls
// inside the tensor (gap == 0, x0 a flat position), otherwise at
// x + (x / cap) * gap with x = x0 + i its stream position.
struct Place {
  int64_t x0, cap, gap;
  double inv_cap;
};

// x / cap: the product is off by less than one for any x that memory holds
// (x < 2^50), so the quotient is right or one off.
__device__ __forceinline__ int64_t bucket_of(const Place& p, int64_t x) {
  const int64_t b = (int64_t)((double)x * p.inv_cap), r = x - b * p.cap;
  return b + (r >= p.cap ? 1 : 0) - (r < 0 ? 1 : 0);
}
template <bool GAPS>
__device__ __forceinline__ int64_t place_at(const Place& p, int64_t i) {
  const int64_t x = p.x0 + i;
  if constexpr (!GAPS)
    return x;
  else
    return x + bucket_of(p, x) * p.gap;
}
// The flat position of element i, and whether elements i to i + n - 1 follow
// each other there.
template <bool GAPS>
__device__ __forceinline__ bool place_run(const Place& p, int64_t i, int n, int64_t& at) {
  const int64_t x = p.x0 + i;
  at = x;
  if constexpr (GAPS) {
    const int64_t b = bucket_of(p, x);
    at += b * p.gap;
    return x - b * p.cap + n <= p.cap;
  }
  return true;
}

// What becomes of a gradient element g (the arithmetic and the flags of
// zero_grad_accumulate): a = scale*g or acc + scale*g, stored, emitted, or both.
struct GradOut {
  float* acc;     // flat accumulator
  uint16_t* out;  // flat bf16 buffer
  Place place;
  float scale;
  uint32_t flags;
};

__device__ __forceinline__ void grad_store(const GradOut& o, int64_t p, float g) {
  const float c = o.scale * g;
  const float a = (o.flags & ZERO_ACC_OVERWRITE) ? c : o.acc[p] + c;
  if (!(o.flags & ZERO_ACC_NO_STORE)) o.acc[p] = a;
  if (o.flags & ZERO_ACC_EMIT_BF16) o.out[p] = (uint16_t)bf16_round(a);
}

// Four consecutive flat positions; `b`: what the accumulator holds there,
// which a kernel may have loaded early (grad_load4).
__device__ __forceinline__ f32x4 grad_load4(const GradOut& o, int64_t p) {
  return (o.flags & ZERO_ACC_OVERWRITE) ? f32x4{0.f, 0.f, 0.f, 0.f} : ld4_stream(o.acc + p);
}
__device__ __forceinline__ void grad_store4(const GradOut& o, int64_t p, f32x4 g, f32x4 b) {
  f32x4 a = {o.scale * g.x, o.scale * g.y, o.scale * g.z, o.scale * g.w};
  if (!(o.flags & ZERO_ACC_OVERWRITE)) a = f32x4{b.x + a.x, b.y + a.y, b.z + a.z, b.w + a.w};
  if (!(o.flags & ZERO_ACC_NO_STORE)) st4_stream(o.acc + p, a);
  if (o.flags & ZERO_ACC_EMIT_BF16)
    *(u32x2_a2*)(o.out + p) = u32x2{bf16_pack2(a.x, a.y), bf16_pack2(a.z, a.w)};
}
__device__ __forceinline__ void grad_store4(const GradOut& o, int64_t p, f32x4 g) {
  grad_store4(o, p, g, grad_load4(o, p));
}

// Exact division of n < 2^31 by d in [1, 2^31): with s = ceil(log2 d) and
// mul = ceil(2^(31+s) / d) the error of n*mul / 2^(31+s) stays below 1/d.
struct FastDiv {
  uint32_t mul, shift, d;
};
__device__ __forceinline__ uint32_t fast_div(uint32_t n, const FastDiv& f) {
  return (uint32_t)(((uint64_t)n * f.mul) >> f.shift);
}

// -------------------------------------------------------------- host side
inline FastDiv make_fast_div(uint32_t d) {
  uint32_t s = 0;
  while (((uint64_t)1 << s) < d) ++s;
  const uint64_t p = (uint64_t)1 << (31 + s);
  return FastDiv{(uint32_t)((p + d - 1) / d), 31 + s, d};
}

// The tensor's place; *lo, *hi: its range in the flat buffer.  The caller has
// checked the tensor index.
inline Place make_place(const zero_layout* L, int32_t t, int64_t* lo, int64_t* hi) {
  zero_layout_tensor_flat(L, t, lo, hi);
  if (*hi - *lo == L->numel[(size_t)t]) return Place{*lo, 1, 0, 1.0};
  return Place{L->tensor_off[(size_t)t], L->cap, L->p_full - L->cap, 1.0 / (double)L->cap};
}

inline bool tensor_ok(const zero_layout* L, int32_t t) {
  return t >= 0 && t < (int32_t)L->numel.size();
}

// Memory of an operand: [p, p + bytes).
struct Bytes {
  const void* p;
  int64_t n;
};
inline Bytes rows_of(const void* p, int64_t rows, int64_t cols, int64_t stride, int64_t elem) {
  return Bytes{p, rows > 0 && cols > 0 ? ((rows - 1) * stride + cols) * elem : 0};
}
inline bool bytes_overlap(const Bytes& a, const Bytes& b) {
  if (!a.p || !b.p || a.n <= 0 || b.n <= 0) return false;
  const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
  return x < y + (uintptr_t)b.n && y < x + (uintptr_t)a.n;
}
// Whether an output meets another output or an input.
template <int NO, int NI>
bool any_overlap(const Bytes (&outs)[NO], const Bytes (&ins)[NI]) {
  for (int a = 0; a < NO; ++a) {
    for (int b = a + 1; b < NO; ++b)
      if (bytes_overlap(outs[a], outs[b])) return true;
    for (int b = 0; b < NI; ++b)
      if (bytes_overlap(outs[a], ins[b])) return true;
  }
  return false;
}

// The flags and buffers of a gradient that covers `numel` elements.
inline int grad_out_ok(uint32_t flags, float scale, const float* acc, const uint16_t* out,
                       int64_t numel) {
  if (flags & ~(ZERO_ACC_OVERWRITE | ZERO_ACC_EMIT_BF16 | ZERO_ACC_NO_STORE)) return ZERO_EINVAL;
  if ((flags & ZERO_ACC_NO_STORE) && !(flags & ZERO_ACC_EMIT_BF16)) return ZERO_EINVAL;
  if (!(scale - scale == 0.0f)) return ZERO_EINVAL;  // not finite
  if (numel == 0) return ZERO_OK;
  const bool acc_used = !(flags & ZERO_ACC_OVERWRITE) || !(flags & ZERO_ACC_NO_STORE);
  if ((acc_used && !acc) || ((flags & ZERO_ACC_EMIT_BF16) && !out)) return ZERO_EINVAL;
  return ZERO_OK;
}
inline bool acc_used(uint32_t flags) {
  return !(flags & ZERO_ACC_OVERWRITE) || !(flags & ZERO_ACC_NO_STORE);
}

inline int launched() { return hipGetLastError() == hipSuccess ? ZERO_OK : ZERO_EHIP; }

}  // namespace zs
