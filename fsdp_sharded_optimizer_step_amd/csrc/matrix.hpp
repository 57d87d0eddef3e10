// What the kernels built on matrix instructions share.
#pragma once

#include <utility>

#include "tensor_place.hpp"

namespace zs {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

typedef __attribute__((address_space(3))) char lds_char;
typedef __attribute__((address_space(3))) u32x4 lds_u32x4;

// Between a wave's LDS accesses where its lanes read what others wrote, or write
// over what others read.  The LDS takes a wave's accesses in order; this keeps
// the compiler, which sees one lane's addresses, from changing that order.  No
// instruction comes of it.
__device__ __forceinline__ void lanes_meet_in_lds() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}

// f(0), f(1) to f(N - 1) with constant arguments: a loop that indexes registers
// and has to be unrolled whatever its size.
template <class F, int... I>
__device__ __forceinline__ void unrolled_of(F f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, class F>
__device__ __forceinline__ void unrolled(F f) {
  unrolled_of(f, std::make_integer_sequence<int, N>{});
}

// Tile number to place: groups of 8 rows of tiles, column by column within a
// group, so that tiles worked on together share their operands in the L2.
__device__ __forceinline__ void tile_place(int32_t tile, int32_t row_tiles, int32_t col_tiles, int32_t& r,
                                           int32_t& c) {
  const int32_t per = 8 * col_tiles, g = tile / per, in = tile - g * per;
  const int32_t h = min(8, row_tiles - g * 8);
  c = in / h;
  r = g * 8 + in - c * h;
}

}  // namespace zs
