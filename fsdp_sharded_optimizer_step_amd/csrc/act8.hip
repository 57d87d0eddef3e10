// zero_act8_pack and zero_act8_unpack: activation checkpoints in 8 bits.
//
// Page "Infra: Data Parallel" (pufanyi.com), section "Zero Redundancy
// Optimizer (ZeRO)": the memory that ZeRO divides among the ranks is that of
// parameters, gradients and optimizer state; activations stay whole on every
// rank, and this format halves those that the backward pass keeps.
//
// Both kernels are HBM streams (pack reads 2 or 4 and writes 1 + 1/128 bytes
// per element, unpack the reverse).  A lane takes 8 consecutive columns, the
// 16 lanes of a DPP row take a block of 128, so the block's maximum needs
// four lane rotations and no LDS.  Codes and scales of a block belong to one
// lane group: the result does not depend on the launch shape.
//
// Cache hints as measured for 8192 x 14336 values: 16-bit and 8-bit loads are
// non-temporal (bf16: pack and unpack together 115 us, 706 MB; temporal 130),
// binary32 loads are not, since two of a lane's instructions share a line
// (pack 107 us against 110), binary32 stores are (unpack 104 against 107).
#include <algorithm>

#include "act8.hpp"

namespace {
using namespace zs;

constexpr int kThreads = 256;
typedef uint32_t u32_a1 __attribute__((aligned(1)));
// (row, block) units of one launch: unit indices stay below 2^31
constexpr int64_t kMaxUnits = (int64_t)1 << 28;

__device__ __forceinline__ void load_row8(float (&x)[8], const uint16_t* p, int n) {
  if (n >= 8) {
    const u32x4 w = __builtin_nontemporal_load((const u32x4_a2*)p);
    x[0] = bf16_lo(w.x); x[1] = bf16_hi(w.x); x[2] = bf16_lo(w.y); x[3] = bf16_hi(w.y);
    x[4] = bf16_lo(w.z); x[5] = bf16_hi(w.z); x[6] = bf16_lo(w.w); x[7] = bf16_hi(w.w);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = k < n ? bf16_one(p[k]) : 0.0f;
  }
}
__device__ __forceinline__ void load_row8(float (&x)[8], const float* p, int n) {
  if (n >= 8) {
    const f32x4 a = *(const f32x4_a4*)p, b = *(const f32x4_a4*)(p + 4);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = k < n ? p[k] : 0.0f;
  }
}

template <class T>
__global__ void __launch_bounds__(kThreads)
    pack_kernel(const T* x, int64_t stride, int64_t cols, FastDiv nb, uint32_t units,
                uint8_t* codes, uint8_t* scales) {
  const uint32_t lane16 = threadIdx.x & 15u;
  const uint32_t step = gridDim.x * (kThreads / 16);
  // every lane of a 16-lane row has the same unit, so the rotations see
  // active lanes only
  for (uint32_t u = blockIdx.x * (kThreads / 16) + (threadIdx.x >> 4); u < units; u += step) {
    const uint32_t r = fast_div(u, nb), b = u - r * nb.d;
    const int64_t c0 = (int64_t)b * kAct8Block + lane16 * 8;
    const int n = (int)min((int64_t)8, cols - c0);  // <= 0: past the row's end
    float v[8];
    load_row8(v, x + (int64_t)r * stride + c0, n);
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) m = max(m, finite_mag(v[k]));
    const uint32_t e = act8_byte(max16(m));
    const float inv = act8_inv(e);
    const u32x2 w = {act8_pack4(v, inv), act8_pack4(v + 4, inv)};
    uint8_t* q = codes + (int64_t)r * cols + c0;
    if (n >= 8) {
      *(u32x2_a1*)q = w;
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < n) q[k] = (uint8_t)((k < 4 ? w.x : w.y) >> (8 * (k & 3)));
    }
    if (lane16 == 0) scales[u] = (uint8_t)e;
  }
}

__device__ __forceinline__ void store_row8(uint16_t* p, u32x2 w, float s, int n) {
  const u32x2 a = act8_bf16x4(w.x, s), b = act8_bf16x4(w.y, s);
  const u32x4 o = {a.x, a.y, b.x, b.y};
  if (n >= 8) {
    *(u32x4_a2*)p = o;
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < n) p[k] = (uint16_t)(o[k >> 1] >> (16 * (k & 1)));
  }
}
__global__ void __launch_bounds__(kThreads)
    unpack_bf16_kernel(const uint8_t* codes, const uint8_t* scales, int64_t cols, FastDiv nb,
                  uint32_t units, uint16_t* out, int64_t stride) {
  const uint32_t lane16 = threadIdx.x & 15u;
  const uint32_t step = gridDim.x * (kThreads / 16);
  for (uint32_t u = blockIdx.x * (kThreads / 16) + (threadIdx.x >> 4); u < units; u += step) {
    const uint32_t r = fast_div(u, nb), b = u - r * nb.d;
    const int64_t c0 = (int64_t)b * kAct8Block + lane16 * 8;
    const int n = (int)min((int64_t)8, cols - c0);
    if (n <= 0) continue;
    const float s = act8_scale(scales[u]);
    const uint8_t* q = codes + (int64_t)r * cols + c0;
    u32x2 w = {0u, 0u};
    if (n >= 8) {
      w = __builtin_nontemporal_load((const u32x2_a1*)q);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < n) {
          if (k < 4) w.x |= (uint32_t)q[k] << (8 * k);
          else w.y |= (uint32_t)q[k] << (8 * (k - 4));
        }
    }
    store_row8(out + (int64_t)r * stride + c0, w, s, n);
  }
}

// Of each half of a block a lane takes 4 columns, so that 16 lanes store 256
// consecutive bytes at a time (8192 x 14336: 104 us; with 8 columns each, two
// stores 32 bytes apart, 130, or 144 through the caches).
__global__ void __launch_bounds__(kThreads)
    unpack_f32_kernel(const uint8_t* codes, const uint8_t* scales, int64_t cols, FastDiv nb,
                      uint32_t units, float* out, int64_t stride) {
  const uint32_t lane16 = threadIdx.x & 15u;
  const uint32_t step = gridDim.x * (kThreads / 16);
  for (uint32_t u = blockIdx.x * (kThreads / 16) + (threadIdx.x >> 4); u < units; u += step) {
    const uint32_t r = fast_div(u, nb), b = u - r * nb.d;
    const float s = act8_scale(scales[u]);
    uint32_t w[2];
    int n[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t c0 = (int64_t)b * kAct8Block + h * 64 + lane16 * 4;
      n[h] = (int)min((int64_t)4, cols - c0);
      const uint8_t* q = codes + (int64_t)r * cols + c0;
      w[h] = 0u;
      if (n[h] >= 4) {
        w[h] = __builtin_nontemporal_load((const u32_a1*)q);
      } else {
#pragma unroll
        for (int k = 0; k < 3; ++k)
          if (k < n[h]) w[h] |= (uint32_t)q[k] << (8 * k);
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const f32x2 lo = act8_f32<false>(w[h], s), hi = act8_f32<true>(w[h], s);
      const f32x4 o = {lo.x, lo.y, hi.x, hi.y};
      float* p = out + (int64_t)r * stride + (int64_t)b * kAct8Block + h * 64 + lane16 * 4;
      if (n[h] >= 4) {
        st4_stream(p, o);
      } else {
#pragma unroll
        for (int k = 0; k < 3; ++k)
          if (k < n[h]) p[k] = o[k];
      }
    }
  }
}

int check(const void* x, int32_t dtype, int64_t rows, int64_t cols, int64_t stride,
          const void* codes, const void* scales) {
  if (dtype != ZERO_DTYPE_BF16 && dtype != ZERO_DTYPE_F32) return ZERO_EINVAL;
  if (rows < 0 || cols < 0) return ZERO_EINVAL;
  if (rows == 0 || cols == 0) return ZERO_OK;
  if (!x || !codes || !scales || stride < cols) return ZERO_EINVAL;
  if (cols > ZERO_MAX_COLS || rows > ZERO_MAX_ROWS || stride > ZERO_MAX_STRIDE) return ZERO_ERANGE;
  return ZERO_OK;
}

template <class F>
int for_row_groups(int64_t rows, int64_t nb, F launch) {
  const int64_t per = std::max<int64_t>(1, kMaxUnits / nb);
  for (int64_t r0 = 0; r0 < rows; r0 += per) {
    const int64_t n = std::min(per, rows - r0);
    const int64_t units = n * nb;
    const int64_t blocks = (units + kThreads / 16 - 1) / (kThreads / 16);
    const int rc = launch(r0, (uint32_t)units, (unsigned)std::min<int64_t>(blocks, 1 << 14));
    if (rc != ZERO_OK) return rc;
  }
  return ZERO_OK;
}

}  // namespace

extern "C" {

int zero_act8_pack(const void* x, int32_t dtype, int64_t rows, int64_t cols, int64_t stride,
                   uint8_t* codes, uint8_t* scales, hipStream_t stream) {
  const int rc = check(x, dtype, rows, cols, stride, codes, scales);
  if (rc != ZERO_OK) return rc;
  if (rows == 0 || cols == 0) return ZERO_OK;
  const int64_t nb = (cols + kAct8Block - 1) / kAct8Block;
  const Bytes ins[] = {rows_of(x, rows, cols, stride, dtype == ZERO_DTYPE_F32 ? 4 : 2)};
  const Bytes outs[] = {Bytes{codes, rows * cols}, Bytes{scales, rows * nb}};
  if (any_overlap(outs, ins)) return ZERO_EOVERLAP;
  if (hip_error_pending()) return ZERO_EHIP;
  const FastDiv d = make_fast_div((uint32_t)nb);
  return for_row_groups(rows, nb, [&](int64_t r0, uint32_t units, unsigned grid) {
    uint8_t* q = codes + r0 * cols;
    uint8_t* s = scales + r0 * nb;
    if (dtype == ZERO_DTYPE_F32)
      hipLaunchKernelGGL(pack_kernel<float>, dim3(grid), dim3(kThreads), 0, stream,
                         (const float*)x + r0 * stride, stride, cols, d, units, q, s);
    else
      hipLaunchKernelGGL(pack_kernel<uint16_t>, dim3(grid), dim3(kThreads), 0, stream,
                         (const uint16_t*)x + r0 * stride, stride, cols, d, units, q, s);
    return launched();
  });
}

int zero_act8_unpack(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols,
                     void* out, int32_t dtype, int64_t stride, hipStream_t stream) {
  const int rc = check(out, dtype, rows, cols, stride, codes, scales);
  if (rc != ZERO_OK) return rc;
  if (rows == 0 || cols == 0) return ZERO_OK;
  const int64_t nb = (cols + kAct8Block - 1) / kAct8Block;
  const Bytes outs[] = {rows_of(out, rows, cols, stride, dtype == ZERO_DTYPE_F32 ? 4 : 2)};
  const Bytes ins[] = {Bytes{codes, rows * cols}, Bytes{scales, rows * nb}};
  if (any_overlap(outs, ins)) return ZERO_EOVERLAP;
  if (hip_error_pending()) return ZERO_EHIP;
  const FastDiv d = make_fast_div((uint32_t)nb);
  return for_row_groups(rows, nb, [&](int64_t r0, uint32_t units, unsigned grid) {
    const uint8_t* q = codes + r0 * cols;
    const uint8_t* s = scales + r0 * nb;
    if (dtype == ZERO_DTYPE_F32)
      hipLaunchKernelGGL(unpack_f32_kernel, dim3(grid), dim3(kThreads), 0, stream, q, s, cols,
                         d, units, (float*)out + r0 * stride, stride);
    else
      hipLaunchKernelGGL(unpack_bf16_kernel, dim3(grid), dim3(kThreads), 0, stream, q, s,
                         cols, d, units, (uint16_t*)out + r0 * stride, stride);
    return launched();
  });
}

}  // extern "C"
