// What the linear layer's kernels share: what becomes of a sum.
#pragma once

#include "activation.hpp"

namespace zs {

// What becomes of a sum.
struct Epilogue {
  const uint16_t* bias;  // flat parameters; null: none
  Place bias_place;
  const uint16_t* add;  // res, or the gradient's other part; null: none
  int64_t add_stride;
  const uint16_t* pre_in;  // input gradient: what the activation was taken of
  uint16_t* pre_out;       // forward: kept for the backward pass
  void* out;
  int64_t out_stride;
  int32_t act, f32, grad;
};

// Eight columns of bias, from column c; `left` of them exist.
__device__ __forceinline__ void bias_at(const Epilogue& e, int32_t c, int left, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j)
    v[j] = e.bias && j < left ? bf16_one(e.bias[place_at<true>(e.bias_place, c + j)]) : 0.f;
}

// What the epilogue reads beside the sums: 8 columns from column c of row r.
// N: the matrix's columns (rows of pre lie densely).
struct Beside {
  u32x4 add, pre;
};
__device__ __forceinline__ Beside beside_at(const Epilogue& e, int32_t N, int64_t r, int32_t c, int left) {
  Beside b{{0u, 0u, 0u, 0u}, {0u, 0u, 0u, 0u}};
  if (e.add) {
    const uint16_t* p = e.add + r * e.add_stride + c;
    b.add = left >= 8 ? *(const u32x4_a2*)p : load_some(p, left);
  }
  if (e.pre_in) {
    const uint16_t* p = e.pre_in + r * N + c;
    b.pre = left >= 8 ? *(const u32x4_a2*)p : load_some(p, left);
  }
  return b;
}

// Eight sums of row r, columns c to c + 7, of which `left` exist.
__device__ __forceinline__ void finish8(const Epilogue& e, int32_t N, int64_t r, int32_t c, int left, float (&v)[8],
                                        const Beside& b, const float (&bias)[8]) {
  float add[8];
  widen8(b.add, add);
  if (e.grad) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += add[j];
    if (e.act != ZERO_ACT_NONE) {
      float s[8];
      widen8(b.pre, s);
      apply8<true>(e.act, s);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= s[j];
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += bias[j];
    if (e.pre_out) {
      uint16_t* p = e.pre_out + r * N + c;
      if (left >= 8)
        *(u32x4_a2*)p = round8(v);
      else
        store_some(p, round8(v), left);
    }
    apply8<false>(e.act, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += add[j];
  }
  if (e.f32) {
    float* o = (float*)e.out + r * e.out_stride + c;
    if (left >= 8) {
      *(f32x4_a4*)o = f32x4{v[0], v[1], v[2], v[3]};
      *(f32x4_a4*)(o + 4) = f32x4{v[4], v[5], v[6], v[7]};
    } else {
#pragma unroll
      for (int j = 0; j < 7; ++j)
        if (j < left) o[j] = v[j];
    }
  } else {
    uint16_t* o = (uint16_t*)e.out + r * e.out_stride + c;
    if (left >= 8)
      *(u32x4_a2*)o = round8(v);
    else
      store_some(o, round8(v), left);
  }
}

// One sum.
__device__ __forceinline__ void finish1(const Epilogue& e, int32_t N, int64_t r, int32_t c, float v) {
  const float add = e.add ? bf16_one(e.add[r * e.add_stride + c]) : 0.f;
  if (e.grad) {
    v += add;
    if (e.act != ZERO_ACT_NONE) v *= apply1<true>(e.act, bf16_one(e.pre_in[r * N + c]));
  } else {
    if (e.bias) v += bf16_one(e.bias[place_at<true>(e.bias_place, c)]);
    if (e.pre_out) e.pre_out[r * N + c] = (uint16_t)round2(v, 0.f);
    v = apply1<false>(e.act, v) + add;
  }
  if (e.f32)
    ((float*)e.out)[r * e.out_stride + c] = v;
  else
    ((uint16_t*)e.out)[r * e.out_stride + c] = (uint16_t)round2(v, 0.f);
}

// The products of few tokens (linear_few.hip).
struct Few {
  const uint16_t *a, *w;  // a: x or dy; w: the flat parameters
  int64_t a_stride;
  Place place;            // the weight's
  int32_t M, N, K;
  Epilogue e;
};
// Whether launch_few is to take a product; copied: the other kernels would have
// to copy the weight first.  Measured (us; outputs x inputs; launch_few, the other
// kernels), the weight from HBM:
//   k adjacent: a block sums 16 outputs alone, 8192 k in 11 us for one token and
//   17 for 16, so long sums for few outputs are split by the others: 2048 x 8192 1
//   token 12.6, 14.9; 16 tokens 17.6, 15.0; 1024 x 16384 20.8, 16.2 and 30.9, 16.0.
//   From 4096 outputs on all CUs have a block: 4096 x 14336 29.9, 39.6 and 41, 40;
//   8192 x 8192 33, 49 and 44, 54.  Very many outputs: 32768 x 512 12.0, 10.0 and
//   14.6, 10.1; 32768 x 4096 55, 69 and 81, 70.  With the copy (a weight at an odd
//   place): 2048 x 4096 16.0, 20.8; 2048 x 8192 27.6, 26.8; 4096 x 32768 143, 181.
//   n adjacent: 1 and 2 tokens, 2048 x 2048 9.2, 10.4 and 10.2, 10.5; 4096 x 4096
//   16.7, 14.2 and 18.4, 14.2; 16384 x 512 8.3, 8.6 and 9.5, 8.4; 4096 x 14336 44,
//   35.  With the copy, 4 tokens: 4096 x 4096 22, 27; 14336 x 4096 50, 68.
constexpr bool is_few(int64_t tokens, int64_t N, int64_t K, bool n_adjacent, bool copied) {
  if (n_adjacent) return copied ? tokens <= 4 : tokens <= 2 && N <= 8192 && N * K <= (int64_t)1 << 23;
  if (tokens > 16) return false;
  if (N < 4096) return (copied ? 40 : tokens + 24) * K <= 28 * 8192;
  return copied || N <= 16384 || (tokens <= 8 && K >= 2048);
}
int64_t few_bytes(int64_t M, int64_t N, int64_t K, bool n_adjacent);
int launch_few(const Few& f, bool n_adjacent, void* workspace, hipStream_t stream);

}  // namespace zs
