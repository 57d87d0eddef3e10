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
// to copy the weight first.  Measured (us, 14336 x 4096; launch_few, the other
// kernels, those with the copy): k adjacent, 16 tokens 38, 38, 73; n adjacent, 2
// tokens 32, 41, 72; 4 tokens 40 to 50, 41, 72.
constexpr bool is_few(int64_t tokens, bool n_adjacent, bool copied) {
  return tokens <= (n_adjacent ? (copied ? 4 : 2) : 16);
}
int64_t few_bytes(int64_t M, int64_t N, int64_t K, bool n_adjacent);
int launch_few(const Few& f, bool n_adjacent, void* workspace, hipStream_t stream);

}  // namespace zs
