// The linear layer's products of few tokens: one pass over the weight.
//
//   C[m, n] = sum over k of A[m, k] * B(k, n), m up to 16
//
// The weight is read once and used M times, so memory bounds both kernels, and
// they take it at any address, also across bucket padding.
//
// k adjacent: a wave takes 16 rows of the weight, a lane 8 neighbouring k of
// one of them, which is a matrix operand as it comes; the tokens' rows are the
// other one.  The waves of a block share the k.
// n adjacent: a lane takes 8 neighbouring n of one k and adds them to its sums,
// times each token's value at that k, which waits in LDS.
// In both, the lanes' and waves' sums are added in a fixed order.
#include <algorithm>

#include "linear.hpp"
#include "matrix.hpp"

namespace {
using namespace zs;

typedef float f32x4v __attribute__((ext_vector_type(4)));

// Elements i to i + 7 of the weight, of which `n` are wanted.
template <bool GAPS>
__device__ __forceinline__ u32x4 weight8(const Few& f, int64_t i, int n) {
  if (n <= 0) return u32x4{0u, 0u, 0u, 0u};
  int64_t at;
  if (place_run<GAPS>(f.place, i, 8, at) && n >= 8) return *(const u32x4_a2*)(f.w + at);
  u32x4 v = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (k < n) v[k >> 1] |= (uint32_t)f.w[place_at<GAPS>(f.place, i + k)] << (16 * (k & 1));
  return v;
}

// ---------------------------------------------------------------- k adjacent
constexpr int kRowWaves = 4, kBlockK = 64;  // k of a wave at a time: a line of each row
constexpr int kRowAhead = 4;                // of which it has that many on the way

template <bool GAPS>
__global__ void __launch_bounds__(kRowWaves * 64) few_rows_kernel(const Few f) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = threadIdx.x & 63;
  const int r = l & 15, g = l >> 4;
  const int32_t n0 = (int32_t)blockIdx.x * 16;
  const int64_t row = (int64_t)min(n0 + r, f.N - 1) * f.K;  // a row past the last one is not stored
  const uint16_t* a = f.a + (int64_t)min(r, f.M - 1) * f.a_stride;
  f32x4v acc = {0.f, 0.f, 0.f, 0.f};
  const int32_t blocks = (f.K + kBlockK - 1) / kBlockK;
  // lane (r, g): k 8g to 8g + 7 of each half of a block
  for (int32_t b0 = wave; b0 < blocks; b0 += kRowWaves * kRowAhead) {
    u32x4 w[kRowAhead][2], x[kRowAhead][2];
#pragma unroll
    for (int u = 0; u < kRowAhead; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int32_t k = (b0 + u * kRowWaves) * kBlockK + 32 * h + 8 * g;
        const int left = f.K - k;
        w[u][h] = weight8<GAPS>(f, row + k, left);
        x[u][h] = u32x4{0u, 0u, 0u, 0u};
        if (left >= 8)
          x[u][h] = *(const u32x4_a2*)(a + k);
        else if (left > 0)
          x[u][h] = load_some(a + k, left);
      }
#pragma unroll
    for (int u = 0; u < kRowAhead; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w[u][h]),
                                                       __builtin_bit_cast(bf16x8, x[u][h]), acc, 0, 0, 0);
  }
  // lane l, value j: row n0 + 4 * (l / 16) + j, token l % 16
  __shared__ f32x4v all[kRowWaves][64];
  all[wave][l] = acc;
  __syncthreads();
  if (wave > 0) return;
#pragma unroll
  for (int k = 1; k < kRowWaves; ++k) acc += all[k][l];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int32_t n = n0 + 4 * g + j;
    if (r < f.M && n < f.N) finish1(f.e, f.N, r, n, acc[j]);
  }
}

// ---------------------------------------------------------------- n adjacent
constexpr int kColWaves = 8, kAcross = 8, kDown = 64 / kAcross;  // a wave: 8 rows of 64 columns
constexpr int kColAhead = 8;
constexpr int kColStep = kColWaves * kDown * kColAhead;          // k of a block at a time

template <int M, bool GAPS>
__global__ void __launch_bounds__(kColWaves * 64) few_columns_kernel(const Few f) {
  __shared__ alignas(16) float x[2][kColStep * M];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = threadIdx.x & 63;
  const int across = l % kAcross, down = wave * kDown + l / kAcross;
  const int32_t n = ((int32_t)blockIdx.x * kAcross + across) * 8;
  const int left = f.N - n;
  float acc[M][8];
#pragma unroll
  for (int t = 0; t < M; ++t)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[t][j] = 0.f;
  int turn = 0;
  for (int32_t k0 = 0; k0 < f.K; k0 += kColStep, turn ^= 1) {
    u32x4 w[kColAhead];
#pragma unroll
    for (int u = 0; u < kColAhead; ++u) {
      const int32_t k = k0 + u * kColWaves * kDown + down;
      w[u] = weight8<GAPS>(f, (int64_t)k * f.N + n, k < f.K ? left : 0);
    }
    // two places in turn: a wave may still read the other one
    for (int i = threadIdx.x; i < kColStep * M; i += kColWaves * 64) {
      const int t = i / kColStep, k = i % kColStep;
      x[turn][k * M + t] = t < f.M && k0 + k < f.K ? bf16_one(f.a[t * f.a_stride + k0 + k]) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kColAhead; ++u) {
      float v[8];
      widen8(w[u], v);
      const float* at = &x[turn][(u * kColWaves * kDown + down) * M];
#pragma unroll
      for (int t = 0; t < M; ++t) {
        const float s = at[t];
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[t][j] = __builtin_fmaf(s, v[j], acc[t][j]);
      }
    }
  }
  // the rows of lanes, then the waves
  __shared__ float all[kColWaves][M][kAcross * 8];
#pragma unroll
  for (int t = 0; t < M; ++t)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float s = acc[t][j];
#pragma unroll
      for (int k = kAcross; k < 64; k *= 2) s += __shfl_xor(s, k, 64);
      if (l < kAcross) all[wave][t][across * 8 + j] = s;
    }
  __syncthreads();
  for (int i = threadIdx.x; i < M * kAcross * 8; i += kColWaves * 64) {
    const int t = i / (kAcross * 8), c = i % (kAcross * 8);
    const int32_t col = (int32_t)blockIdx.x * kAcross * 8 + c;
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < kColWaves; ++k) s += all[k][t][c];
    if (t < f.M && col < f.N) finish1(f.e, f.N, t, col, s);
  }
}

template <int M>
void launch_columns(const Few& f, hipStream_t s) {
  const dim3 grid((unsigned)((f.N + kAcross * 8 - 1) / (kAcross * 8)));
  if (f.place.gap)
    hipLaunchKernelGGL((few_columns_kernel<M, true>), grid, dim3(kColWaves * 64), 0, s, f);
  else
    hipLaunchKernelGGL((few_columns_kernel<M, false>), grid, dim3(kColWaves * 64), 0, s, f);
}

}  // namespace

namespace zs {

int launch_few(const Few& f, bool n_adjacent, hipStream_t s) {
  if (n_adjacent) {
    if (f.M == 1) launch_columns<1>(f, s);
    else if (f.M == 2) launch_columns<2>(f, s);
    else if (f.M <= 4) launch_columns<4>(f, s);
    else launch_columns<8>(f, s);
    return launched();
  }
  const dim3 grid((unsigned)((f.N + 15) / 16));
  if (f.place.gap)
    hipLaunchKernelGGL(few_rows_kernel<true>, grid, dim3(kRowWaves * 64), 0, s, f);
  else
    hipLaunchKernelGGL(few_rows_kernel<false>, grid, dim3(kRowWaves * 64), 0, s, f);
  return launched();
}

}  // namespace zs
