// The linear layer's products of few tokens: one pass over the weight.
//
//   C[m, n] = sum over k of A[m, k] * B(k, n)
//
// The weight is read once and used M times, so memory bounds both kernels, and
// they take it at any address, also across bucket padding.
//
// k adjacent: a wave takes 16 rows of the weight, a lane 8 neighbouring k of
// one of them, which is a matrix operand as it comes; the tokens' rows are the
// other one.  The waves of a block share the k.
// n adjacent: a lane takes 8 neighbouring n of one k and adds them to its sums,
// times each token's value at that k, which waits in LDS; where the columns
// are few the k are split over blocks, whose sums a second launch adds up.
// In both, all sums are added in a fixed order.
#include <algorithm>

#include "linear.hpp"
#include "matrix.hpp"

namespace {
using namespace zs;

// 8 elements from p.  ODD: p may lie between two words of 4 bytes.  A load of 16
// bytes from there takes more than twice the time (1 token, 14336 x 4096: 63 us
// against 28; of words 40, 50 of a weight that no cache holds), so it is made of words, each of which holds an
// element that belongs to the operand: `inside` says that those next to the 8
// do.
template <bool ODD>
__device__ __forceinline__ u32x4 eight_at(const uint16_t* p, bool inside) {
  if constexpr (ODD) {
    typedef uint32_t u32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));
    const uint32_t odd = (uint32_t)(uintptr_t)p & 2u;
    if (!odd || inside) {
      const uint32_t* q = (const uint32_t*)((uintptr_t)p & ~(uintptr_t)3);
      const u32x4 a = *(const u32x4_a4*)q;
      const uint32_t b = odd ? q[4] : 0u;
      return u32x4{__builtin_amdgcn_alignbyte(a.y, a.x, odd), __builtin_amdgcn_alignbyte(a.z, a.y, odd),
                   __builtin_amdgcn_alignbyte(a.w, a.z, odd), __builtin_amdgcn_alignbyte(b, a.w, odd)};
    }
  }
  return *(const u32x4_a2*)p;
}

// Elements i to i + 7 of the weight, of which `n` are wanted.
template <bool GAPS, bool ODD>
__device__ __forceinline__ u32x4 weight8(const Few& f, int64_t i, int n) {
  if (n <= 0) return u32x4{0u, 0u, 0u, 0u};
  int64_t at;
  if (place_run<GAPS>(f.place, i, 8, at) && n >= 8) return eight_at<ODD>(f.w + at, i > 0 && n > 8);
  u32x4 v = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (k < n) v[k >> 1] |= (uint32_t)f.w[place_at<GAPS>(f.place, i + k)] << (16 * (k & 1));
  return v;
}

// ---------------------------------------------------------------- k adjacent
// Measured (us; 1 token, 14336 x 4096 and 4096 x 14336) with 8 waves and 4
// blocks ahead: 25.7 and 23.7; 4 waves 26.8 and 31.8; 8 waves, 2 ahead 26.8 and
// 24.6; 4 waves, 8 ahead 26.7 and 27.7.  Two loads take a line's halves, so they
// go through the caches (non-temporal, with 4 waves: 28.2 and 31.5).
constexpr int kRowWaves = 8, kBlockK = 64;  // k of a wave at a time: a line of each row
constexpr int kRowAhead = 4;                // of which it has that many on the way

template <bool GAPS, bool ODD>
__global__ void __launch_bounds__(kRowWaves * 64) few_rows_kernel(const Few f) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = threadIdx.x & 63;
  const int r = l & 15, g = l >> 4;
  const int32_t n0 = (int32_t)blockIdx.x * 16;
  // rows and tokens past the last one are not stored
  const int64_t row = (int64_t)min(n0 + r, f.N - 1) * f.K;
  const uint16_t* a = f.a + (int64_t)min(r, f.M - 1) * f.a_stride;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
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
        w[u][h] = weight8<GAPS, ODD>(f, row + k, left);
        x[u][h] = u32x4{0u, 0u, 0u, 0u};
        if (left >= 8)
          x[u][h] = eight_at<ODD>(a + k, k > 0 && left > 8);
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
  __shared__ f32x4 all[kRowWaves][64];
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
// Loads go to any address: 1 token, 14336 x 4096, 38.6 us at an odd place, 39.1 at
// one of 16 bytes.
constexpr int kColStep = kColWaves * kDown * kColAhead;          // k of a block at a time

// per_split: k of a block of one split; partial: its sums (splits x tokens x
// columns), where there is more than one
template <int M, bool GAPS>
__global__ void __launch_bounds__(kColWaves * 64) few_columns_kernel(const Few f, int32_t per_split, float* partial) {
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
  const int32_t ka = (int32_t)blockIdx.y * per_split, kz = min(f.K, ka + per_split);
  int turn = 0;
  for (int32_t k0 = ka; k0 < kz; k0 += kColStep, turn ^= 1) {
    u32x4 w[kColAhead];
#pragma unroll
    for (int u = 0; u < kColAhead; ++u) {
      const int32_t k = k0 + u * kColWaves * kDown + down;
      w[u] = weight8<GAPS, false>(f, (int64_t)k * f.N + n, k < kz ? left : 0);
    }
    // two places in turn: a wave may still read the other one
    for (int i = threadIdx.x; i < kColStep * M; i += kColWaves * 64) {
      const int t = i / kColStep, k = i % kColStep;
      x[turn][k * M + t] = t < f.M && k0 + k < kz ? bf16_one(f.a[t * f.a_stride + k0 + k]) : 0.f;
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
    if (t >= f.M || col >= f.N) continue;
    if (partial)
      partial[((int64_t)blockIdx.y * f.M + t) * f.N + col] = s;
    else
      finish1(f.e, f.N, t, col, s);
  }
}

constexpr int kSumThreads = 256;
__global__ void __launch_bounds__(kSumThreads) few_sum_kernel(const Few f, int32_t splits, const float* partial) {
  const int32_t n = (int32_t)(blockIdx.x * kSumThreads + threadIdx.x), t = (int32_t)blockIdx.y;
  if (n >= f.N) return;
  float s = 0.f;
#pragma unroll 8
  for (int k = 0; k < splits; ++k) s += partial[((int64_t)k * f.M + t) * f.N + n];
  finish1(f.e, f.N, t, n, s);
}

// ------------------------------------------------------------------ host
// About 384 blocks, 512 k each at least: 4096 x 14336, one token, in 64 blocks
// takes 77 us.
struct Split {
  int64_t blocks, splits, per_split;
};
Split split_of(int64_t N, int64_t K) {
  Split p;
  p.blocks = (N + kAcross * 8 - 1) / (kAcross * 8);
  p.splits = std::max<int64_t>(1, std::min((K + kColStep - 1) / kColStep, 384 / p.blocks));
  p.per_split = ((K + p.splits - 1) / p.splits + 63) / 64 * 64;
  p.splits = (K + p.per_split - 1) / p.per_split;
  return p;
}

template <int M>
void launch_columns(const Few& f, const Split& p, float* partial, hipStream_t s) {
  const dim3 grid((unsigned)p.blocks, (unsigned)p.splits);
  if (f.place.gap)
    hipLaunchKernelGGL((few_columns_kernel<M, true>), grid, dim3(kColWaves * 64), 0, s, f, (int32_t)p.per_split,
                       partial);
  else
    hipLaunchKernelGGL((few_columns_kernel<M, false>), grid, dim3(kColWaves * 64), 0, s, f, (int32_t)p.per_split,
                       partial);
}
void launch_rows(const Few& f, hipStream_t s) {
  const dim3 grid((unsigned)((f.N + 15) / 16)), block(kRowWaves * 64);
  const bool odd = (((uintptr_t)f.w >> 1) + (uintptr_t)f.place.x0) % 2 != 0 || f.K % 2 != 0 ||
                   ((uintptr_t)f.a >> 1) % 2 != 0 || f.a_stride % 2 != 0;
  if (f.place.gap)
    hipLaunchKernelGGL((few_rows_kernel<true, false>), grid, block, 0, s, f);
  else if (odd)
    hipLaunchKernelGGL((few_rows_kernel<false, true>), grid, block, 0, s, f);
  else
    hipLaunchKernelGGL((few_rows_kernel<false, false>), grid, block, 0, s, f);
}

}  // namespace

namespace zs {

int64_t few_bytes(int64_t M, int64_t N, int64_t K, bool n_adjacent) {
  if (!n_adjacent) return 0;
  const Split p = split_of(N, K);
  return p.splits > 1 ? p.splits * M * N * 4 : 0;
}

int launch_few(const Few& f, bool n_adjacent, void* workspace, hipStream_t s) {
  if (!n_adjacent) {
    launch_rows(f, s);
    return launched();
  }
  const Split p = split_of(f.N, f.K);
  float* partial = p.splits > 1 ? (float*)workspace : nullptr;
  if (f.M == 1) launch_columns<1>(f, p, partial, s);
  else if (f.M == 2) launch_columns<2>(f, p, partial, s);
  else launch_columns<4>(f, p, partial, s);
  const int rc = launched();
  if (rc != ZERO_OK || !partial) return rc;
  hipLaunchKernelGGL(few_sum_kernel, dim3((unsigned)((f.N + kSumThreads - 1) / kSumThreads), (unsigned)f.M),
                     dim3(kSumThreads), 0, s, f, (int32_t)p.splits, partial);
  return launched();
}

}  // namespace zs
