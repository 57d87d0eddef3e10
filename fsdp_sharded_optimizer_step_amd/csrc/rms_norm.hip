// zero_rms_norm and zero_rms_norm_grad.
//
// Page "Infra: Data Parallel" (pufanyi.com), section "Zero Redundancy
// Optimizer (ZeRO)": the norm's weight is read from the flat buffer of
// gathered parameters; section "Naive Data Parallelism": its gradient is
// added to the rank's sum over micro-batches.
//
//   forward   h = bf16(x + r);  R = 1 / sqrt(mean(h^2) + eps);  y = act8(h*R*w)
//   backward  g = dy*w;  n = h*R;  dx = bf16(dh + R*(g - n*mean(g*n)))
//             dw = sum over rows of dy*n
// (the rounding of y to 8 bits is passed straight through).  Between the
// loads and the stores the forward pass is binary64, the backward binary32.
//
// Both are HBM streams: each row is read once and stays in registers between
// its statistics and its output, 8 consecutive columns per lane and piece; 16
// lanes of a DPP row hold one block of 128 columns of the 8-bit output.  A
// row takes 16 to 1024 threads, so that a thread keeps at most 32 columns.
// The threads are chosen by the width alone, with as few idle as a thread's
// pieces allow: a backward pass of one row of 768 columns and 128
// threads a block takes 109 us for 32768 rows, of eight rows of 64 threads 44.
// The weight's gradient is summed over groups of rows whose number follows
// from the shape, and over the groups, in order, by a second launch: the same
// sum in every run.
#include <algorithm>

#include "act8.hpp"

namespace {
using namespace zs;

constexpr int kMaxNormCols = ZERO_MAX_NORM_COLS;

// Cache hints, measured for both kernels with all four settings of loads and
// stores: the forward pass (two streams in, four out) is fastest with
// non-temporal stores alone (16384 x 8192: 211 us; none 224, loads 243, both
// 216), the backward pass (three in, one out) with non-temporal loads alone
// (16384 x 4096: 102 us; none 114, stores 111, both 104).
//
// 8 bf16 values, as loaded.
struct Piece8 {
  u32x4 w;
};
template <bool NT>
__device__ __forceinline__ Piece8 load8(const uint16_t* p, int n) {
  if (n >= 8) {
    if constexpr (NT)
      return Piece8{__builtin_nontemporal_load((const u32x4_a2*)p)};
    else
      return Piece8{*(const u32x4_a2*)p};
  }
  u32x4 w = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (k < n) w[k >> 1] |= (uint32_t)p[k] << (16 * (k & 1));
  return Piece8{w};
}
template <bool NT>
__device__ __forceinline__ void store8(uint16_t* p, u32x4 w, int n) {
  if (n >= 8) {
    if constexpr (NT)
      __builtin_nontemporal_store(w, (u32x4_a2*)p);
    else
      *(u32x4_a2*)p = w;
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < n) p[k] = (uint16_t)(w[k >> 1] >> (16 * (k & 1)));
  }
}
__device__ __forceinline__ float at8(const Piece8& p, int k) {
  return (k & 1) ? bf16_hi(p.w[k >> 1]) : bf16_lo(p.w[k >> 1]);
}
__device__ __forceinline__ u32x4 round8(const float (&x)[8]) {
  return u32x4{bf16_pack2(x[0], x[1]), bf16_pack2(x[2], x[3]), bf16_pack2(x[4], x[5]),
               bf16_pack2(x[6], x[7])};
}
template <bool GAPS>
__device__ __forceinline__ Piece8 weight8(const uint16_t* params, const Place& pl, int c0, int n) {
  int64_t at;
  if (place_run<GAPS>(pl, c0, 8, at) || !GAPS) return load8<false>(params + at, n);
  u32x4 w = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (k < n) w[k >> 1] |= (uint32_t)params[place_at<GAPS>(pl, c0 + k)] << (16 * (k & 1));
  return Piece8{w};
}

// Sum over the NT threads of a row; `slot`: NT/64 values of LDS of this row,
// not read by anyone else until the next barrier.
template <int NT, class T>
__device__ __forceinline__ T row_sum(T x, T* slot) {
#pragma unroll
  for (int k = (NT < 64 ? NT : 64) / 2; k; k >>= 1) x += __shfl_xor(x, k, 64);
  if constexpr (NT > 64) {
    const int w = (threadIdx.x % NT) >> 6;
    if ((threadIdx.x & 63) == 0) slot[w] = x;
    __syncthreads();
    x = 0;
#pragma unroll
    for (int k = 0; k < NT / 64; ++k) x += slot[k];
  }
  return x;
}

// Threads of a block for a row of NT threads: rows of up to one wave share a
// block.
template <int NT>
constexpr int kBlock = NT < 256 ? 256 : NT;

struct NormArgs {
  const uint16_t *params, *x, *res;
  int64_t x_stride, res_stride;
  Place place;
  uint16_t *h, *y;
  float* rstd;
  uint8_t *codes, *scales;
  int64_t rows;
  int32_t cols, nb;
  double eps;
};

// x in binary32, 21 bits of it, the last one set if x has any below: what is
// rounded to fewer bits later comes out as if x itself were rounded, ties
// included.
__device__ __forceinline__ float round_to_odd(double x) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x);
  const uint32_t hi = (uint32_t)(b >> 32) | ((uint32_t)b != 0u ? 1u : 0u);
  return (float)__builtin_bit_cast(double, (uint64_t)hi << 32);
}

// The statistics and the products are binary64: a code is the rounding of one
// exact product h*w (16 bits) times 1/rms, not of a value already rounded,
// which near a code's border would come out one code off.  The kernel waits
// for memory all the same: 16384 rows of 8192 columns with every output (1.21
// GB) take 211 us, 5.7 TB/s; in binary32 alone it gains under 2 %.
template <int NT, int NP, bool GAPS>
__global__ void __launch_bounds__(kBlock<NT>, 4) norm_kernel(const NormArgs A) {
  constexpr int kRows = kBlock<NT> / NT;
  __shared__ double red[2][kBlock<NT> / 64];
  const int tid = threadIdx.x % NT, sub = threadIdx.x / NT;
  Piece8 w[NP];
#pragma unroll
  for (int k = 0; k < NP; ++k) {
    const int c0 = (k * NT + tid) * 8;
    w[k] = weight8<GAPS>(A.params, A.place, c0, A.cols - c0);
  }
  int turn = 0;
  for (int64_t r0 = (int64_t)blockIdx.x * kRows; r0 < A.rows; r0 += (int64_t)gridDim.x * kRows) {
    const int64_t r = r0 + sub;
    const bool live = r < A.rows;
    Piece8 h[NP];
    double ss = 0;
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      const int c0 = (k * NT + tid) * 8, n = live ? A.cols - c0 : 0;
      h[k] = load8<false>(A.x + r * A.x_stride + c0, n);
      if (A.res) {
        const Piece8 b = load8<false>(A.res + r * A.res_stride + c0, n);
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = at8(h[k], j) + at8(b, j);
        h[k].w = round8(v);
      }
      if (A.h) store8<true>(A.h + r * A.cols + c0, h[k].w, n);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const double d = at8(h[k], j);
        ss = __builtin_fma(d, d, ss);
      }
    }
    // two slots in turn: a wave may write the next row's sum while another
    // still reads this one's
    ss = row_sum<NT>(ss, &red[turn][0]);
    turn ^= 1;
    const double rstd = 1.0 / __builtin_sqrt(ss / A.cols + A.eps);
    if (live && tid == 0) A.rstd[r] = (float)rstd;
    // rstd = rf * r2, r2 a power of two: h*r2 is a normed value's size, so
    // that its product with w is exact in binary32 (16 bits) for any row size
    const int rexp = min(max((int)((__double2hiint(rstd) >> 20) & 0x7ff) - 1022, -126), 127);
    const float r2 = __uint_as_float((uint32_t)(rexp + 127) << 23);
    const double rf = rstd * __builtin_bit_cast(double, (uint64_t)(1023 - rexp) << 52);
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      const int c0 = (k * NT + tid) * 8, n = live ? A.cols - c0 : 0;
      float v[8];
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[j] = round_to_odd((double)(at8(h[k], j) * r2 * at8(w[k], j)) * rf);
        m = max(m, j < n ? finite_mag(v[j]) : 0u);
      }
      const uint32_t e = act8_byte(max16(m));
      const float inv = act8_inv(e);
      const u32x2 q = {act8_pack4(v, inv), act8_pack4(v + 4, inv)};
      uint8_t* qp = A.codes + r * A.cols + c0;
      if (n >= 8) {
        __builtin_nontemporal_store(q, (u32x2_a1*)qp);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < n) qp[j] = (uint8_t)((j < 4 ? q.x : q.y) >> (8 * (j & 3)));
      }
      if ((tid & 15) == 0 && n > 0) A.scales[r * A.nb + (c0 >> 7)] = (uint8_t)e;
      if (A.y) {
        const float s = act8_scale(e);
        const u32x2 a = act8_bf16x4(q.x, s), b = act8_bf16x4(q.y, s);
        store8<true>(A.y + r * A.cols + c0, u32x4{a.x, a.y, b.x, b.y}, n);
      }
    }
  }
}

// ------------------------------------------------------------------ backward
struct NormGradArgs {
  const uint16_t *params, *dy, *dh, *h;
  int64_t dy_stride, dh_stride;
  Place place;
  const float* rstd;
  uint16_t* dx;
  float* partial;  // groups x cols
  int64_t rows, rows_per_group;
  int32_t cols;
};

// The operands of one row, and its 1/rms.
template <int NP>
struct GradRow {
  Piece8 dy[NP], h[NP], dh[NP];
  float R;
};
template <int NT, int NP>
__device__ __forceinline__ GradRow<NP> load_row(const NormGradArgs& A, int64_t r, bool live, int t) {
  // at any address, which a scalar load of a row's one value would not be
  typedef float any __attribute__((aligned(1)));
  GradRow<NP> x;
  x.R = live ? ((const any*)A.rstd)[r] : 0.f;
#pragma unroll
  for (int k = 0; k < NP; ++k) {
    const int c0 = (k * NT + t) * 8, n = live ? A.cols - c0 : 0;
    x.dy[k] = load8<true>(A.dy + r * A.dy_stride + c0, n);
    x.h[k] = load8<true>(A.h + r * A.cols + c0, n);
    if (A.dh) x.dh[k] = load8<true>(A.dh + r * A.dh_stride + c0, n);
  }
  return x;
}
// Keeps a piece packed: its widened values are not carried past this point.
__device__ __forceinline__ void keep(Piece8& p) { asm volatile("" : "+v"(p.w)); }

// One block per group of consecutive rows, WAYS rows at a time, each by NT
// threads; the ways' sums for the weight are added in order at the end.  What
// it needs is loads in flight: 16 waves on a CU, from several rows a block
// where a row is short (65536 x 256: 195 us with a wave a block, 29 here; 1M x
// 128: 2950, 190).  The next row's loads before this row's sum were no faster
// (16384 x 4096: 108 us, 100 here) for the registers that they hold.
// Rows of more than two pieces a thread keep the weight's sums in LDS, each
// thread its own, 16 bytes apart: in registers they spill (4096 x 32768: 639
// us, 209 here; 4096 x 12288: 90 in registers of 1024 threads, 84 here).
template <int NT, int NP, int WAYS, bool GAPS>
__global__ void __launch_bounds__(NT* WAYS, 4) norm_grad_kernel(const NormGradArgs A) {
  constexpr int kWidth = NT * NP * 8;
  constexpr bool kInLds = NP > 2;
  static_assert(WAYS == 1 || !kInLds, "the sums of the ways take the same LDS");
  __shared__ float red[2][(NT * WAYS + 63) / 64];
  __shared__ alignas(16) float sum[WAYS > 1 || kInLds ? WAYS * kWidth : 1];
  const int t = WAYS > 1 ? threadIdx.x % NT : threadIdx.x, way = WAYS > 1 ? threadIdx.x / NT : 0;
  f32x4* mine = (f32x4*)sum + t;
  Piece8 w[NP];
  float dw[NP][8];
#pragma unroll
  for (int k = 0; k < NP; ++k) {
    const int c0 = (k * NT + t) * 8;
    w[k] = weight8<GAPS>(A.params, A.place, c0, A.cols - c0);
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[k][j] = 0.f;
    if constexpr (kInLds) mine[2 * k * NT] = mine[(2 * k + 1) * NT] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  const int64_t ra = (int64_t)blockIdx.x * A.rows_per_group;
  const int64_t rz = min(A.rows, ra + A.rows_per_group);
  int turn = 0;
  for (int64_t r0 = ra; r0 < rz; r0 += WAYS) {
    const int64_t r = r0 + way;
    GradRow<NP> x = load_row<NT, NP>(A, r, r < rz, t);
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      if constexpr (kInLds) keep(w[k]);
      f32x4 lo, hi;
      if constexpr (kInLds) lo = mine[2 * k * NT], hi = mine[(2 * k + 1) * NT];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float d = at8(x.dy[k], j), n = at8(x.h[k], j) * x.R;
        s += d * at8(w[k], j) * n;
        if constexpr (!kInLds) dw[k][j] += d * n;
        else if (j < 4) lo[j] += d * n;
        else hi[j - 4] += d * n;
      }
      if constexpr (kInLds) mine[2 * k * NT] = lo, mine[(2 * k + 1) * NT] = hi;
    }
    s = row_sum<NT>(s, &red[turn][way * NT / 64]);
    turn ^= 1;
    const float c = s / (float)A.cols;
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      const int c0 = (k * NT + t) * 8, n = r < rz ? A.cols - c0 : 0;
      if constexpr (kInLds) keep(w[k]), keep(x.dy[k]), keep(x.h[k]);
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float g = at8(x.dy[k], j) * at8(w[k], j);
        const float d = x.R * (g - c * (at8(x.h[k], j) * x.R));
        v[j] = A.dh ? at8(x.dh[k], j) + d : d;
      }
      store8<false>(A.dx + r * A.cols + c0, round8(v), n);
    }
  }
  if constexpr (WAYS > 1) {
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      float* p = &sum[way * kWidth + (k * NT + t) * 8];
      *(f32x4*)p = f32x4{dw[k][0], dw[k][1], dw[k][2], dw[k][3]};
      *(f32x4*)(p + 4) = f32x4{dw[k][4], dw[k][5], dw[k][6], dw[k][7]};
    }
    __syncthreads();
    for (int c = threadIdx.x; c < A.cols; c += NT * WAYS) {
      float v = 0.f;
#pragma unroll
      for (int k = 0; k < WAYS; ++k) v += sum[k * kWidth + c];
      A.partial[(int64_t)blockIdx.x * A.cols + c] = v;
    }
    return;
  }
#pragma unroll
  for (int k = 0; k < NP; ++k) {
    const int c0 = (k * NT + t) * 8, n = A.cols - c0;
    float* p = A.partial + (int64_t)blockIdx.x * A.cols + c0;
    if constexpr (kInLds) {
#pragma unroll
      for (int j = 0; j < 8; ++j) dw[k][j] = mine[(2 * k + j / 4) * NT][j & 3];
    }
    if (n >= 8) {
      *(f32x4_a4*)p = f32x4{dw[k][0], dw[k][1], dw[k][2], dw[k][3]};
      *(f32x4_a4*)(p + 4) = f32x4{dw[k][4], dw[k][5], dw[k][6], dw[k][7]};
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < n) p[j] = dw[k][j];
    }
  }
}

// Sum over the groups: 32 columns per block, 32 threads per column, each
// taking every 32nd group in order; then the 32 sums in order.
constexpr int kSumCols = 32, kSumWays = 32;
template <bool GAPS>
__global__ void __launch_bounds__(kSumCols* kSumWays)
    norm_sum_kernel(const float* partial, int32_t groups, int32_t cols, const GradOut out) {
  __shared__ float part[kSumWays][kSumCols + 1];
  const int c = threadIdx.x % kSumCols, way = threadIdx.x / kSumCols;
  const int32_t col = (int32_t)blockIdx.x * kSumCols + c;
  float s = 0.f;
  if (col < cols) {
#pragma unroll 4
    for (int32_t g = way; g < groups; g += kSumWays) s += partial[(int64_t)g * cols + col];
  }
  part[way][c] = s;
  __syncthreads();
  if (way == 0 && col < cols) {
    float t = 0.f;
#pragma unroll
    for (int k = 0; k < kSumWays; ++k) t += part[k][c];
    grad_store(out, place_at<GAPS>(out.place, col), t);
  }
}

// ------------------------------------------------------------------ host
// Rows that a block of the backward pass takes at a time.
int64_t grad_ways(int64_t cols) {
  return cols <= 128 ? 32 : cols <= 256 ? 16 : cols <= 1024 ? 8 : cols <= 2048 ? 4 : cols <= 4096 ? 2 : 1;
}
// Row groups of the weight's gradient: a function of the shape alone, so the
// order of the sum is too.  Two blocks per CU, or one where its LDS leaves no
// room for another (4096 x 32768 in 512 groups: 227 us, in 256 209).
int64_t rows_per_group(int64_t rows, int64_t cols) {
  const int64_t groups = cols <= 16384 ? 512 : 256;
  return std::max({(int64_t)4, grad_ways(cols), (rows + groups - 1) / groups});
}
int64_t groups_of(int64_t rows, int64_t cols) {
  const int64_t n = rows_per_group(rows, cols);
  return rows == 0 ? 0 : (rows + n - 1) / n;
}

int shape_ok(const zero_layout* L, int32_t tensor, int64_t rows) {
  if (!L || rows < 0) return ZERO_EINVAL;
  if (!tensor_ok(L, tensor)) return ZERO_ERANGE;
  const int64_t cols = L->numel[(size_t)tensor];
  if (cols > kMaxNormCols || rows > ZERO_MAX_ROWS) return ZERO_ERANGE;
  return ZERO_OK;
}

template <int NT, int NP>
int launch_norm(const NormArgs& A, hipStream_t s) {
  constexpr int kRows = kBlock<NT> / NT;
  const unsigned grid = (unsigned)std::min<int64_t>((A.rows + kRows - 1) / kRows, 1 << 14);
  if (A.place.gap)
    hipLaunchKernelGGL((norm_kernel<NT, NP, true>), dim3(grid), dim3(kBlock<NT>), 0, s, A);
  else
    hipLaunchKernelGGL((norm_kernel<NT, NP, false>), dim3(grid), dim3(kBlock<NT>), 0, s, A);
  return launched();
}
template <int NT, int NP, int WAYS>
int launch_norm_grad(const NormGradArgs& A, int64_t groups, hipStream_t s) {
  const dim3 grid((unsigned)groups), block(NT * WAYS);
  if (A.place.gap)
    hipLaunchKernelGGL((norm_grad_kernel<NT, NP, WAYS, true>), grid, block, 0, s, A);
  else
    hipLaunchKernelGGL((norm_grad_kernel<NT, NP, WAYS, false>), grid, block, 0, s, A);
  return launched();
}

}  // namespace

extern "C" {

int zero_rms_norm(const zero_layout* L, int32_t tensor, const uint16_t* params_flat,
                  const uint16_t* x, int64_t x_stride, const uint16_t* res, int64_t res_stride,
                  int64_t rows, double eps, uint16_t* h, float* rstd, uint8_t* codes,
                  uint8_t* scales, uint16_t* y, hipStream_t stream) {
  const int rc = shape_ok(L, tensor, rows);
  if (rc != ZERO_OK) return rc;
  if (!(eps >= 0.0) || !(eps - eps == 0.0)) return ZERO_EINVAL;
  const int64_t cols = L->numel[(size_t)tensor];
  if (rows == 0 || cols == 0) return ZERO_OK;
  if (!params_flat || !x || !rstd || !codes || !scales || (res && !h)) return ZERO_EINVAL;
  if (x_stride < cols || (res && res_stride < cols)) return ZERO_EINVAL;
  if (x_stride > ZERO_MAX_STRIDE || (res && res_stride > ZERO_MAX_STRIDE)) return ZERO_ERANGE;
  NormArgs A;
  int64_t lo, hi;
  A.place = make_place(L, tensor, &lo, &hi);
  const int64_t nb = (cols + kAct8Block - 1) / kAct8Block;
  const Bytes outs[] = {Bytes{h, 2 * rows * cols}, Bytes{y, 2 * rows * cols}, Bytes{rstd, 4 * rows},
                        Bytes{codes, rows * cols}, Bytes{scales, rows * nb}};
  const Bytes ins[] = {Bytes{params_flat + lo, 2 * (hi - lo)}, rows_of(x, rows, cols, x_stride, 2),
                       rows_of(res, rows, cols, res_stride, 2)};
  if (any_overlap(outs, ins)) return ZERO_EOVERLAP;
  if (hip_error_pending()) return ZERO_EHIP;
  A.params = params_flat;
  A.x = x;
  A.res = res;
  A.x_stride = x_stride;
  A.res_stride = res_stride;
  A.h = h;
  A.y = y;
  A.rstd = rstd;
  A.codes = codes;
  A.scales = scales;
  A.rows = rows;
  A.cols = (int32_t)cols;
  A.nb = (int32_t)nb;
  A.eps = eps;
  if (cols <= 128) return launch_norm<16, 1>(A, stream);
  if (cols <= 256) return launch_norm<32, 1>(A, stream);
  if (cols <= 512) return launch_norm<64, 1>(A, stream);
  if (cols <= 1024) return launch_norm<64, 2>(A, stream);
  if (cols <= 2048) return launch_norm<256, 1>(A, stream);
  if (cols <= 4096) return launch_norm<256, 2>(A, stream);
  if (cols <= 6144) return launch_norm<256, 3>(A, stream);
  if (cols <= 8192) return launch_norm<256, 4>(A, stream);
  if (cols <= 12288) return launch_norm<512, 3>(A, stream);
  if (cols <= 16384) return launch_norm<1024, 2>(A, stream);
  if (cols <= 24576) return launch_norm<1024, 3>(A, stream);
  return launch_norm<1024, 4>(A, stream);
}

int64_t zero_rms_norm_grad_workspace(const zero_layout* L, int32_t tensor, int64_t rows) {
  const int rc = shape_ok(L, tensor, rows);
  if (rc != ZERO_OK) return rc;
  return groups_of(rows, L->numel[(size_t)tensor]) * L->numel[(size_t)tensor] * 4;
}

int zero_rms_norm_grad(const zero_layout* L, int32_t tensor, const uint16_t* params_flat,
                       const uint16_t* dy, int64_t dy_stride, const uint16_t* dh,
                       int64_t dh_stride, const uint16_t* h, const float* rstd, int64_t rows,
                       float scale, uint32_t flags, uint16_t* dx, float* acc_flat,
                       uint16_t* bf16_flat, void* workspace, int64_t workspace_bytes,
                       hipStream_t stream) {
  int rc = shape_ok(L, tensor, rows);
  if (rc != ZERO_OK) return rc;
  const int64_t cols = L->numel[(size_t)tensor];
  rc = grad_out_ok(flags, scale, acc_flat, bf16_flat, cols);
  if (rc != ZERO_OK) return rc;
  // without rows the gradient is zero, which changes something only where
  // the flags ask for an overwrite or an emission
  if (cols == 0 || (rows == 0 && !(flags & (ZERO_ACC_OVERWRITE | ZERO_ACC_EMIT_BF16)))) return ZERO_OK;
  const int64_t groups = groups_of(rows, cols), need = groups * cols * 4;
  if (rows > 0) {
    if (!params_flat || !dy || !h || !rstd || !dx || !workspace) return ZERO_EINVAL;
    if (dy_stride < cols || (dh && dh_stride < cols)) return ZERO_EINVAL;
    if (dy_stride > ZERO_MAX_STRIDE || (dh && dh_stride > ZERO_MAX_STRIDE)) return ZERO_ERANGE;
    if (workspace_bytes < need || ((uintptr_t)workspace & 15u)) return ZERO_EINVAL;
  }
  NormGradArgs A;
  GradOut out;
  int64_t lo, hi;
  out.place = A.place = make_place(L, tensor, &lo, &hi);
  const Bytes outs[] = {Bytes{dx, 2 * rows * cols},
                        Bytes{acc_used(flags) ? acc_flat + lo : nullptr, 4 * (hi - lo)},
                        Bytes{(flags & ZERO_ACC_EMIT_BF16) ? bf16_flat + lo : nullptr, 2 * (hi - lo)},
                        Bytes{workspace, need}};
  const Bytes ins[] = {Bytes{params_flat ? params_flat + lo : nullptr, 2 * (hi - lo)},
                       rows_of(dy, rows, cols, dy_stride, 2), rows_of(dh, rows, cols, dh_stride, 2),
                       Bytes{h, 2 * rows * cols}, Bytes{rstd, 4 * rows}};
  if (any_overlap(outs, ins)) return ZERO_EOVERLAP;
  if (hip_error_pending()) return ZERO_EHIP;
  if (rows > 0) {
    A.params = params_flat;
    A.dy = dy;
    A.dh = dh;
    A.h = h;
    A.dy_stride = dy_stride;
    A.dh_stride = dh_stride;
    A.rstd = rstd;
    A.dx = dx;
    A.partial = (float*)workspace;
    A.rows = rows;
    A.rows_per_group = rows_per_group(rows, cols);
    A.cols = (int32_t)cols;
    if (cols <= 128) rc = launch_norm_grad<16, 1, 32>(A, groups, stream);
    else if (cols <= 256) rc = launch_norm_grad<32, 1, 16>(A, groups, stream);
    else if (cols <= 512) rc = launch_norm_grad<64, 1, 8>(A, groups, stream);
    else if (cols <= 1024) rc = launch_norm_grad<64, 2, 8>(A, groups, stream);
    else if (cols <= 2048) rc = launch_norm_grad<128, 2, 4>(A, groups, stream);
    else if (cols <= 4096) rc = launch_norm_grad<256, 2, 2>(A, groups, stream);
    else if (cols <= 8192) rc = launch_norm_grad<512, 2, 1>(A, groups, stream);
    else if (cols <= 12288) rc = launch_norm_grad<512, 3, 1>(A, groups, stream);
    else if (cols <= 16384) rc = launch_norm_grad<512, 4, 1>(A, groups, stream);
    else if (cols <= 24576) rc = launch_norm_grad<1024, 3, 1>(A, groups, stream);
    else rc = launch_norm_grad<1024, 4, 1>(A, groups, stream);
    if (rc != ZERO_OK) return rc;
  }
  out.acc = acc_flat;
  out.out = bf16_flat;
  out.scale = scale;
  out.flags = flags;
  const unsigned grid = (unsigned)((cols + kSumCols - 1) / kSumCols);
  if (out.place.gap)
    hipLaunchKernelGGL(norm_sum_kernel<true>, dim3(grid), dim3(kSumCols * kSumWays), 0, stream,
                       (const float*)workspace, (int32_t)groups, (int32_t)cols, out);
  else
    hipLaunchKernelGGL(norm_sum_kernel<false>, dim3(grid), dim3(kSumCols * kSumWays), 0, stream,
                       (const float*)workspace, (int32_t)groups, (int32_t)cols, out);
  return launched();
}

}  // extern "C"
