// zero_bias_grad: the gradient through a layer's own activation, and the
// bias's gradient, a sum over the rows.
//
// Page "Infra: Data Parallel" (pufanyi.com), section "Naive Data
// Parallelism": a micro-batch's gradients are added to the rank's sum, scaled.
//
//   g = dy * act'(pre);  db[c] = sum over rows t of g[t, c];  dpre = bf16(g)
//
// An HBM stream: a lane takes 8 neighbouring columns, 16 bytes of a row, and
// keeps their sums; a block's rows are summed in LDS, the blocks' sums by a
// second launch, both in order.
#include <algorithm>

#include "activation.hpp"

namespace {
using namespace zs;

constexpr int kThreads = 256;
constexpr int kAhead = 4;  // rows that a lane has in flight

struct Args {
  const uint16_t *dy, *pre;
  uint16_t* dpre;
  int64_t dy_stride, rows, rows_per_group;
  int32_t cols, act;
  float* partial;  // groups x cols
};

__device__ __forceinline__ u32x4 load8(const uint16_t* p, int n) {
  return n >= 8 ? __builtin_nontemporal_load((const u32x4_a2*)p) : load_some(p, n);
}

// ACROSS lanes along a row (8 columns each), the rest of the block down.  Bound by
// HBM: 16384 x 14336 through an activation takes 272 us and the sum's launch 5,
// 5.1 TB/s (439 where the normal distribution's function came from the math
// library); 1000 x 2304 without one 3.8 + 3.0.  At an odd place 339; rows of 14337
// columns 380, of 14335 568.
template <int ACROSS, bool ACT>
__global__ void __launch_bounds__(kThreads) bias_kernel(const Args A) {
  constexpr int kDown = kThreads / ACROSS;  // rows at a time
  const int across = threadIdx.x % ACROSS, down = threadIdx.x / ACROSS;
  const int32_t c = ((int32_t)blockIdx.x * ACROSS + across) * 8;
  const int n = min(8, A.cols - c);
  const int64_t ra = (int64_t)blockIdx.y * A.rows_per_group, rz = min(A.rows, ra + A.rows_per_group);
  float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int64_t r0 = ra + down; r0 < rz; r0 += kDown * kAhead) {
    u32x4 dy[kAhead], pre[ACT ? kAhead : 1];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int64_t r = r0 + k * kDown;
      const int m = r < rz ? n : 0;
      dy[k] = load8(A.dy + r * A.dy_stride + c, m);
      if constexpr (ACT) pre[k] = load8(A.pre + r * A.cols + c, m);
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int64_t r = r0 + k * kDown;
      float g[8];
      widen8(dy[k], g);
      if constexpr (ACT) {
        if (r >= rz) continue;
        float s[8];
        widen8(pre[k], s);
        apply8<true>(A.act, s);
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] *= s[j];
      }
      if (A.dpre && r < rz) {
        uint16_t* p = A.dpre + r * A.cols + c;
        if (n >= 8)
          __builtin_nontemporal_store(round8(g), (u32x4_a2*)p);
        else
          store_some(p, round8(g), n);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[j] += g[j];
    }
  }
  __shared__ alignas(16) f32x4 all[kThreads * 2];
  all[threadIdx.x * 2] = f32x4{sum[0], sum[1], sum[2], sum[3]};
  all[threadIdx.x * 2 + 1] = f32x4{sum[4], sum[5], sum[6], sum[7]};
  __syncthreads();
  // thread k sums 4 columns (k / 2, k % 2) over the rows of threads
  if (threadIdx.x >= ACROSS * 2) return;
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
  for (int d = 0; d < kDown; ++d) v = v + all[d * ACROSS * 2 + threadIdx.x];
  const int32_t at = (int32_t)blockIdx.x * ACROSS * 8 + (int)threadIdx.x * 4;
  float* p = A.partial + (int64_t)blockIdx.y * A.cols + at;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (at + j < A.cols) p[j] = v[j];
}

// Sum over the groups: 32 columns per block, 32 threads per column, each
// taking every 32nd group in order; then the 32 sums in order.
constexpr int kSumCols = 32, kSumWays = 32;
__global__ void __launch_bounds__(kSumCols* kSumWays)
    bias_sum_kernel(const float* partial, int32_t groups, int32_t cols, const GradOut out) {
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
    grad_store(out, place_at<true>(out.place, col), t);
  }
}

// ------------------------------------------------------------------ host
// Threads along a row: 64 of a block's 256 where the rows are long, fewer where
// they are short; groups of rows so that about 2048 blocks have work.  A function
// of the shape alone, and so is the order of the sums.
struct Plan {
  int across;
  int64_t col_blocks, rows_per_group, groups, bytes;
};
Plan make_plan(int64_t rows, int64_t cols) {
  Plan p;
  p.across = cols > 512 ? 64 : cols > 128 ? 32 : 8;
  p.col_blocks = (cols + p.across * 8 - 1) / (p.across * 8);
  const int64_t at_least = (int64_t)kThreads / p.across * kAhead;
  const int64_t wanted = std::max<int64_t>(1, 2048 / std::max<int64_t>(1, p.col_blocks));
  p.rows_per_group = std::max(at_least, (rows + wanted - 1) / wanted);
  p.groups = rows == 0 ? 0 : (rows + p.rows_per_group - 1) / p.rows_per_group;
  p.bytes = p.groups * cols * 4;
  return p;
}

int shape_ok(const zero_layout* L, int32_t tensor, int64_t rows) {
  if (!L || rows < 0) return ZERO_EINVAL;
  if (!tensor_ok(L, tensor)) return ZERO_ERANGE;
  if (L->numel[(size_t)tensor] > ZERO_MAX_COLS || rows > ZERO_MAX_ROWS) return ZERO_ERANGE;
  return ZERO_OK;
}

template <int ACROSS>
void launch(const Args& A, const Plan& p, hipStream_t s) {
  const dim3 grid((unsigned)p.col_blocks, (unsigned)p.groups);
  if (A.pre)
    hipLaunchKernelGGL((bias_kernel<ACROSS, true>), grid, dim3(kThreads), 0, s, A);
  else
    hipLaunchKernelGGL((bias_kernel<ACROSS, false>), grid, dim3(kThreads), 0, s, A);
}

}  // namespace

extern "C" {

int64_t zero_bias_grad_workspace(const zero_layout* L, int32_t tensor, int64_t rows) {
  const int rc = shape_ok(L, tensor, rows);
  if (rc != ZERO_OK) return rc;
  return make_plan(rows, L->numel[(size_t)tensor]).bytes;
}

int zero_bias_grad(const zero_layout* L, int32_t tensor, const uint16_t* dy, int64_t dy_stride,
                   const uint16_t* pre, int32_t activation, int64_t rows, float scale, uint32_t flags,
                   uint16_t* dpre, float* acc_flat, uint16_t* bf16_flat, void* workspace,
                   int64_t workspace_bytes, hipStream_t stream) {
  int rc = shape_ok(L, tensor, rows);
  if (rc != ZERO_OK) return rc;
  if (!activation_ok(activation)) return ZERO_EINVAL;
  const int64_t cols = L->numel[(size_t)tensor];
  rc = grad_out_ok(flags, scale, acc_flat, bf16_flat, cols);
  if (rc != ZERO_OK) return rc;
  if (cols == 0 || (rows == 0 && !(flags & (ZERO_ACC_OVERWRITE | ZERO_ACC_EMIT_BF16)))) return ZERO_OK;
  const Plan p = make_plan(rows, cols);
  if (rows > 0) {
    if (!dy || (activation != ZERO_ACT_NONE) != (pre != nullptr) || dy_stride < cols) return ZERO_EINVAL;
    if (dy_stride > ZERO_MAX_STRIDE) return ZERO_ERANGE;
    if (!workspace || workspace_bytes < p.bytes || ((uintptr_t)workspace & 15u)) return ZERO_EINVAL;
  }
  GradOut out{acc_flat, bf16_flat, {}, scale, flags};
  int64_t lo, hi;
  out.place = make_place(L, tensor, &lo, &hi);
  const Bytes outs[] = {Bytes{dpre, 2 * rows * cols}, Bytes{acc_used(flags) ? acc_flat + lo : nullptr, 4 * (hi - lo)},
                        Bytes{(flags & ZERO_ACC_EMIT_BF16) ? bf16_flat + lo : nullptr, 2 * (hi - lo)},
                        Bytes{workspace, p.bytes}};
  const Bytes ins[] = {rows_of(dy, rows, cols, dy_stride, 2), Bytes{pre, 2 * rows * cols}};
  if (any_overlap(outs, ins)) return ZERO_EOVERLAP;
  if (hip_error_pending()) return ZERO_EHIP;
  if (rows > 0) {
    const Args A{dy,   pre,  dpre, dy_stride, rows, p.rows_per_group, (int32_t)cols, activation, (float*)workspace};
    if (p.across == 64) launch<64>(A, p, stream);
    else if (p.across == 32) launch<32>(A, p, stream);
    else launch<8>(A, p, stream);
    rc = launched();
    if (rc != ZERO_OK) return rc;
  }
  hipLaunchKernelGGL(bias_sum_kernel, dim3((unsigned)((cols + kSumCols - 1) / kSumCols)), dim3(kSumCols * kSumWays),
                     0, stream, (const float*)workspace, (int32_t)p.groups, (int32_t)cols, out);
  return launched();
}

}  // extern "C"
