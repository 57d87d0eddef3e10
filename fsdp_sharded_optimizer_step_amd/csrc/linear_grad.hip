// zero_linear_grad: a linear weight's gradient from the output gradient (bf16)
// and the layer's input, kept as an 8-bit checkpoint.
//
// Page "Infra: Data Parallel" (pufanyi.com), section "Naive Data
// Parallelism": a micro-batch's gradients are added to the rank's local sum,
// scaled; here the product is added to that sum as it leaves the registers.
//
//   dW[o, i] = sum over t of dY[t, o] * X[t, i],  X the values the 8-bit codes
//   stand for (weights kept as (in, out) take the transpose)
//
// The sum runs over the tokens, the slow index of both operands, while a
// matrix instruction wants consecutive tokens of one column in a lane.  So
// the tiles go to LDS as they lie in memory, 32 columns to a panel of 64-byte
// token rows, and are read back with the transposing LDS read: 16 lanes read
// 4 token rows of 16 columns and each gets one column's 4 tokens.  A panel
// read of a wave is 512 consecutive bytes, free of bank conflicts.  Codes
// become bf16 on their way into LDS, exactly (their scale is a power of two,
// and every value is a normal bf16 number), with one conversion per two
// codes; products of bf16 are exact in binary32, sums are binary32.
#include <algorithm>

#include "act8.hpp"

namespace {
using namespace zs;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kThreads = 256;            // 4 waves, two by two over the tile
constexpr int kStep = 64;                // tokens of one LDS tile
constexpr int kPanelBytes = kStep * 64 + 64;  // 64 bytes apart: writes of one token row spread over the banks

struct Args {
  const uint16_t* dy;
  int64_t dy_stride;
  const uint8_t* codes;
  const uint8_t* scales;
  int64_t tokens, tokens_per_split;
  int32_t O, I, nb;
  int32_t rows, cols;           // of the gradient: (O, I), or (I, O) when transposed
  int32_t row_tiles, col_tiles;
  int32_t splits;
  float* partial;               // splits x rows x cols where the result does not go out directly
  GradOut out;
};

// Chunks of dY: 8 columns of one token; of X: 16 columns.
template <int TC>
struct DyTile {
  static constexpr int kPerRow = TC / 8, kRows = kThreads / kPerRow, kN = kStep / kRows;
  u32x4 v[kN];
  __device__ __forceinline__ void load(const Args& A, int64_t t0, int64_t tz, int32_t c0) {
    const int col = c0 + (threadIdx.x % kPerRow) * 8;
#pragma unroll
    for (int k = 0; k < kN; ++k) {
      const int64_t t = t0 + k * kRows + threadIdx.x / kPerRow;
      const uint16_t* p = A.dy + t * A.dy_stride + col;
      const int n = t < tz ? A.O - col : 0;
      v[k] = u32x4{0u, 0u, 0u, 0u};
      if (n >= 8) {
        v[k] = *(const u32x4_a2*)p;
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < n) v[k][j >> 1] |= (uint32_t)p[j] << (16 * (j & 1));
      }
    }
  }
  __device__ __forceinline__ void store(char* lds) const {
    const int c = (threadIdx.x % kPerRow) * 8;
#pragma unroll
    for (int k = 0; k < kN; ++k) {
      const int t = k * kRows + threadIdx.x / kPerRow;
      *(u32x4*)(lds + (c >> 5) * kPanelBytes + t * 64 + (c & 31) * 2) = v[k];
    }
  }
};

template <int TC>
struct XTile {
  static constexpr int kPerRow = TC / 16, kRows = kThreads / kPerRow, kN = kStep / kRows;
  u32x4 v[kN];
  uint32_t e[kN];
  __device__ __forceinline__ void load(const Args& A, int64_t t0, int64_t tz, int32_t c0) {
    const int col = c0 + (threadIdx.x % kPerRow) * 16;
#pragma unroll
    for (int k = 0; k < kN; ++k) {
      const int64_t t = t0 + k * kRows + threadIdx.x / kPerRow;
      const uint8_t* p = A.codes + t * A.I + col;
      const int n = t < tz ? A.I - col : 0;
      v[k] = u32x4{0u, 0u, 0u, 0u};
      e[k] = 127u;
      if (n > 0) e[k] = A.scales[t * A.nb + (col >> 7)];
      if (n >= 16) {
        v[k] = *(const u32x4_a1*)p;
      } else {
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (j < n) v[k][j >> 2] |= (uint32_t)p[j] << (8 * (j & 3));
      }
    }
  }
  __device__ __forceinline__ void store(char* lds) const {
    const int c = (threadIdx.x % kPerRow) * 16;
#pragma unroll
    for (int k = 0; k < kN; ++k) {
      const int t = k * kRows + threadIdx.x / kPerRow;
      char* p = lds + (c >> 5) * kPanelBytes + t * 64 + (c & 31) * 2;
      const float s = act8_scale(e[k]);
      const u32x2 a = act8_bf16x4(v[k].x, s), b = act8_bf16x4(v[k].y, s);
      const u32x2 d = act8_bf16x4(v[k].z, s), f = act8_bf16x4(v[k].w, s);
      *(u32x4*)p = u32x4{a.x, a.y, b.x, b.y};
      *(u32x4*)(p + 16) = u32x4{d.x, d.y, f.x, f.y};
    }
  }
};

// 32 columns x 16 tokens of a panel as a matrix operand: lane l holds column
// l % 32, tokens 4*(l / 32) + {0..3, 8..11}.
__device__ __forceinline__ bf16x8 frag(const char* panel) {
  typedef __attribute__((address_space(3))) s16x4 lds_t;
  const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_t*)panel);
  const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_t*)(panel + 512));
  return __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}
__device__ __forceinline__ int frag_offset() {
  const int l = threadIdx.x & 63, g = l >> 4, i = l & 15;
  return ((i >> 2) + 4 * (g >> 1)) * 64 + (g & 1) * 32 + (i & 3) * 8;
}

// W: 32-column panels of a wave along each side; the block's tile is 2W
// panels wide and high.  TR: rows of the gradient are X's columns.
template <int W, bool TR>
__global__ void __launch_bounds__(kThreads) grad_kernel(const Args A) {
  constexpr int kSide = 64 * W;
  __shared__ __align__(16) char lds[2][2 * W * kPanelBytes];  // rows' operand, columns' operand
  const int tile = blockIdx.x;
  const int32_t r0 = (tile / A.col_tiles) * kSide, c0 = (tile % A.col_tiles) * kSide;
  const int64_t ta = (int64_t)blockIdx.y * A.tokens_per_split;
  const int64_t tz = min(A.tokens, ta + A.tokens_per_split);
  const int wave = threadIdx.x >> 6, wm = wave >> 1, wn = wave & 1, lane = threadIdx.x & 63;
  f32x16 acc[W][W];
#pragma unroll
  for (int a = 0; a < W; ++a)
#pragma unroll
    for (int b = 0; b < W; ++b)
#pragma unroll
      for (int k = 0; k < 16; ++k) acc[a][b][k] = 0.f;

  DyTile<kSide> dy;
  XTile<kSide> x;
  const char* fa = lds[0] + wm * W * kPanelBytes + frag_offset();
  const char* fb = lds[1] + wn * W * kPanelBytes + frag_offset();
  for (int64_t t = ta; t < tz; t += kStep) {
    dy.load(A, t, tz, TR ? c0 : r0);
    x.load(A, t, tz, TR ? r0 : c0);
    __syncthreads();
    dy.store(lds[TR ? 1 : 0]);
    x.store(lds[TR ? 0 : 1]);
    __syncthreads();
#pragma unroll
    for (int s = 0; s < kStep / 16; ++s) {
      bf16x8 a[W], b[W];
#pragma unroll
      for (int k = 0; k < W; ++k) {
        a[k] = frag(fa + k * kPanelBytes + s * 1024);
        b[k] = frag(fb + k * kPanelBytes + s * 1024);
      }
#pragma unroll
      for (int m = 0; m < W; ++m)
#pragma unroll
        for (int n = 0; n < W; ++n)
          acc[m][n] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[m], b[n], acc[m][n], 0, 0, 0);
    }
  }
  // lane l, register k: row 8*(k/4) + 4*(l/32) + k%4, column l%32
#pragma unroll
  for (int n = 0; n < W; ++n) {
    const int32_t c = c0 + (wn * W + n) * 32 + (lane & 31);
    if (c >= A.cols) continue;
#pragma unroll
    for (int m = 0; m < W; ++m)
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const int32_t r = r0 + (wm * W + m) * 32 + 8 * (k >> 2) + 4 * (lane >> 5) + (k & 3);
        if (r >= A.rows) continue;
        const int64_t i = (int64_t)r * A.cols + c;
        if (A.partial)
          A.partial[(int64_t)blockIdx.y * A.rows * A.cols + i] = acc[m][n][k];
        else
          grad_store(A.out, A.out.place.x0 + i, acc[m][n][k]);
      }
  }
}

// Adds up the splits, in order, and hands the sum on.
template <bool GAPS>
__global__ void __launch_bounds__(kThreads)
    sum_kernel(const float* partial, int32_t splits, int64_t numel, const GradOut out) {
  const int64_t T = (int64_t)gridDim.x * kThreads;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i * 4 < numel; i += T) {
    const int64_t e = i * 4;
    const int n = (int)min((int64_t)4, numel - e);
    f32x4 s = {0.f, 0.f, 0.f, 0.f};
    for (int k = 0; k < splits; ++k) {
      const float* p = partial + (int64_t)k * numel + e;
      if (n >= 4) {
        s += *(const f32x4_a4*)p;
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (j < n) s[j] += p[j];
      }
    }
    if (!GAPS && n >= 4) {
      grad_store4(out, place_at<GAPS>(out.place, e), s);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < n) grad_store(out, place_at<GAPS>(out.place, e + j), s[j]);
    }
  }
}

// ------------------------------------------------------------------ host
struct Plan {
  int64_t row_tiles, col_tiles, splits, tokens_per_split, bytes;
};

// Tiles of 128 x 128.  Fewer tiles than the chip takes at once (256 CUs, two
// blocks each) leave the sum over tokens to several blocks, 256 tokens each
// at least.  Where padding falls inside the tensor the result goes through
// the workspace too, and the sum places it.
Plan make_plan(const zero_layout* L, int32_t tensor, int64_t rows, int64_t cols, int64_t tokens) {
  int64_t lo, hi;
  const bool gaps = make_place(L, tensor, &lo, &hi).gap != 0;
  Plan p;
  p.row_tiles = (rows + 127) / 128;
  p.col_tiles = (cols + 127) / 128;
  const int64_t tiles = std::max<int64_t>(1, p.row_tiles * p.col_tiles);
  const int64_t most = std::max<int64_t>(1, (tokens + 255) / 256);
  p.splits = std::max<int64_t>(1, std::min<int64_t>({most, 512 / tiles, 32}));
  p.tokens_per_split = (tokens + p.splits * kStep - 1) / (p.splits * kStep) * kStep;
  if (p.tokens_per_split == 0) p.tokens_per_split = kStep;
  p.splits = std::max<int64_t>(1, (tokens + p.tokens_per_split - 1) / p.tokens_per_split);
  p.bytes = p.splits > 1 || gaps ? p.splits * rows * cols * 4 : 0;
  return p;
}

int shape_ok(const zero_layout* L, int32_t tensor, int64_t O, int64_t I, int64_t tokens) {
  if (!L || O < 0 || I < 0 || tokens < 0) return ZERO_EINVAL;
  if (!tensor_ok(L, tensor)) return ZERO_ERANGE;
  if (O > ZERO_MAX_COLS || I > ZERO_MAX_COLS || tokens > ZERO_MAX_ROWS) return ZERO_ERANGE;
  if (O * I != L->numel[(size_t)tensor]) return ZERO_EINVAL;
  return ZERO_OK;
}

}  // namespace

extern "C" {

int64_t zero_linear_grad_workspace(const zero_layout* L, int32_t tensor, int32_t transposed,
                                   int64_t out_features, int64_t in_features, int64_t tokens) {
  const int rc = shape_ok(L, tensor, out_features, in_features, tokens);
  if (rc != ZERO_OK) return rc;
  if (transposed != 0 && transposed != 1) return ZERO_EINVAL;
  return make_plan(L, tensor, transposed ? in_features : out_features,
                   transposed ? out_features : in_features, tokens)
      .bytes;
}

int zero_linear_grad(const zero_layout* L, int32_t tensor, int32_t transposed, const uint16_t* dy,
                     int64_t dy_stride, const uint8_t* codes, const uint8_t* scales,
                     int64_t tokens, int64_t out_features, int64_t in_features, float scale,
                     uint32_t flags, float* acc_flat, uint16_t* bf16_flat, void* workspace,
                     int64_t workspace_bytes, hipStream_t stream) {
  int rc = shape_ok(L, tensor, out_features, in_features, tokens);
  if (rc != ZERO_OK) return rc;
  if (transposed != 0 && transposed != 1) return ZERO_EINVAL;
  const int64_t O = out_features, I = in_features, numel = O * I;
  rc = grad_out_ok(flags, scale, acc_flat, bf16_flat, numel);
  if (rc != ZERO_OK) return rc;
  if (numel == 0 || (tokens == 0 && !(flags & (ZERO_ACC_OVERWRITE | ZERO_ACC_EMIT_BF16))))
    return ZERO_OK;
  if (tokens > 0 && (!dy || !codes || !scales || dy_stride < O)) return ZERO_EINVAL;
  if (dy_stride > ZERO_MAX_STRIDE) return ZERO_ERANGE;
  const int64_t rows = transposed ? I : O, cols = transposed ? O : I;
  const Plan p = make_plan(L, tensor, rows, cols, tokens);
  if (p.bytes > 0 && (!workspace || workspace_bytes < p.bytes || ((uintptr_t)workspace & 15u)))
    return ZERO_EINVAL;
  if (p.row_tiles * p.col_tiles > ((int64_t)1 << 23)) return ZERO_ERANGE;
  Args A;
  int64_t lo, hi;
  A.out.place = make_place(L, tensor, &lo, &hi);
  const int64_t nb = (I + kAct8Block - 1) / kAct8Block;
  const Bytes outs[] = {Bytes{acc_used(flags) ? acc_flat + lo : nullptr, 4 * (hi - lo)},
                        Bytes{(flags & ZERO_ACC_EMIT_BF16) ? bf16_flat + lo : nullptr, 2 * (hi - lo)},
                        Bytes{workspace, p.bytes}};
  const Bytes ins[] = {rows_of(dy, tokens, O, dy_stride, 2), Bytes{codes, tokens * I},
                       Bytes{scales, tokens * nb}};
  if (any_overlap(outs, ins)) return ZERO_EOVERLAP;
  if (hip_error_pending()) return ZERO_EHIP;
  A.dy = dy;
  A.dy_stride = dy_stride;
  A.codes = codes;
  A.scales = scales;
  A.tokens = tokens;
  A.tokens_per_split = p.tokens_per_split;
  A.O = (int32_t)O;
  A.I = (int32_t)I;
  A.nb = (int32_t)nb;
  A.rows = (int32_t)rows;
  A.cols = (int32_t)cols;
  A.row_tiles = (int32_t)p.row_tiles;
  A.col_tiles = (int32_t)p.col_tiles;
  A.splits = (int32_t)p.splits;
  A.partial = p.bytes > 0 ? (float*)workspace : nullptr;
  A.out.acc = acc_flat;
  A.out.out = bf16_flat;
  A.out.scale = scale;
  A.out.flags = flags;
  const dim3 grid((unsigned)(p.row_tiles * p.col_tiles), (unsigned)p.splits);
  if (transposed)
    hipLaunchKernelGGL((grad_kernel<2, true>), grid, dim3(kThreads), 0, stream, A);
  else
    hipLaunchKernelGGL((grad_kernel<2, false>), grid, dim3(kThreads), 0, stream, A);
  rc = launched();
  if (rc != ZERO_OK || !A.partial) return rc;
  const unsigned sgrid = (unsigned)std::min<int64_t>((numel / 4 + kThreads) / kThreads, 1 << 14);
  if (A.out.place.gap)
    hipLaunchKernelGGL(sum_kernel<true>, dim3(sgrid), dim3(kThreads), 0, stream, A.partial,
                       A.splits, numel, A.out);
  else
    hipLaunchKernelGGL(sum_kernel<false>, dim3(sgrid), dim3(kThreads), 0, stream, A.partial,
                       A.splits, numel, A.out);
  return launched();
}

}  // extern "C"
