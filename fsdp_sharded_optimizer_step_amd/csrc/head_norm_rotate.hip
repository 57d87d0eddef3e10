// zero_head_norm_rotate and zero_head_norm_rotate_grad.
//
// Page "Infra: Data Parallel" (pufanyi.com), section "Zero Redundancy
// Optimizer (ZeRO)": the norms' weights are read from the flat buffer of
// gathered parameters; section "Naive Data Parallelism": their gradients are
// added to the rank's sum over micro-batches.
//
//   forward   n = x / sqrt(mean(x^2) + eps), u = n*w over a head's d columns;
//             a pair (a, b) of its first columns becomes
//             (a cos - b sin, a sin + b cos), angle = position[axis] * frequency
//   backward  u' = dy turned back, g = u'*w:  dx = R*(g - n*mean(g*n)),
//             dw = sum over tokens and heads of u'*n          (R = 1/sqrt(...))
//
// HBM streams, 4 bytes an element forward and 6 backward.  A head's row lies
// in NL neighbouring lanes, 8 pairs (16 columns) each, so the two columns of a
// pair meet in one lane, and a lane's cosines and sines stay in its registers
// for all the heads of a token that the lane works on.  The sums over a row go
// through data-parallel moves between the lanes.
#include <algorithm>
#include <cfloat>

#include "act8.hpp"
#include "activation.hpp"
#include "matrix.hpp"

namespace {
using namespace zs;

constexpr int kThreads = 256;
constexpr int kMaxAxes = ZERO_MAX_AXES;

// How a lane's 8 pairs lie in a row: two vectors of 8 columns, the pairs'
// first and second ones (kHalves: rotation of d/2 apart columns), two vectors
// of 4 whole pairs each (kNeighbours), or column by column (kSingle: every
// layout that whole vectors do not fit).
enum : int { kHalves = 0, kNeighbours = 1, kSingle = 2 };

struct View {
  char* p;
  int64_t token, head;  // strides in elements
};
struct Heads {
  View x, dy, out;
  Place place;
  int32_t heads, normed;
  int32_t log_across;  // a wave's rows at a time: 2^log_across heads of a token, the rest tokens
  int32_t per_chunk;   // heads of a block
};
struct Args {
  Heads side[2];
  const uint16_t* params;
  const void* positions;
  const double* freqs;
  int64_t tokens;
  float* partial;
  int32_t wide;               // positions of 8 bytes
  int32_t d, half;            // columns of a head, pairs that turn
  int32_t upto[kMaxAxes];     // pairs below upto[a] (and not below upto[a - 1]) turn by axis a
  int32_t neighbours;         // pairs are neighbouring columns
  int32_t chunks;             // of the first side
  float eps;
};

// Sum over NL neighbouring lanes, in every one of them.
template <int CTRL>
__device__ __forceinline__ float moved(float x) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(x), CTRL, 0xf, 0xf, true));
}
template <int NL>
__device__ __forceinline__ float lanes_sum(float x) {
  if constexpr (NL > 1) x += moved<0xB1>(x);   // lanes 1 0 3 2 of four
  if constexpr (NL > 2) x += moved<0x4E>(x);   // lanes 2 3 0 1
  if constexpr (NL > 4) x += moved<0x141>(x);  // eight lanes mirrored
  if constexpr (NL > 8) x += moved<0x140>(x);  // sixteen lanes mirrored
  if constexpr (NL > 16) {
    const uint32_t b = __float_as_uint(x);
    const auto w = __builtin_amdgcn_permlane16_swap(b, b, false, false);
    x = __uint_as_float(w[0]) + __uint_as_float(w[1]);
  }
  return x;
}

// One rounding, and one instruction where a product and a sum are two: the columns'
// parts of each other, chosen for every pair, and the division of what is summed
// cost as many.
__device__ __forceinline__ float plus_product(float s, float a, float b) { return __builtin_fmaf(a, b, s); }

// A lane's place in a row.
struct Cols {
  int32_t a, b;    // first columns of its two vectors, or its first pair
  int32_t na, nb;  // whether the vectors lie in the row
};
template <int NL, int MODE>
__device__ __forceinline__ Cols cols_of(const Args& A, int lane) {
  Cols c{};
  if constexpr (MODE == kHalves) {
    const int turning = A.half >> 3;  // lanes whose pairs turn
    c.a = lane < turning ? 8 * lane : 2 * A.half + 16 * (lane - turning);
    c.b = lane < turning ? A.half + 8 * lane : c.a + 8;
  } else if constexpr (MODE == kNeighbours) {
    c.a = 16 * lane;
    c.b = c.a + 8;
  }
  c.na = c.a < A.d;
  c.nb = c.b < A.d;
  return c;
}
// Pair m of a lane; those from A.half on do not turn.
template <int NL, int MODE>
__device__ __forceinline__ int pair_of(const Args& A, int lane, int m) {
  if constexpr (MODE == kHalves)
    return lane < (A.half >> 3) ? 8 * lane + m : A.half;
  else if constexpr (MODE == kNeighbours)
    return 8 * lane + m;
  else
    return lane + NL * m;
}
// Columns of pair j where columns go one by one; d and more: none.
__device__ __forceinline__ void pair_cols(const Args& A, int j, int& x, int& y) {
  if (j >= A.half || A.neighbours) {
    x = 2 * j;
    y = 2 * j + 1;
  } else {
    x = j;
    y = A.half + j;
  }
}

// A row's values as loaded; x and y are the two columns of a lane's 8 pairs.
struct Row {
  u32x4 a, b;
};
template <int MODE, int NL>
__device__ __forceinline__ Row load_row(const Args& A, const uint16_t* p, const Cols& c, int lane, bool live) {
  Row r{{0u, 0u, 0u, 0u}, {0u, 0u, 0u, 0u}};
  if constexpr (MODE == kSingle) {
#pragma unroll
    for (int m = 0; m < 8; ++m) {
      int x, y;
      pair_cols(A, pair_of<NL, MODE>(A, lane, m), x, y);
      if (live && x < A.d) r.a[m >> 1] |= (uint32_t)p[x] << (16 * (m & 1));
      if (live && y < A.d) r.b[m >> 1] |= (uint32_t)p[y] << (16 * (m & 1));
    }
  } else {
    if (live && c.na) r.a = __builtin_nontemporal_load((const u32x4_a2*)(p + c.a));
    if (live && c.nb) r.b = __builtin_nontemporal_load((const u32x4_a2*)(p + c.b));
  }
  return r;
}
__device__ __forceinline__ float half_of(uint32_t w, int k) { return k & 1 ? bf16_hi(w) : bf16_lo(w); }
__device__ __forceinline__ float weight(const u32x4& w, int m) { return half_of(w[m >> 1], m); }
template <int MODE>
__device__ __forceinline__ void widen(const Row& r, float (&x)[8], float (&y)[8]) {
#pragma unroll
  for (int m = 0; m < 8; ++m) {
    if constexpr (MODE == kNeighbours) {
      const uint32_t w = m < 4 ? r.a[m & 3] : r.b[m & 3];
      x[m] = bf16_lo(w);
      y[m] = bf16_hi(w);
    } else {
      x[m] = half_of(r.a[m >> 1], m);
      y[m] = half_of(r.b[m >> 1], m);
    }
  }
}
template <int MODE, int NL>
__device__ __forceinline__ void store_row(const Args& A, uint16_t* p, const Cols& c, int lane, bool live,
                                          const float (&x)[8], const float (&y)[8]) {
  if constexpr (MODE == kSingle) {
#pragma unroll
    for (int m = 0; m < 8; ++m) {
      int i, j;
      pair_cols(A, pair_of<NL, MODE>(A, lane, m), i, j);
      const uint32_t w = round2(x[m], y[m]);  // the instruction: fewer registers here than bf16_round
      if (live && i < A.d) p[i] = (uint16_t)w;
      if (live && j < A.d) p[j] = (uint16_t)(w >> 16);
    }
  } else {
    u32x4 a, b;
    if constexpr (MODE == kNeighbours) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        a[k] = bf16_pack2(x[k], y[k]);
        b[k] = bf16_pack2(x[4 + k], y[4 + k]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        a[k] = bf16_pack2(x[2 * k], x[2 * k + 1]);
        b[k] = bf16_pack2(y[2 * k], y[2 * k + 1]);
      }
    }
    if (live && c.na) __builtin_nontemporal_store(a, (u32x4_a2*)(p + c.a));
    if (live && c.nb) __builtin_nontemporal_store(b, (u32x4_a2*)(p + c.b));
  }
}

// Cosine and sine of pair m of lane `lane` of a row for token t.  The angle is
// counted in turns in 64 bits, where whole turns fall away without loss:
// position 10^6 at frequency 1 is off by 10^-10 of a turn.
template <int NL, int MODE>
__device__ __forceinline__ f32x2 turn(const Args& A, int64_t t, int lane, int m) {
  const int j = pair_of<NL, MODE>(A, lane, m);
  if (j >= A.half) return f32x2{1.f, 0.f};
  int axis = 0;
#pragma unroll
  for (int a = 0; a < kMaxAxes - 1; ++a) axis += j >= A.upto[a] ? 1 : 0;
  const int64_t at = axis * A.tokens + t;
  const double pos = A.wide ? (double)((const int64_t*)A.positions)[at] : (double)((const int32_t*)A.positions)[at];
  const double x = pos * (A.freqs[j] * 0.15915494309189533577);
  float si, co;
  sincospif(2.f * (float)(x - __builtin_rint(x)), &si, &co);
  return f32x2{co, si};
}

// What a column of pair m gives to the other one: nothing where the pair does
// not turn, since an infinity or a NaN times a sine of zero would be a NaN.
template <int NL, int MODE>
__device__ __forceinline__ float crossing(const Args& A, int lane, int m, float x) {
  return pair_of<NL, MODE>(A, lane, m) < A.half ? x : 0.f;
}

// A side's weights in LDS in the lanes' order: x's of a lane, then y's.
template <int NL, int MODE>
__device__ __forceinline__ void weights_to_lds(const Args& A, const Heads& s, uint16_t* w) {
  for (int k = threadIdx.x; k < NL * 16; k += kThreads) {
    const int lane = k >> 4, m = k & 7;
    int x, y;
    if constexpr (MODE == kSingle) {
      pair_cols(A, pair_of<NL, MODE>(A, lane, m), x, y);
    } else if constexpr (MODE == kHalves) {
      const Cols c = cols_of<NL, MODE>(A, lane);
      x = c.a + m;
      y = c.b + m;
    } else {
      x = 16 * lane + 2 * m;
      y = x + 1;
    }
    const int col = (k & 8) ? y : x;
    w[k] = col < A.d ? A.params[place_at<true>(s.place, col)] : (uint16_t)0;
  }
}

// Bound by HBM where there are many rows.  Measured (us; 16384 tokens, heads of
// 128): 64 + 8 heads forward 111, 5.4 TB/s (without the non-temporal hints 125);
// 32 + 8 heads backward 107 with the sum's launch (4 us), 4.9 TB/s (four rows in
// flight instead of two 142; four waves a SIMD, at which all of them spill
// 22 registers and more, 226).  Rows at an odd place, the same vectors: 177 for
// 125, backward 132 for 111 (calls alone in a graph).  Element by element
// (kSingle), 32 + 8 heads of 96 with 24 columns turning: 104, 2.4 TB/s, backward
// 289, 1.3 TB/s; these kernels are bound by their instructions and spill up to 8
// registers.  One token takes 4.5 us: the angles' chain of binary64 and the rows'
// trip to memory.
template <int NL, int MODE, bool GRAD>
__global__ void __launch_bounds__(kThreads, GRAD ? 3 : 4) rotate_kernel(const Args A) {
  constexpr int kAhead = GRAD ? 2 : 4;  // rows whose loads a lane has in flight
  constexpr int kGroups = 64 / NL, kWaves = kThreads / 64;
  constexpr int kLane = 17;  // a lane's 16 sums, apart by one against bank conflicts
  // the weights at first, then each wave's cosines and sines, at last the sums
  constexpr int kTable = kGroups * NL * 8;  // of 512 pairs at most
  __shared__ alignas(16) char shared[GRAD && kThreads * kLane * 4 > kWaves * kTable * 8 ? kThreads * kLane * 4
                                                                                        : kWaves * kTable * 8];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = threadIdx.x & 63;
  const int lane = l % NL, group = l / NL;
  const int side = (int)blockIdx.y >= A.chunks ? 1 : 0;
  const Heads& s = A.side[side];
  const int chunk = side ? (int)blockIdx.y - A.chunks : (int)blockIdx.y;
  const int across = 1 << s.log_across, down = kGroups >> s.log_across;
  const int head_in = group & (across - 1), token_in = group >> s.log_across;
  const int h0 = chunk * s.per_chunk, h1 = min(s.heads, h0 + s.per_chunk);
  const Cols c = cols_of<NL, MODE>(A, lane);
  const bool normed = s.normed;
  u32x4 wx = {0u, 0u, 0u, 0u}, wy = wx;  // bf16, widened where they are used
  if (normed) {
    weights_to_lds<NL, MODE>(A, s, (uint16_t*)shared);
    __syncthreads();
    wx = ((const u32x4*)shared)[lane * 2];
    wy = ((const u32x4*)shared)[lane * 2 + 1];
    __syncthreads();
  }
  float dwx[8], dwy[8];
  if constexpr (GRAD) {
#pragma unroll
    for (int m = 0; m < 8; ++m) dwx[m] = dwy[m] = 0.f;
  }
  f32x2* const table = (f32x2*)shared + wave * kTable;
  // Means are sums of what is divided by d first: where the mean of the squares
  // is a binary32 number, their sum need not be.
  const float inv_d = 1.f / (float)A.d;
  // all lanes of a wave stay in the loops together: their rows' sums meet
  for (int64_t t0 = ((int64_t)blockIdx.x * kWaves + wave) * down; t0 < A.tokens;
       t0 += (int64_t)gridDim.x * kWaves * down) {
    const int64_t t = t0 + token_in;
    const bool here = t < A.tokens;
    float co[8], si[8];
    if (A.half > 0) {
      // The pairs of the wave's tokens are dealt to its lanes, and collected
      // by those that need them.
      for (int v = l; v < down * NL * 8; v += 64) {
        const int64_t u = t0 + v / (NL * 8);
        table[v] = u < A.tokens ? turn<NL, MODE>(A, u, v / 8 % NL, v % 8) : f32x2{1.f, 0.f};
      }
      lanes_meet_in_lds();
#pragma unroll
      for (int m = 0; m < 8; ++m) {
        const f32x2 q = table[(token_in * NL + lane) * 8 + m];
        co[m] = q.x;
        si[m] = q.y;
      }
      lanes_meet_in_lds();
    } else {
#pragma unroll
      for (int m = 0; m < 8; ++m) co[m] = 1.f, si[m] = 0.f;
    }
    const uint16_t* px = (const uint16_t*)s.x.p + t * s.x.token;
    const uint16_t* py = GRAD ? (const uint16_t*)s.dy.p + t * s.dy.token : nullptr;
    uint16_t* po = (uint16_t*)s.out.p + t * s.out.token;
    for (int hb = h0; hb < h1; hb += kAhead * across) {
      Row rx[kAhead], ry[GRAD ? kAhead : 1];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int h = hb + k * across + head_in;
        const bool live = here && h < h1;
        if (!GRAD || normed) rx[k] = load_row<MODE, NL>(A, px + h * s.x.head, c, lane, live);
        if constexpr (GRAD) ry[k] = load_row<MODE, NL>(A, py + h * s.dy.head, c, lane, live);
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        if (hb + k * across >= h1) break;
        const int h = hb + k * across + head_in;
        float x[8], y[8], ox[8], oy[8];
        // Which pairs turn is found anew for each row: kept from row to row, in two
        // scalar registers a pair, it makes the element-by-element kernels spill
        // (16384 tokens, 32 + 8 heads of 96, 24 columns turning: 112 us against 104).
        int own = lane;
        if constexpr (MODE == kSingle) asm volatile("" : "+v"(own));
        if constexpr (!GRAD) {
          widen<MODE>(rx[k], x, y);
          if (normed) {
            float ss = 0.f;
#pragma unroll
            for (int m = 0; m < 8; ++m) ss = plus_product(plus_product(ss, x[m] * inv_d, x[m]), y[m] * inv_d, y[m]);
            const float r = 1.f / __builtin_sqrtf(lanes_sum<NL>(ss) + A.eps);
#pragma unroll
            for (int m = 0; m < 8; ++m) x[m] = x[m] * r * weight(wx, m), y[m] = y[m] * r * weight(wy, m);
          }
#pragma unroll
          for (int m = 0; m < 8; ++m) {
            ox[m] = plus_product(x[m] * co[m], -crossing<NL, MODE>(A, own, m, y[m]), si[m]);
            oy[m] = plus_product(y[m] * co[m], crossing<NL, MODE>(A, own, m, x[m]), si[m]);
          }
        } else {
          float gx[8], gy[8];
          widen<MODE>(ry[k], gx, gy);
#pragma unroll
          for (int m = 0; m < 8; ++m) {
            ox[m] = plus_product(gx[m] * co[m], crossing<NL, MODE>(A, own, m, gy[m]), si[m]);
            oy[m] = plus_product(gy[m] * co[m], -crossing<NL, MODE>(A, own, m, gx[m]), si[m]);
          }
          if (normed) {
            widen<MODE>(rx[k], x, y);
            float ss = 0.f, sg = 0.f;
#pragma unroll
            for (int m = 0; m < 8; ++m) {
              const float xd = x[m] * inv_d, yd = y[m] * inv_d;
              ss = plus_product(plus_product(ss, xd, x[m]), yd, y[m]);
              sg = plus_product(plus_product(sg, ox[m] * weight(wx, m), xd), oy[m] * weight(wy, m), yd);
            }
            // lanes without a row, whose values are zeros, count for nothing
            const float rms = __builtin_sqrtf(lanes_sum<NL>(ss) + A.eps);
            const float r = here && h < h1 ? 1.f / rms : 0.f;
            const float mean = lanes_sum<NL>(sg) * r;  // of g*n
#pragma unroll
            for (int m = 0; m < 8; ++m) {
              const float nx = x[m] * r, ny = y[m] * r;
              dwx[m] += ox[m] * nx;
              dwy[m] += oy[m] * ny;
              ox[m] = r * (ox[m] * weight(wx, m) - nx * mean);
              oy[m] = r * (oy[m] * weight(wy, m) - ny * mean);
            }
          }
        }
        store_row<MODE, NL>(A, po + h * s.out.head, c, lane, here && h < h1, ox, oy);
      }
    }
  }
  if constexpr (GRAD) {
    if (!normed) return;
    // the groups' sums, in order
    __syncthreads();
    float* sum = (float*)shared;
#pragma unroll
    for (int m = 0; m < 8; ++m) {
      sum[threadIdx.x * kLane + m] = dwx[m];
      sum[threadIdx.x * kLane + 8 + m] = dwy[m];
    }
    __syncthreads();
    float* to = A.partial + ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * (NL * 16);
    for (int k = threadIdx.x; k < NL * 16; k += kThreads) {
      float v = 0.f;
      for (int g = 0; g < kThreads / NL; ++g) v += sum[(g * NL + (k >> 4)) * kLane + (k & 15)];
      to[k] = v;
    }
  }
}

// Sums the blocks' parts of one side (or both, where they share a weight) and
// hands them on: 32 columns a block, 32 threads a column, each taking every
// 32nd part in order, then the 32 sums in order.
constexpr int kSumCols = 32, kSumWays = 32;
struct SumArgs {
  const float* partial;
  int32_t parts;  // of `width` values each
  int32_t width;
  int32_t mode, d, half, neighbours;
  GradOut out;
};
// The column of value k of a part (lane k / 16; its x's, then its y's).
__device__ __forceinline__ int column_of(const SumArgs& S, int k) {
  const int lane = k >> 4, m = k & 7, nl = S.width >> 4;
  const bool second = k & 8;
  if (S.mode == kHalves) {
    const int turning = S.half >> 3;
    const int a = lane < turning ? 8 * lane : 2 * S.half + 16 * (lane - turning);
    const int b = lane < turning ? S.half + 8 * lane : a + 8;
    return (second ? b : a) + m;
  }
  if (S.mode == kNeighbours) return 16 * lane + 2 * m + (second ? 1 : 0);
  const int j = lane + nl * m;
  if (j >= S.half || S.neighbours) return 2 * j + (second ? 1 : 0);
  return second ? S.half + j : j;
}
struct BothSums {
  SumArgs side[2];
};
__global__ void __launch_bounds__(kSumCols* kSumWays) rotate_sum_kernel(const BothSums both) {
  const SumArgs& S = both.side[blockIdx.y];
  __shared__ float part[kSumWays][kSumCols + 1];
  const int c = threadIdx.x % kSumCols, way = threadIdx.x / kSumCols;
  const int k = (int)blockIdx.x * kSumCols + c;
  float s = 0.f;
  if (k < S.width) {
#pragma unroll 8
    for (int32_t g = way; g < S.parts; g += kSumWays) s += S.partial[(int64_t)g * S.width + k];
  }
  part[way][c] = s;
  __syncthreads();
  if (way == 0 && k < S.width) {
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < kSumWays; ++w) t += part[w][c];
    const int col = column_of(S, k);
    if (col < S.d) grad_store(S.out, place_at<true>(S.out.place, col), t);
  }
}

// ------------------------------------------------------------------ host
int lanes_for(int32_t d) {
  int n = 1;
  while (n * 16 < d) n *= 2;
  return n;
}

// The launch.  A wave works on neighbouring heads of a token, so that what it
// reads and writes at a time lies together, and on several tokens where there
// are fewer heads than its groups of lanes.  All heads of a token go to one
// block, or, where that leaves fewer than kBlocks, parts of them to several.
// Backward, at most kMaxAlong blocks share the tokens.  A function of the shape
// alone, and so is the order of the weights' sums.
constexpr int64_t kBlocks = 1024, kMaxAlong = 512;
struct Plan {
  int nl;
  int32_t log_across[2], per_chunk[2], chunks[2];
  int64_t along, bytes;
};
Plan make_plan(int64_t tokens, int32_t d, const int32_t (&heads)[2], bool grad) {
  Plan p;
  p.nl = lanes_for(d);
  const int groups = 64 / p.nl;
  int64_t need[2] = {1, 1};
  p.along = 1;
  for (int n = 0; n < 2; ++n) {
    p.log_across[n] = 0;
    while ((1 << p.log_across[n]) < std::min<int64_t>(heads[n], groups)) ++p.log_across[n];
    const int64_t at_once = (int64_t)(kThreads / 64) * (groups >> p.log_across[n]);
    need[n] = std::max<int64_t>(1, (tokens + at_once - 1) / at_once);
    if (heads[n] > 0) p.along = std::max(p.along, need[n]);
  }
  p.along = std::min(p.along, grad ? kMaxAlong : (int64_t)1 << 22);
  for (int n = 0; n < 2; ++n) {
    const int64_t turns = ((int64_t)heads[n] + (1 << p.log_across[n]) - 1) >> p.log_across[n];
    const int64_t parts = std::min(std::max<int64_t>(1, turns), (kBlocks + p.along - 1) / p.along);
    const int64_t per = (turns + parts - 1) / parts;
    p.per_chunk[n] = (int32_t)std::max<int64_t>(1, per << p.log_across[n]);
    p.chunks[n] = (heads[n] + p.per_chunk[n] - 1) / p.per_chunk[n];
  }
  p.bytes = (int64_t)(p.chunks[0] + p.chunks[1]) * p.along * p.nl * 16 * 4;
  return p;
}

constexpr int64_t kMaxHeadStride = (int64_t)1 << 40;

int64_t extent(const zero_head_view& v, int64_t tokens, int64_t heads, int64_t d) {
  return (tokens - 1) * v.token_stride + (heads - 1) * v.head_stride + d;
}
int view_ok(const zero_head_view& v, int64_t tokens, int64_t heads, int64_t d, bool output) {
  if (!v.data_dev) return ZERO_EINVAL;
  if (v.token_stride < 0 || v.head_stride < 0) return ZERO_EINVAL;
  if (v.token_stride > kMaxHeadStride || v.head_stride > kMaxHeadStride) return ZERO_ERANGE;
  if ((double)tokens * (double)v.token_stride + (double)heads * (double)v.head_stride > 0x1p50) return ZERO_ERANGE;
  if (!output) return ZERO_OK;
  // rows of an output do not meet: tokens of heads, or heads of tokens
  const int64_t ts = tokens > 1 ? v.token_stride : kMaxHeadStride * 2, hs = heads > 1 ? v.head_stride : 0;
  const bool by_token = (heads <= 1 || v.head_stride >= d) && (tokens <= 1 || ts >= (heads - 1) * hs + d);
  const bool by_head = (tokens <= 1 || v.token_stride >= d) &&
                       (heads <= 1 || v.head_stride >= (tokens - 1) * (tokens > 1 ? v.token_stride : 0) + d);
  return by_token || by_head ? ZERO_OK : ZERO_EINVAL;
}

// Whether two views of rows meet.  Parts of one buffer whose rows take turns
// do not: equal strides of tokens (or heads), and what a token (a head) of one
// covers lies beside the other's.
bool views_meet(const zero_head_view& a, int64_t heads_a, const zero_head_view& b, int64_t heads_b,
                int64_t tokens, int64_t d) {
  const Bytes x{a.data_dev, 2 * extent(a, tokens, heads_a, d)}, y{b.data_dev, 2 * extent(b, tokens, heads_b, d)};
  if (!bytes_overlap(x, y)) return false;
  const int64_t diff = (int64_t)((uintptr_t)b.data_dev - (uintptr_t)a.data_dev);
  const auto beside = [&](int64_t stride_a, int64_t stride_b, int64_t covers_a, int64_t covers_b) {
    if (stride_a != stride_b || stride_a <= 0) return false;
    const int64_t s = 2 * stride_a, off = ((diff % s) + s) % s;
    return off >= 2 * covers_a && off + 2 * covers_b <= s;
  };
  return !(beside(a.token_stride, b.token_stride, (heads_a - 1) * a.head_stride + d,
                  (heads_b - 1) * b.head_stride + d) ||
           beside(a.head_stride, b.head_stride, (tokens - 1) * a.token_stride + d,
                  (tokens - 1) * b.token_stride + d));
}

// Everything but the memory of the two sides.
int shape_ok(const zero_layout* L, int64_t tokens, int32_t d, const zero_heads* const (&side)[2]) {
  if (!L || tokens < 0 || d < 1) return ZERO_EINVAL;
  for (const zero_heads* s : side) {
    if (!s) continue;
    if (s->heads < 0 || s->tensor < -1) return ZERO_EINVAL;
    if (s->tensor >= 0 && !tensor_ok(L, s->tensor)) return ZERO_ERANGE;
    if (s->heads > ZERO_MAX_HEADS) return ZERO_ERANGE;
    if (s->tensor >= 0 && L->numel[(size_t)s->tensor] != d) return ZERO_EINVAL;
  }
  if (d > ZERO_MAX_HEAD_DIM || tokens > ZERO_MAX_ROWS) return ZERO_ERANGE;
  return ZERO_OK;
}
int rotation_ok(const zero_rotation* r, int64_t tokens, int32_t d, int32_t* pairs) {
  *pairs = 0;
  if (!r) return ZERO_OK;
  if (r->n_axes < 0 || r->n_axes > kMaxAxes || (r->interleaved != 0 && r->interleaved != 1)) return ZERO_EINVAL;
  if (r->position_bytes != 4 && r->position_bytes != 8) return ZERO_EINVAL;
  int64_t n = 0;
  for (int a = 0; a < r->n_axes; ++a) {
    if (r->sections[a] < 0) return ZERO_EINVAL;
    n += r->sections[a];
  }
  if (2 * n > d) return ZERO_EINVAL;
  if (n > 0 && tokens > 0 && (!r->positions_dev || !r->freqs_dev)) return ZERO_EINVAL;
  *pairs = (int32_t)n;
  return ZERO_OK;
}

int mode_for(int32_t d, int32_t pairs, bool neighbours) {
  if (d % 8) return kSingle;
  if (pairs == 0) return kNeighbours;
  if (neighbours) return kNeighbours;
  return pairs % 8 ? kSingle : kHalves;
}

template <int NL, bool GRAD>
int launch(const Args& A, int mode, dim3 grid, hipStream_t s) {
  if (mode == kHalves)
    hipLaunchKernelGGL((rotate_kernel<NL, kHalves, GRAD>), grid, dim3(kThreads), 0, s, A);
  else if (mode == kNeighbours)
    hipLaunchKernelGGL((rotate_kernel<NL, kNeighbours, GRAD>), grid, dim3(kThreads), 0, s, A);
  else
    hipLaunchKernelGGL((rotate_kernel<NL, kSingle, GRAD>), grid, dim3(kThreads), 0, s, A);
  return launched();
}
template <bool GRAD>
int launch(const Args& A, int nl, int mode, dim3 grid, hipStream_t s) {
  switch (nl) {
    case 1: return launch<1, GRAD>(A, mode, grid, s);
    case 2: return launch<2, GRAD>(A, mode, grid, s);
    case 4: return launch<4, GRAD>(A, mode, grid, s);
    case 8: return launch<8, GRAD>(A, mode, grid, s);
    case 16: return launch<16, GRAD>(A, mode, grid, s);
    default: return launch<32, GRAD>(A, mode, grid, s);
  }
}

struct GradCall {
  float scale;
  uint32_t flags;
  float* acc;
  uint16_t* out;
  void* workspace;
  int64_t workspace_bytes;
};

// The checks and the launch of both directions; g: backward.
int run(const zero_layout* L, const uint16_t* params, int64_t tokens, int32_t d, double eps,
        const zero_rotation* rot, const zero_heads* q, const zero_heads* k, const GradCall* g, hipStream_t stream) {
  const zero_heads* const side[2] = {q, k};
  int rc = shape_ok(L, tokens, d, side);
  if (rc != ZERO_OK) return rc;
  if (!(eps >= 0.0) || eps > (double)FLT_MAX) return ZERO_EINVAL;
  int32_t pairs;
  rc = rotation_ok(rot, tokens, d, &pairs);
  if (rc != ZERO_OK) return rc;
  const int32_t heads[2] = {q ? q->heads : 0, k ? k->heads : 0};
  bool normed[2];  // a side whose weight counts, with or without tokens
  for (int n = 0; n < 2; ++n) normed[n] = side[n] && side[n]->tensor >= 0 && (g || (heads[n] > 0 && tokens > 0));
  if (g) {
    rc = grad_out_ok(g->flags, g->scale, g->acc, g->out, normed[0] || normed[1] ? d : 0);
    if (rc != ZERO_OK) return rc;
  }
  const bool work = tokens > 0 && heads[0] + heads[1] > 0;
  const bool clears = g && (normed[0] || normed[1]) && (g->flags & (ZERO_ACC_OVERWRITE | ZERO_ACC_EMIT_BF16));
  if (!work && !clears) return ZERO_OK;
  const Plan p = make_plan(tokens, d, heads, g != nullptr);
  const bool sums = g && work && (normed[0] || normed[1]);
  Args A{};
  int64_t lo[2] = {0, 0}, hi[2] = {0, 0};
  for (int n = 0; n < 2; ++n)
    if (normed[n]) A.side[n].place = make_place(L, side[n]->tensor, &lo[n], &hi[n]);
  if (work) {
    for (int n = 0; n < 2; ++n) {
      if (heads[n] == 0) continue;
      const bool needs_x = !g || normed[n];
      if (needs_x && (rc = view_ok(side[n]->x, tokens, heads[n], d, false)) != ZERO_OK) return rc;
      if (g && (rc = view_ok(side[n]->dy, tokens, heads[n], d, false)) != ZERO_OK) return rc;
      if ((rc = view_ok(side[n]->out, tokens, heads[n], d, true)) != ZERO_OK) return rc;
      if (normed[n] && !params) return ZERO_EINVAL;
    }
    if (sums && (!g->workspace || g->workspace_bytes < p.bytes || ((uintptr_t)g->workspace & 15u)))
      return ZERO_EINVAL;
  }
  // memory: outputs against inputs and each other
  const auto range = [&](const zero_head_view& v, int n) { return Bytes{v.data_dev, 2 * extent(v, tokens, heads[n], d)}; };
  Bytes ins[8];
  int n_ins = 0;
  if (work) {
    for (int n = 0; n < 2; ++n) {
      if (heads[n] == 0) continue;
      if (!g || normed[n]) ins[n_ins++] = range(side[n]->x, n);
      if (g) ins[n_ins++] = range(side[n]->dy, n);
      if (normed[n]) ins[n_ins++] = Bytes{params + lo[n], 2 * (hi[n] - lo[n])};
    }
    if (pairs > 0) {
      ins[n_ins++] = Bytes{rot->positions_dev, (int64_t)rot->position_bytes * tokens * rot->n_axes};
      ins[n_ins++] = Bytes{rot->freqs_dev, 8 * (int64_t)pairs};
    }
  }
  Bytes flat[5];
  int n_flat = 0;
  if (g) {
    const bool shared = normed[0] && normed[1] && side[0]->tensor == side[1]->tensor;
    for (int n = 0; n < (shared ? 1 : 2); ++n) {
      if (!normed[n]) continue;
      if (acc_used(g->flags)) flat[n_flat++] = Bytes{g->acc + lo[n], 4 * (hi[n] - lo[n])};
      if (g->flags & ZERO_ACC_EMIT_BF16) flat[n_flat++] = Bytes{g->out + lo[n], 2 * (hi[n] - lo[n])};
    }
    if (sums) flat[n_flat++] = Bytes{g->workspace, p.bytes};
  }
  for (int a = 0; a < n_flat; ++a) {
    for (int b = a + 1; b < n_flat; ++b)
      if (bytes_overlap(flat[a], flat[b])) return ZERO_EOVERLAP;
    for (int b = 0; b < n_ins; ++b)
      if (bytes_overlap(flat[a], ins[b])) return ZERO_EOVERLAP;
  }
  if (work) {
    for (int n = 0; n < 2; ++n) {
      if (heads[n] == 0) continue;
      const Bytes out = range(side[n]->out, n);
      for (int b = 0; b < n_flat; ++b)
        if (bytes_overlap(out, flat[b])) return ZERO_EOVERLAP;
      for (int b = 0; b < n_ins; ++b)
        if (bytes_overlap(out, ins[b])) return ZERO_EOVERLAP;
    }
    if (heads[0] > 0 && heads[1] > 0 && views_meet(q->out, heads[0], k->out, heads[1], tokens, d))
      return ZERO_EOVERLAP;
  }
  if (hip_error_pending()) return ZERO_EHIP;

  const bool neighbours = rot && rot->interleaved;
  const int mode = mode_for(d, pairs, neighbours);
  if (work) {
    for (int n = 0; n < 2; ++n) {
      Heads& s = A.side[n];
      s.heads = heads[n];
      s.normed = normed[n] ? 1 : 0;
      s.log_across = p.log_across[n];
      s.per_chunk = p.per_chunk[n];
      if (heads[n] == 0) continue;
      s.x = View{(char*)side[n]->x.data_dev, side[n]->x.token_stride, side[n]->x.head_stride};
      s.dy = View{(char*)side[n]->dy.data_dev, side[n]->dy.token_stride, side[n]->dy.head_stride};
      s.out = View{(char*)side[n]->out.data_dev, side[n]->out.token_stride, side[n]->out.head_stride};
    }
    A.params = params;
    A.tokens = tokens;
    A.d = d;
    A.half = pairs;
    A.neighbours = neighbours;
    if (pairs > 0) {
      A.positions = rot->positions_dev;
      A.freqs = rot->freqs_dev;
      A.wide = rot->position_bytes == 8;
      int32_t n = 0;
      for (int a = 0; a < kMaxAxes; ++a) {
        if (a < rot->n_axes) n += rot->sections[a];
        A.upto[a] = n;
      }
    }
    A.chunks = p.chunks[0];
    // one too small for binary32 still keeps rows of zeros from 0 / 0
    A.eps = eps > 0.0 ? std::max((float)eps, FLT_TRUE_MIN) : 0.f;
    A.partial = sums ? (float*)g->workspace : nullptr;
    const dim3 grid((unsigned)p.along, (unsigned)(p.chunks[0] + p.chunks[1]));
    rc = g ? launch<true>(A, p.nl, mode, grid, stream) : launch<false>(A, p.nl, mode, grid, stream);
    if (rc != ZERO_OK) return rc;
  }
  if (!g) return ZERO_OK;
  const int width = p.nl * 16;
  const bool shared = normed[0] && normed[1] && side[0]->tensor == side[1]->tensor;
  const int64_t parts[2] = {work ? p.chunks[0] * p.along : 0, work ? p.chunks[1] * p.along : 0};
  BothSums both;
  unsigned sides = 0;
  for (int n = 0; n < 2; ++n) {
    if (!normed[n] || (shared && n == 1)) continue;
    SumArgs& S = both.side[sides];
    S.parts = (int32_t)(shared ? parts[0] + parts[1] : parts[n]);
    if (S.parts == 0 && !(g->flags & (ZERO_ACC_OVERWRITE | ZERO_ACC_EMIT_BF16))) continue;
    S.partial = (const float*)g->workspace + (n == 1 ? parts[0] * width : 0);
    S.width = width;
    S.mode = mode;
    S.d = d;
    S.half = pairs;
    S.neighbours = neighbours;
    S.out = GradOut{g->acc, g->out, A.side[n].place, g->scale, g->flags};
    ++sides;
  }
  if (sides == 0) return ZERO_OK;
  hipLaunchKernelGGL(rotate_sum_kernel, dim3((unsigned)((width + kSumCols - 1) / kSumCols), sides),
                     dim3(kSumCols * kSumWays), 0, stream, both);
  return launched();
}

}  // namespace

extern "C" {

int zero_head_norm_rotate(const zero_layout* L, const uint16_t* params_flat, int64_t tokens, int32_t head_dim,
                          double eps, const zero_rotation* rotation, const zero_heads* q, const zero_heads* k,
                          hipStream_t stream) {
  return run(L, params_flat, tokens, head_dim, eps, rotation, q, k, nullptr, stream);
}

int64_t zero_head_norm_rotate_grad_workspace(const zero_layout* L, int64_t tokens, int32_t head_dim,
                                             const zero_heads* q, const zero_heads* k) {
  const zero_heads* const side[2] = {q, k};
  const int rc = shape_ok(L, tokens, head_dim, side);
  if (rc != ZERO_OK) return rc;
  const int32_t heads[2] = {q ? q->heads : 0, k ? k->heads : 0};
  const bool normed = (q && q->tensor >= 0) || (k && k->tensor >= 0);
  if (!normed || tokens == 0 || heads[0] + heads[1] == 0) return 0;
  return make_plan(tokens, head_dim, heads, true).bytes;
}

int zero_head_norm_rotate_grad(const zero_layout* L, const uint16_t* params_flat, int64_t tokens,
                               int32_t head_dim, double eps, const zero_rotation* rotation, const zero_heads* q,
                               const zero_heads* k, float scale, uint32_t flags, float* acc_flat,
                               uint16_t* bf16_flat, void* workspace, int64_t workspace_bytes,
                               hipStream_t stream) {
  const GradCall g{scale, flags, acc_flat, bf16_flat, workspace, workspace_bytes};
  return run(L, params_flat, tokens, head_dim, eps, rotation, q, k, &g, stream);
}

}  // extern "C"
