// zero_linear and zero_linear_input_grad: products with a weight that lies in
// the flat buffer of gathered parameters.
//
// Page "Infra: Data Parallel" (pufanyi.com), section "Zero Redundancy
// Optimizer (ZeRO)": parameters are gathered before forward and backward; the
// products read them where the gather put them.
//
//   forward     pre = x W^T + b;  out = act(pre) + res
//   input grad  dx = (dy W + add) * act'(pre)
//
// Both are C[m, n] = sum over k of A[m, k] * B(k, n), m a token, A (x or dy)
// with k adjacent.  B has k adjacent where the weight is kept as (out, in)
// and x is multiplied, or (in, out) and dy; n adjacent in the other two.
//
// A block's tiles of A and B go from memory straight to LDS, 16 bytes a lane,
// 64 k a step: the next step but one is requested as places become free.  A
// request puts a wave's 1024 bytes next to each other in LDS, 8 rows of 128
// bytes; which 16 bytes of its row a lane fetches is permuted, so that the rows
// that a fragment read meets at a time use all banks.  A fragment of k adjacent
// is one 16-byte read a lane, one of n adjacent two transposing reads of 8
// bytes.  Products of bf16 are exact in binary32, sums are binary32.
//
// Requests of 16 bytes need addresses of 16 bytes and rows of whole chunks.
// An operand that has not (an odd width, a tensor at an odd place of the flat
// buffer, padding inside it) is first copied to the workspace.
#include <algorithm>

#include "linear.hpp"
#include "linear_plan.hpp"
#include "matrix.hpp"

namespace {
using namespace zs;

// For closures: called out of line, what they capture would go through memory.
#define ZERO_INLINE __attribute__((always_inline))

constexpr int kThreads = 256;
constexpr int kStep = kTileStep;  // k of an LDS buffer: 128 bytes of a row

struct Args {
  const uint16_t *a, *b;
  int64_t a_stride, b_stride;  // elements
  int32_t M, N, K;             // K: whole chunks of 8 where k is adjacent
  int32_t Kb;                  // rows of a B with n adjacent
  int32_t row_tiles, col_tiles;
  int32_t whole;               // tiles of one block each
  int32_t splits, per_split;   // blocks of each further tile, steps of each
  float* partial;
  Epilogue e;
};

// The shape of a block's tile: 64*W rows and columns, four waves two by two.
template <int W_>
struct Shape {
  static constexpr int W = W_, kSide = tile_side(W);
  static constexpr int kOperand = kSide * 128;  // bytes of a step
  static constexpr int kB = 3 * kOperand;       // A has three places in LDS, behind them are B's two
  static constexpr int kLoads = 2 * W;  // requests of a wave for an operand
  // The way out: a strip of 32 rows of a wave's sums, of which 16 lanes write 16
  // bytes to as many rows and meet all banks, and what the epilogue reads beside
  // them, 16 bytes a lane and piece of 8 columns.
  static constexpr int kCols = W * 32, kRow = kCols + 4;
  static constexpr int kAcross = kCols / 8, kDown = 64 / kAcross, kVecs = 32 / kDown;
  static constexpr int kStrip = 32 * kRow * 4, kWay = kStrip + 2 * kVecs * 1024;
  static constexpr int kLds = 5 * kOperand;
  static_assert(kLds >= 4 * kWay);
};

// An address that is the same in all lanes, in scalar registers.
__device__ __forceinline__ const char* uniform(const char* p) {
  const uint64_t x = (uint64_t)p;
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)x), hi = __builtin_amdgcn_readfirstlane((uint32_t)(x >> 32));
  return (const char*)((uint64_t)hi << 32 | lo);
}

// 16 bytes a lane from base + off to LDS at `lds` + 16 * lane.  Written out:
// the compiler does not know that the address is read at issue and would wait
// for the data before the next LDS read.  No vector register is written; the wait
// is requests_done().  m0 is a reserved register, of which the compiler warns: what
// it keeps there itself it writes right before its use.  With memory declared it
// keeps requests and LDS accesses in the order written, and the loop got faster
// (8192 x 14336 x 4096: 660 us, 643 with it; 16384 x 4096 x 14336: 1400, 1373).
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void request(const void* base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
               :
               : "s"(lds), "v"(off), "s"(base)
               : "m0", "memory");
}
#pragma clang diagnostic pop
// All but the last N of them.
template <int N = 0>
__device__ __forceinline__ void requests_done() {
  asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}

// One wave's requests for an operand with k adjacent: rows 8 * (wave * kLoads +
// j) to + 7 of the tile; in LDS chunk c of row r lies at c ^ (r / 2 % 8), so
// that the 16 rows of which 16 lanes read one chunk each fill the 64 banks.
template <class S>
struct KRows {
  uint32_t off[S::kLoads];
  // the chunk that a lane fetches in request j (kLoads is even)
  static __device__ __forceinline__ int chunk(int j) {
    return (threadIdx.x & 7) ^ (((threadIdx.x >> 4) & 3) + 4 * (j & 1));
  }
  __device__ __forceinline__ void set(int32_t r0, int32_t rows, int64_t stride) {
    const int wave = threadIdx.x >> 6;
#pragma unroll
    for (int j = 0; j < S::kLoads; ++j) {
      const int r = min((wave * S::kLoads + j) * 8 + (int)((threadIdx.x >> 3) & 7), rows - 1 - r0);
      off[j] = (uint32_t)(r * stride) * 2u + chunk(j) * 16;
    }
  }
  // `left`: k of this step that there are (kStep: all)
  __device__ __forceinline__ uint32_t at(int j, int left) const {
    return left >= kStep || chunk(j) * 8 < left ? off[j] : off[j] - chunk(j) * 16;
  }
  static __device__ __forceinline__ bool missing(int j, int left) { return chunk(j) * 8 >= left; }
  static __device__ __forceinline__ int64_t step_bytes(int64_t) { return kStep * 2; }
  // fragment s of a panel of ROWS (16 or 32): 512 / ROWS k; lane l holds row l %
  // ROWS, k 8 * (l / ROWS) to + 7
  template <int ROWS>
  static __device__ __forceinline__ int frag_offset() {
    return (threadIdx.x & (ROWS - 1)) * 128;
  }
  template <int ROWS>
  static __device__ __forceinline__ bf16x8 frag(const lds_char* p, int panel, int s) {
    const int c = (64 / ROWS * s + (int)((threadIdx.x & 63) / ROWS)) ^ (int)((threadIdx.x >> 1) & 7);
    typedef __attribute__((address_space(3))) bf16x8 lds_t;
    return *(const lds_t*)(p + panel * (128 * ROWS) + c * 16);
  }
};

// The same for an operand with n adjacent, in panels of 64 columns: request j
// of a wave is rows 8 * (i % 8) to + 7 of panel i / 8, i = wave * kLoads + j;
// lane l fetches chunk (l % 8) ^ 2 * (row % 4) of its row.
template <class S>
struct NRows {
  uint32_t off[S::kLoads];
  static __device__ __forceinline__ int chunk() { return ((threadIdx.x & 7) ^ (2 * ((threadIdx.x >> 3) & 3))); }
  static __device__ __forceinline__ int row(int j) {
    return (((int)(threadIdx.x >> 6) * S::kLoads + j) & 7) * 8 + (int)((threadIdx.x >> 3) & 7);
  }
  int64_t stride;
  __device__ __forceinline__ void set(int32_t n0, int32_t cols, int64_t stride_) {
    stride = stride_;
#pragma unroll
    for (int j = 0; j < S::kLoads; ++j) {
      const int panel = ((int)(threadIdx.x >> 6) * S::kLoads + j) >> 3;
      const int c = min(n0 + panel * 64 + chunk() * 8, (cols - 1) & ~7) - n0;
      off[j] = (uint32_t)(row(j) * stride + c) * 2u;
    }
  }
  __device__ __forceinline__ uint32_t at(int j, int left) const {
    return row(j) < left ? off[j] : off[j] - (uint32_t)((row(j) - left + 1) * stride) * 2u;
  }
  static __device__ __forceinline__ bool missing(int j, int left) { return row(j) >= left; }
  static __device__ __forceinline__ int64_t step_bytes(int64_t stride) { return kStep * stride * 2; }
  // 16 lanes read 4 rows of 16 columns and each gets a column's 4 rows
  template <int COLS>
  static __device__ __forceinline__ int frag_offset() {
    return 0;
  }
  template <int COLS>
  static __device__ __forceinline__ bf16x8 frag(const lds_char* p, int panel, int s) {
    static_assert(COLS == 32);
    typedef __attribute__((address_space(3))) s16x4 lds_t;
    const int l = threadIdx.x & 63, g = l >> 4, i = l & 15;
    const int k = i >> 2;  // row % 4 of both reads
    const int c = (panel & 1) * 4 + (g & 1) * 2 + ((i & 3) >> 1);
    const lds_char* q = p + (panel >> 1) * 8192 + (16 * s + 8 * (g >> 1) + k) * 128 + (c ^ (2 * k)) * 16 + (i & 1) * 8;
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_t*)q);
    const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_t*)(q + 512));
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
  }
};

// The matrix instructions: panels of 16 rows and columns and 32 k take less power
// a product, since a sum is read and written half as often, and so run at a
// higher clock (16384 x 4096 x 14336: 1490 us, of 32 rows and 16 k 1555).  With n
// adjacent the compiler moves the sums of the smaller panels about (2190).
template <bool NC>
struct Panels {
  static constexpr int kSide = 16, kQuads = 1;
  typedef f32x4 Sums;
  // lane l, value j: row l % 16 of a, row 4 * (l / 16) + j of b
  static __device__ __forceinline__ Sums multiply(bf16x8 a, bf16x8 b, Sums c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(b, a, c, 0, 0, 0);
  }
  static __device__ __forceinline__ f32x4 quad(const Sums& c, int) { return c; }
};
template <>
struct Panels<true> {
  static constexpr int kSide = 32, kQuads = 4;
  typedef f32x16 Sums;
  // lane l, value j: row l % 32 of a, row 8 * (j / 4) + 4 * (l / 32) + j % 4 of b
  static __device__ __forceinline__ Sums multiply(bf16x8 a, bf16x8 b, Sums c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(b, a, c, 0, 0, 0);
  }
  static __device__ __forceinline__ f32x4 quad(const Sums& c, int q) {
    return f32x4{c[4 * q], c[4 * q + 1], c[4 * q + 2], c[4 * q + 3]};
  }
};

// A block's tile of the result, or its share of a split tile.  The matrix cores
// bound the loop, at the clock that their power allows: beside each product
// stands its share of the next fragments' reads and of the requests two steps
// on, so that no wave waits for either.  Sides of 256 read LDS half as often a
// product as sides of 128 and fill a CU alone, so nothing computes while a block
// begins and ends (13 to 15 us; results and what the epilogue reads cross HBM
// then); sides of 128 stand two to a CU.  Measured (us): 8192 x 14336 x 4096
// (tokens, sum, columns) 643, 1496 TFLOP/s, with n adjacent 717; 16384 x 4096 x
// 14336 1373, with n adjacent 1497; with everything in the epilogue 674 (K of
// 14336), through the activation's gradient and with n adjacent 1648.  On the
// way there (cards differ by 4 %): A's and B's steps in two places each, all requests beside a
// quarter of a step's products 775 (1560 for sums over 4096), beside two quarters
// 724 (1550), smaller panels of k adjacent 690 (1425); tiles in groups of 4 or 16 rows
// instead of 8 within 3 % either way.  Without requests, for timing, 528 of the 690;
// requests that always hit L2 611; without LDS reads 679.
template <class S, bool NC>
__global__ void __launch_bounds__(kThreads, S::W == 4 ? 1 : 2) product_kernel(const Args A) {
  constexpr int W = S::W, kSide = S::kSide;
  using BRows = std::conditional_t<NC, NRows<S>, KRows<S>>;
  using Matrix = Panels<NC>;
  constexpr int kPanel = Matrix::kSide, P = S::kCols / kPanel;  // panels of a wave's side
  constexpr int kStretches = kStep * kPanel / 512;              // of a step, each of an instruction's k
  __shared__ __align__(1024) char shared[S::kLds];
  lds_char* lds = (lds_char*)shared;
  const uint32_t lds_base = (uint32_t)(uintptr_t)lds;

  // whole tiles first, dealt to the XCDs (block b runs on XCD b % 8) in runs
  const int32_t all_steps = (max(A.K, NC ? A.Kb : 0) + kStep - 1) / kStep;
  int32_t tile, split = 0, sa = 0, sz = all_steps;
  if ((int32_t)blockIdx.x < A.whole) {
    tile = (A.whole & 7) ? (int32_t)blockIdx.x
                         : (int32_t)(blockIdx.x & 7) * (A.whole >> 3) + (int32_t)(blockIdx.x >> 3);
  } else {
    // quotients come from the vector unit; what follows from them is one
    // value for the wave
    const int32_t x = (int32_t)blockIdx.x - A.whole, t = __builtin_amdgcn_readfirstlane(x / A.splits);
    split = x - t * A.splits;
    tile = A.whole + t;
    sa = split * A.per_split;
    sz = min(all_steps, sa + A.per_split);
  }
  int32_t r0, c0;
  tile_place(tile, A.row_tiles, A.col_tiles, r0, c0);
  r0 = __builtin_amdgcn_readfirstlane(r0) * kSide;
  c0 = __builtin_amdgcn_readfirstlane(c0) * kSide;

  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wm = wave >> 1, wn = wave & 1;
  const int lane = threadIdx.x & 63;
  typename Matrix::Sums acc[P][P];
#pragma unroll
  for (int m = 0; m < P; ++m)
#pragma unroll
    for (int n = 0; n < P; ++n) acc[m][n] = typename Matrix::Sums{};

  KRows<S> ra;
  BRows rb;
  ra.set(r0, A.M, A.a_stride);
  rb.set(c0, A.N, A.b_stride);
  const char* const pa = uniform((const char*)(A.a + r0 * A.a_stride));
  const char* const pb = uniform((const char*)(A.b + (NC ? (int64_t)c0 : c0 * A.b_stride)));
  const int32_t steps = sz - sa;
  // The step that may not be whole, the last one of k, is a block's first: the
  // others need no checks.  at: the number in k of a block's step i.
  const bool has_end = sz == all_steps;
  const auto at = [&](int32_t i) ZERO_INLINE { return has_end ? (i == 0 ? all_steps - 1 : sa + i - 1) : sa + i; };
  const uint32_t mine = lds_base + wave * S::kLoads * 1024;
  // request j of A or B for the step at a_at or b_at; `to`: its place
  const auto fetch_a = [&](const char* a_at, int to, auto index) ZERO_INLINE {
    constexpr int j = decltype(index)::value;
    request(a_at, ra.off[j], mine + to + j * 1024);
  };
  const auto fetch_b = [&](const char* b_at, int to, auto index) ZERO_INLINE {
    constexpr int j = decltype(index)::value;
    request(b_at, rb.off[j], mine + S::kB + to + j * 1024);
  };
  const auto a_of = [&](int32_t i) ZERO_INLINE { return uniform(pa + (int64_t)at(i) * KRows<S>::step_bytes(A.a_stride)); };
  const auto b_of = [&](int32_t i) ZERO_INLINE { return uniform(pb + (int64_t)at(i) * BRows::step_bytes(A.b_stride)); };
  // The first step, its k from `left` on replaced by zeros, and what step 0 does
  // not request of the second.
  constexpr int kEarly = kStretches > 2 ? S::kLoads / 2 : S::kLoads;  // of B's requests
  const auto fetch_first = [&]() ZERO_INLINE {
    const char *a_at = a_of(0), *b_at = b_of(0);
    const int left_a = A.K - at(0) * kStep, left_b = (NC ? A.Kb : A.K) - at(0) * kStep;
#pragma unroll
    for (int j = 0; j < S::kLoads; ++j) {
      request(a_at, ra.at(j, left_a), mine + j * 1024);
      request(b_at, rb.at(j, left_b), mine + S::kB + j * 1024);
    }
    if (steps > 1) {
      const char *a_1 = a_of(1), *b_1 = b_of(1);
      unrolled<S::kLoads>([&](auto j) ZERO_INLINE { fetch_a(a_1, S::kOperand, j); });
      unrolled<kEarly>([&](auto j) ZERO_INLINE { fetch_b(b_1, S::kOperand, j); });
      requests_done<S::kLoads + kEarly>();
    } else {
      requests_done();
    }
    if (left_a < kStep || left_b < kStep) {
      lds_char* p = lds + wave * S::kLoads * 1024 + lane * 16;
#pragma unroll 1
      for (int j = 0; j < S::kLoads; ++j) {
        if (KRows<S>::missing(j, left_a)) *(lds_u32x4*)(p + j * 1024) = u32x4{0u, 0u, 0u, 0u};
        if (BRows::missing(j, left_b)) *(lds_u32x4*)(p + S::kB + j * 1024) = u32x4{0u, 0u, 0u, 0u};
      }
    }
  };

  const lds_char* const fa = lds + wm * W * 4096 + KRows<S>::template frag_offset<kPanel>();
  const lds_char* const fb = lds + S::kB + wn * W * 4096 + BRows::template frag_offset<kPanel>();
  bf16x8 a[2][P], b[2][P];  // two sets of fragments
  const auto read1 = [&](auto set, int pa, int pb, int s, auto index) ZERO_INLINE {
    constexpr int to = decltype(set)::value, j = decltype(index)::value;
    if constexpr (j < P)
      a[to][j] = KRows<S>::template frag<kPanel>(fa + pa, j, s);
    else
      b[to][j - P] = BRows::template frag<kPanel>(fb + pb, j - P, s);
  };
  // The products of one stretch; after each of them `beside` puts its share of
  // other work.
  constexpr int kM = P * P;
  const auto multiply = [&](auto set, auto beside) ZERO_INLINE {
    constexpr int from = decltype(set)::value;
    unrolled<kM>([&](auto index) ZERO_INLINE {
      constexpr int i = decltype(index)::value;
      acc[i / P][i % P] = Matrix::multiply(a[from][i / P], b[from][i % P], acc[i / P][i % P]);
      beside(index);
      __builtin_amdgcn_sched_barrier(0);
    });
  };
  // f(j) for those of N things, dealt to the products from FROM to TO - 1, that
  // go beside product I
  const auto share = [](auto index, auto from, auto to, auto count, auto f) ZERO_INLINE {
    constexpr int len = decltype(to)::value - decltype(from)::value, n = decltype(count)::value;
    constexpr int i = decltype(index)::value - decltype(from)::value;
    if constexpr (i >= 0 && i < len) {
      constexpr int first = (i * n + len - 1) / len, next = ((i + 1) * n + len - 1) / len;
      unrolled<next - first>([&](auto j) ZERO_INLINE { f(std::integral_constant<int, first + decltype(j)::value>{}); });
    }
  };
  constexpr std::integral_constant<int, 0> k0;
  constexpr std::integral_constant<int, kM> kAll;
  constexpr std::integral_constant<int, kStretches == 2 ? kM / 2 : kM> kRead;  // the products that reads go beside
  constexpr std::integral_constant<int, 2 * P> kReads;
  // Step i, in places p0 of A and q0 of B; p1: A's next place, p2: the free one.
  // kNext: steps that follow (2: or more).  B's place is free once the last
  // stretch is read, which is when the waves meet.  A CU takes 64 bytes a cycle, a
  // request of a wave in 16, and one that has to wait holds its wave's
  // products up: so the requests for step i + 2 are dealt over the whole step, A's
  // before the waves meet, B's after that (and, where a step has four stretches,
  // half of them with the next step's first).
  const auto step = [&](auto next, int32_t i, int p0, int p1, int p2, int q0) ZERO_INLINE {
    constexpr int kNext = decltype(next)::value;
    const int q1 = q0 ^ S::kOperand;
    const char *a_at = pa, *b_at = pb;
    if constexpr (kNext > 1) a_at = a_of(i + 2);
    unrolled<kStretches - 1>([&](auto stretch) ZERO_INLINE {
      constexpr int s = decltype(stretch)::value;
      if constexpr (s == 0 && kNext > 0 && kStretches > 2) b_at = b_of(i + 1);
      multiply(std::integral_constant<int, s % 2>{}, [&](auto index) ZERO_INLINE {
        share(index, k0, kRead, kReads,
              [&](auto j) ZERO_INLINE { read1(std::integral_constant<int, (s + 1) % 2>{}, p0, q0, s + 1, j); });
        if constexpr (kStretches == 2) {
          if constexpr (kNext > 1)
            share(index, k0, kAll, std::integral_constant<int, S::kLoads>{},
                  [&](auto j) ZERO_INLINE { fetch_a(a_at, p2, j); });
        } else if constexpr (s == 0) {
          if constexpr (kNext > 0)
            share(index, k0, kAll, std::integral_constant<int, S::kLoads - kEarly>{}, [&](auto j) ZERO_INLINE {
              fetch_b(b_at, q1, std::integral_constant<int, kEarly + decltype(j)::value>{});
            });
        } else if constexpr (kNext > 1) {
          share(index, k0, kAll, std::integral_constant<int, S::kLoads / 2>{}, [&](auto j) ZERO_INLINE {
            fetch_a(a_at, p2, std::integral_constant<int, (s - 1) * (S::kLoads / 2) + decltype(j)::value>{});
          });
        }
      });
    });
    // all but A's of step i + 2
    if constexpr (kNext > 0) requests_done<(kNext > 1 ? S::kLoads : 0)>();
    __syncthreads();
    constexpr std::integral_constant<int, (kStretches - 1) % 2> kLast;
    if constexpr (kNext > 1) b_at = b_of(i + 2);
    multiply(kLast, [&](auto index) ZERO_INLINE {
      if constexpr (kNext > 0) share(index, k0, kRead, kReads, [&](auto j) ZERO_INLINE { read1(k0, p1, q1, 0, j); });
      if constexpr (kNext > 1)
        share(index, k0, kAll, std::integral_constant<int, kEarly>{}, [&](auto j) ZERO_INLINE { fetch_b(b_at, q0, j); });
    });
  };
  if (steps > 0) {
    fetch_first();
    __syncthreads();
    unrolled<2 * P>([&](auto j) ZERO_INLINE { read1(k0, 0, 0, 0, j); });
    int32_t i = 0;
    int p0 = 0, p1 = S::kOperand, p2 = 2 * S::kOperand, q0 = 0;
    const auto turn = [&]() ZERO_INLINE {
      const int p = p0;
      p0 = p1;
      p1 = p2;
      p2 = p;
      q0 ^= S::kOperand;
      ++i;
    };
#pragma unroll 1
    for (; i + 2 < steps; turn()) step(std::integral_constant<int, 2>{}, i, p0, p1, p2, q0);
    if (i + 1 < steps) {
      step(std::integral_constant<int, 1>{}, i, p0, p1, p2, q0);
      turn();
    }
    step(std::integral_constant<int, 0>{}, i, p0, p1, p2, q0);
  }

  if (tile >= A.whole) {
    // to the workspace as they lie, for sum_kernel
    const int64_t part = (int64_t)(tile - A.whole) * A.splits + split;
    float* const to = A.partial + (part * 4 + wave) * (kSide * kSide / 4) + lane * 4;
#pragma unroll
    for (int m = 0; m < P; ++m)
#pragma unroll
      for (int n = 0; n < P; ++n)
#pragma unroll
        for (int q = 0; q < Matrix::kQuads; ++q)
          *(f32x4*)(to + ((m * P + n) * Matrix::kQuads + q) * 256) = Matrix::quad(acc[m][n], q);
    return;
  }
  // A wave's sums leave 32 rows at a time through LDS of its own, from where a
  // lane gets 8 columns of a row.  What the epilogue reads of the next 32 rows is
  // on its way meanwhile; it waits in LDS too, so that the activations stand in
  // a loop and not in every piece's code.
  constexpr int kVecs = S::kVecs, kDown = S::kDown, kRow = S::kRow;
  typedef __attribute__((address_space(3))) float lds_f32;
  typedef __attribute__((address_space(3))) f32x4 lds_f32x4;
  lds_char* const way = lds + wave * S::kWay;
  lds_f32* const strip = (lds_f32*)way;
  lds_u32x4* const kept = (lds_u32x4*)(way + S::kStrip) + lane;
  const int down = lane / S::kAcross, across = lane % S::kAcross * 8;
  const int32_t c = c0 + wn * S::kCols + across;
  const int left = A.N - c;
  const bool reads = A.e.add || A.e.pre_in;
  float bias[8];
  bias_at(A.e, c, left, bias);
  Beside beside[kVecs];
  const auto fetch_beside = [&](int m) ZERO_INLINE {
    if (!reads) return;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int32_t r = r0 + (wm * W + m) * 32 + i * kDown + down;
      beside[i] = beside_at(A.e, A.N, r, c, r < A.M ? left : 0);
    }
  };
  fetch_beside(0);
  __syncthreads();
  unrolled<W>([&](auto index) ZERO_INLINE {
    constexpr int m = decltype(index)::value, kDeep = 32 / kPanel;
#pragma unroll
    for (int h = 0; h < kDeep; ++h)
#pragma unroll
      for (int n = 0; n < P; ++n)
#pragma unroll
        for (int q = 0; q < Matrix::kQuads; ++q)
          *(lds_f32x4*)(strip + (h * kPanel + lane % kPanel) * kRow + n * kPanel + 8 * q + lane / kPanel * 4) =
              Matrix::quad(acc[m * kDeep + h][n], q);
    if (reads) {
#pragma unroll
      for (int i = 0; i < kVecs; ++i) {
        kept[i * 128] = beside[i].add;
        kept[i * 128 + 64] = beside[i].pre;
      }
    }
    lanes_meet_in_lds();
    if constexpr (m + 1 < W) fetch_beside(m + 1);
    const int32_t rb = r0 + (wm * W + m) * 32 + down;
    // Not unrolled: a tile runs this code once, and the more of it there is the
    // longer a CU waits for it (16384 x 4096 x 14336 with everything in the
    // epilogue: 1580 us, by 2 1610, by 4 1710, by 8 1855).
#pragma unroll 1
    for (int i = 0; i < kVecs; ++i) {
      const lds_f32x4* p = (const lds_f32x4*)(strip + (i * kDown + down) * kRow + across);
      const f32x4 lo = p[0], hi = p[1];
      float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
      Beside x{{0u, 0u, 0u, 0u}, {0u, 0u, 0u, 0u}};
      if (reads) x = Beside{kept[i * 128], kept[i * 128 + 64]};
      const int32_t r = rb + i * kDown;
      if (r < A.M && left > 0) finish8(A.e, A.N, r, c, left, v, x, bias);
    }
    lanes_meet_in_lds();
  });
}

// Adds up a tile's splits, in order, and finishes the sums: `parts` blocks to
// a tile.  The 32 pieces of 8 columns in which 64 lanes hold 4 sums each are 32
// neighbouring threads'.
template <class S, bool NC>
__global__ void __launch_bounds__(kThreads) sum_kernel(const Args A, int32_t parts) {
  constexpr int SIDE = S::kSide, kWave = SIDE * SIDE / 4, kPanel = Panels<NC>::kSide, P = S::kCols / kPanel;
  constexpr int kQuads = Panels<NC>::kQuads;
  const int32_t at = (int32_t)blockIdx.x / parts, part = (int32_t)blockIdx.x % parts;
  int32_t r0, c0;
  tile_place(A.whole + at, A.row_tiles, A.col_tiles, r0, c0);
  const float* from = A.partial + (int64_t)at * A.splits * SIDE * SIDE;
  const int per = SIDE * SIDE / 8 / parts;
  for (int g = part * per + threadIdx.x; g < (part + 1) * per; g += kThreads) {
    const int wave = g / (kWave / 8), unit = g / 32 % (kWave / 256), x = g % 32;
    const int m = unit / (P * kQuads), n = unit / kQuads % P, q = unit % kQuads;
    const int row = x % kPanel, eight = kQuads * (x / kPanel) + q;  // of a panel
    const int32_t r = r0 * SIDE + wave / 2 * S::kCols + m * kPanel + row;
    const int32_t c = c0 * SIDE + wave % 2 * S::kCols + n * kPanel + 8 * eight;
    const int left = A.N - c;
    if (r >= A.M || left <= 0) continue;
    const Beside b = beside_at(A.e, A.N, r, c, left);
    float bias[8];
    bias_at(A.e, c, left, bias);
    f32x4 lo = {0.f, 0.f, 0.f, 0.f}, hi = {0.f, 0.f, 0.f, 0.f};
    const float* p = from + wave * kWave + unit * 256 + (row + 2 * kPanel * (x / kPanel)) * 4;
#pragma unroll 8
    for (int k = 0; k < A.splits; ++k, p += SIDE * SIDE) {
      lo += *(const f32x4*)p;
      hi += *(const f32x4*)(p + 4 * kPanel);
    }
    float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    finish8(A.e, A.N, r, c, left, v, b, bias);
  }
}

// Copies of operands that requests cannot take, rows filled up with zeros to
// whole chunks: the weight from its places in the flat buffer, then A.
struct Copy {
  const uint16_t* from;
  uint16_t* to;
  Place place;     // the weight's; A: x0 0, no gap
  int64_t stride;  // of the source
  int64_t rows;
  int32_t cols, chunks;
};
__global__ void __launch_bounds__(kThreads) copy_kernel(const Copy w, const Copy a) {
  const int64_t nw = w.rows * w.chunks, n = nw + a.rows * a.chunks;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kThreads) {
    const bool first = i < nw;
    const Copy& c = first ? w : a;
    const int64_t j = first ? i : i - nw;
    const int64_t r = j / c.chunks;
    const int32_t col = (int32_t)(j - r * c.chunks) * 8;
    const int left = c.cols - col;
    u32x4 v = {0u, 0u, 0u, 0u};
    int64_t at;
    if (place_run<true>(c.place, r * c.stride + col, 8, at) && left >= 8) {
      v = *(const u32x4_a2*)(c.from + at);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < left)
          v[k >> 1] |= (uint32_t)c.from[place_at<true>(c.place, r * c.stride + col + k)] << (16 * (k & 1));
    }
    *(u32x4*)(c.to + (r * c.chunks * 8 + col)) = v;
  }
}

// ------------------------------------------------------------------ host
constexpr int64_t kMaxStride = (int64_t)1 << 22;  // a tile's rows lie within 32 bits

struct Plan : TilePlan {
  bool few;                        // the kernels of few tokens
  int64_t w_bytes, a_bytes, bytes;  // copies, and everything
};

typedef Shape<4> Large;
typedef Shape<2> Small;

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

// A call's sizes: M tokens, N columns of the result, K of the sum.  n_adjacent:
// B's neighbouring elements differ in n.
struct Sizes {
  int64_t M, N, K;
  bool n_adjacent;
  int64_t w_rows, w_cols;
};
Sizes sizes_of(int64_t tokens, int64_t out_f, int64_t in_f, bool transposed, bool grad) {
  Sizes z;
  z.M = tokens;
  z.N = grad ? in_f : out_f;
  z.K = grad ? out_f : in_f;
  z.n_adjacent = transposed != grad;
  z.w_rows = transposed ? in_f : out_f;
  z.w_cols = transposed ? out_f : in_f;
  return z;
}

Plan make_plan(const zero_layout* L, int32_t tensor, const Sizes& z, const uint16_t* params, const uint16_t* a,
               int64_t a_stride) {
  int64_t lo, hi;
  const Place pl = make_place(L, tensor, &lo, &hi);
  const bool copy_w = pl.gap != 0 || z.w_cols % 8 || !aligned16(params + lo);
  if (is_few(z.M, z.N, z.K, z.n_adjacent, copy_w)) {
    Plan p{};
    p.few = true;
    p.bytes = few_bytes(z.M, z.N, z.K, z.n_adjacent);
    return p;
  }
  Plan p{plan_of(z.M, z.N, z.K)};
  const bool copy_a = z.K % 8 || a_stride % 8 || a_stride > kMaxStride || !aligned16(a);
  p.w_bytes = copy_w ? z.w_rows * ((z.w_cols + 7) / 8) * 16 : 0;
  p.a_bytes = copy_a ? z.M * ((z.K + 7) / 8) * 16 : 0;
  p.bytes = p.w_bytes + p.a_bytes + p.further * p.splits * p.side * p.side * 4;
  return p;
}

int shape_ok(const zero_layout* L, int32_t tensor, int32_t transposed, int64_t O, int64_t I, int64_t tokens) {
  if (!L || O < 0 || I < 0 || tokens < 0 || (transposed != 0 && transposed != 1)) return ZERO_EINVAL;
  if (!tensor_ok(L, tensor)) return ZERO_ERANGE;
  if (O > ZERO_MAX_FEATURES || I > ZERO_MAX_FEATURES || tokens > ZERO_MAX_ROWS) return ZERO_ERANGE;
  if (O * I != L->numel[(size_t)tensor]) return ZERO_EINVAL;
  return ZERO_OK;
}
// The dispatch grids count work-items in 32 bits.
int plan_ok(const Plan& p) { return p.row_tiles * p.col_tiles > ((int64_t)1 << 23) ? ZERO_ERANGE : ZERO_OK; }

template <class S>
int launch(const Args& A, const Plan& p, bool n_adjacent, hipStream_t s) {
  const dim3 grid((unsigned)(p.whole + p.further * p.splits));
  if (n_adjacent)
    hipLaunchKernelGGL((product_kernel<S, true>), grid, dim3(kThreads), 0, s, A);
  else
    hipLaunchKernelGGL((product_kernel<S, false>), grid, dim3(kThreads), 0, s, A);
  const int rc = launched();
  if (rc != ZERO_OK || p.further == 0) return rc;
  int32_t parts = S::kSide * S::kSide / 2048;
  while (parts > 1 && parts * p.further > 2048) parts >>= 1;
  const dim3 sums((unsigned)(p.further * parts));
  if (n_adjacent)
    hipLaunchKernelGGL((sum_kernel<S, true>), sums, dim3(kThreads), 0, s, A, parts);
  else
    hipLaunchKernelGGL((sum_kernel<S, false>), sums, dim3(kThreads), 0, s, A, parts);
  return launched();
}

int64_t workspace_of(const zero_layout* L, int32_t tensor, int32_t transposed, const uint16_t* params,
                     const uint16_t* a, int64_t a_stride, int64_t tokens, int64_t O, int64_t I, bool grad) {
  const int rc = shape_ok(L, tensor, transposed, O, I, tokens);
  if (rc != ZERO_OK) return rc;
  if (O == 0 || I == 0 || tokens == 0) return 0;
  const Sizes z = sizes_of(tokens, O, I, transposed != 0, grad);
  if (a_stride < z.K) return ZERO_EINVAL;
  const Plan p = make_plan(L, tensor, z, params, a, a_stride);
  return plan_ok(p) == ZERO_OK ? p.bytes : ZERO_ERANGE;
}

// What both directions do once their own arguments are checked and the
// epilogue is filled in.  The memory of the outputs is in `outs`, what the
// epilogue reads in `ins`.
int run(const zero_layout* L, int32_t tensor, const uint16_t* params, const uint16_t* a, int64_t a_stride,
        const Sizes& z, const Epilogue& e, const Bytes (&out)[2], const Bytes (&in)[3], void* workspace,
        int64_t workspace_bytes, hipStream_t stream) {
  const Plan p = make_plan(L, tensor, z, params, a, a_stride);
  if (plan_ok(p) != ZERO_OK) return ZERO_ERANGE;
  if (p.bytes > 0 && (!workspace || workspace_bytes < p.bytes || ((uintptr_t)workspace & 15u))) return ZERO_EINVAL;
  int64_t lo, hi;
  const Place place = make_place(L, tensor, &lo, &hi);
  const Bytes outs[] = {out[0], out[1], Bytes{workspace, p.bytes}};
  const Bytes ins[] = {in[0], in[1], in[2], Bytes{params + lo, 2 * (hi - lo)}, rows_of(a, z.M, z.K, a_stride, 2)};
  if (any_overlap(outs, ins)) return ZERO_EOVERLAP;
  if (hip_error_pending()) return ZERO_EHIP;
  if (p.few)
    return launch_few(Few{a, params, a_stride, place, (int32_t)z.M, (int32_t)z.N, (int32_t)z.K, e}, z.n_adjacent,
                      workspace, stream);
  Args A{};
  A.M = (int32_t)z.M;
  A.N = (int32_t)z.N;
  A.K = (int32_t)((z.K + 7) / 8 * 8);
  A.Kb = (int32_t)z.K;
  A.row_tiles = (int32_t)p.row_tiles;
  A.col_tiles = (int32_t)p.col_tiles;
  A.whole = (int32_t)p.whole;
  A.splits = (int32_t)p.splits;
  A.per_split = (int32_t)p.per_split;
  A.e = e;
  char* ws = (char*)workspace;
  A.a = p.a_bytes ? (const uint16_t*)(ws + p.w_bytes) : a;
  A.a_stride = p.a_bytes ? A.K : a_stride;
  const int64_t w_stride = (z.w_cols + 7) / 8 * 8;
  A.b = p.w_bytes ? (const uint16_t*)ws : params + lo;
  A.b_stride = p.w_bytes ? w_stride : z.w_cols;
  A.partial = (float*)(ws + p.w_bytes + p.a_bytes);
  if (p.w_bytes || p.a_bytes) {
    // without padding every run of elements lies in one piece
    const Place plain{0, (int64_t)1 << 62, 0, 0.0}, whole{place.x0, plain.cap, 0, 0.0};
    const Copy w{params, (uint16_t*)ws, place.gap ? place : whole, z.w_cols, p.w_bytes ? z.w_rows : 0, (int32_t)z.w_cols,
                 (int32_t)((z.w_cols + 7) / 8)};
    const Copy c{a, (uint16_t*)(ws + p.w_bytes), plain, a_stride, p.a_bytes ? z.M : 0, (int32_t)z.K,
                 (int32_t)((z.K + 7) / 8)};
    const int64_t n = w.rows * w.chunks + c.rows * c.chunks;
    const unsigned grid = (unsigned)std::min<int64_t>((n + kThreads - 1) / kThreads, 16 * kCus);
    hipLaunchKernelGGL(copy_kernel, dim3(grid), dim3(kThreads), 0, stream, w, c);
    const int rc = launched();
    if (rc != ZERO_OK) return rc;
  }
  return p.side == Large::kSide ? launch<Large>(A, p, z.n_adjacent, stream)
                                : launch<Small>(A, p, z.n_adjacent, stream);
}

}  // namespace

extern "C" {

int64_t zero_linear_workspace(const zero_layout* L, int32_t tensor, int32_t transposed,
                              const uint16_t* params_flat, const uint16_t* x, int64_t x_stride, int64_t tokens,
                              int64_t out_features, int64_t in_features) {
  return workspace_of(L, tensor, transposed, params_flat, x, x_stride, tokens, out_features, in_features, false);
}

int zero_linear(const zero_layout* L, int32_t tensor, int32_t transposed, int32_t bias_tensor,
                const uint16_t* params_flat, const uint16_t* x, int64_t x_stride, int64_t tokens,
                int64_t out_features, int64_t in_features, int32_t activation, const uint16_t* res,
                int64_t res_stride, void* out, int64_t out_stride, int32_t out_dtype, uint16_t* pre,
                void* workspace, int64_t workspace_bytes, hipStream_t stream) {
  const int rc = shape_ok(L, tensor, transposed, out_features, in_features, tokens);
  if (rc != ZERO_OK) return rc;
  const int64_t O = out_features, I = in_features;
  if (bias_tensor < -1 || !activation_ok(activation)) return ZERO_EINVAL;
  if (out_dtype != ZERO_DTYPE_BF16 && out_dtype != ZERO_DTYPE_F32) return ZERO_EINVAL;
  if (bias_tensor >= 0) {
    if (!tensor_ok(L, bias_tensor)) return ZERO_ERANGE;
    if (L->numel[(size_t)bias_tensor] != O) return ZERO_EINVAL;
  }
  // a sum over nothing would still be the bias: not a layer
  if (I == 0 && O > 0 && tokens > 0) return ZERO_EINVAL;
  if (tokens == 0 || O == 0) return ZERO_OK;
  if (!params_flat || !x || !out || x_stride < I || out_stride < O || (res && res_stride < O)) return ZERO_EINVAL;
  if (x_stride > ZERO_MAX_STRIDE || out_stride > ZERO_MAX_STRIDE || (res && res_stride > ZERO_MAX_STRIDE))
    return ZERO_ERANGE;
  Epilogue e{};
  int64_t lo = 0, hi = 0;
  if (bias_tensor >= 0) {
    e.bias = params_flat;
    e.bias_place = make_place(L, bias_tensor, &lo, &hi);
  }
  e.add = res;
  e.add_stride = res_stride;
  e.pre_out = pre;
  e.out = out;
  e.out_stride = out_stride;
  e.act = activation;
  e.f32 = out_dtype == ZERO_DTYPE_F32;
  const Bytes outs[2] = {rows_of(out, tokens, O, out_stride, e.f32 ? 4 : 2), Bytes{pre, 2 * tokens * O}};
  const Bytes ins[3] = {rows_of(res, tokens, O, res_stride, 2), Bytes{params_flat + lo, 2 * (hi - lo)}, Bytes{}};
  return run(L, tensor, params_flat, x, x_stride, sizes_of(tokens, O, I, transposed != 0, false), e, outs, ins,
             workspace, workspace_bytes, stream);
}

int64_t zero_linear_input_grad_workspace(const zero_layout* L, int32_t tensor, int32_t transposed,
                                         const uint16_t* params_flat, const uint16_t* dy, int64_t dy_stride,
                                         int64_t tokens, int64_t out_features, int64_t in_features) {
  return workspace_of(L, tensor, transposed, params_flat, dy, dy_stride, tokens, out_features, in_features, true);
}

int zero_linear_input_grad(const zero_layout* L, int32_t tensor, int32_t transposed, const uint16_t* params_flat,
                           const uint16_t* dy, int64_t dy_stride, int64_t tokens, int64_t out_features,
                           int64_t in_features, int32_t activation, const uint16_t* pre, const uint16_t* add,
                           int64_t add_stride, uint16_t* dx, int64_t dx_stride, void* workspace,
                           int64_t workspace_bytes, hipStream_t stream) {
  const int rc = shape_ok(L, tensor, transposed, out_features, in_features, tokens);
  if (rc != ZERO_OK) return rc;
  const int64_t O = out_features, I = in_features;
  if (!activation_ok(activation)) return ZERO_EINVAL;
  if (O == 0 && I > 0 && tokens > 0) return ZERO_EINVAL;
  if (tokens == 0 || I == 0) return ZERO_OK;
  if (!params_flat || !dy || !dx || dy_stride < O || dx_stride < I || (add && add_stride < I)) return ZERO_EINVAL;
  if ((activation != ZERO_ACT_NONE) != (pre != nullptr)) return ZERO_EINVAL;
  if (dy_stride > ZERO_MAX_STRIDE || dx_stride > ZERO_MAX_STRIDE || (add && add_stride > ZERO_MAX_STRIDE))
    return ZERO_ERANGE;
  Epilogue e{};
  e.add = add;
  e.add_stride = add_stride;
  e.pre_in = pre;
  e.out = dx;
  e.out_stride = dx_stride;
  e.act = activation;
  e.grad = 1;
  const Bytes outs[2] = {rows_of(dx, tokens, I, dx_stride, 2), Bytes{}};
  const Bytes ins[3] = {rows_of(add, tokens, I, add_stride, 2), Bytes{pre, 2 * tokens * I}, Bytes{}};
  return run(L, tensor, params_flat, dy, dy_stride, sizes_of(tokens, O, I, transposed != 0, true), e, outs, ins,
             workspace, workspace_bytes, stream);
}

}  // extern "C"
