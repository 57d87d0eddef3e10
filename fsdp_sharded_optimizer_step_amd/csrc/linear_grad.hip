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
#include "matrix.hpp"

namespace {
using namespace zs;

// The shape of a block: G groups of 4 waves; the waves of a group lie two by
// two over the tile, W panels of 32 columns along each side of a wave, and
// each group sums 64 of the 64*G tokens of an LDS tile.
template <int W_, int G_>
struct Shape {
  static constexpr int W = W_, G = G_;
  static constexpr int kSide = 64 * W;
  static constexpr int kThreads = 256 * G;
  static constexpr int kStep = 64 * G;  // tokens of one LDS tile
  // A panel: kStep tokens of 32 columns in bf16, 64 bytes to a token.  Panels
  // lie 64 bytes further apart than they are long, so that the writes of one
  // token row, which go to as many panels as the tile is wide, spread over
  // the banks.
  static constexpr int kPanelBytes = kStep * 64 + 64;
  static constexpr int kOperand = 2 * W * kPanelBytes, kBuffer = 2 * kOperand;
};
typedef Shape<4, 1> Large;
typedef Shape<2, 2> Small;
constexpr int kSumThreads = 256;

struct Args {
  const uint16_t* dy;
  int64_t dy_stride;
  const uint8_t* codes;
  const uint8_t* scales;
  int64_t tokens;
  int32_t O, I, nb;
  int32_t rows, cols;  // of the gradient: (O, I), or (I, O) when transposed
  int32_t row_tiles, col_tiles;
  int32_t whole;       // tiles that one block sums over all tokens
  int32_t splits;      // blocks of each further tile
  int64_t tokens_per_split;
  int64_t fast_tokens; // tokens before this one can be read in whole chunks
  int32_t direct;      // whole tiles go straight to the gradient (else: like split ones)
  float* partial;      // per split and further tile, a tile of binary32 sums
  GradOut out;
};

// One thread's part of a tile of kSide columns and kStep tokens: chunks of 8
// columns of dY or 16 of X (16 bytes each, at any alignment).  fast() takes
// whole chunks of whole steps.  A chunk that begins past the last column is
// read from the last chunk, and the last chunk of a row may run on into the
// next row: what it finds there enters only sums that are not stored.  part()
// does the same for a step that is not whole, with zeros for the tokens from
// `lim` on.  The matrix's last tokens, from where a chunk would run out of the
// matrix (15 at most), are put into LDS by finish(), element by element.
template <class S>
struct DyTile {
  static constexpr int kPerRow = S::kSide / 8, kRows = S::kThreads / kPerRow, kN = S::kStep / kRows;
  u32x4 v[kN];
  static __device__ __forceinline__ int col() { return (threadIdx.x % kPerRow) * 8; }
  static __device__ __forceinline__ int row() { return threadIdx.x / kPerRow; }
  static __device__ __forceinline__ uint32_t fast_offset(const Args& A, int32_t c0) {
    return (uint32_t)(row() * A.dy_stride + min(c0 + col(), (A.O - 1) & ~7)) * 2u;
  }
  __device__ __forceinline__ void fast1(const Args& A, int64_t t0, uint32_t off, int k) {
    const char* p = (const char*)(A.dy + (t0 + k * kRows) * A.dy_stride);
    v[k] = *(const u32x4_a2*)(p + off);
  }
  __device__ __forceinline__ void fast(const Args& A, int64_t t0, uint32_t off) {
#pragma unroll
    for (int k = 0; k < kN; ++k) fast1(A, t0, off, k);
  }
  __device__ __forceinline__ void part(const Args& A, int64_t t0, int64_t lim, uint32_t off) {
#pragma unroll
    for (int k = 0; k < kN; ++k) {
      v[k] = u32x4{0u, 0u, 0u, 0u};
      if (t0 + k * kRows + row() < lim) fast1(A, t0, off, k);
    }
  }
  static __device__ __forceinline__ void finish(const Args& A, int64_t t0, int64_t from, int64_t tz,
                                                int32_t c0, lds_char* lds) {
    const int c = c0 + col();
#pragma unroll 1
    for (int k = 0; k < kN; ++k) {
      const int64_t t = t0 + k * kRows + row();
      if (t < from || t >= tz) continue;
      const uint16_t* p = A.dy + t * A.dy_stride + c;
      u32x4 w = {0u, 0u, 0u, 0u};
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < A.O - c) w[j >> 1] |= (uint32_t)p[j] << (16 * (j & 1));
      *(lds_u32x4*)(lds + (col() >> 5) * S::kPanelBytes + (k * kRows + row()) * 64 + (col() & 31) * 2) = w;
    }
  }
  __device__ __forceinline__ void store1(lds_char* lds, int k) const {
    *(lds_u32x4*)(lds + (col() >> 5) * S::kPanelBytes + (k * kRows + row()) * 64 + (col() & 31) * 2) = v[k];
  }
  __device__ __forceinline__ void store(lds_char* lds) const {
#pragma unroll
    for (int k = 0; k < kN; ++k) store1(lds, k);
  }
};

template <class S>
struct XTile {
  static constexpr int kPerRow = S::kSide / 16, kRows = S::kThreads / kPerRow, kN = S::kStep / kRows;
  u32x4 v[kN];
  uint32_t e[kN];
  static __device__ __forceinline__ int col() { return (threadIdx.x % kPerRow) * 16; }
  static __device__ __forceinline__ int row() { return threadIdx.x / kPerRow; }
  static __device__ __forceinline__ uint32_t fast_offset(const Args& A, int32_t c0) {
    return (uint32_t)(row() * A.I + min(c0 + col(), (A.I - 1) & ~15));
  }
  static __device__ __forceinline__ uint32_t fast_scale_offset(const Args& A, int32_t c0) {
    return (uint32_t)(row() * A.nb + (min(c0 + col(), (A.I - 1) & ~15) >> 7));
  }
  __device__ __forceinline__ void fast1(const Args& A, int64_t t0, uint32_t off, uint32_t soff,
                                        int k) {
    const uint8_t* p = A.codes + (t0 + k * kRows) * A.I;
    const uint8_t* s = A.scales + (t0 + k * kRows) * A.nb;
    v[k] = *(const u32x4_a1*)(p + off);
    e[k] = s[soff];
  }
  __device__ __forceinline__ void fast(const Args& A, int64_t t0, uint32_t off, uint32_t soff) {
#pragma unroll
    for (int k = 0; k < kN; ++k) fast1(A, t0, off, soff, k);
  }
  // A chunk's 32 bytes go to LDS as two writes.  Eight lanes write at a time,
  // to four panels, of which those two apart share their banks: the lanes of
  // the further two write their second half first.
  static __device__ __forceinline__ void put(lds_char* to, const u32x4& v, uint32_t byte) {
    const bool swap = (col() >> 6) & 1;
    const float s = act8_scale(byte);
    const u32x2 first = swap ? u32x2{v.z, v.w} : u32x2{v.x, v.y};
    const u32x2 second = swap ? u32x2{v.x, v.y} : u32x2{v.z, v.w};
    const u32x2 a = act8_bf16x4(first.x, s), b = act8_bf16x4(first.y, s);
    const u32x2 d = act8_bf16x4(second.x, s), f = act8_bf16x4(second.y, s);
    *(lds_u32x4*)(to + (swap ? 16 : 0)) = u32x4{a.x, a.y, b.x, b.y};
    *(lds_u32x4*)(to + (swap ? 0 : 16)) = u32x4{d.x, d.y, f.x, f.y};
  }
  __device__ __forceinline__ void part(const Args& A, int64_t t0, int64_t lim, uint32_t off,
                                       uint32_t soff) {
#pragma unroll
    for (int k = 0; k < kN; ++k) {
      v[k] = u32x4{0u, 0u, 0u, 0u};
      e[k] = 127u;
      if (t0 + k * kRows + row() < lim) fast1(A, t0, off, soff, k);
    }
  }
  static __device__ __forceinline__ void finish(const Args& A, int64_t t0, int64_t from, int64_t tz,
                                                int32_t c0, lds_char* lds) {
    const int c = c0 + col();
#pragma unroll 1
    for (int k = 0; k < kN; ++k) {
      const int64_t t = t0 + k * kRows + row();
      if (t < from || t >= tz) continue;
      const uint8_t* p = A.codes + t * A.I + c;
      u32x4 w = {0u, 0u, 0u, 0u};
      uint32_t b = 127u;
      if (c < A.I) b = A.scales[t * A.nb + (c >> 7)];
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if (j < A.I - c) w[j >> 2] |= (uint32_t)p[j] << (8 * (j & 3));
      put(lds + (col() >> 5) * S::kPanelBytes + (k * kRows + row()) * 64 + (col() & 31) * 2, w, b);
    }
  }
  __device__ __forceinline__ void store1(lds_char* lds, int k) const {
    put(lds + (col() >> 5) * S::kPanelBytes + (k * kRows + row()) * 64 + (col() & 31) * 2, v[k], e[k]);
  }
  __device__ __forceinline__ void store(lds_char* lds) const {
#pragma unroll
    for (int k = 0; k < kN; ++k) store1(lds, k);
  }
};

// 32 columns x 16 tokens of a panel as a matrix operand: lane l holds column
// l % 32, tokens 4*(l / 32) + {0..3, 8..11}.
__device__ __forceinline__ bf16x8 frag(const lds_char* panel) {
  typedef __attribute__((address_space(3))) s16x4 lds_t;
  const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_t*)panel);
  const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_t*)(panel + 512));
  return __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}
__device__ __forceinline__ int frag_offset() {
  const int l = threadIdx.x & 63, g = l >> 4, i = l & 15;
  return ((i >> 2) + 4 * (g >> 1)) * 64 + (g & 1) * 32 + (i & 3) * 8;
}

// Instruction order of a stretch of MF matrix instructions: the LDS reads (DR)
// beside the first half of them, so that the next stretch finds its
// fragments, LDS writes (DW) and global loads (GL) beside the second half.
template <int MF, int DR, int DW, int GL>
__device__ __forceinline__ void interleave() {
#pragma unroll
  for (int k = 0; k < MF / 2; ++k) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x100, 2 * DR / MF, 0);
  }
#pragma unroll
  for (int k = 0; k < MF / 2; ++k) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    if constexpr (DW > 0) __builtin_amdgcn_sched_group_barrier(0x200, 2 * DW / MF, 0);
    if constexpr (GL > 0) __builtin_amdgcn_sched_group_barrier(0x020, 2 * GL / MF, 0);
  }
  __builtin_amdgcn_sched_barrier(0);
}

__device__ __forceinline__ void tile_at(const Args& A, int32_t tile, int32_t& r, int32_t& c) {
  tile_place(tile, A.row_tiles, A.col_tiles, r, c);
}

// The workspace's tiles: those that do not go out directly.
__device__ __forceinline__ int64_t slot_of(const Args& A, int32_t tile, int32_t split) {
  const int64_t kept = A.direct ? 0 : A.whole;
  return tile < A.whole ? tile : kept + (int64_t)(tile - A.whole) * A.splits + split;
}

// TR: rows of the gradient are X's columns.
//
// Two LDS buffers and two sets of registers.  A step is four stretches of 16
// tokens (of a group's 64).  While the matrix cores work on a stretch the
// fragments of the next are read; in the first two stretches the next step's
// chunks are converted and written to the other buffer, and those of the step
// three ahead are requested.  One barrier a step, before its last stretch,
// whose fragments are already in registers.
//
// Measured (16384 tokens, 14336 x 4096): 1.47 to 1.54 ms from card to card, 1310
// to 1250 TFLOP/s, against 1.91 to 1.96 ms of a library bf16 product of that
// shape alone.  The matrix cores are busy 71 % of the cycles, at a clock that the
// load itself brings down to about 1.75 GHz: when it took 1.59 ms, it took 1.35
// without the global loads, 1.42 without the LDS reads, 1.06 without either and
// without the LDS writes (for timing only).  Requests two steps ahead instead of
// three take the same time; fragments two stretches ahead spill at this tile
// (2.36 ms) and gain nothing at the smaller one.  As it is, 32 of this tile's
// registers are spilled, none of them inside the loop of whole steps.
// The smaller tile (4000 tokens, 1024 x 4096: 41 us) takes 11 us at the ends and
// 1.02 us for 128 tokens, in which the matrix cores and the LDS are busy for
// about 0.45 us each.
template <class S, bool TR>
__global__ void __launch_bounds__(S::kThreads, 1) grad_kernel(const Args A) {
  constexpr int W = S::W, G = S::G, kSide = S::kSide, kStep = S::kStep;
  constexpr int kPanelBytes = S::kPanelBytes, kOperand = S::kOperand, kBuffer = S::kBuffer;
  __shared__ __align__(16) char shared[2 * kBuffer];
  lds_char* lds = (lds_char*)shared;

  // whole tiles first, dealt to the XCDs (block b runs on XCD b % 8) in runs
  int32_t tile, split = 0;
  int64_t ta = 0, tz = A.tokens;
  if ((int32_t)blockIdx.x < A.whole) {
    tile = (A.whole & 7) ? (int32_t)blockIdx.x
                         : (int32_t)(blockIdx.x & 7) * (A.whole >> 3) + (int32_t)(blockIdx.x >> 3);
  } else {
    const int32_t x = (int32_t)blockIdx.x - A.whole;
    split = x % A.splits;
    tile = A.whole + x / A.splits;
    ta = split * A.tokens_per_split;
    tz = min(A.tokens, ta + A.tokens_per_split);
  }
  int32_t r0, c0;
  tile_at(A, tile, r0, c0);
  r0 *= kSide;
  c0 *= kSide;

  const int wave = threadIdx.x >> 6, wm = (wave >> 1) & 1, wn = wave & 1, group = wave >> 2;
  const int lane = threadIdx.x & 63;
  f32x16 acc[W][W];
#pragma unroll
  for (int a = 0; a < W; ++a)
#pragma unroll
    for (int b = 0; b < W; ++b)
#pragma unroll
      for (int k = 0; k < 16; ++k) acc[a][b][k] = 0.f;

  DyTile<S> dy[2];
  XTile<S> x[2];
  const int32_t dy_c = TR ? c0 : r0, x_c = TR ? r0 : c0;
  const uint32_t dy_off = DyTile<S>::fast_offset(A, dy_c),
                 x_off = XTile<S>::fast_offset(A, x_c),
                 s_off = XTile<S>::fast_scale_offset(A, x_c);
  lds_char* const dy_lds = lds + (TR ? kOperand : 0);
  lds_char* const x_lds = lds + (TR ? 0 : kOperand);
  // a group's 64 tokens: 4096 bytes of a panel
  const lds_char* const fa = lds + wm * W * kPanelBytes + group * 4096 + frag_offset();
  const lds_char* const fb = lds + kOperand + wn * W * kPanelBytes + group * 4096 + frag_offset();

  const int64_t steps = (tz - ta + kStep - 1) / kStep;
  // tokens and whole steps that chunk loads can take
  const int64_t lim = min(tz, A.fast_tokens);
  const int64_t full = max((int64_t)0, lim - ta) / kStep;
  // step k waits in set k % 2 of the registers
  auto load = [&](int64_t k, int set) {
    const int64_t t0 = ta + k * kStep;
    if (k < full) {
      dy[set].fast(A, t0, dy_off);
      x[set].fast(A, t0, x_off, s_off);
    } else {
      dy[set].part(A, t0, lim, dy_off);
      x[set].part(A, t0, lim, x_off, s_off);
    }
  };
  bf16x8 a[2][W], b[2][W];
  auto read = [&](int to, int buf, int s) {
#pragma unroll
    for (int k = 0; k < W; ++k) {
      a[to][k] = frag(fa + buf * kBuffer + k * kPanelBytes + s * 1024);
      b[to][k] = frag(fb + buf * kBuffer + k * kPanelBytes + s * 1024);
    }
  };
  auto multiply = [&](int from) {
#pragma unroll
    for (int m = 0; m < W; ++m)
#pragma unroll
      for (int n = 0; n < W; ++n)
        acc[m][n] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[from][m], b[from][n], acc[m][n], 0, 0, 0);
  };
  // step k from set k % 2 to buffer k % 2 (so both are `set`)
  auto store = [&](int64_t k, int set) {
    dy[set].store(dy_lds + set * kBuffer);
    x[set].store(x_lds + set * kBuffer);
    if (ta + (k + 1) * kStep > lim && lim < tz) {
      // the same thread writes the same places: in order
      DyTile<S>::finish(A, ta + k * kStep, lim, tz, dy_c, dy_lds + set * kBuffer);
      XTile<S>::finish(A, ta + k * kStep, lim, tz, x_c, x_lds + set * kBuffer);
    }
  };
  // Step k, in buffer `buf`: its products; step k + 1 goes from the registers
  // to the other buffer, step k + 3 is requested into the same registers.
  auto step = [&](int64_t k, int buf) {
    constexpr int kM = W * W, kR = 4 * W, kX = XTile<S>::kN, kDy = DyTile<S>::kN;
    const int set = buf ^ 1;
    read(1, buf, 1);
    x[set].store(x_lds + (buf ^ 1) * kBuffer);
    x[set].fast(A, ta + (k + 3) * kStep, x_off, s_off);
    multiply(0);
    interleave<kM, kR, 2 * kX, 2 * kX>();
    read(0, buf, 2);
    dy[set].store(dy_lds + (buf ^ 1) * kBuffer);
    dy[set].fast(A, ta + (k + 3) * kStep, dy_off);
    multiply(1);
    interleave<kM, kR, kDy, kDy>();
    read(1, buf, 3);
    multiply(0);
    interleave<kM, kR, 0, 0>();
    __syncthreads();
    read(0, buf ^ 1, 0);
    multiply(1);
    interleave<kM, kR, 0, 0>();
  };

  if (steps > 0) {
    load(0, 0);
    if (steps > 1) load(1, 1);
    store(0, 0);
    if (steps > 2) load(2, 0);
    __syncthreads();
    read(0, 0, 0);
    int64_t k = 0;
    for (; k + 4 < full; k += 2) {
      step(k, 0);
      step(k + 1, 1);
    }
    // the last steps
    for (; k < steps; ++k) {
      const int buf = (int)(k & 1);
      read(1, buf, 1);
      multiply(0);
      read(0, buf, 2);
      multiply(1);
      read(1, buf, 3);
      multiply(0);
      if (k + 1 < steps) {
        if (buf)
          store(k + 1, 0);
        else
          store(k + 1, 1);
      }
      if (k + 3 < steps) {
        if (buf)
          load(k + 3, 0);
        else
          load(k + 3, 1);
      }
      __syncthreads();
      if (k + 1 < steps) read(0, buf ^ 1, 0);
      multiply(1);
    }
  }

  // Two groups: each keeps one half of its rows of blocks and gets the other
  // group's sums of it through LDS.
  constexpr int kMine = W / G;  // rows of blocks of a wave
  const int m0 = group * kMine;
  if constexpr (G == 2) {
    typedef __attribute__((address_space(3))) float lds_float;
    lds_float* const box = (lds_float*)lds + (threadIdx.x & 255);
    constexpr int kHalf = kMine * W * 16 * 256;  // what one group sends
    static_assert(2 * kHalf * 4 <= 2 * kBuffer, "both fit the buffers");
    __syncthreads();
#pragma unroll
    for (int g = 0; g < 2; ++g)
      if (group == g) {
#pragma unroll
        for (int m = 0; m < kMine; ++m)
#pragma unroll
          for (int n = 0; n < W; ++n)
#pragma unroll
            for (int k = 0; k < 16; ++k)
              box[g * kHalf + ((m * W + n) * 16 + k) * 256] = acc[(1 - g) * kMine + m][n][k];
      }
    __syncthreads();
#pragma unroll
    for (int g = 0; g < 2; ++g)
      if (group == g) {
#pragma unroll
        for (int m = 0; m < kMine; ++m)
#pragma unroll
          for (int n = 0; n < W; ++n)
#pragma unroll
            for (int k = 0; k < 16; ++k)
              acc[m][n][k] = acc[g * kMine + m][n][k] + box[(1 - g) * kHalf + ((m * W + n) * 16 + k) * 256];
      }
  }

  // lane l, register k: row 8*(k/4) + 4*(l/32) + k%4, column l%32
  if (A.direct && tile < A.whole) {
    // A wave's sums leave 32 rows at a time, through LDS of its own (the
    // buffers are free), from where a lane gets 4 columns of a row; the
    // accumulator's values of the next strip are requested before this one's
    // are stored.  Single values from the registers to memory left half of its
    // rate unused: 1024 tokens, 8192 x 8192, added 294 us, 239 here, overwritten
    // 231, 172; 16384 tokens, 14336 x 4096: 1541, 1499.
    constexpr int kCols = W * 32, kStride = kCols + 8;  // 4 rows are 32 banks apart
    constexpr int kAcross = kCols / 4, kDown = 64 / kAcross, kVecs = 32 / kDown;
    static_assert(S::kThreads / 64 * 32 * kStride * 4 <= 2 * kBuffer, "the strips fit the buffers");
    typedef __attribute__((address_space(3))) float lds_f32;
    typedef __attribute__((address_space(3))) f32x4 lds_f32x4;
    __syncthreads();
    lds_f32* const strip = (lds_f32*)lds + (threadIdx.x >> 6) * 32 * kStride;
    const int down = lane / kAcross, across = lane % kAcross * 4;
    auto put = [&](auto index) {
      constexpr int m = decltype(index)::value;
#pragma unroll
      for (int n = 0; n < W; ++n)
#pragma unroll
        for (int k = 0; k < 16; ++k)
          strip[(8 * (k >> 2) + (k & 3) + 4 * (lane >> 5)) * kStride + n * 32 + (lane & 31)] = acc[m][n][k];
    };
    auto get = [&](int i) {
      return *(const lds_f32x4*)(strip + (i * kDown + down) * kStride + across);
    };
    const uint32_t lane_off = (uint32_t)down * (uint32_t)A.cols + across;
    const bool add = !(A.out.flags & ZERO_ACC_OVERWRITE);
    const bool keep = !(A.out.flags & ZERO_ACC_NO_STORE), emit = A.out.flags & ZERO_ACC_EMIT_BF16;
    f32x4 v[2][kVecs];
    // CHECKED: the tile goes past the matrix's last row or column
    auto out = [&](auto checked) {
      constexpr bool kChecked = decltype(checked)::value;
      const int32_t cb = c0 + wn * kCols;
      // f(i, position, columns left): vector i of strip m
      auto each = [&](int m, auto f) {
        const int32_t rb = r0 + (wm * W + m0 + m) * 32;
        const int64_t at = A.out.place.x0 + (int64_t)rb * A.cols + cb;
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
          int left = 4;
          if (kChecked) left = rb + i * kDown + down < A.rows ? A.cols - cb - across : 0;
          if (!kChecked || left > 0) f(i, at + (int64_t)(i * kDown) * A.cols, left);
        }
      };
      auto fetch = [&](int m) {
        each(m, [&](int i, int64_t at, int left) {
          const float* q = A.out.acc + at + lane_off;
          if (left >= 4) {
            v[m & 1][i] = __builtin_nontemporal_load((const f32x4_a4*)q);
          } else {
#pragma unroll
            for (int j = 0; j < 3; ++j)
              if (j < left) v[m & 1][i][j] = q[j];
          }
        });
      };
      if (add) fetch(0);
      unrolled<kMine>([&](auto index) {
        constexpr int m = decltype(index)::value;
        put(index);
        lanes_meet_in_lds();
        if (add && m + 1 < kMine) fetch(m + 1);
        each(m, [&](int i, int64_t at, int left) {
          const f32x4 s = get(i);
          f32x4 x = {A.out.scale * s.x, A.out.scale * s.y, A.out.scale * s.z, A.out.scale * s.w};
          if (add) {
            const f32x4 b = v[m & 1][i];
            x = f32x4{b.x + x.x, b.y + x.y, b.z + x.z, b.w + x.w};
          }
          float* q = A.out.acc + at + lane_off;
          uint16_t* o = A.out.out + at + lane_off;
          if (left >= 4) {
            if (keep) __builtin_nontemporal_store(x, (f32x4_a4*)q);
            if (emit) *(u32x2_a2*)o = u32x2{bf16_pack2(x.x, x.y), bf16_pack2(x.z, x.w)};
          } else {
#pragma unroll
            for (int j = 0; j < 3; ++j)
              if (j < left) {
                if (keep) q[j] = x[j];
                if (emit) o[j] = (uint16_t)bf16_round(x[j]);
              }
          }
        });
        lanes_meet_in_lds();
      });
    };
    if (r0 + kSide <= A.rows && c0 + kSide <= A.cols)
      out(std::false_type{});
    else
      out(std::true_type{});
    return;
  }
  // a tile of the workspace, rows of kSide columns (through LDS no faster: 1000
  // tokens, 2304 x 768, 25 us against 22)
  float* const to = A.partial + slot_of(A, tile, split) * kSide * kSide + 4 * (lane >> 5) * kSide + (lane & 31);
#pragma unroll
  for (int m = 0; m < kMine; ++m)
#pragma unroll
    for (int n = 0; n < W; ++n)
#pragma unroll
      for (int k = 0; k < 16; ++k)
        to[((wm * W + m0 + m) * 32 + 8 * (k >> 2) + (k & 3)) * kSide + (wn * W + n) * 32] = acc[m][n][k];
}

// Adds up a tile's splits, in order, and hands the sum on: blocks over the
// tiles from `first`, `parts` to a tile.
template <int SIDE, bool GAPS>
__global__ void __launch_bounds__(kSumThreads) sum_kernel(const Args A, int32_t first,
                                                          int32_t parts) {
  const int32_t tile = first + (int32_t)blockIdx.x / parts;
  const int32_t part = (int32_t)blockIdx.x % parts;
  int32_t r0, c0;
  tile_at(A, tile, r0, c0);
  r0 *= SIDE;
  c0 *= SIDE;
  const int32_t n_splits = tile < A.whole ? 1 : A.splits;
  const float* from = A.partial + slot_of(A, tile, 0) * SIDE * SIDE;
  const int per = SIDE * SIDE / 4 / parts;  // groups of 4 columns
  for (int g = part * per + threadIdx.x; g < (part + 1) * per; g += kSumThreads) {
    const int32_t r = r0 + g / (SIDE / 4), c = c0 + (g % (SIDE / 4)) * 4;
    const int n = min(4, A.cols - c);
    if (r >= A.rows || n <= 0) continue;
    f32x4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
    for (int k = 0; k < n_splits; ++k) s += *(const f32x4*)(from + (int64_t)k * SIDE * SIDE + g * 4);
    const int64_t e = (int64_t)r * A.cols + c;
    int64_t at;
    if (n >= 4 && place_run<GAPS>(A.out.place, e, 4, at)) {
      grad_store4(A.out, at, s);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < n) grad_store(A.out, place_at<GAPS>(A.out.place, e + j), s[j]);
    }
  }
}

// ------------------------------------------------------------------ host
struct Plan {
  int64_t side, row_tiles, col_tiles, whole, further, splits, tokens_per_split, slots, bytes;
  double us;
  bool direct;
};

// Tiles that fill the chip's 256 CUs are summed by one block each; the rest of
// the tiles, fewer than 256, share the CUs, each tile's tokens being split
// over as many blocks as there is room for, kMinSplit tokens each at least.
// Where padding falls inside the tensor every tile goes through the
// workspace, and the sum places it.  The number of CUs is the card's, and a
// constant: the splits, and with them the order of a sum and the workspace's
// size, follow from the sizes alone.
constexpr int64_t kCus = 256, kMinSplit = 256, kGrain = 128, kMaxSplits = 32;

template <class S>
Plan plan_for(bool direct, int64_t rows, int64_t cols, int64_t tokens) {
  Plan p;
  p.direct = direct;
  p.side = S::kSide;
  p.row_tiles = (rows + p.side - 1) / p.side;
  p.col_tiles = (cols + p.side - 1) / p.side;
  const int64_t tiles = p.row_tiles * p.col_tiles;
  p.whole = tiles / kCus * kCus;
  p.further = tiles - p.whole;
  p.splits = 1;
  p.tokens_per_split = std::max<int64_t>(tokens, 1);
  if (p.further > 0) {
    const int64_t most = std::max<int64_t>(1, tokens / kMinSplit);
    p.splits = std::max<int64_t>(1, std::min({most, kCus / p.further, kMaxSplits}));
    p.tokens_per_split = std::max<int64_t>(1, (tokens + p.splits * kGrain - 1) / (p.splits * kGrain)) * kGrain;
    p.splits = std::max<int64_t>(1, (tokens + p.tokens_per_split - 1) / p.tokens_per_split);
    if (p.splits == 1) {  // nothing to split
      p.whole = tiles;
      p.further = 0;
    }
  }
  p.slots = (p.direct ? 0 : p.whole) + p.further * p.splits;
  p.bytes = p.slots * p.side * p.side * 4;
  // Time in us, from what one block was measured to take: a step of an LDS
  // tile, and 8 bytes for each accumulator or workspace element at 4.7 TB/s.
  const double step = S::kSide == 256 ? 1.53 : 1.02;
  const double tile_io = (double)(p.side * p.side) * 8 / 4.7e6;
  const auto steps = [](int64_t t) { return (double)((t + S::kStep - 1) / S::kStep); };
  const double rounds = (double)((p.whole + kCus - 1) / kCus);
  p.us = rounds * (steps(tokens) * step + kCus * tile_io);
  if (p.further > 0)
    p.us += steps(p.tokens_per_split) * step + (double)(p.further * (p.splits + 1)) * tile_io + 4;
  return p;
}

// The larger tile does twice the products per byte of LDS, the smaller one
// leaves fewer CUs idle and fewer sums to the workspace.  Measured, 256 against
// 128 columns (us): 8192 tokens, 4096 x 4096: 229, 288; 16384 tokens, 1024 x
// 4096: 129, 135; 64 tokens, 4096 x 4096: 27, 34; 4000 tokens, 1024 x 4096: 57,
// 41; 4096 tokens, 2048 x 2048: 57, 42; 1024 tokens, 768 x 768: 22, 15.  The
// estimate takes the faster one in 14 of 15 sizes tried (not for 512 tokens, 8192
// x 8192: 196, 186).
Plan make_plan(const zero_layout* L, int32_t tensor, int64_t rows, int64_t cols, int64_t tokens) {
  int64_t lo, hi;
  const bool direct = make_place(L, tensor, &lo, &hi).gap == 0;
  const Plan a = plan_for<Large>(direct, rows, cols, tokens);
  const Plan b = plan_for<Small>(direct, rows, cols, tokens);
  return a.us <= b.us ? a : b;
}

int shape_ok(const zero_layout* L, int32_t tensor, int64_t O, int64_t I, int64_t tokens) {
  if (!L || O < 0 || I < 0 || tokens < 0) return ZERO_EINVAL;
  if (!tensor_ok(L, tensor)) return ZERO_ERANGE;
  if (O > ZERO_MAX_COLS || I > ZERO_MAX_COLS || tokens > ZERO_MAX_ROWS) return ZERO_ERANGE;
  if (O * I != L->numel[(size_t)tensor]) return ZERO_EINVAL;
  return ZERO_OK;
}

// The dispatch grids count work-items in 32 bits: 2^22 tiles of 512 threads.
// Any weight of up to 2^35 elements has fewer.
int plan_ok(const Plan& p) {
  return p.row_tiles * p.col_tiles > ((int64_t)1 << 22) ? ZERO_ERANGE : ZERO_OK;
}

template <class S, bool TR>
int launch(const Args& A, const Plan& p, hipStream_t s) {
  hipLaunchKernelGGL((grad_kernel<S, TR>), dim3((unsigned)(p.whole + p.further * p.splits)),
                     dim3(S::kThreads), 0, s, A);
  const int rc = launched();
  if (rc != ZERO_OK || p.slots == 0) return rc;
  const int32_t first = p.direct ? (int32_t)p.whole : 0;
  // about 2048 blocks, a power of two for each tile, 4 KB of sums each at least
  const int64_t n = p.whole + p.further - first;
  int32_t parts = S::kSide * S::kSide / 1024;
  while (parts > 1 && parts * n > 2048) parts >>= 1;
  const unsigned grid = (unsigned)(n * parts);
  if (A.out.place.gap)
    hipLaunchKernelGGL((sum_kernel<S::kSide, true>), dim3(grid), dim3(kSumThreads), 0, s, A, first,
                       parts);
  else
    hipLaunchKernelGGL((sum_kernel<S::kSide, false>), dim3(grid), dim3(kSumThreads), 0, s, A, first,
                       parts);
  return launched();
}
template <class S>
int launch(const Args& A, const Plan& p, bool tr, hipStream_t s) {
  return tr ? launch<S, true>(A, p, s) : launch<S, false>(A, p, s);
}

}  // namespace

extern "C" {

int64_t zero_linear_grad_workspace(const zero_layout* L, int32_t tensor, int32_t transposed,
                                   int64_t out_features, int64_t in_features, int64_t tokens) {
  const int rc = shape_ok(L, tensor, out_features, in_features, tokens);
  if (rc != ZERO_OK) return rc;
  if (transposed != 0 && transposed != 1) return ZERO_EINVAL;
  const Plan p = make_plan(L, tensor, transposed ? in_features : out_features,
                           transposed ? out_features : in_features, tokens);
  return plan_ok(p) == ZERO_OK ? p.bytes : ZERO_ERANGE;
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
  if (plan_ok(p) != ZERO_OK) return ZERO_ERANGE;
  if (p.bytes > 0 && (!workspace || workspace_bytes < p.bytes || ((uintptr_t)workspace & 15u)))
    return ZERO_EINVAL;
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
  A.whole = (int32_t)p.whole;
  // a row's last chunk reaches up to 7 (15) elements past its end
  const int64_t past_dy = (O + 7) / 8 * 8 - O, past_x = (I + 15) / 16 * 16 - I;
  const int64_t short_dy = (past_dy + std::max<int64_t>(dy_stride, 1) - 1) / std::max<int64_t>(dy_stride, 1);
  const int64_t short_x = (past_x + I - 1) / I;
  A.fast_tokens = tokens - std::max(short_dy, short_x);
  A.direct = p.direct;
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
  return p.side == Large::kSide ? launch<Large>(A, p, transposed != 0, stream)
                                : launch<Small>(A, p, transposed != 0, stream);
}

}  // extern "C"
