// zero_embedding_lookup and zero_embedding_grad.
//
// Page "Infra: Data Parallel" (pufanyi.com), section "Zero Redundancy
// Optimizer (ZeRO)": the updated 16-bit parameters are gathered into one flat
// buffer before the forward pass, where the lookup reads the table's rows;
// section "Naive Data Parallelism": without synchronisation a micro-batch's
// gradients are added to the rank's own sum, which is where the table's
// gradient goes.
//
// lookup: out[t] = scale * E[id_t].  A stream of 2*cols bytes in and out per
// token with whole rows, so no LDS.  16384 tokens of 8192 columns take 91 us
// (467 MB, 5.1 TB/s) with non-temporal stores, 98 with temporal ones or with
// non-temporal loads as well.
//
// gradient: dE[v] = sum over the t with id_t = v of dY[t], t ascending, so
// that the result is the same in every run.  Three launches:
//   plan   the tokens grouped by id, in ascending order within an id.  The
//          ids are dealt to slices (slice = id mod S, so that frequent
//          neighbours fall into different ones); one block per slice reads all
//          n ids, counts its own and those of lower slices, which gives its
//          place in the order without talking to other blocks, and places its
//          tokens in a second pass.  n ids are read from the L2 by S blocks:
//          12 us for 16384 ids, 6 us for 1000.  Of more ids a slice's block
//          reads its own alone, put together by two launches before it (131072
//          ids: 16 us in all, 80 without them).
//   sums   an id of up to kPiece tokens is summed and added to its row of the
//          accumulator; one with more is cut into pieces of kPiece, summed
//          apart in binary32, so that a frequent token does not keep one row
//          of threads busy alone.  Once for each distinct id, or for every row
//          of the table where the flags ask for the whole gradient (an absent
//          id's is zero).
//   join   the pieces of a long id, in order
#include <algorithm>

#include "tensor_place.hpp"

namespace {
using namespace zs;

constexpr int kThreads = 256;

// An id at any address.  Saying so matters where all lanes read the same one:
// the scalar load that the compiler then takes ignores the address's last two bits.
template <class T>
__device__ __forceinline__ T id_at(const void* ids, int64_t t) {
  typedef T any __attribute__((aligned(1)));
  return ((const any*)ids)[t];
}

// ------------------------------------------------------------------ lookup
struct LookupArgs {
  const uint16_t* params;
  const void* ids;
  void* out;
  int64_t out_stride;
  Place place;
  int64_t vocab;
  int32_t n, cols;
  FastDiv pieces;     // threads of a row
  int32_t rows_per_block;
  float scale;
};

// Columns of a thread: 16 bytes of output, so that a wave's store is one run of
// them (to binary32, 16384 rows of 4096 columns: 59 us, with 8 columns and two
// stores 32 bytes apart 97; of 8192 columns 166 and 153).
template <class OUT>
constexpr int kPerThread = 16 / (int)sizeof(OUT);

__device__ __forceinline__ void put(uint16_t* p, const float (&x)[8], int n) {
  if (n >= 8) {
    const u32x4 w = {bf16_pack2(x[0], x[1]), bf16_pack2(x[2], x[3]), bf16_pack2(x[4], x[5]),
                     bf16_pack2(x[6], x[7])};
    __builtin_nontemporal_store(w, (u32x4_a2*)p);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < n) p[k] = (uint16_t)bf16_round(x[k]);
  }
}
__device__ __forceinline__ void put(float* p, const float (&x)[4], int n) {
  if (n >= 4) {
    st4_stream(p, f32x4{x[0], x[1], x[2], x[3]});
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k < n) p[k] = x[k];
  }
}

template <class ID, class OUT, bool GAPS>
__global__ void __launch_bounds__(kThreads) lookup_kernel(const LookupArgs A) {
  constexpr int kN = kPerThread<OUT>;
  const int64_t t0 = (int64_t)blockIdx.x * A.rows_per_block;
  const uint32_t units = (uint32_t)A.rows_per_block * A.pieces.d;
  for (uint32_t u = threadIdx.x; u < units; u += kThreads) {
    const uint32_t r = fast_div(u, A.pieces);
    const int32_t c0 = (int32_t)(u - r * A.pieces.d) * kN;
    const int64_t t = t0 + r;
    if (t >= A.n) break;
    const int n = min(kN, A.cols - c0);
    const int64_t id = id_at<ID>(A.ids, t);
    float x[kN];
#pragma unroll
    for (int k = 0; k < kN; ++k) x[k] = 0.f;
    if (id >= 0 && id < A.vocab) {
      const int64_t i = id * A.cols + c0;
      int64_t at;
      if (n >= kN && place_run<GAPS>(A.place, i, kN, at)) {
        typedef uint32_t words __attribute__((ext_vector_type(kN / 2), aligned(2)));
        const words w = *(const words*)(A.params + at);
#pragma unroll
        for (int k = 0; k < kN; k += 2) x[k] = bf16_lo(w[k >> 1]), x[k + 1] = bf16_hi(w[k >> 1]);
      } else {
#pragma unroll
        for (int k = 0; k < kN; ++k)
          if (k < n) x[k] = bf16_one(A.params[place_at<GAPS>(A.place, i + k)]);
      }
#pragma unroll
      for (int k = 0; k < kN; ++k) x[k] = A.scale * x[k];
    }
    put((OUT*)A.out + t * A.out_stride + c0, x, n);
  }
}

// ------------------------------------------------------------------ plan
// One entry per place in the order.
struct Entry {
  int32_t token, row;  // token index, its id
  int32_t rel, count;  // place among the id's tokens, and how many these are
};
static_assert(sizeof(Entry) == 16, "entry");

constexpr int kPlanThreads = 1024;
constexpr int kPlanWaves = kPlanThreads / 64;
constexpr int kMaxLocal = 1024;  // ids of one slice: 16 waves x 1024 counters, 64 KiB of LDS
constexpr int kMinSlices = 256;  // one block per CU
constexpr int kBatch = 16;

struct PlanArgs {
  const void* ids;
  int32_t vocab, n, local;  // rows of the table; tokens; ids per slice
  uint32_t slice_bits;      // S = 2^slice_bits slices
  int32_t* start;           // S*local + 1 places: first place of (slice, id / S)
  Entry* order;
  // many tokens only: dealt to their slices by an earlier launch
  int32_t chunk;       // tokens of one of its blocks
  int32_t* counts;     // chunks x kMinSlices
  int32_t* slice_at;   // kMinSlices + 1 places in `dealt`
  struct Token* dealt;
};
struct Token {
  int32_t token, id;
};

// The id at t as a number below vocab, or -1 (vocab <= 2^30).
template <class ID>
__device__ __forceinline__ int32_t token_at(const PlanArgs& A, int64_t t, int64_t tz) {
  if (t >= tz) return -1;
  const ID id = id_at<ID>(A.ids, t);
  if constexpr (sizeof(ID) == 8) {
    if ((uint64_t)id >> 32) return -1;
  }
  return (uint32_t)id < (uint32_t)A.vocab ? (int32_t)id : -1;
}

// The lanes of `on` whose key of BITS bits is this lane's.
template <int BITS>
__device__ __forceinline__ uint64_t same_key(uint64_t on, int32_t key) {
  uint32_t lo = (uint32_t)on, hi = (uint32_t)(on >> 32);
#pragma unroll
  for (int b = 0; b < BITS; ++b) {
    const uint32_t x = (uint32_t)((int32_t)((uint32_t)key << (31 - b)) >> 31);
    const uint64_t ones = __ballot(x != 0u);
    lo &= ~((uint32_t)ones ^ x);
    hi &= ~((uint32_t)(ones >> 32) ^ x);
  }
  return (uint64_t)hi << 32 | lo;
}
// A place for each lane that is `on`: the key's next free ones, by lane.  The
// lanes of a few frequent keys are found one key at a time, the others by the
// keys' bits.
template <int BITS>
__device__ __forceinline__ int32_t take_place(int32_t* next, bool on, int32_t key, int lane) {
  const uint64_t me = (uint64_t)1 << lane;
  uint64_t todo = __ballot(on), same = me;
  for (int k = 0; todo && k < 3; ++k) {
    const int32_t k0 = __builtin_amdgcn_readlane(key, __ffsll((unsigned long long)todo) - 1);
    const uint64_t m = __ballot(key == k0) & todo;
    if (m & me) same = m;
    todo &= ~m;
  }
  if (todo) {
    const uint64_t m = same_key<BITS>(todo, key);
    if (todo & me) same = m;
  }
  const int lead = __ffsll((unsigned long long)same) - 1;
  int32_t p = 0;
  if (on && lane == lead) p = atomicAdd(&next[key], (int32_t)__popcll(same));
  return __shfl(p, lead, 64) + (int32_t)__popcll(same & (me - 1));
}
// The same additions where the places are not asked for: one for the lanes of
// the first lane's key, which may be most, one for each other lane.
__device__ __forceinline__ void count_keys(int32_t* cnt, bool on, int32_t key, int lane) {
  const uint64_t all = __ballot(on);
  if (!all) return;
  const int lead = __ffsll((unsigned long long)all) - 1;
  const uint64_t m = __ballot(key == __builtin_amdgcn_readlane(key, lead)) & all;
  if ((m >> lane) & 1) {
    if (lane == lead) atomicAdd(&cnt[key], (int32_t)__popcll(m));
  } else if (on) {
    atomicAdd(&cnt[key], 1);
  }
}

// Many tokens: dealt to the slices first, in order, so that a slice's block
// reads its own alone.  count_kernel counts a chunk's tokens of each slice;
// deal_kernel adds those of the chunks before its own and of the lower slices,
// and places its tokens.
constexpr int kMaxChunks = 256;
template <class ID>
__global__ void __launch_bounds__(kPlanThreads) count_kernel(const PlanArgs A) {
  __shared__ int32_t cnt[kMinSlices];
  const int tid = threadIdx.x;
  const int64_t ta = (int64_t)blockIdx.x * A.chunk, tz = min((int64_t)A.n, ta + A.chunk);
  if (tid < kMinSlices) cnt[tid] = 0;
  __syncthreads();
#pragma unroll 4
  for (int64_t t = ta + tid; t < tz; t += kPlanThreads) {
    const int32_t id = token_at<ID>(A, t, tz);
    if (id >= 0) atomicAdd(&cnt[id & (kMinSlices - 1)], 1);
  }
  __syncthreads();
  if (tid < kMinSlices) A.counts[(int64_t)blockIdx.x * kMinSlices + tid] = cnt[tid];
}

template <class ID>
__global__ void __launch_bounds__(kPlanThreads) deal_kernel(const PlanArgs A) {
  constexpr int kParts = kPlanThreads / kMinSlices;
  __shared__ int32_t cnt[kPlanWaves][kMinSlices];  // counts, later the next free place
  __shared__ int32_t part[2][kParts][kMinSlices];  // chunks before this one; all
  __shared__ int32_t wsum[kMinSlices / 64];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int s = tid % kMinSlices, q = tid / kMinSlices;
  const int64_t ca = (int64_t)blockIdx.x * A.chunk, cz = min((int64_t)A.n, ca + A.chunk);
  // a wave takes consecutive tokens (the chunk is a multiple of 1024)
  const int64_t ta = ca + (int64_t)wave * (A.chunk / kPlanWaves);
  const int64_t tz = min(cz, ta + A.chunk / kPlanWaves);
  for (int w = q; w < kPlanWaves; w += kParts) cnt[w][s] = 0;
  int32_t before = 0, all = 0;
#pragma unroll 8
  for (int c = q; c < (int)gridDim.x; c += kParts) {
    const int32_t k = A.counts[(int64_t)c * kMinSlices + s];
    all += k;
    if (c < (int)blockIdx.x) before += k;
  }
  part[0][q][s] = before;
  part[1][q][s] = all;
  __syncthreads();
  for (int64_t t = ta + lane; t < tz; t += 64) {
    const int32_t id = token_at<ID>(A, t, tz);
    if (id >= 0) atomicAdd(&cnt[wave][id & (kMinSlices - 1)], 1);
  }
  int32_t run = 0, total = 0;
  if (q == 0) {
    for (int k = 0; k < kParts; ++k) total += part[1][k][s];
    run = total;
    for (int k = 1; k < 64; k <<= 1) {
      const int32_t up = __shfl_up(run, k, 64);
      if (lane >= k) run += up;
    }
    if (lane == 63) wsum[wave] = run;
  }
  __syncthreads();
  if (q == 0) {
    for (int w = 0; w < wave; ++w) run += wsum[w];
    if (blockIdx.x == 0) {
      A.slice_at[s] = run - total;
      if (s == kMinSlices - 1) A.slice_at[kMinSlices] = run;
    }
    int32_t next = run - total;
    for (int k = 0; k < kParts; ++k) next += part[0][k][s];
    for (int w = 0; w < kPlanWaves; ++w) {
      const int32_t k = cnt[w][s];
      cnt[w][s] = next;
      next += k;
    }
  }
  __syncthreads();
  for (int64_t t0 = ta; t0 < tz; t0 += 64) {
    const int32_t id = token_at<ID>(A, t0 + lane, tz);
    const int32_t p = take_place<8>(cnt[wave], id >= 0, id & (kMinSlices - 1), lane);
    if (id >= 0) A.dealt[p] = Token{(int32_t)(t0 + lane), id};
  }
}
static_assert(kMinSlices == 1 << 8, "take_place's bits");

// DEALT: the slice's tokens come from A.dealt, none are another slice's.
template <class ID, bool DEALT>
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanArgs A) {
  __shared__ int32_t cnt[kPlanWaves][kMaxLocal];  // counts, later the next free place
  __shared__ int32_t tot[kMaxLocal];              // an id's tokens
  __shared__ int32_t first[kMaxLocal];            // its first place
  __shared__ int32_t wsum[kPlanWaves], wlow[kPlanWaves];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int32_t slice = (int32_t)blockIdx.x;
  const int32_t mask = (int32_t)((1u << A.slice_bits) - 1u);
  // each wave counts its own contiguous part of the tokens, kBatch loads at a
  // time: the readings are bound by their latency
  const int64_t na = DEALT ? A.slice_at[slice] : 0, nz = DEALT ? A.slice_at[slice + 1] : A.n;
  const int64_t per = (nz - na + kPlanThreads - 1) / kPlanThreads * 64;
  const int64_t ta = na + wave * per, tz = min(nz, ta + per);
  int32_t id[kBatch], token[kBatch];
  auto read = [&](int64_t t0) {
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int64_t t = t0 + k * 64 + lane;
      if constexpr (DEALT) {
        const Token x = t < tz ? A.dealt[t] : Token{-1, -1};
        id[k] = x.id, token[k] = x.token;
      } else {
        id[k] = token_at<ID>(A, t, tz);
      }
    }
  };
  if (ta < tz) read(ta);
  if (tid < A.local)
    for (int w = 0; w < kPlanWaves; ++w) cnt[w][tid] = 0;
  __syncthreads();
  int32_t low = 0;
  for (int64_t t0 = ta; t0 < tz; t0 += 64 * kBatch) {
    if (t0 != ta) read(t0);
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int32_t s = id[k] & mask;
      if (!DEALT && id[k] >= 0 && s < slice) ++low;
      const bool own = id[k] >= 0 && s == slice;
      if (DEALT)
        count_keys(cnt[wave], own, id[k] >> A.slice_bits, lane);
      else if (own)
        atomicAdd(&cnt[wave][id[k] >> A.slice_bits], 1);
    }
  }
  for (int k = 32; k; k >>= 1) low += __shfl_xor(low, k, 64);
  if (lane == 0) wlow[wave] = low;
  __syncthreads();
  // one id per thread (local <= kMaxLocal = kPlanThreads): its total, then
  // the running sum over the slice's ids
  int32_t base = (int32_t)na;
  for (int w = 0; w < kPlanWaves; ++w) base += wlow[w];
  int32_t mine = 0;
  if (tid < A.local)
    for (int w = 0; w < kPlanWaves; ++w) mine += cnt[w][tid];
  int32_t run = mine;
  for (int k = 1; k < 64; k <<= 1) {
    const int32_t up = __shfl_up(run, k, 64);
    if (lane >= k) run += up;
  }
  if (lane == 63) wsum[wave] = run;
  __syncthreads();
  int32_t before = base;
  for (int w = 0; w < wave; ++w) before += wsum[w];
  const int32_t at = before + run - mine;
  if (tid < A.local) {
    tot[tid] = mine;
    first[tid] = at;
    A.start[(int64_t)slice * A.local + tid] = at;
    int32_t next = at;
    for (int w = 0; w < kPlanWaves; ++w) {
      const int32_t c = cnt[w][tid];
      cnt[w][tid] = next;
      next += c;
    }
    if (slice == mask && tid == A.local - 1) A.start[((int64_t)mask + 1) * A.local] = next;
  }
  __syncthreads();
  // tokens of this slice go to their places, in order (a wave walks its
  // tokens upwards; equal ids among 64 tokens by lane)
  for (int64_t t0 = ta; t0 < tz; t0 += 64 * kBatch) {
    if (tz - ta > 64 * kBatch) read(t0);  // one batch: still in registers
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (DEALT && t0 + k * 64 >= tz) break;
      const bool own = id[k] >= 0 && (id[k] & mask) == slice;
      const int32_t loc = own ? id[k] >> A.slice_bits : -1;
      if constexpr (DEALT) {
        const int32_t p = take_place<10>(cnt[wave], own, loc, lane);
        if (own) A.order[p] = Entry{token[k], id[k], p - first[loc], tot[loc]};
        continue;
      }
      uint64_t todo = __ballot(own);
      while (todo) {
        const int lead = __ffsll((unsigned long long)todo) - 1;
        const int32_t l = __builtin_amdgcn_readlane(loc, lead);
        const uint64_t same = __ballot(loc == l);
        int32_t p0 = 0;
        if (lane == lead) p0 = atomicAdd(&cnt[wave][l], (int32_t)__popcll(same));
        p0 = __builtin_amdgcn_readlane(p0, lead);
        if (loc == l) {
          const int32_t p = p0 + __popcll(same & (((uint64_t)1 << lane) - 1));
          A.order[p] = Entry{(int32_t)(t0 + k * 64 + lane), id[k], p - first[l], tot[l]};
        }
        todo &= ~same;
      }
    }
  }
}
static_assert(kMaxLocal == 1 << 10, "take_place's bits");

// ------------------------------------------------------------------ sums
// Tokens summed by one thread without a break; more go to pieces.
constexpr int kPiece = 16;
static_assert(kPiece <= 64, "a window fits a wave");
// Tokens from which on an id's pieces are joined by blocks of 64 columns.
constexpr int kLong = 1024;

struct GradArgs {
  const void* dy;
  int64_t dy_stride;
  const int32_t* start;
  const Entry* order;
  float* partial;  // 2 * (n / kPiece + 1) rows of cols
  GradOut out;
  int64_t vocab;
  int32_t n, cols, local;
  uint32_t slice_bits;
  FastDiv pieces;  // pieces of 4 columns per row
  int32_t rows_per_block;
  uint32_t piece_blocks;
  FastDiv chunks;       // blocks of a row (or of rows_per_block rows)
  uint32_t row_blocks;  // groups of rows that the grid covers at once
  uint32_t table_rows;   // of a wave
  uint32_t window_rows;  // windows of pieces that it covers at once
  unsigned long_blocks;  // of the join, for ids of kLong tokens or more
};

// The partial row of the piece that begins at place p: among the places of a
// window of kPiece there is at most one first piece of a long id and at most
// one later piece.
__device__ __forceinline__ int64_t slot_of(int32_t p, bool first) {
  return 2 * (int64_t)(p / kPiece) + (first ? 1 : 0);
}

// Columns [c0, c0 + n) of a token, n <= 4.  FULL: n is 4 for the whole thread,
// known outside of any loop; a branch at each load would make each of them
// wait for the one before.
template <class DY, bool FULL>
__device__ __forceinline__ f32x4 dy4(const GradArgs& A, int32_t token, int32_t c0, int n) {
  const DY* p = (const DY*)A.dy + (int64_t)token * A.dy_stride + c0;
  if constexpr (FULL) {
    if constexpr (sizeof(DY) == 2) {
      const u32x2 w = __builtin_nontemporal_load((const u32x2_a2*)p);
      return f32x4{bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y)};
    } else {
      return *(const f32x4_a4*)p;
    }
  }
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (k < n) v[k] = sizeof(DY) == 2 ? bf16_one(((const uint16_t*)p)[k]) : ((const float*)p)[k];
  return v;
}

// s and N tokens, token_of(0) to token_of(m - 1) of them, in order; 1 <= m <= N.
// All loads go out before the first sum.
template <class DY, bool FULL, int N, class F>
__device__ __forceinline__ f32x4 add_tokens(const GradArgs& A, f32x4 s, F token_of, int m,
                                            int32_t c0, int n) {
  f32x4 v[N];
#pragma unroll
  for (int u = 0; u < N; ++u) v[u] = dy4<DY, FULL>(A, token_of(min(u, m - 1)), c0, n);
#pragma unroll
  for (int u = 0; u < N; ++u)
    if (u < m) s += v[u];
  return s;
}

// The sum of one id's tokens, or of one piece of them: `first` and the m - 1
// that token_of(0) and so on give, in order; 1 <= m <= kPiece.  N loads at a
// time: a kernel that streams keeps N small, for its registers.
template <class DY, bool FULL, int N, class F>
__device__ __forceinline__ f32x4 sum_tokens(const GradArgs& A, int32_t first, F token_of, int m,
                                            int32_t c0, int n) {
  f32x4 s = dy4<DY, FULL>(A, first, c0, n);
  for (int j = 0; j + 1 < m; j += N)
    s = add_tokens<DY, FULL, N>(A, s, [=](int u) { return token_of(j + u); }, min(N, m - 1 - j), c0, n);
  return s;
}
template <class DY, int N, class F>
__device__ __forceinline__ f32x4 sum_tokens(const GradArgs& A, int32_t first, F token_of, int m,
                                            int32_t c0, int n) {
  return n >= 4 ? sum_tokens<DY, true, N>(A, first, token_of, m, c0, n)
                : sum_tokens<DY, false, N>(A, first, token_of, m, c0, n);
}
// The tokens at places [p, p + m).  Five loads at a time: 134 us for the case
// at places_kernel, against 138 with two, 137 with three, 140 with eight.
template <class DY>
__device__ __forceinline__ f32x4 sum_places(const GradArgs& A, int32_t first, int32_t p, int m,
                                            int32_t c0, int n) {
  const Entry* rest = A.order + p + 1;
  return sum_tokens<DY, 5>(A, first, [=](int u) { return rest[u].token; }, m, c0, n);
}

// Columns [c0, c0 + n) of row v, n <= 4.
template <bool GAPS>
__device__ __forceinline__ void row_out(const GradArgs& A, int64_t v, int32_t c0, int n, f32x4 s) {
  const int64_t i = v * A.cols + c0;
  int64_t at;
  if (n >= 4 && place_run<GAPS>(A.out.place, i, 4, at)) {
    grad_store4(A.out, at, s);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k < n) grad_store(A.out, place_at<GAPS>(A.out.place, i + k), s[k]);
  }
}

__device__ __forceinline__ void piece_out(const GradArgs& A, int32_t p, bool first, int32_t c0,
                                          int n, f32x4 s) {
  float* to = A.partial + slot_of(p, first) * A.cols + c0;
  if (n >= 4) {
    *(f32x4_a4*)to = s;
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k < n) to[k] = s[k];
  }
}

// The first place of the window from w0 that begins a piece of a long id: the
// id's first piece, or a later one.  -1: none.  For a whole wave.
__device__ __forceinline__ int32_t piece_in_window(const GradArgs& A, int32_t total, int32_t w0,
                                                   bool first) {
  const int lane = threadIdx.x & 63;
  bool here = false;
  if (lane < kPiece && w0 + lane < total) {
    const Entry e = A.order[w0 + lane];
    here = e.count > kPiece && e.rel % kPiece == 0 && (e.rel == 0) == first;
  }
  const uint64_t found = __ballot(here);
  return found ? w0 + __ffsll((unsigned long long)found) - 1 : -1;
}

// One row per distinct id or piece, found at its first place; 4 columns per
// thread, the blocks of a row one after another.  Nearly every id of a batch
// occurs once, so the row's accumulator and its first token are requested
// together, before any of the sum.  Measured for 16384 tokens of 4096 columns
// and 12000 distinct ids (520 MB), all three kernels at 134 us (127 with what
// came later): 8 columns per thread cost 18 us more, a row's blocks spread over
// the grid 9, temporal accesses 5, pieces of 32 and 64 tokens 10 and 25.
template <class DY, bool GAPS>
__global__ void __launch_bounds__(kThreads) places_kernel(const GradArgs A) {
  const int32_t total = A.start[((int64_t)1 << A.slice_bits) * A.local];
  const uint32_t units = (uint32_t)A.rows_per_block * A.pieces.d;
  const uint32_t bx = fast_div(blockIdx.x, A.chunks);
  const uint32_t u = (blockIdx.x - bx * A.chunks.d) * kThreads + threadIdx.x;
  if (u >= units) return;
  const uint32_t r = fast_div(u, A.pieces);
  const int32_t c0 = (int32_t)(u - r * A.pieces.d) * 4;
  const int n = min(4, A.cols - c0);
  for (int64_t x = (int64_t)bx * A.rows_per_block + r; x < total;
       x += (int64_t)A.row_blocks * A.rows_per_block) {
    const Entry e = A.order[x];
    if (e.rel % kPiece != 0) continue;
    int64_t at;
    const bool vec = place_run<GAPS>(A.out.place, (int64_t)e.row * A.cols + c0, 4, at) && n >= 4;
    const bool whole = e.count <= kPiece;
    f32x4 base = {0.f, 0.f, 0.f, 0.f};
    if (vec && whole) base = grad_load4(A.out, at);
    const f32x4 s = sum_places<DY>(A, e.token, (int32_t)x, min(kPiece, e.count - e.rel), c0, n);
    if (!whole)
      piece_out(A, (int32_t)x, e.rel == 0, c0, n, s);
    else if (vec)
      grad_store4(A.out, at, s, base);
    else
      row_out<GAPS>(A, e.row, c0, n, s);
  }
}

// The same for rows of more than 124 columns: a wave takes 256 columns of kRun
// places, of which only those that begin a row or a piece cost more than their
// share of one load.  With threads for each place, those that found nothing to
// do took most of the time where ids repeat.  In runs of 4, one by one, in twos
// and in eights (us): 12000 tokens of 4096 columns and 600 ids 52, 64, 56, 50;
// 16384 tokens and 12700 ids 132, 130, 130, 133; 65536 tokens of 768 columns and
// 36600 ids 88, 98, 90, 90; 131072 tokens 128, 155, 134, 127.  Narrow rows stay
// with the kernel above: 65536 tokens of 64 columns took 28 us there, 32 here.
// The places' entries lie in the first lanes, and all lanes read them, also
// those past the row's end: a lane's registers are only sure to hold its values
// for others while it is active itself.
constexpr uint32_t kMinWide = 32;  // pieces of 4 columns
constexpr int kRun = 4;
template <class DY, bool GAPS>
__global__ void __launch_bounds__(kThreads) wide_places_kernel(const GradArgs A) {
  const int32_t total = A.start[((int64_t)1 << A.slice_bits) * A.local];
  const int lane = threadIdx.x & 63;
  const uint32_t wave = blockIdx.x * (kThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t bx = fast_div(wave, A.chunks);
  if (bx >= A.row_blocks) return;
  const int32_t c0 = (int32_t)((wave - bx * A.chunks.d) * 64 + lane) * 4;
  const int n = min(4, A.cols - c0);
  for (int64_t x0 = (int64_t)bx * kRun; x0 < total; x0 += (int64_t)A.row_blocks * kRun) {
    Entry mine = {0, 0, 1, 0};
    if (lane < kRun && x0 + lane < total) mine = A.order[x0 + lane];
    uint64_t todo = __ballot(lane < kRun && x0 + lane < total && mine.rel % kPiece == 0);
    while (todo) {
      const int i = __ffsll((unsigned long long)todo) - 1;
      todo &= todo - 1;
      const Entry e = {__builtin_amdgcn_readlane(mine.token, i), __builtin_amdgcn_readlane(mine.row, i),
                       __builtin_amdgcn_readlane(mine.rel, i), __builtin_amdgcn_readlane(mine.count, i)};
      if (n <= 0) continue;  // this lane only; it takes part in the next entry's reads
      const int32_t x = (int32_t)x0 + i;
      int64_t at;
      const bool vec = place_run<GAPS>(A.out.place, (int64_t)e.row * A.cols + c0, 4, at) && n >= 4;
      const bool whole = e.count <= kPiece;
      f32x4 base = {0.f, 0.f, 0.f, 0.f};
      if (vec && whole) base = grad_load4(A.out, at);
      const f32x4 s = sum_places<DY>(A, e.token, x, min(kPiece, e.count - e.rel), c0, n);
      if (!whole)
        piece_out(A, x, e.rel == 0, c0, n, s);
      else if (vec)
        grad_store4(A.out, at, s, base);
      else
        row_out<GAPS>(A, e.row, c0, n, s);
    }
  }
}

// Every row of the table but those of long ids, whose pieces the first
// piece_blocks blocks sum.
template <class DY, bool GAPS>
__global__ void __launch_bounds__(kThreads) table_kernel(const GradArgs A) {
  if (blockIdx.x < A.piece_blocks) {
    const int32_t total = A.start[((int64_t)1 << A.slice_bits) * A.local];
    for (int64_t b = blockIdx.x; (b >> 1) * kPiece < total; b += A.piece_blocks) {
      const bool first = (b & 1) != 0;
      const int32_t p = piece_in_window(A, total, (int32_t)(b >> 1) * kPiece, first);
      if (p < 0) continue;
      const Entry e = A.order[p];
      for (int32_t c0 = (int32_t)threadIdx.x * 4; c0 < A.cols; c0 += kThreads * 4) {
        const int n = min(4, A.cols - c0);
        piece_out(A, p, first, c0, n,
                  sum_places<DY>(A, e.token, p, min(kPiece, e.count - e.rel), c0, n));
      }
    }
    return;
  }
  const uint32_t units = (uint32_t)A.rows_per_block * A.pieces.d;
  const int64_t mask = ((int64_t)1 << A.slice_bits) - 1;
  for (int64_t b = blockIdx.x - A.piece_blocks; b * A.rows_per_block < A.vocab;
       b += gridDim.x - A.piece_blocks) {
    for (uint32_t u = threadIdx.x; u < units; u += kThreads) {
      const uint32_t r = fast_div(u, A.pieces);
      const int32_t c0 = (int32_t)(u - r * A.pieces.d) * 4;
      const int64_t v = b * A.rows_per_block + r;
      if (v >= A.vocab) break;
      const int32_t* at = A.start + (v & mask) * A.local + (v >> A.slice_bits);
      const int32_t p = at[0], count = at[1] - p;
      if (count > kPiece) continue;
      const int n = min(4, A.cols - c0);
      f32x4 s = {0.f, 0.f, 0.f, 0.f};
      if (count > 0) s = sum_places<DY>(A, A.order[p].token, p, count, c0, n);
      row_out<GAPS>(A, v, c0, n, s);
    }
  }
}

// row_out for a table that is written whole.  Where that is all (no sum read,
// no bf16) it goes through the caches.  So, and with non-temporal stores (us, of
// 16384 tokens): 128256 x 2048 218 and 228, 61036 x 4096 264 and 276, 32000 x
// 8192 308 and 329, 50257 x 768 59 and 57.
template <bool GAPS>
__device__ __forceinline__ void table_out(const GradArgs& A, int64_t v, int32_t c0, int n, f32x4 s) {
  int64_t at;
  if ((A.out.flags & (ZERO_ACC_OVERWRITE | ZERO_ACC_NO_STORE | ZERO_ACC_EMIT_BF16)) != ZERO_ACC_OVERWRITE ||
      n < 4 || !place_run<GAPS>(A.out.place, v * A.cols + c0, 4, at))
    return row_out<GAPS>(A, v, c0, n, s);
  const float m = A.out.scale;
  *(f32x4_a4*)(A.out.acc + at) = f32x4{m * s.x, m * s.y, m * s.z, m * s.w};
}

// The same for rows of more than 124 columns, 256 columns per wave (all lanes
// of which read the entries, as in wide_places_kernel): the waves
// of the first piece_blocks blocks take a window each, the others table_rows
// rows of the table, whose places and first tokens are requested together.
// 16384 tokens, 50257 x 768, overwritten: 58 us, with a thread's rows one after
// another, each with its three loads in turn, 71.
template <class DY, bool GAPS>
__global__ void __launch_bounds__(kThreads) wide_table_kernel(const GradArgs A) {
  const int lane = threadIdx.x & 63;
  const uint32_t wave = blockIdx.x * (kThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t piece_waves = A.piece_blocks * (kThreads / 64);
  const bool pieces = wave < piece_waves;
  const uint32_t wid = pieces ? wave : wave - piece_waves, bx = fast_div(wid, A.chunks);
  const int32_t c0 = (int32_t)((wid - bx * A.chunks.d) * 64 + lane) * 4;
  const int n = min(4, A.cols - c0);
  if (pieces) {
    const int32_t total = A.start[((int64_t)1 << A.slice_bits) * A.local];
    if (bx >= A.window_rows) return;
    for (int64_t w0 = (int64_t)bx * kPiece; w0 < total; w0 += (int64_t)A.window_rows * kPiece) {
      Entry mine = {0, 0, 1, 0};
      if (lane < kPiece && w0 + lane < total) mine = A.order[w0 + lane];
      uint64_t todo = __ballot(mine.count > kPiece && mine.rel % kPiece == 0);
      while (todo) {
        const int i = __ffsll((unsigned long long)todo) - 1;
        todo &= todo - 1;
        const int32_t token = __builtin_amdgcn_readlane(mine.token, i),
                      rel = __builtin_amdgcn_readlane(mine.rel, i),
                      count = __builtin_amdgcn_readlane(mine.count, i);
        const int32_t p = (int32_t)w0 + i;
        if (n > 0)
          piece_out(A, p, rel == 0, c0, n,
                    sum_places<DY>(A, token, p, min(kPiece, count - rel), c0, n));
      }
    }
    return;
  }
  if (bx >= A.row_blocks) return;
  const int64_t mask = ((int64_t)1 << A.slice_bits) - 1;
  for (int64_t v0 = (int64_t)bx * A.table_rows; v0 < A.vocab; v0 += (int64_t)A.row_blocks * A.table_rows) {
    int32_t p0 = 0, count0 = 0, token0 = 0;
    if (lane < A.table_rows && v0 + lane < A.vocab) {
      const int64_t v = v0 + lane;
      const int32_t* at = A.start + (v & mask) * A.local + (v >> A.slice_bits);
      p0 = at[0], count0 = at[1] - p0;
      if (count0 > 0) token0 = A.order[p0].token;
    }
    // waited for here, once, and not in the loop, where it would be for the
    // stores of the rows before too (65536 tokens, 32000 x 2048: 145 us, 155)
    asm volatile("" : "+v"(p0), "+v"(count0), "+v"(token0));
    const int rows = (int)min((int64_t)A.table_rows, A.vocab - v0);
    for (int i = 0; i < rows; ++i) {
      const int32_t count = __builtin_amdgcn_readlane(count0, i);
      if (count > kPiece) continue;
      if (count > 0) {
        const int32_t token = __builtin_amdgcn_readlane(token0, i), p = __builtin_amdgcn_readlane(p0, i);
        if (n > 0) table_out<GAPS>(A, v0 + i, c0, n, sum_places<DY>(A, token, p, count, c0, n));
      } else if (n > 0) {
        table_out<GAPS>(A, v0 + i, c0, n, f32x4{0.f, 0.f, 0.f, 0.f});
      }
    }
  }
}

// Four columns of the pieces of `count` tokens from place p, N loads at once.
template <int N>
__device__ __forceinline__ void join_pieces(const GradArgs& A, int32_t p, int32_t count, int32_t c0,
                                            f32x4& s) {
  const int32_t last = (count - 1) / kPiece * kPiece;
  for (int32_t j0 = 0; j0 <= last; j0 += N * kPiece) {
    f32x4 v[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {  // behind the last piece: that one again
      const int32_t j = min(j0 + k * kPiece, last);
      v[k] = *(const f32x4_a4*)(A.partial + slot_of(p + j, j == 0) * A.cols + c0);
    }
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (j0 + k * kPiece <= last) s += v[k];
  }
}

// The row of the long id that begins in the window from w0, from its pieces,
// in order.  Little data, so what counts is how many loads wait for
// one another: the window's entries are read before the number of places is
// known (behind it they hold nothing that is used), the accumulator before the
// pieces.
template <bool GAPS>
__device__ __forceinline__ void join_window(const GradArgs& A, int32_t w0, int32_t c0,
                                            int32_t total) {
  const int n = min(4, A.cols - c0), lane = threadIdx.x & 63;
  Entry e = {0, 0, 1, 0};
  if (lane < kPiece && w0 + lane < A.n) e = A.order[w0 + lane];
  const uint64_t found =
      __ballot(w0 + lane < total && e.rel == 0 && e.count > kPiece && e.count < kLong);
  if (!found) return;
  const int at = __ffsll((unsigned long long)found) - 1;
  const int32_t p = w0 + at, count = __builtin_amdgcn_readlane(e.count, at),
                row = __builtin_amdgcn_readlane(e.row, at);
  if (n <= 0) return;
  int64_t to;
  const bool vec = place_run<GAPS>(A.out.place, (int64_t)row * A.cols + c0, 4, to) && n >= 4;
  f32x4 base = {0.f, 0.f, 0.f, 0.f}, s = base;
  if (vec) base = grad_load4(A.out, to);
  if (n >= 4) {
    if (count <= 4 * kPiece)
      join_pieces<4>(A, p, count, c0, s);
    else
      join_pieces<8>(A, p, count, c0, s);
  } else {
    for (int32_t j = 0; j < count; j += kPiece) {
      const float* q = A.partial + slot_of(p + j, j == 0) * A.cols + c0;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (k < n) s[k] += q[k];
    }
  }
  if (vec)
    grad_store4(A.out, to, s, base);
  else
    row_out<GAPS>(A, row, c0, n, s);
}

// 64 columns of a row of kLong tokens or more: the block loads 64 pieces at a
// time, one wave adds them, in order, a column per lane, while the next are
// on their way (an id of 21600 tokens of 64 columns: 26 us, 350 with a thread's
// own loads of its columns).  The row is that whose places hold place `m`, a
// multiple of kLong, and no lower one.
template <bool GAPS>
__device__ __forceinline__ void join_long(const GradArgs& A, int32_t m, int32_t cb, int32_t total,
                                          float (&stage)[64][64]) {
  if (cb >= A.cols || m >= total) return;
  const Entry e = A.order[m];
  if (e.count < kLong || e.rel >= kLong) return;
  const int32_t p = m - e.rel, pieces = (e.count + kPiece - 1) / kPiece;
  const int col = threadIdx.x & 63, part = threadIdx.x >> 6;
  constexpr int kParts = kThreads / 64, kEach = 64 / kParts;
  const bool live = cb + col < A.cols;
  float v[kEach], s = 0.f;
  auto load = [&](int32_t j0) {
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      const int32_t j = j0 + k * kParts + part;
      v[k] = live && j < pieces ? A.partial[slot_of(p + j * kPiece, j == 0) * A.cols + cb + col] : 0.f;
    }
  };
  load(0);
  for (int32_t j0 = 0; j0 < pieces; j0 += 64) {
#pragma unroll
    for (int k = 0; k < kEach; ++k) stage[k * kParts + part][col] = v[k];
    __syncthreads();
    if (j0 + 64 < pieces) load(j0 + 64);
    if (part == 0) {
      const int rest = min(64, pieces - j0);
      if (rest == 64) {
#pragma unroll
        for (int k = 0; k < 64; ++k) s += stage[k][col];
      } else {
        for (int k = 0; k < rest; ++k) s += stage[k][col];
      }
    }
    __syncthreads();
  }
  if (part == 0 && live)
    grad_store(A.out, place_at<GAPS>(A.out.place, (int64_t)e.row * A.cols + cb + col), s);
}

__host__ __device__ inline bool join_narrow(const GradArgs& A) { return A.pieces.d <= 64; }

// The first long_blocks of a row of the grid are for the longest ids, kSub
// blocks of 64 columns each, the others for windows.
template <bool GAPS>
__global__ void __launch_bounds__(kThreads) join_kernel(const GradArgs A) {
  constexpr int kSub = kThreads * 4 / 64;
  __shared__ float stage[64][64];
  const int32_t total = A.start[((int64_t)1 << A.slice_bits) * A.local];
  if (blockIdx.x < A.long_blocks) {
    const int32_t cb = (int32_t)(blockIdx.y * kSub + blockIdx.x % kSub) * 64;
    for (int64_t m = (int64_t)(blockIdx.x / kSub) * kLong; m < A.n; m += (int64_t)(A.long_blocks / kSub) * kLong)
      join_long<GAPS>(A, (int32_t)m, cb, total, stage);
    return;
  }
  // a window for each wave where a wave covers a row, for each block otherwise
  const bool narrow = join_narrow(A);
  const int32_t c0 = narrow ? (threadIdx.x & 63) * 4 : (blockIdx.y * kThreads + threadIdx.x) * 4;
  const int per = narrow ? kThreads / 64 : 1;
  const int64_t step = (int64_t)(gridDim.x - A.long_blocks) * per * kPiece;
  for (int64_t w0 = ((int64_t)(blockIdx.x - A.long_blocks) * per + (narrow ? threadIdx.x >> 6 : 0)) * kPiece;
       w0 < A.n; w0 += step)
    join_window<GAPS>(A, (int32_t)w0, c0, total);
}

// ------------------------------------------------------------------ few tokens
// Up to kFew tokens, added to the accumulator alone: one launch and no
// workspace.  A block takes one token and 1024 columns; it reads every id, and
// if its token is the first with its id, lists the others in order and sums
// them as the kernels above do (pieces of kPiece, then over the pieces), for
// the same bits.  512 tokens of 1000 columns: 8 us against 14 through the plan,
// nearly all of it the launches; should all 512 have one id, 37 us against 24,
// which is why it ends there.
constexpr int kFew = 512;
template <class ID, class DY, bool GAPS>
__global__ void __launch_bounds__(kThreads)
    few_kernel(const GradArgs A, const void* ids, uint32_t column_blocks) {
  __shared__ int32_t list[kFew];
  __shared__ int32_t counts[kFew / 64];
  const uint32_t token = blockIdx.x / column_blocks;
  const int64_t id = id_at<ID>(ids, token);
  if (id < 0 || id >= A.vocab) return;
  constexpr int kRounds = kFew / kThreads;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  bool mine[kRounds];
  uint64_t same[kRounds];
  bool earlier = false;
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    const int32_t k = r * kThreads + (int32_t)threadIdx.x;
    mine[r] = k < A.n && id_at<ID>(ids, k) == id;
    earlier = earlier || (mine[r] && k < (int32_t)token);
    same[r] = __ballot(mine[r]);
    if (lane == 0) counts[r * (kThreads / 64) + wave] = (int32_t)__popcll(same[r]);
  }
  if (__syncthreads_or(earlier)) return;
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    int32_t at = 0;
    for (int w = 0; w < r * (kThreads / 64) + wave; ++w) at += counts[w];
    if (mine[r])
      list[at + __popcll(same[r] & (((uint64_t)1 << lane) - 1))] = r * kThreads + (int32_t)threadIdx.x;
  }
  int32_t count = 0;
#pragma unroll
  for (int w = 0; w < kFew / 64; ++w) count += counts[w];
  __syncthreads();
  const int32_t c0 = (int32_t)((blockIdx.x - token * column_blocks) * kThreads + threadIdx.x) * 4;
  const int n = min(4, A.cols - c0);
  if (n <= 0) return;
  int64_t at;
  const bool vec = place_run<GAPS>(A.out.place, id * A.cols + c0, 4, at) && n >= 4;
  f32x4 base = {0.f, 0.f, 0.f, 0.f}, sum = base;
  if (vec) base = grad_load4(A.out, at);
  for (int32_t p = 0; p < count; p += kPiece) {
    const int32_t m = min(kPiece, count - p);
    const int32_t* rest = list + p + 1;
    const f32x4 s =
        sum_tokens<DY, kPiece - 1>(A, list[p], [=](int u) { return rest[u]; }, m, c0, n);
    sum = p == 0 ? s : sum + s;
  }
  if (vec)
    grad_store4(A.out, at, sum, base);
  else
    row_out<GAPS>(A, id, c0, n, sum);
}

// ------------------------------------------------------------------ host
struct Plan {
  uint32_t slice_bits;
  int64_t slices, local;
  int64_t chunk, chunks;  // of the dealing launches, 0: none
  int64_t start_bytes, order_bytes, partial_bytes, bytes;
};
int64_t up16(int64_t n) { return (n + 15) & ~(int64_t)15; }

// Up to this many tokens every slice's block reads all ids; more are dealt to
// the slices first, which costs two launches, but where each id is read 3 times
// instead of 512.  The whole call, 64 columns, direct and dealt: 16384 tokens
// 17 and 23 us, 24576 25 and 23, 65536 48 and 27, 2^20 905 and 203.
// Tables of more than 2^18 rows have more than kMinSlices slices and are not
// dealt: a row more costs 65536 tokens of 128 columns 84 us instead of 38, 2^20
// tokens of 64 columns 1588 instead of 214.
constexpr int64_t kMaxDirect = 16384;
Plan make_plan(int64_t vocab, int64_t cols, int64_t n) {
  Plan p;
  p.slice_bits = 8;
  while (((int64_t)kMaxLocal << p.slice_bits) < vocab) ++p.slice_bits;
  p.slices = (int64_t)1 << p.slice_bits;
  p.local = std::max<int64_t>(1, (vocab + p.slices - 1) / p.slices);
  p.start_bytes = up16((p.slices * p.local + 1) * 4);
  p.order_bytes = n * (int64_t)sizeof(Entry);
  p.chunk = p.chunks = 0;
  int64_t dealt_bytes = 0;
  if (n > kMaxDirect && p.slices == kMinSlices) {
    p.chunk = (n + kMaxChunks * kPlanThreads - 1) / (kMaxChunks * kPlanThreads) * kPlanThreads;
    p.chunks = (n + p.chunk - 1) / p.chunk;
    dealt_bytes = (p.chunks + 1) * kMinSlices * 4 + 16 + n * (int64_t)sizeof(Token);
  }
  // the dealt tokens are read before the first partial sum is written
  p.partial_bytes = std::max(2 * (n / kPiece + 1) * cols * 4, dealt_bytes);
  p.bytes = p.start_bytes + p.order_bytes + p.partial_bytes;
  return p;
}
static_assert(kMinSlices == 1 << 8, "slice_bits starts at 8");

// Flags that ask for a value of every row of the table.
bool whole_table(uint32_t flags) { return (flags & (ZERO_ACC_OVERWRITE | ZERO_ACC_EMIT_BF16)) != 0; }

int shape_ok(const zero_layout* L, int32_t tensor, int64_t cols, int64_t n) {
  if (!L || cols < 1 || n < 0) return ZERO_EINVAL;
  if (!tensor_ok(L, tensor)) return ZERO_ERANGE;
  const int64_t numel = L->numel[(size_t)tensor];
  if (numel % cols != 0) return ZERO_EINVAL;
  if (cols > ZERO_MAX_COLS || n > ZERO_MAX_ROWS || numel / cols > ZERO_MAX_ROWS) return ZERO_ERANGE;
  return ZERO_OK;
}

// Rows of a block, 1 at least: about 4 units per thread, or 1 where that leaves
// fewer than 2048 blocks (8 for each CU).
int32_t rows_per_block(int64_t rows, int64_t units_per_row) {
  const int64_t units = std::max<int64_t>(1, units_per_row);
  const int64_t per_thread = rows * units >= (int64_t)2048 * 4 * kThreads ? 4 : 1;
  return (int32_t)std::max<int64_t>(1, per_thread * kThreads / units);
}

template <class ID, class OUT, bool GAPS>
int launch_lookup(const LookupArgs& A, hipStream_t s) {
  const int64_t blocks = ((int64_t)A.n + A.rows_per_block - 1) / A.rows_per_block;
  // the dispatch grid counts work-items in 32 bits
  constexpr int64_t kMaxBlocks = (int64_t)1 << 20;
  LookupArgs B = A;
  for (int64_t b0 = 0; b0 < blocks; b0 += kMaxBlocks) {
    const int64_t t0 = b0 * A.rows_per_block;
    B.ids = (const ID*)A.ids + t0;
    B.out = (OUT*)A.out + t0 * A.out_stride;
    B.n = (int32_t)(A.n - t0);
    hipLaunchKernelGGL((lookup_kernel<ID, OUT, GAPS>), dim3((unsigned)std::min(kMaxBlocks, blocks - b0)),
                       dim3(kThreads), 0, s, B);
    const int rc = launched();
    if (rc != ZERO_OK) return rc;
  }
  return ZERO_OK;
}
template <class ID, class OUT>
int launch_lookup(const LookupArgs& A, hipStream_t s) {
  return A.place.gap ? launch_lookup<ID, OUT, true>(A, s) : launch_lookup<ID, OUT, false>(A, s);
}

template <class DY, bool GAPS>
int launch_sums(const GradArgs& B, bool dense, hipStream_t s) {
  GradArgs A = B;
  const int64_t windows = (A.n + kPiece - 1) / kPiece;
  const bool pieces = A.n > kPiece;
  const bool wide = A.pieces.d >= kMinWide;
  constexpr int64_t kWaves = kThreads / 64, kMaxWaves = (int64_t)1 << 24;
  if (dense && wide) {
    A.chunks = make_fast_div((A.pieces.d + 63) / 64);
    const int64_t most = std::max<int64_t>(1, kMaxWaves / A.chunks.d);
    A.window_rows = pieces ? (uint32_t)std::min(windows, most) : 0u;
    A.piece_blocks = (unsigned)((A.window_rows * (int64_t)A.chunks.d + kWaves - 1) / kWaves);
    // 4 rows a wave, or fewer where that leaves less than three waves for each
    // of the 8192 that the card's 256 CUs hold at once (16384 tokens overwritten,
    // 4, 2 and 1 rows: 128256 x 2048 218, 277 and 334 us, 50257 x 768 59, 61 and
    // 70, 20000 x 256 29, 26 and 27, 5000 x 256 25, 21 and 19)
    A.table_rows = 4;
    while (A.table_rows > 1 && A.vocab * A.chunks.d < A.table_rows * (int64_t)(3 * 8192)) A.table_rows /= 2;
    A.row_blocks = (uint32_t)std::min((A.vocab + A.table_rows - 1) / A.table_rows, most);
    hipLaunchKernelGGL((wide_table_kernel<DY, GAPS>),
                       dim3(A.piece_blocks +
                            (unsigned)((A.row_blocks * (int64_t)A.chunks.d + kWaves - 1) / kWaves)),
                       dim3(kThreads), 0, s, A);
  } else if (dense) {
    A.piece_blocks = pieces ? (unsigned)std::min<int64_t>(2 * windows, 1 << 12) : 0u;
    const int64_t blocks = (A.vocab + A.rows_per_block - 1) / A.rows_per_block;
    hipLaunchKernelGGL((table_kernel<DY, GAPS>),
                       dim3(A.piece_blocks + (unsigned)std::min<int64_t>(blocks, 1 << 20)),
                       dim3(kThreads), 0, s, A);
  } else {
    const int64_t per = wide ? kRun : A.rows_per_block;
    const int64_t units = wide ? A.pieces.d : (int64_t)A.rows_per_block * A.pieces.d;
    const int each = wide ? 64 : kThreads;  // a chunk's threads
    A.chunks = make_fast_div((uint32_t)((units + each - 1) / each));
    A.row_blocks = (uint32_t)std::min<int64_t>((A.n + per - 1) / per,
                                               std::max<int64_t>(1, (1 << 22) * (kThreads / each) / A.chunks.d));
    const dim3 grid((unsigned)(((int64_t)A.row_blocks * A.chunks.d * each + kThreads - 1) / kThreads));
    if (wide)
      hipLaunchKernelGGL((wide_places_kernel<DY, GAPS>), grid, dim3(kThreads), 0, s, A);
    else
      hipLaunchKernelGGL((places_kernel<DY, GAPS>), grid, dim3(kThreads), 0, s, A);
  }
  const int rc = launched();
  if (rc != ZERO_OK || !pieces) return rc;
  const int64_t per = join_narrow(A) ? kThreads / 64 : 1;
  A.long_blocks = kThreads * 4 / 64 * (unsigned)std::min<int64_t>(A.n / kLong, 1 << 12);
  hipLaunchKernelGGL(join_kernel<GAPS>,
                     dim3(A.long_blocks + (unsigned)std::min<int64_t>((windows + per - 1) / per, 1 << 16),
                          (A.pieces.d + kThreads - 1) / kThreads),
                     dim3(kThreads), 0, s, A);
  return launched();
}

template <class ID, class DY>
int launch_few(const GradArgs& A, const void* ids, hipStream_t s) {
  const uint32_t column_blocks = (A.pieces.d + kThreads - 1) / kThreads;
  const dim3 grid((unsigned)A.n * column_blocks);  // 512 * 2^14 at most
  if (A.out.place.gap)
    hipLaunchKernelGGL((few_kernel<ID, DY, true>), grid, dim3(kThreads), 0, s, A, ids, column_blocks);
  else
    hipLaunchKernelGGL((few_kernel<ID, DY, false>), grid, dim3(kThreads), 0, s, A, ids, column_blocks);
  return launched();
}
template <class ID>
int launch_few(const GradArgs& A, const void* ids, bool f32, hipStream_t s) {
  return f32 ? launch_few<ID, float>(A, ids, s) : launch_few<ID, uint16_t>(A, ids, s);
}

template <class ID>
int launch_plan(const PlanArgs& P, const Plan& p, hipStream_t s) {
  const dim3 slices((unsigned)p.slices), chunks((unsigned)p.chunks), block(kPlanThreads);
  if (p.chunks == 0) {
    hipLaunchKernelGGL((plan_kernel<ID, false>), slices, block, 0, s, P);
  } else {
    hipLaunchKernelGGL(count_kernel<ID>, chunks, block, 0, s, P);
    hipLaunchKernelGGL(deal_kernel<ID>, chunks, block, 0, s, P);
    hipLaunchKernelGGL((plan_kernel<ID, true>), slices, block, 0, s, P);
  }
  return launched();
}

template <class DY>
int launch_grad(const GradArgs& A, bool dense, hipStream_t s) {
  return A.out.place.gap ? launch_sums<DY, true>(A, dense, s) : launch_sums<DY, false>(A, dense, s);
}

}  // namespace

extern "C" {

int zero_embedding_lookup(const zero_layout* L, int32_t tensor, int64_t cols,
                          const uint16_t* params_flat, const void* ids, int32_t id_bytes,
                          int64_t n_ids, float scale, void* out, int64_t out_stride,
                          int32_t out_dtype, hipStream_t stream) {
  const int rc = shape_ok(L, tensor, cols, n_ids);
  if (rc != ZERO_OK) return rc;
  if ((id_bytes != 4 && id_bytes != 8) || (out_dtype != ZERO_DTYPE_BF16 && out_dtype != ZERO_DTYPE_F32))
    return ZERO_EINVAL;
  if (!(scale - scale == 0.0f)) return ZERO_EINVAL;
  if (n_ids == 0) return ZERO_OK;
  const int64_t numel = L->numel[(size_t)tensor];
  if (!ids || !out || (numel > 0 && !params_flat) || out_stride < cols) return ZERO_EINVAL;
  if (out_stride > ZERO_MAX_STRIDE) return ZERO_ERANGE;
  LookupArgs A;
  int64_t lo, hi;
  A.place = make_place(L, tensor, &lo, &hi);
  const Bytes outs[] = {rows_of(out, n_ids, cols, out_stride, out_dtype == ZERO_DTYPE_F32 ? 4 : 2)};
  const Bytes ins[] = {Bytes{params_flat ? params_flat + lo : nullptr, 2 * (hi - lo)},
                       Bytes{ids, n_ids * id_bytes}};
  if (any_overlap(outs, ins)) return ZERO_EOVERLAP;
  if (hip_error_pending()) return ZERO_EHIP;
  A.params = params_flat;
  A.ids = ids;
  A.out = out;
  A.out_stride = out_stride;
  A.vocab = numel / cols;
  A.n = (int32_t)n_ids;
  A.cols = (int32_t)cols;
  const int64_t per = out_dtype == ZERO_DTYPE_F32 ? kPerThread<float> : kPerThread<uint16_t>;
  A.pieces = make_fast_div((uint32_t)((cols + per - 1) / per));
  A.rows_per_block = rows_per_block(n_ids, A.pieces.d);
  A.scale = scale;
  if (id_bytes == 4)
    return out_dtype == ZERO_DTYPE_F32 ? launch_lookup<int32_t, float>(A, stream)
                                       : launch_lookup<int32_t, uint16_t>(A, stream);
  return out_dtype == ZERO_DTYPE_F32 ? launch_lookup<int64_t, float>(A, stream)
                                     : launch_lookup<int64_t, uint16_t>(A, stream);
}

int64_t zero_embedding_grad_workspace(const zero_layout* L, int32_t tensor, int64_t cols,
                                      int64_t n_ids, uint32_t flags) {
  const int rc = shape_ok(L, tensor, cols, n_ids);
  if (rc != ZERO_OK) return rc;
  if (n_ids <= kFew && !whole_table(flags)) return 0;
  return make_plan(L->numel[(size_t)tensor] / cols, cols, n_ids).bytes;
}

int zero_embedding_grad(const zero_layout* L, int32_t tensor, int64_t cols, const void* ids,
                        int32_t id_bytes, int64_t n_ids, const void* dy, int64_t dy_stride,
                        int32_t dy_dtype, float scale, uint32_t flags, float* acc_flat,
                        uint16_t* bf16_flat, void* workspace, int64_t workspace_bytes,
                        hipStream_t stream) {
  int rc = shape_ok(L, tensor, cols, n_ids);
  if (rc != ZERO_OK) return rc;
  if ((id_bytes != 4 && id_bytes != 8) || (dy_dtype != ZERO_DTYPE_BF16 && dy_dtype != ZERO_DTYPE_F32))
    return ZERO_EINVAL;
  const int64_t numel = L->numel[(size_t)tensor];
  rc = grad_out_ok(flags, scale, acc_flat, bf16_flat, numel);
  if (rc != ZERO_OK) return rc;
  const bool dense = whole_table(flags), few = n_ids <= kFew && !dense;
  if (numel == 0 || (n_ids == 0 && !dense)) return ZERO_OK;
  if (n_ids > 0 && (!ids || !dy || dy_stride < cols)) return ZERO_EINVAL;
  if (dy_stride > ZERO_MAX_STRIDE) return ZERO_ERANGE;
  const Plan p = make_plan(numel / cols, cols, n_ids);
  const int64_t need = few ? 0 : p.bytes;
  if (need > 0 && (!workspace || workspace_bytes < need || ((uintptr_t)workspace & 15u)))
    return ZERO_EINVAL;
  GradArgs A;
  int64_t lo, hi;
  A.out.place = make_place(L, tensor, &lo, &hi);
  const Bytes outs[] = {Bytes{acc_used(flags) ? acc_flat + lo : nullptr, 4 * (hi - lo)},
                        Bytes{(flags & ZERO_ACC_EMIT_BF16) ? bf16_flat + lo : nullptr, 2 * (hi - lo)},
                        Bytes{workspace, need}};
  const Bytes ins[] = {Bytes{ids, n_ids * id_bytes},
                       rows_of(dy, n_ids, cols, dy_stride, dy_dtype == ZERO_DTYPE_F32 ? 4 : 2)};
  if (any_overlap(outs, ins)) return ZERO_EOVERLAP;
  if (hip_error_pending()) return ZERO_EHIP;

  A.dy = dy;
  A.dy_stride = dy_stride;
  A.out.acc = acc_flat;
  A.out.out = bf16_flat;
  A.out.scale = scale;
  A.out.flags = flags;
  A.vocab = numel / cols;
  A.n = (int32_t)n_ids;
  A.cols = (int32_t)cols;
  A.pieces = make_fast_div((uint32_t)((cols + 3) / 4));
  A.rows_per_block = rows_per_block(dense ? A.vocab : n_ids, A.pieces.d);
  if (few)
    return id_bytes == 4 ? launch_few<int32_t>(A, ids, dy_dtype == ZERO_DTYPE_F32, stream)
                         : launch_few<int64_t>(A, ids, dy_dtype == ZERO_DTYPE_F32, stream);

  PlanArgs P;
  P.ids = ids;
  P.vocab = (int32_t)(numel / cols);
  P.n = (int32_t)n_ids;
  P.local = (int32_t)p.local;
  P.slice_bits = p.slice_bits;
  P.start = (int32_t*)workspace;
  P.order = (Entry*)((char*)workspace + p.start_bytes);
  P.chunk = (int32_t)p.chunk;
  P.counts = (int32_t*)((char*)workspace + p.start_bytes + p.order_bytes);
  P.slice_at = P.counts + p.chunks * kMinSlices;
  P.dealt = (Token*)(P.slice_at + kMinSlices + 4);
  rc = id_bytes == 4 ? launch_plan<int32_t>(P, p, stream) : launch_plan<int64_t>(P, p, stream);
  if (rc != ZERO_OK) return rc;

  A.start = P.start;
  A.order = P.order;
  A.partial = (float*)((char*)workspace + p.start_bytes + p.order_bytes);
  A.local = P.local;
  A.slice_bits = P.slice_bits;
  return dy_dtype == ZERO_DTYPE_F32 ? launch_grad<float>(A, dense, stream)
                                    : launch_grad<uint16_t>(A, dense, stream);
}

}  // extern "C"
