// zero_shard_step_moments8, zero_moments8_pack and zero_moments8_unpack.
//
// Page "Infra: Data Parallel" (pufanyi.com), section "Zero Redundancy
// Optimizer (ZeRO)": the optimizer's state is what a rank holds most of, 12
// bytes a parameter (master weight and two moments in binary32).  With a code
// of 8 bits for each moment it is 6, and the step moves 2*N_d + 14 bytes an
// element instead of 2*N_d + 26 (and two scale bytes for 128 elements).
//
//   g = sum over ranks of G_q / N_d;  m' = B1*m + C1*g;  v' = B2*v + C2*g*g
//   th' = a_wd*th - s * m' / (sqrt(v')*rho + E)
//
// binary32 with every operation rounded, the arithmetic of zero_shard_step,
// on the values that the codes stand for; th' uses m' and v' before they are
// rounded to codes again.
//
// One pass: a wave takes 512 consecutive elements of a bucket's slice, each
// lane two pieces of 4, so that every load and store of a wave covers
// consecutive bytes; the 128 elements of a block are 32 lanes, whose largest
// magnitudes meet in registers.  Vectors go to any address, so a slice may
// begin anywhere.
#include <algorithm>

#include "adamw.hpp"
#include "layout.hpp"
#include "moments8.hpp"

namespace {
using namespace zs;

constexpr int kUnit = 512;  // elements of a wave
constexpr int kThreads = 256;
constexpr int64_t kCus = 256;

// Where the units of a launch lie: two runs of equal buckets (the full ones
// and the last), or a table of slices that follow each other in the shard.
struct Run {
  int64_t shard, flat, scale, len, stride, blocks;  // of its first bucket; len: a slice's elements
  FastDiv units;                                    // of a bucket
};
struct Runs {
  uint32_t total, first1;  // units; the second run's first one
  Run run[2];
};
template <int N>
struct Table {
  uint32_t total;
  int32_t count;
  uint32_t first[N + 1];
  int64_t shard[N + 1], flat[N], scale[N];
};
struct Spot {
  int64_t i, f, s;  // first element in the shard and in a flat buffer, first scale byte
  int n;            // elements, kUnit or less
};

__device__ __forceinline__ Spot spot(const Runs& g, uint32_t u) {
  const bool second = u >= g.first1;
  const Run& r = g.run[second ? 1 : 0];
  const uint32_t v = second ? u - g.first1 : u;
  const uint32_t b = fast_div(v, r.units);
  const int64_t e = (int64_t)(v - b * r.units.d) * kUnit;
  return Spot{r.shard + b * r.len + e, r.flat + b * r.stride + e, r.scale + b * r.blocks + e / kMomentBlock,
              (int)min((int64_t)kUnit, r.len - e)};
}
template <int N>
__device__ __forceinline__ Spot spot(const Table<N>& g, uint32_t u) {
  int lo = 0, hi = g.count;  // first[lo] <= u < first[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (g.first[mid] <= u) lo = mid;
    else hi = mid;
  }
  const int64_t e = (int64_t)(u - g.first[lo]) * kUnit;
  return Spot{g.shard[lo] + e, g.flat[lo] + e, g.scale[lo] + e / kMomentBlock,
              (int)min((int64_t)kUnit, g.shard[lo + 1] - g.shard[lo] - e)};
}

struct Codes {
  uint8_t *m, *me, *v, *ve;
};

template <int NP>
struct StepArgs {
  const void* g[NP];
  float* master;
  uint16_t* pout;
  Codes q;
  Scalars k;
  Random rnd;
  float nd_f, inv_nd;
  int32_t nd, pow2, flat_grad, slot_out;
};
// Rank counts of their own; 0: any.
constexpr int pointers(int nd) { return nd > 0 ? nd : ZERO_MAX_ND; }
// Slices of a table launch, within 4 KB of kernel arguments.
constexpr int table_size(int nd) { return nd == 0 ? 56 : nd >= 64 ? 108 : 120; }

// 4 consecutive values at any address, `cnt` of them real (4: a whole piece).
__device__ __forceinline__ f32x4 get4(const float* p, int cnt) {
  if (cnt >= 4) return ld4_stream(p);
  f32x4 x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int k = 0; k < 3; ++k)
    if (k < cnt) x[k] = p[k];
  return x;
}
__device__ __forceinline__ void put4(float* p, f32x4 x, int cnt) {
  if (cnt >= 4) {
    st4_stream(p, x);
    return;
  }
#pragma unroll
  for (int k = 0; k < 3; ++k)
    if (k < cnt) p[k] = x[k];
}
__device__ __forceinline__ f32x4 get4(const uint16_t* p, int cnt) {
  u32x2 w = {0u, 0u};
  if (cnt >= 4) {
    w = __builtin_nontemporal_load((const u32x2_a2*)p);
  } else {
#pragma unroll
    for (int k = 0; k < 3; ++k)
      if (k < cnt) w[k >> 1] |= (uint32_t)p[k] << (16 * (k & 1));
  }
  return f32x4{bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y)};
}
__device__ __forceinline__ void put4(uint16_t* p, f32x4 x, int cnt) {
  if (cnt >= 4) {
    __builtin_nontemporal_store(u32x2{bf16_pack2(x.x, x.y), bf16_pack2(x.z, x.w)}, (u32x2_a2*)p);
    return;
  }
#pragma unroll
  for (int k = 0; k < 3; ++k)
    if (k < cnt) p[k] = (uint16_t)bf16_round(x[k]);
}
typedef uint32_t u32_a1 __attribute__((aligned(1)));
__device__ __forceinline__ uint32_t get_codes(const uint8_t* p, int cnt) {
  if (cnt >= 4) return __builtin_nontemporal_load((const u32_a1*)p);
  uint32_t w = 0u;
#pragma unroll
  for (int k = 0; k < 3; ++k)
    if (k < cnt) w |= (uint32_t)p[k] << (8 * k);
  return w;
}
__device__ __forceinline__ void put_codes(uint8_t* p, uint32_t w, int cnt) {
  if (cnt >= 4) {
    __builtin_nontemporal_store(w, (u32_a1*)p);
    return;
  }
#pragma unroll
  for (int k = 0; k < 3; ++k)
    if (k < cnt) p[k] = (uint8_t)(w >> (8 * k));
}

__device__ __forceinline__ f32x4 m8_values(uint32_t w, uint32_t e) {
  const float s = act8_scale(e);
  const f32x2 a = act8_f32<false>(w, s), b = act8_f32<true>(w, s);
  return f32x4{a.x, a.y, b.x, b.y};
}
__device__ __forceinline__ f32x4 v8_values(uint32_t w, uint32_t e) {
  const float s = act8_scale(e);
  return f32x4{v8_value(w & 255u, s), v8_value((w >> 8) & 255u, s), v8_value((w >> 16) & 255u, s),
               v8_value(w >> 24, s)};
}

// A block's codes and scales, 4 elements a lane (32 lanes together); s: its
// scale byte's place.  Values past the slice's end are zeros here.
template <class R>
__device__ __forceinline__ void put_moments(const Codes& q, int64_t i, int64_t s, f32x4 m, f32x4 v,
                                            const R (&r)[4], int lane, int cnt) {
  uint32_t am = 0u, av = 0u;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    am = max(am, finite_mag(m[k]));
    av = max(av, finite_mag(v[k]));
  }
  const uint32_t em = act8_byte(max32(am)), ev = v8_byte(max32(av));
  const float im = act8_inv(em), iv = act8_inv(ev);
  uint32_t wm = 0u, wv = 0u;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    wm |= m8_code(m[k], im, r[k]) << (8 * k);
    wv |= v8_code(v[k], iv, r[k]) << (8 * k);
  }
  put_codes(q.m + i, wm, cnt);
  put_codes(q.v + i, wv, cnt);
  if ((lane & 31) == 0 && cnt > 0) {
    q.me[s] = (uint8_t)em;
    q.ve[s] = (uint8_t)ev;
  }
}

template <class T, int ND, class Args>
__device__ __forceinline__ void reduce(const Args& A, const int64_t (&at)[2], const int (&cnt)[2], f32x4 (&a)[2]) {
  const T* p0 = (const T*)A.g[0];
#pragma unroll
  for (int h = 0; h < 2; ++h) a[h] = get4(p0 + at[h], cnt[h]);
  if constexpr (ND > 0) {
    constexpr int kGroup = ND < 9 ? ND : 8;
#pragma unroll
    for (int q0 = 1; q0 < ND; q0 += kGroup) {
      f32x4 w[kGroup][2];
#pragma unroll
      for (int u = 0; u < kGroup; ++u)
        if (q0 + u < ND)
#pragma unroll
          for (int h = 0; h < 2; ++h) w[u][h] = get4((const T*)A.g[q0 + u] + at[h], cnt[h]);
#pragma unroll
      for (int u = 0; u < kGroup; ++u)
        if (q0 + u < ND)
#pragma unroll
          for (int h = 0; h < 2; ++h) a[h] = a[h] + w[u][h];
    }
  } else {
#pragma unroll 4
    for (int q = 1; q < A.nd; ++q)
#pragma unroll
      for (int h = 0; h < 2; ++h) a[h] = a[h] + get4((const T*)A.g[q] + at[h], cnt[h]);
  }
}

template <class T, int ND, class Args>
__device__ __forceinline__ void step_unit(const Args& A, const Spot& x, const int (&cnt)[2], int lane) {
  int64_t i[2], g[2], o[2], s[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t e = 256 * h + 4 * lane;
    i[h] = x.i + e;
    g[h] = (A.flat_grad ? x.f : x.i) + e;
    o[h] = (A.slot_out ? x.f : x.i) + e;
    s[h] = x.s + 2 * h + (lane >> 5);
  }
  f32x4 th[2];
  uint32_t wm[2], wv[2], em[2], ev[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    th[h] = get4(A.master + i[h], cnt[h]);
    wm[h] = get_codes(A.q.m + i[h], cnt[h]);
    wv[h] = get_codes(A.q.v + i[h], cnt[h]);
    em[h] = cnt[h] > 0 ? A.q.me[s[h]] : 0u;
    ev[h] = cnt[h] > 0 ? A.q.ve[s[h]] : 0u;
  }
  f32x4 a[2];
  reduce<T, ND>(A, g, cnt, a);
  uint32_t seed = random_seed(A.rnd, i[0]);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    f32x4 m = m8_values(wm[h], em[h]), v = v8_values(wv[h], ev[h]);
    AtRandom r[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float gk = (ND > 0 && (ND & (ND - 1)) == 0) || A.pow2 ? a[h][k] * A.inv_nd : a[h][k] / A.nd_f;
      float t = th[h][k], mk = m[k], vk = v[k];
      adamw(gk, t, mk, vk, A.k);
      th[h][k] = t;
      // elements past the end count for nothing
      m[k] = k < cnt[h] ? mk : 0.f;
      v[k] = k < cnt[h] ? vk : 0.f;
      // the product's lower half wraps with the index's
      const int64_t j = x.i + 256 * h + 4 * lane + k;
      const bool wrapped = (uint32_t)j < (uint32_t)i[0];
      r[k].h = random_bits(A.rnd, seed + (uint32_t)(256 * h + k) * kMulLow + (wrapped ? kMulHigh : 0u));
    }
    put4(A.master + i[h], th[h], cnt[h]);
    put4(A.pout + o[h], th[h], cnt[h]);
    put_moments(A.q, i[h], s[h], m, v, r, lane, cnt[h]);
  }
}

// HBM bounds it: 262M elements of 30 bytes at N_d = 8 take 1.52 ms, 5.2 TB/s (a
// copy reached 4.6 to 4.8); without the update or the hash, for timing, it took
// the same.  Other counts of ranks (TB/s; bf16, binary32 contributions): 2 4.8, 5.2;
// 4 5.2, 4.8; 6, by the loop of any count, 4.1, 4.1; 16 5.0, 5.1; 32 5.1, 5.3; 64
// 2.5, 5.4: the loads of 64 ranks move far ahead, 412 registers, so one wave a SIMD
// (512 and 233 spilled of binary32).  Slices that begin anywhere, vectors at odd
// addresses: 3.7 to 4.2 (bf16, 4 to 16 ranks).
template <class T, int ND, class Geo>
__global__ void __launch_bounds__(kThreads) step8_kernel(const StepArgs<pointers(ND)> A, const Geo G) {
  const int lane = threadIdx.x & 63;
  const uint32_t waves = gridDim.x * (kThreads / 64);
  uint32_t u = __builtin_amdgcn_readfirstlane(blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6));
  for (; u < G.total; u += waves) {
    const Spot x = spot(G, u);
    if (x.n == kUnit) {
      const int cnt[2] = {4, 4};
      step_unit<T, ND>(A, x, cnt, lane);
    } else {
      const int cnt[2] = {min(max(x.n - 4 * lane, 0), 4), min(max(x.n - 256 - 4 * lane, 0), 4)};
      step_unit<T, ND>(A, x, cnt, lane);
    }
  }
}

// Conversion of binary32 moments and back, 10 bytes an element.  Measured (2^28
// elements): to 8 bits 0.53 ms, 5.1 TB/s; back 0.50 ms, 5.3 TB/s.
struct ConvertArgs {
  float *m, *v;
  Codes q;
};
template <bool PACK, class Geo>
__global__ void __launch_bounds__(kThreads) convert_kernel(const ConvertArgs A, const Geo G) {
  const int lane = threadIdx.x & 63;
  const uint32_t waves = gridDim.x * (kThreads / 64);
  uint32_t u = __builtin_amdgcn_readfirstlane(blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6));
  for (; u < G.total; u += waves) {
    const Spot x = spot(G, u);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t i = x.i + 256 * h + 4 * lane, s = x.s + 2 * h + (lane >> 5);
      const int cnt = min(max(x.n - 256 * h - 4 * lane, 0), 4);
      if constexpr (PACK) {
        f32x4 m = get4(A.m + i, cnt), v = get4(A.v + i, cnt);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = v[k] < 0.f ? 0.f : v[k];
        const ToNearest r[4] = {};
        put_moments(A.q, i, s, m, v, r, lane, cnt);
      } else {
        const uint32_t wm = get_codes(A.q.m + i, cnt), wv = get_codes(A.q.v + i, cnt);
        const uint32_t em = cnt > 0 ? A.q.me[s] : 0u, ev = cnt > 0 ? A.q.ve[s] : 0u;
        put4(A.m + i, m8_values(wm, em), cnt);
        put4(A.v + i, v8_values(wv, ev), cnt);
      }
    }
  }
}

// ------------------------------------------------------------------ host
int64_t blocks_of(int64_t n) { return (n + kMomentBlock - 1) / kMomentBlock; }
int64_t units_of(int64_t n) { return (n + kUnit - 1) / kUnit; }

// Calls f(geometry) for launches that cover buckets [b0, b1), which hold at
// least one element.  N: slices of a table launch.
template <int N, class F>
int each_launch(const zero_layout* L, int64_t b0, int64_t b1, F f) {
  constexpr int64_t kMost = (int64_t)1 << 30;  // units of a launch
  const int64_t r = L->rank;
  if (L->fixed()) {
    Runs G{};
    const int64_t full = std::min(b1, L->nb - 1) - std::min(b0, L->nb - 1);
    const bool last = b1 == L->nb;
    const int64_t uf = full > 0 ? units_of(L->s_full) : 0, ul = last ? units_of(L->s_last) : 0;
    // int64 sizes of 2^63 elements do not occur; units of 2^30 are 2^39 elements
    if (uf > kMost || ul > kMost || full * uf + ul > kMost) return ZERO_ERANGE;
    G.first1 = (uint32_t)(full * uf);
    G.total = (uint32_t)(full * uf + ul);
    G.run[0] = Run{b0 * L->s_full, b0 * L->p_full + r * L->s_full, b0 * blocks_of(L->s_full), L->s_full,
                   L->p_full, blocks_of(L->s_full), make_fast_div((uint32_t)std::max<int64_t>(1, uf))};
    const int64_t n = L->nb - 1;
    G.run[1] = Run{n * L->s_full, n * L->p_full + r * L->s_last, n * blocks_of(L->s_full), L->s_last,
                   L->p_last, blocks_of(L->s_last), make_fast_div((uint32_t)std::max<int64_t>(1, ul))};
    return f(G);
  }
  Table<N> T;
  T.total = 0;
  T.count = 0;
  int64_t scale = 0;
  for (int64_t b = 0; b < b0; ++b) scale += blocks_of(L->bucket_slice(b));
  for (int64_t b = b0; b < b1; ++b)
    if (units_of(L->bucket_slice(b)) > kMost) return ZERO_ERANGE;
  for (int64_t b = b0; b < b1; ++b) {
    const int64_t n = L->bucket_slice(b), units = units_of(n);
    if (n == 0) continue;
    if (T.count == N || T.total + units > kMost) {
      const int rc = f(T);
      if (rc != ZERO_OK) return rc;
      T.count = 0;
      T.total = 0;
    }
    const int k = T.count++;
    T.first[k] = T.total;
    T.shard[k] = L->bucket_shard_off(b);
    T.flat[k] = L->bucket_padded_off(b) + r * n;
    T.scale[k] = scale;
    T.total += (uint32_t)units;
    T.first[k + 1] = T.total;
    T.shard[k + 1] = T.shard[k] + n;
    scale += blocks_of(n);
  }
  return T.count > 0 ? f(T) : ZERO_OK;
}

unsigned grid_for(uint32_t units, int64_t blocks_per_cu) {
  const int64_t need = (units + kThreads / 64 - 1) / (kThreads / 64);
  return (unsigned)std::max<int64_t>(1, std::min(need, blocks_per_cu * kCus));
}

// Waves a CU, four to a block: few that each have 24 loads in flight.  Measured
// (us, 262M elements, N_d = 8): the step with 4 waves 1618, 8 1520, 16 1606 to
// 1660; the next unit's loads requested before this one's stores 1525.
constexpr int64_t kStepBlocks = 2, kConvertBlocks = 5;

struct Call {
  const void* const* g;
  float* master;
  uint16_t* pout;
  Codes q;
  Scalars k;
  Random rnd;
  bool flat_grad, slot_out;
};

template <class T, int ND>
int launch_step(const zero_layout* L, int64_t b0, int64_t b1, const Call& c, hipStream_t s) {
  StepArgs<pointers(ND)> A;
  const int32_t nd = L->n_d;
  for (int32_t q = 0; q < pointers(ND); ++q) A.g[q] = q < nd ? c.g[q] : nullptr;
  A.master = c.master;
  A.pout = c.pout;
  A.q = c.q;
  A.k = c.k;
  A.rnd = c.rnd;
  A.nd = nd;
  A.nd_f = (float)nd;
  A.inv_nd = 1.0f / (float)nd;
  A.pow2 = (nd & (nd - 1)) == 0;
  A.flat_grad = c.flat_grad;
  A.slot_out = c.slot_out;
  return each_launch<table_size(ND)>(L, b0, b1, [&](const auto& G) {
    using Geo = std::decay_t<decltype(G)>;
    static_assert(sizeof(A) + sizeof(Geo) + 16 <= 4096, "kernel arguments");
    hipLaunchKernelGGL((step8_kernel<T, ND, Geo>), dim3(grid_for(G.total, kStepBlocks)), dim3(kThreads), 0, s, A, G);
    return launched();
  });
}
template <class T>
int launch_step(const zero_layout* L, int64_t b0, int64_t b1, const Call& c, hipStream_t s) {
  switch (L->n_d) {
    case 1: return launch_step<T, 1>(L, b0, b1, c, s);
    case 2: return launch_step<T, 2>(L, b0, b1, c, s);
    case 4: return launch_step<T, 4>(L, b0, b1, c, s);
    case 8: return launch_step<T, 8>(L, b0, b1, c, s);
    case 16: return launch_step<T, 16>(L, b0, b1, c, s);
    case 32: return launch_step<T, 32>(L, b0, b1, c, s);
    case 64: return launch_step<T, 64>(L, b0, b1, c, s);
    default: return launch_step<T, 0>(L, b0, b1, c, s);
  }
}

template <bool PACK>
int convert(const zero_layout* L, float* m, float* v, const Codes& q, hipStream_t s) {
  if (!L) return ZERO_EINVAL;
  const int64_t S = L->S, nb = zero_layout_moment_blocks(L);
  if (S == 0) return ZERO_OK;
  if (!m || !v || !q.m || !q.me || !q.v || !q.ve) return ZERO_EINVAL;
  const Bytes codes[] = {Bytes{q.m, S}, Bytes{q.me, nb}, Bytes{q.v, S}, Bytes{q.ve, nb}};
  const Bytes reals[] = {Bytes{m, 4 * S}, Bytes{v, 4 * S}};
  if (PACK ? any_overlap(codes, reals) : any_overlap(reals, codes)) return ZERO_EOVERLAP;
  if (hip_error_pending()) return ZERO_EHIP;
  const ConvertArgs A{m, v, q};
  return each_launch<120>(L, 0, L->nb, [&](const auto& G) {
    using Geo = std::decay_t<decltype(G)>;
    hipLaunchKernelGGL((convert_kernel<PACK, Geo>), dim3(grid_for(G.total, kConvertBlocks)), dim3(kThreads), 0, s, A,
                       G);
    return launched();
  });
}

}  // namespace

extern "C" {

int64_t zero_layout_moment_blocks(const zero_layout* L) {
  if (!L) return -1;
  if (L->S == 0) return 0;
  if (L->fixed()) return (L->nb - 1) * blocks_of(L->s_full) + blocks_of(L->s_last);
  int64_t n = 0;
  for (int64_t b = 0; b < L->nb; ++b) n += blocks_of(L->bucket_slice(b));
  return n;
}

int zero_shard_step_moments8(const zero_layout* L, const zero_adamw* hp, int64_t t, int64_t bucket_begin,
                             int64_t bucket_end, const void* const* rank_grads, int32_t grad_dtype,
                             int32_t grad_layout, float* master, uint8_t* m_codes, uint8_t* m_scales,
                             uint8_t* v_codes, uint8_t* v_scales, uint16_t* param_out, int32_t out_mode,
                             uint64_t seed, hipStream_t stream) {
  if (!L || !hp || !rank_grads || t < 1 || !hp_ok(*hp)) return ZERO_EINVAL;
  if (grad_dtype != ZERO_DTYPE_BF16 && grad_dtype != ZERO_DTYPE_F32) return ZERO_EINVAL;
  if (grad_layout != ZERO_GRAD_COMPACT && grad_layout != ZERO_GRAD_FLAT) return ZERO_EINVAL;
  if (out_mode != ZERO_OUT_AG_SLOT && out_mode != ZERO_OUT_SHARD) return ZERO_EINVAL;
  if (bucket_begin < 0 || bucket_end > L->nb || bucket_begin > bucket_end) return ZERO_ERANGE;
  if (L->S == 0 || bucket_begin == bucket_end) return ZERO_OK;
  if (!master || !m_codes || !m_scales || !v_codes || !v_scales || !param_out) return ZERO_EINVAL;
  const int64_t S = L->S, nb = zero_layout_moment_blocks(L);
  const int64_t n_in = (grad_layout == ZERO_GRAD_FLAT ? L->P : S) * (grad_dtype == ZERO_DTYPE_F32 ? 4 : 2);
  for (int32_t q = 0; q < L->n_d; ++q)
    if (!rank_grads[q]) return ZERO_EINVAL;
  const Bytes outs[] = {Bytes{master, 4 * S}, Bytes{m_codes, S}, Bytes{m_scales, nb}, Bytes{v_codes, S},
                        Bytes{v_scales, nb},
                        Bytes{param_out, 2 * (out_mode == ZERO_OUT_AG_SLOT ? L->P : S)}};
  for (int32_t q = 0; q < L->n_d; ++q) {
    const Bytes in[] = {Bytes{rank_grads[q], n_in}};
    if (any_overlap(outs, in)) return ZERO_EOVERLAP;
  }
  if (hip_error_pending()) return ZERO_EHIP;
  const Call c{rank_grads, master, param_out, Codes{m_codes, m_scales, v_codes, v_scales}, make_scalars(*hp, t),
               random_of(seed, t), grad_layout == ZERO_GRAD_FLAT, out_mode == ZERO_OUT_AG_SLOT};
  return grad_dtype == ZERO_DTYPE_F32 ? launch_step<float>(L, bucket_begin, bucket_end, c, stream)
                                      : launch_step<uint16_t>(L, bucket_begin, bucket_end, c, stream);
}

int zero_moments8_pack(const zero_layout* L, const float* exp_avg, const float* exp_avg_sq, uint8_t* m_codes,
                       uint8_t* m_scales, uint8_t* v_codes, uint8_t* v_scales, hipStream_t stream) {
  return convert<true>(L, const_cast<float*>(exp_avg), const_cast<float*>(exp_avg_sq),
                       Codes{m_codes, m_scales, v_codes, v_scales}, stream);
}

int zero_moments8_unpack(const zero_layout* L, const uint8_t* m_codes, const uint8_t* m_scales,
                         const uint8_t* v_codes, const uint8_t* v_scales, float* exp_avg, float* exp_avg_sq,
                         hipStream_t stream) {
  return convert<false>(L, exp_avg, exp_avg_sq,
                        Codes{const_cast<uint8_t*>(m_codes), const_cast<uint8_t*>(m_scales),
                              const_cast<uint8_t*>(v_codes), const_cast<uint8_t*>(v_scales)},
                        stream);
}

}  // extern "C"
