// Which tiles the linear layer's products are cut into (host only).
//
// Tiles that fill the chip's 256 CUs are summed by one block each; the k of the
// rest may be split over several blocks each, where an estimate of the time
// says so.  The number of CUs is a constant: the order of a sum and the
// workspace's size follow from the sizes alone.
#pragma once

#include <algorithm>
#include <cstdint>

namespace zs {

constexpr int64_t kCus = 256, kMaxSplits = 32;
constexpr int kTileStep = 64;                        // k of a step
constexpr int tile_side(int W) { return 64 * W; }  // rows and columns of a block's tile

struct TilePlan {
  int64_t side, row_tiles, col_tiles, whole, further, splits, per_split;
  double us;
};

// What a block was measured to take (us): a step of 64 k, alone on its CU or
// beside another; its beginning and end; a split's part of a tile, written and
// read again; the launch that adds the parts up.
template <int W>
struct TileCost;
template <>
struct TileCost<4> {
  static constexpr double step[2] = {1.42, 1.42}, ends = 13, part = 0.054, sum = 2.7;
};
template <>
struct TileCost<2> {
  static constexpr double step[2] = {0.49, 0.80}, ends = 6, part = 0.0134, sum = 2.7;
};

// Measured (us) in splits of the smaller tile: 1000 x 2304 x 768 (tokens, outputs,
// inputs) 1: 11.0, 2: 20.1; 1000 x 768 x 2304 1: 25.2, 3: 16.2, 4: 16.5, 8: 21.8; 333
// x 8192 x 1024 1: 12.6, 2: 23.4; 300 x 300 x 8192 1: 57, 4: 17.8, 8: 12.8, 16: 12.8,
// 26: 15.4; 512 x 4096 x 4096 1: 38, 2: 31.7, 3: 38.5.  The estimate takes 1, 4, 1, 26
// and 2.  1000 x 4160 x 4100: the smaller tile in 2 83, the larger in 3 69.
template <int W>
TilePlan plan_for(int64_t M, int64_t N, int64_t K) {
  using C = TileCost<W>;
  TilePlan p{};
  p.side = tile_side(W);
  p.row_tiles = (M + p.side - 1) / p.side;
  p.col_tiles = (N + p.side - 1) / p.side;
  const int64_t tiles = p.row_tiles * p.col_tiles, steps = std::max<int64_t>(1, (K + kTileStep - 1) / kTileStep);
  const int64_t per_cu = W == 4 ? 1 : 2, at_once = kCus * per_cu;
  p.whole = tiles / at_once * at_once;
  p.further = tiles - p.whole;
  p.splits = 1;
  p.per_split = steps;
  p.us = (double)(p.whole / at_once) * ((double)steps * C::step[per_cu - 1] + C::ends);
  if (p.further == 0) return p;
  double best = 0;
  for (int64_t n = 1; n <= std::min(kMaxSplits, steps) && (n == 1 || n * p.further <= at_once); ++n) {
    const int64_t per = (steps + n - 1) / n, splits = (steps + per - 1) / per, blocks = splits * p.further;
    double us = C::ends + (double)per * C::step[blocks > kCus ? 1 : 0];
    if (splits > 1) us += C::sum + (double)blocks * C::part;
    if (n == 1 || us < best) {
      best = us;
      p.splits = splits;
      p.per_split = per;
    }
  }
  p.us += best;
  if (p.splits == 1) {
    p.whole = tiles;
    p.further = 0;
  }
  return p;
}

// The tile that is estimated to take less time.
inline TilePlan plan_of(int64_t M, int64_t N, int64_t K) {
  const TilePlan x = plan_for<4>(M, N, K), y = plan_for<2>(M, N, K);
  return x.us <= y.us ? x : y;
}

}  // namespace zs
