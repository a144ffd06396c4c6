// Which tile a dense product takes and into how many runs its k is cut
// (dense.hip). Host code without HIP, so that a test can ask it which kernel a
// shape reaches.
#pragma once

#include <stdint.h>

#include <algorithm>

namespace swimba {

constexpr int kBK = 32;  // k elements of a tile's step

// Tile and number of k runs of a product, by an estimate of its time in us. A
// tile's k step takes `alone` us by itself (its copies and LDS reads waited for)
// and at least `busy` us per tile that shares the CU, of which there are up to
// `most`; `rest` is what a tile adds (first copies, epilogue, stores). Fitted to
// products of 999 x 1016 x 480 and 4096 x 1024 x 1024 with each tile and of
// 32768 x 8192 x 2048. fp32 stages of 256 rows do not fit LDS.
// (At 14 sizes drawn at random, 77 to 13483 tokens and widths of 64 to 5024 in both
// types, the planned tile took 3 to 5 % longer than the best one on average over
// each kind of product, 23 % at worst: fp32 6855 x 352 -> 2 x 440, 55 against 45 us.)
struct TileCost {
  int rows, cols, most;
  double busy, alone, rest;
  double split;  // factor of a step with hi and lo
};
constexpr TileCost kBf16Tiles[] = {{256, 256, 1, 0.90, 0.90, 10, 1.8},
                                   {256, 192, 1, 0.72, 0.72, 9, 1.9},
                                   {128, 128, 2, 0.31, 0.35, 6, 1.6},
                                   {64, 64, 4, 0.16, 0.20, 4, 1.8},
                                   {32, 64, 6, 0.10, 0.20, 4, 1.8}};
constexpr TileCost kBf16Gated[] = {{256, 256, 1, 0.90, 0.90, 12, 1},
                                   {128, 128, 2, 0.31, 0.35, 7, 1},
                                   {64, 128, 3, 0.19, 0.22, 5, 1}};
constexpr TileCost kF32Tiles[] = {{128, 128, 1, 2.0, 2.0, 8, 1},
                                  {64, 64, 2, 0.52, 0.65, 6, 1},
                                  {32, 64, 3, 0.25, 0.40, 5, 1}};
constexpr TileCost kF32Gated[] = {{128, 128, 2, 1.8, 2.0, 8, 1}, {64, 128, 1, 1.0, 1.0, 6, 1},
                                  {32, 128, 2, 0.50, 0.65, 6, 1}};

struct Plan {
  int tile, splits;  // tile: rows * 1000 + columns
};
// most: the largest number of k runs; their partial sums are written, read and
// summed at about 4 TB/s by one more launch.
inline Plan plan(bool is_bf16, bool split, bool gated, int64_t R, int64_t S, int64_t K, int64_t most) {
  Plan best{0, 1};
  double tbest = 1e30;
  const TileCost* tiles =
      is_bf16 ? (gated ? kBf16Gated : kBf16Tiles) : (gated ? kF32Gated : kF32Tiles);
  const int nt = is_bf16 ? (gated ? 3 : 5) : 3;
  for (int i = 0; i < nt; ++i) {
    const TileCost& c = tiles[i];
    const double steps = (double)((K + kBK - 1) / kBK) * (split ? c.split : 1.0);
    const int64_t units = (R + c.rows - 1) / c.rows * ((S + c.cols - 1) / c.cols);
    if (i > 0 && units > (1 << 20)) continue;  // (a launch's threads are counted in 32 bits)
    for (int64_t n = 1; n <= most; ++n) {
      auto round = [&](int64_t per_cu) {
        return steps / n * std::max(c.alone, per_cu * c.busy) + c.rest;
      };
      const int64_t full = units * n / (256 * c.most), left = units * n % (256 * c.most);
      double t = full * round(c.most) + (left ? round((left + 255) / 256) : 0.0);
      if (n > 1) t += 4 + (double)(n + 1) * R * S * 4e-6 / 4;
      if (t < tbest) {
        tbest = t;
        best = Plan{c.rows * 1000 + c.cols, (int)n};
      }
      if (full > 3) break;  // more runs only add partial sums
    }
  }
  return best;
}

// The k runs of a product, at least 256 long and 64 at most (for few tokens, or
// a weight gradient of many tokens and few columns). Of a weight gradient every
// run's operand rows also stay below 2 GiB.
struct Runs {
  int tile, splits, ksplit;
};
inline Runs runs_of(bool is_bf16, bool split, bool tn, int R, int S, int K) {
  const Plan p = plan(is_bf16, split, false, R, S, K,
                      std::max<int64_t>(1, std::min<int64_t>(64, K / 256)));
  int64_t n = p.splits;
  if (tn) {
    const int64_t row = (int64_t)(R > S ? R : S) * (is_bf16 ? 2 : 4);
    n = std::max<int64_t>(n, (K * row + (int64_t(1) << 30) - 1) >> 30);
  }
  Runs r{p.tile, 1, 0};
  r.ksplit = (int)(((K + n - 1) / n + kBK - 1) / kBK * kBK);
  r.splits = (K + r.ksplit - 1) / r.ksplit;
  return r;
}

}  // namespace swimba
