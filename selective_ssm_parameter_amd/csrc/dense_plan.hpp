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
// (The factors of three numbers are fitted by themselves, to which tile a product should
// take: over dx and dw of 17 sizes of the cross entropy, 64 to 16384 tokens and 500 to
// 131072 words, the planned tile takes 1.3 % longer than the best one on average, 15 % at
// worst; by the factors of two, carried on, 3.3 %.)
struct TileCost {
  int rows, cols, most;
  double busy, alone, rest;
  double split;  // factor of a step whose a is two numbers
  double three = 1;  // and of one whose a is three
};
constexpr TileCost kBf16Tiles[] = {{256, 256, 1, 0.90, 0.90, 10, 1.8, 2.0},
                                   {256, 192, 1, 0.72, 0.72, 9, 1.9, 1.9},
                                   {128, 128, 2, 0.31, 0.35, 6, 1.6, 2.0},
                                   {64, 64, 4, 0.16, 0.20, 4, 1.8, 3.5},
                                   {32, 64, 6, 0.10, 0.20, 4, 1.8, 2.6}};
constexpr TileCost kBf16Gated[] = {{256, 256, 1, 0.90, 0.90, 12, 1},
                                   {128, 128, 2, 0.31, 0.35, 7, 1},
                                   {64, 128, 3, 0.19, 0.22, 5, 1}};
constexpr TileCost kF32Tiles[] = {{128, 128, 1, 2.0, 2.0, 8, 1},
                                  {64, 64, 2, 0.52, 0.65, 6, 1},
                                  {32, 64, 3, 0.25, 0.40, 5, 1}};
constexpr TileCost kF32Gated[] = {{128, 128, 2, 1.8, 2.0, 8, 1}, {64, 128, 1, 1.0, 1.0, 6, 1},
                                  {32, 128, 2, 0.50, 0.65, 6, 1}};
// The cross entropy's in fp32: the same loop, but an epilogue that is light on small tiles.
// (Forward and backward at 16 sizes, 1 to 16384 tokens and 500 to 50000 words: 0.4 % longer
// than with the best tile on average, 7 % at worst; by the gated products' costs 1.6 and
// 13 %, at 999 x 480 over 10007 words 456 instead of 403 us. 64 x 128 is nowhere the best.)
constexpr TileCost kF32Xent[] = {{128, 128, 2, 1.8, 2.0, 8, 1}, {32, 128, 2, 0.45, 0.55, 6, 1}};

struct Plan {
  int tile, splits;  // tile: rows * 1000 + columns
};
// most: the largest number of k runs; their partial sums are written, read and
// summed at about 4 TB/s by one more launch. more: numbers that a is the sum of,
// beyond the first.
inline Plan plan_of(const TileCost* tiles, int nt, int more, int64_t R, int64_t S, int64_t K,
                    int64_t most) {
  Plan best{0, 1};
  double tbest = 1e30;
  for (int i = 0; i < nt; ++i) {
    const TileCost& c = tiles[i];
    const double steps = (double)((K + kBK - 1) / kBK) * (more == 0 ? 1.0 : more == 1 ? c.split : c.three);
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

inline Plan plan(bool is_bf16, int more, bool gated, int64_t R, int64_t S, int64_t K, int64_t most) {
  const TileCost* tiles =
      is_bf16 ? (gated ? kBf16Gated : kBf16Tiles) : (gated ? kF32Gated : kF32Tiles);
  return plan_of(tiles, is_bf16 && !gated ? 5 : 3, more, R, S, K, most);
}

// The k runs of a product, at least 256 long and 64 at most (for few tokens, or
// a weight gradient of many tokens and few columns). Of a weight gradient every
// run's operand rows also stay below 2 GiB.
struct Runs {
  int tile, splits, ksplit;
};
inline Runs runs_of(bool is_bf16, int more, bool tn, int R, int S, int K) {
  const Plan p = plan(is_bf16, more, false, R, S, K,
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

// The tile of the cross entropy's z (tokens x vocabulary rows); in bf16 by the costs of
// the gated products' tiles, whose kernel it shares up to the epilogue.
inline int xent_tile(bool is_bf16, int64_t R, int64_t S, int64_t K) {
  if (!is_bf16) return plan_of(kF32Xent, 2, 0, R, S, K, 1).tile;
  return plan(true, 0, true, R, S, K, 1).tile;
}

}  // namespace swimba
