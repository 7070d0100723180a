// How the products of an expert's layer are launched, from the sizes alone.
// `rows` is what the experts' counts add up to at most: rows of padding between
// aligned segments are in no tile.
// Host code without HIP, so that it can be run and tested anywhere.
#pragma once

#include <limits.h>
#include <math.h>
#include <stddef.h>
#include <stdint.h>

#include <initializer_list>

namespace ep {

constexpr int kTileCols = 256;  // columns of a tile
constexpr int kTileStep = 32;   // contraction step
constexpr int kXcds = 8;
constexpr int kCusPerXcd = 32;

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Tiles of one product.
struct LinearPlan {
  int mi;  // 32-row sub-tiles of a wave: tiles of 64 mi rows; 0: the kernel for few rows
  int run;  // tiles that an XCD takes in a row
  unsigned blocks;
};

// Blocks of a launch with up to `tiles` tiles in runs of `run`: whole rounds
// of runs over the XCDs, or of an eighth of the tiles.
inline unsigned blocks_of(int64_t tiles, int64_t run) {
  if (run > ceil_div(tiles, kXcds)) run = ceil_div(tiles, kXcds);
  return static_cast<unsigned>(ceil_div(tiles, kXcds * run) * kXcds * run);
}

inline int64_t row_tiles(int64_t rows, int E, int bm) { return ceil_div(rows, bm) + (rows < E ? rows : E); }

// A product whose tiles' rows are the experts' `rows` rows, by nt column tiles.
inline LinearPlan plan_rows(int64_t rows, int E, int64_t nt) {
  // Tile height by the rounds of tiles over the CUs and their height, for rows
  // that the router spread at random: an expert then has its share and about
  // two standard deviations more.  A tile costs its rows and as much as 64 more,
  // for its start, its stores and the weights that it loads whatever its rows
  // (over 13 layers 32, 64 and 128 give the same times to 1%; 0 takes 4% more
  // forward and 2% in grad_x, 2.64 ms against 2.28 with 256 experts of 256 rows).
  const double avg = static_cast<double>(rows) / E;
  const double most = avg + 2.0 * sqrt(avg * (E - 1) / E);
  int best = 0;
  double least = 0.0;
  for (int mi : {2, 4, 5}) {
    const int64_t mt = ceil_div(static_cast<int64_t>(ceil(most)), 64 * mi);
    const double per = static_cast<double>(ceil_div(ceil_div(static_cast<int64_t>(ceil(most)), mt), 32) * 32);
    // two blocks of 128 rows share a CU
    const int64_t places = kXcds * kCusPerXcd * (mi == 2 ? 2 : 1);
    const int64_t tiles = mt * E * nt;
    const int64_t turns = ceil_div(tiles, places) * (mi == 2 && tiles > places / 2 ? 2 : 1);
    const double cost = static_cast<double>(turns) * (per + 64.0);
    if (best == 0 || cost < least) {
      best = mi;
      least = cost;
    }
  }
  // Runs of 32, one tile a CU: all XCDs work on neighbouring tiles, whose rows
  // and weights meet in the memory-side cache (65,536 rows x 7168 -> 2048 of 32
  // experts: 1.81 ms, one run an XCD 1.87).  Where weights are read once, one
  // run an XCD streams them faster (64 experts of 4 rows: 260 us against 270;
  // of 64 rows 396 against 459).
  const int run = best == 2 ? INT_MAX : kCusPerXcd;
  return {best, run, blocks_of(row_tiles(rows, E, 64 * best) * nt, run)};
}

// The forward product of N outputs.
inline LinearPlan plan_forward(int64_t rows, int E, int N, bool gated) {
  // Up to 4 rows an expert, or few enough 16 x 64 pieces that the tiles of
  // 128 rows and more would leave most CUs idle (8 experts of 127 rows, 1032 ->
  // 520: 13.5 us against 24).  Where tiles overtake it depends on the layer
  // (here against tiles of 128 rows, us, at 2, 4, 8 and 12 rows an expert: 64
  // experts, 4096 -> 2 x 2048: 320/348, 402/376, 422/378, 376/380; 2048 -> 4096:
  // 157/170, 177/177, 188/184, 207/185; 256 experts, 7168 -> 2048: 1034/1081,
  // 1180/1234, 1225/1260, 1285/1276; 8 experts, 4096 -> 14,336: 148/163, 154/167,
  // 156/169, 179/173): from 3 rows to 10, at 7% on either side.
  const int64_t few_nt = ceil_div(N, gated ? 32 : 64);
  if (rows <= 4 * static_cast<int64_t>(E) || ceil_div(ceil_div(rows, E), 16) * E * few_nt <= 1024)
    return {0, INT_MAX, blocks_of(row_tiles(rows, E, 16) * few_nt, INT_MAX)};
  return plan_rows(rows, E, ceil_div(N, gated ? kTileCols / 2 : kTileCols));
}

// Parts of each expert's rows in the weight gradient, and their workspace.
struct LinearGeom {
  int splits;
  size_t part_bytes;  // 16 at least
};
inline LinearGeom linear_geom(int64_t rows, int E, int H, int W) {
  LinearGeom g;
  const int64_t tiles = ceil_div(W, 256) * ceil_div(H, kTileCols) * E;
  // Rows in as many parts as cost least, in us as measured for even rows: 8 a
  // tile and 0.9 for every 32 of its rows, a tile a CU at once, against writing
  // and reading the fp32 parts at 6 TB/s and 5 for the join.  (2048 rows x 2048
  // -> 2048 of one expert: 56.6 us whole, 42.6 in 4 parts, 64.8 in 8; 16,384 x
  // 1024 -> 1024: 399 whole, 55.6 in 16; 8192 x 4096 -> 4096: 233 whole, 280 in 2.)
  constexpr int64_t kCus = kXcds * kCusPerXcd;
  g.splits = 1;
  double least = 0.0;
  for (int64_t s = 1; s == 1 || (s * tiles <= 2 * kCus && s * 64 <= rows / E); s += s < 8 ? 1 : s / 8) {
    const int64_t steps = ceil_div(ceil_div(rows, E * s), kTileStep);
    double cost = static_cast<double>(ceil_div(tiles * s, kCus)) * (0.9 * static_cast<double>(steps) + 8.0);
    if (s > 1) cost += 5.0 + 8.0 * static_cast<double>((static_cast<int64_t>(W) * H + W) * E * s) / 6.0e6;
    if (s == 1 || cost < least) {
      least = cost;
      g.splits = static_cast<int>(s);
    }
  }
  g.part_bytes = g.splits > 1 ? (static_cast<size_t>(W) * H + W) * E * g.splits * 4 : 16;
  return g;
}

// Both gradients.
struct GradsPlan {
  LinearPlan x, w;  // blocks 0: that one is not wanted
  bool by_expert;   // w's runs are whole experts, if the device finds their rows even
  bool together;    // in one launch
};
inline GradsPlan plan_grads(int64_t rows, int E, int H, int W, int splits, bool x, bool w) {
  GradsPlan p = {};
  if (x) p.x = plan_rows(rows, E, ceil_div(H, kTileCols));
  if (!w) return p;
  // Where experts have few rows, starting a tile and writing it take the time:
  // 128 x 256 tiles, two blocks a CU (64 experts of 4 rows, 2.1 GB of gradients:
  // 358 us, 256 x 256 tiles 460; of 64 rows 500 and 594; of 256 rows 985 and 948).
  // So too where grad_x has few tiles and takes those, for one launch of both
  // (8 experts of 260 rows, 1712 -> 2440: 90 -> 59 us; 4 of 500, 1024 -> 1024: 42
  // -> 24; 61 of 197, 520 -> 264: 36.7 -> 37.3).
  const int64_t avg = rows / E;
  const bool half = avg <= 128 || (x && p.x.mi == 2);
  const int64_t per_expert = ceil_div(W, half ? 128 : 256) * ceil_div(H, kTileCols) * splits;
  p.w.mi = half ? 2 : 4;
  // Runs of 32 tiles spread every expert over the XCDs.  Where an expert's rows
  // fit an L2 (4 MiB) and there are many experts, an XCD takes a whole expert,
  // whose rows are then read by one XCD and not by all (64 experts of 256 rows,
  // 8192 columns in all: 0.95 ms against 1.08), if the experts have much the
  // same rows: with rows by a Zipf law of exponent 1.2 the XCD of the largest
  // takes 1.41 ms, runs of 32 1.05.  The rows are known on the device alone.
  p.by_expert = splits == 1 && avg >= 128 && E >= 32 && avg * (W + H) * 2 <= (4 << 20);
  p.w.run = p.by_expert ? static_cast<int>(per_expert) : kCusPerXcd;
  // whole rounds of either run
  p.w.blocks = blocks_of(blocks_of(per_expert * E, p.w.run), kCusPerXcd);
  // One launch for both (509 rows x 1032 -> 520, top-2 of 8: 31.2 -> 23.3 us in
  // all; 64 experts by a Zipf law of 1.2: 1870 -> 1785; 32 experts of 2048 rows,
  // 2048 -> 7168: 3.86 -> 3.88 ms), where the blocks of both have one occupancy.
  p.together = x && (p.x.mi == 2) == half && p.x.blocks + p.w.blocks < (1u << 22);
  return p;
}

// Tiles of the largest launch of these sizes, at most.
inline int64_t linear_max_tiles(int64_t rows, int E, int H, int W) {
  // columns of 128 (gated) or 256, rows of 128 at least
  const int64_t by_rows = row_tiles(rows, E, 128) * ceil_div(W > H ? W : H, 128);
  // (rows are split where that makes no more than 1024)
  const int64_t by_weights = ceil_div(W, 128) * ceil_div(H, kTileCols) * E;
  const int64_t few = rows <= 4 * static_cast<int64_t>(E) ? row_tiles(rows, E, 16) * ceil_div(W, 64) : 0;
  const int64_t tiles = by_rows > by_weights ? by_rows : by_weights;
  return few > tiles ? few : tiles;
}

}  // namespace ep
