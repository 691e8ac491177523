// int8_plan.h -- how an int8 product of 5 rows and more is cut into work
// (host code, no device types: the tests compile it alone).
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace nvfp4 {

constexpr int kInt8MaxWG = 256;  // workgroups: one per CU
constexpr int kInt8UnitK = 128;

// Up to 64 rows: groups of `slots` slots of columns (32 of one matrix, 16 of
// gate and up each), which go to the workgroups in turn; or, where there are
// few, each in `parts` parts along K, a workgroup each.  (Parts beside whole
// groups do not pay: the sums that a part leaves in memory hold up the
// transfers behind them, 10 us.)
struct Int8Plan {
  int mt;      // 16-row tiles: 1, 2 or 4
  int slots;
  int groups;
  int units;   // units of K
  int parts;   // of a group
  int nwg;
  size_t partial_bytes;
};
constexpr int kInt8RingRows = 64;
constexpr int kInt8MaxSlots = 6;
constexpr int kInt8RingParts = 16;

constexpr size_t int8_piece_bytes(int mt, int slots) { return (size_t)slots * 32 * 16 * mt * 4; }

inline Int8Plan int8_plan_of(int slots, int parts, int m, int n, int k, int nmat) {
  Int8Plan p{};
  p.mt = m <= 16 ? 1 : m <= 32 ? 2 : 4;
  p.slots = slots;
  const int cols = 32 / nmat * slots;
  p.groups = (n + cols - 1) / cols;
  p.units = (k + kInt8UnitK - 1) / kInt8UnitK;
  p.parts = (int64_t)p.groups * parts > kInt8MaxWG || parts > p.units ? 1 : parts;
  const int64_t pairs = (int64_t)p.groups * p.parts;
  p.nwg = (int)(pairs < kInt8MaxWG ? pairs : kInt8MaxWG);
  p.partial_bytes = p.parts > 1 ? (size_t)pairs * int8_piece_bytes(p.mt, slots) : 0;
  return p;
}
// In microseconds, as measured: a unit of a workgroup takes 0.1 and 0.0185 for
// each KB of it, all weights come at 5.8 TB/s (the shorter of the two counts a
// little: nothing overlaps quite); then what it costs to join parts.
inline double int8_cost(const Int8Plan &p, int n, int k, int nmat) {
  const double unit = 0.1 + 0.0185 * (4.0 * p.slots + 2.0 * p.mt);
  const int pairs = p.groups * p.parts;
  const double busiest = (double)((pairs + p.nwg - 1) / p.nwg) * ((p.units + p.parts - 1) / p.parts) * unit;
  const double memory = (double)nmat * n * k / 5.8e6;
  return (busiest > memory ? busiest + 0.2 * memory : memory + 0.2 * busiest) + (p.parts > 1 ? 1.5 + 0.3 * p.parts : 0.0);
}
inline Int8Plan int8_plan(int m, int n, int k, int nmat) {
  Int8Plan best{};
  double least = 0;
  for (int slots = 1; slots <= kInt8MaxSlots; ++slots)
    for (int parts = 1; parts <= kInt8RingParts; ++parts) {
      const Int8Plan p = int8_plan_of(slots, parts, m, n, k, nmat);
      if (p.parts != parts) continue;
      const double cost = int8_cost(p, n, k, nmat);
      if ((slots == 1 && parts == 1) || cost < least) best = p, least = cost;
    }
  return best;
}

// Many rows: tiles of the output.  Whole rounds of tiles go one to a
// workgroup; the tiles of the last round, where they do not fill it, may be
// cut along K into `parts` parts each.  The (tile, part) pairs are numbered
// part by part, so that the tiles that share rows or columns read the same K
// at the same time, and dealt to the workgroups in turn; the last part of a
// tile to end joins them.
struct Int8TilePlan {
  int shape;           // of a tile: kInt8Tiles[shape]
  int columns;         // of the output, from the first that is not planned before
  int row_blocks, groups, units;  // tiles along rows and columns, units of K
  int nwg;
  int whole;           // tiles that go whole, the first ones
  int parts;           // of each of the others
  size_t partial_bytes;
};
// What a round of tiles costs, and a split of one, in microseconds (measured
// at K of 4096 to 17408, where several row blocks share the weights): a unit
// of K, the rest of a tile (its first unit's way from memory, its end), and to
// join its parts, each.  What a single row block waits for memory is not in
// it, nor that a join finds the parts in a cache (66 rows of 5120 x 17408: 33.6
// by these, 29.5 measured; 333 rows of 7001 x 4128: 23.9 and 25 to 32; 2048 of
// 17408 x 5120: 177 and 186 to 205).
struct Int8Tile {
  int rows, cols;  // (cols: half of them gate and half up, with two matrices)
  double unit, tile, join;
};
constexpr int kInt8TileK = 128;
constexpr int kInt8Shapes = 4;
constexpr Int8Tile kInt8Tiles[kInt8Shapes] = {
    {256, 256, 1.75, 7.3, 10}, {256, 128, 0.95, 6.9, 5}, {128, 256, 0.96, 6.1, 5}, {128, 128, 0.53, 6.4, 2.5}};
constexpr double kInt8Launch = 4;  // one more launch
constexpr int kInt8MaxParts = 8;
constexpr int kInt8MaxPairs = 2 * kInt8MaxWG;  // of tiles and parts: two rounds

// The tiles left over by whole rounds in `parts` parts (1: no split).
inline Int8TilePlan int8_tile_plan_of(int shape, int parts, int m, int n, int k, int nmat) {
  const Int8Tile t = kInt8Tiles[shape];
  Int8TilePlan p{};
  p.shape = shape;
  p.columns = n;
  p.row_blocks = (m + t.rows - 1) / t.rows;
  p.groups = (n + t.cols / nmat - 1) / (t.cols / nmat);
  p.units = (k + kInt8TileK - 1) / kInt8TileK;
  const int64_t tiles = (int64_t)p.row_blocks * p.groups;
  int64_t rest = parts > 1 ? tiles % kInt8MaxWG : 0;
  if (rest * parts > kInt8MaxPairs || parts > p.units) rest = 0;
  p.whole = (int)(tiles - rest);
  p.parts = rest ? parts : 1;
  const int64_t pairs = rest * p.parts, most = p.whole > pairs ? p.whole : pairs;
  p.nwg = (int)(most < kInt8MaxWG ? most : kInt8MaxWG);
  p.partial_bytes = (size_t)pairs * t.rows * t.cols * 4;
  return p;
}
inline double int8_tile_cost(const Int8TilePlan &p) {
  const Int8Tile t = kInt8Tiles[p.shape];
  const int pairs = (p.row_blocks * p.groups - p.whole) * p.parts;
  double cost = (double)((p.whole + p.nwg - 1) / p.nwg) * (p.units * t.unit + t.tile);
  if (pairs)
    cost += (double)((pairs + p.nwg - 1) / p.nwg) * ((p.units + p.parts - 1) / p.parts * t.unit + t.tile) + p.parts * t.join;
  return cost;
}

// One launch, or two: whole rounds of tiles of one shape for the first
// columns, and the others in a shape (and split) of their own.
struct Int8TilePlans {
  int count;
  Int8TilePlan part[2];
};
inline Int8TilePlans int8_tile_plan(int m, int n, int k, int nmat) {
  Int8TilePlans best{};
  double least = 0;
  auto one = [&](int columns, double *cost) {
    Int8TilePlan p{};
    for (int shape = 0; shape < kInt8Shapes; ++shape)
      for (int parts = 1; parts <= kInt8MaxParts; ++parts) {
        const Int8TilePlan q = int8_tile_plan_of(shape, parts, m, columns, k, nmat);
        const double c = int8_tile_cost(q);
        if ((shape == 0 && parts == 1) || c < *cost) p = q, *cost = c;
      }
    return p;
  };
  best.count = 1;
  best.part[0] = one(n, &least);
  for (int shape = 0; shape < kInt8Shapes; ++shape) {
    const Int8TilePlan all = int8_tile_plan_of(shape, 1, m, n, k, nmat);
    const int64_t tiles = (int64_t)all.row_blocks * all.groups, rounds = tiles / kInt8MaxWG;
    const int64_t groups = rounds * kInt8MaxWG / all.row_blocks;
    if (groups == 0 || groups >= all.groups) continue;
    const int columns = (int)groups * (kInt8Tiles[shape].cols / nmat);
    const Int8TilePlan first = int8_tile_plan_of(shape, 1, m, columns, k, nmat);
    double cost = 0;
    const Int8TilePlan second = one(n - columns, &cost);
    cost += int8_tile_cost(first) + kInt8Launch;
    if (cost < least) least = cost, best.count = 2, best.part[0] = first, best.part[1] = second;
  }
  return best;
}
inline size_t int8_tile_partial_bytes(const Int8TilePlans &p) {
  const size_t a = p.part[0].partial_bytes, b = p.count > 1 ? p.part[1].partial_bytes : 0;
  return a > b ? a : b;
}

// No plan for m rows or fewer has more partial sums than these.
inline size_t int8_partial_bound(int m, int n, int k, int nmat) {
  size_t most = 0;
  auto more = [&](size_t b) { most = b > most ? b : most; };
  for (int rows = 16; rows <= kInt8RingRows; rows *= 2)
    if (rows == 16 || rows / 2 < m) more(int8_plan(rows, n, k, nmat).partial_bytes);
  for (int shape = 0; shape < kInt8Shapes && m > kInt8RingRows; ++shape) {
    const Int8TilePlan p = int8_tile_plan_of(shape, 1, m, n, k, nmat);
    const int64_t pairs = (int64_t)p.row_blocks * p.groups * kInt8MaxParts;
    more((size_t)(pairs < kInt8MaxPairs ? pairs : kInt8MaxPairs) * kInt8Tiles[shape].rows * kInt8Tiles[shape].cols * 4);
  }
  return most;
}

}  // namespace nvfp4
