// int8_plan.h -- how an int8 product of 5 rows and more is cut into work
// (host code, no device types: the tests compile it alone).
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace nvfp4 {

// Columns come in groups and K in units; the (group, unit) pairs, group by
// group, are dealt to the workgroups in equal runs, one workgroup per CU.  A
// group whose units lie in several runs is summed from their pieces by the
// last of them to end.
struct Int8Plan {
  int mt;        // 16-row tiles of a workgroup: 1, 2, 4, 8 or 16
  int groups;    // column groups
  int units;     // units of K in a group
  int nwg;       // workgroups
  size_t partial_bytes;
};

constexpr int kInt8UnitK = 128;
constexpr int kInt8MaxWG = 256;
constexpr int kInt8MinUnits = 4;  // units of a workgroup, at least
// columns of a group: of one matrix, or 64 of gate and the same 64 of up
constexpr int kInt8GroupCols = 128;

inline size_t int8_piece_bytes(int mt) { return (size_t)kInt8GroupCols * 16 * mt * 4; }

inline Int8Plan int8_plan(int m, int n, int k, int nmat) {
  Int8Plan p{};
  p.mt = m <= 16 ? 1 : m <= 32 ? 2 : m <= 64 ? 4 : m <= 128 ? 8 : 16;
  const int cols = kInt8GroupCols / nmat;
  p.groups = (n + cols - 1) / cols;
  p.units = (k + kInt8UnitK - 1) / kInt8UnitK;
  const int64_t all = (int64_t)p.groups * p.units;
  const int64_t want = (all + kInt8MinUnits - 1) / kInt8MinUnits;
  p.nwg = want < kInt8MaxWG ? (int)want : kInt8MaxWG;
  p.partial_bytes = (size_t)p.nwg * 2 * int8_piece_bytes(p.mt);
  return p;
}

// Many rows: tiles of the output.  Whole rounds of tiles go one to a
// workgroup; the tiles of the last round, where they do not fill it, may be
// cut along K into equal runs over all workgroups, as above.
struct Int8TilePlan {
  int shape;           // of a tile: kInt8Tiles[shape]
  int columns;         // of the output, from the first that is not planned before
  int row_blocks, groups, units;  // tiles along rows and columns, units of K
  int nwg;
  int whole;           // tiles that go whole, the first ones
  size_t partial_bytes;
};
// What a round of tiles costs, and a split of one, in microseconds (measured
// at K of 4096 to 17408): a unit of K, the rest of a tile (its first unit's
// way from memory, its end), and the pieces' way to the workgroup that joins
// them.
struct Int8Tile {
  int rows, cols;  // (cols: half of them gate and half up, with two matrices)
  double unit, tile, join;
};
constexpr int kInt8TileK = 128;
constexpr int kInt8Shapes = 4;
constexpr Int8Tile kInt8Tiles[kInt8Shapes] = {
    {256, 256, 1.75, 7.3, 55}, {256, 128, 0.95, 6.9, 25}, {128, 256, 0.96, 6.1, 25}, {128, 128, 0.53, 6.4, 12}};
constexpr double kInt8Launch = 4;  // one more launch

inline Int8TilePlan int8_tile_plan_of(int shape, bool split, int m, int n, int k, int nmat) {
  const Int8Tile t = kInt8Tiles[shape];
  Int8TilePlan p{};
  p.shape = shape;
  p.columns = n;
  p.row_blocks = (m + t.rows - 1) / t.rows;
  p.groups = (n + t.cols / nmat - 1) / (t.cols / nmat);
  p.units = (k + kInt8TileK - 1) / kInt8TileK;
  const int64_t tiles = (int64_t)p.row_blocks * p.groups;
  // (every workgroup has to have units of a split: the last to end counts them all)
  int64_t rest = split ? tiles % kInt8MaxWG : 0;
  if (tiles >= kInt8MaxWG && rest * p.units < (int64_t)kInt8MaxWG * kInt8MinUnits) rest = 0;
  p.whole = (int)(tiles - rest);
  int64_t nwg = tiles;
  if (rest) nwg = p.whole ? kInt8MaxWG : (rest * p.units + kInt8MinUnits - 1) / kInt8MinUnits;
  p.nwg = (int)(nwg < kInt8MaxWG ? nwg : kInt8MaxWG);
  p.partial_bytes = rest ? (size_t)p.nwg * 2 * t.rows * t.cols * 4 : 0;
  return p;
}
inline double int8_tile_cost(const Int8TilePlan &p) {
  const Int8Tile t = kInt8Tiles[p.shape];
  const int64_t rest = (int64_t)p.row_blocks * p.groups - p.whole;
  double cost = (double)((p.whole + p.nwg - 1) / p.nwg) * (p.units * t.unit + t.tile);
  if (rest) cost += (double)rest * p.units / p.nwg * t.unit + t.tile + t.join;
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
      for (int split = 0; split < 2; ++split) {
        const Int8TilePlan q = int8_tile_plan_of(shape, split, m, columns, k, nmat);
        const double c = int8_tile_cost(q);
        if ((shape == 0 && !split) || c < *cost) p = q, *cost = c;
      }
    return p;
  };
  best.count = 1;
  best.part[0] = one(n, &least);
  for (int shape = 0; shape < kInt8Shapes; ++shape) {
    const Int8TilePlan all = int8_tile_plan_of(shape, false, m, n, k, nmat);
    const int64_t tiles = (int64_t)all.row_blocks * all.groups, rounds = tiles / kInt8MaxWG;
    const int64_t groups = rounds * kInt8MaxWG / all.row_blocks;
    if (groups == 0 || groups >= all.groups) continue;
    const int columns = (int)groups * (kInt8Tiles[shape].cols / nmat);
    const Int8TilePlan first = int8_tile_plan_of(shape, false, m, columns, k, nmat);
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
  for (int rows = 16; rows <= 256; rows *= 2)
    if (rows == 16 || rows / 2 < m) more(int8_plan(rows, n, k, nmat).partial_bytes);
  for (int shape = 0; shape < kInt8Shapes && m > 256; ++shape) {
    const Int8TilePlan p = int8_tile_plan_of(shape, false, m, n, k, nmat);
    const int64_t tiles = (int64_t)p.row_blocks * p.groups;
    const int64_t wgs = ((tiles < kInt8MaxWG ? tiles : kInt8MaxWG) * p.units + kInt8MinUnits - 1) / kInt8MinUnits;
    more((size_t)(wgs < kInt8MaxWG ? wgs : kInt8MaxWG) * 2 * kInt8Tiles[shape].rows * kInt8Tiles[shape].cols * 4);
  }
  return most;
}

// first pair of workgroup w's run, and the workgroup whose run holds pair u
#if defined(__HIPCC__)
#define INT8_PLAN_FN __host__ __device__ inline
#else
#define INT8_PLAN_FN inline
#endif
INT8_PLAN_FN int int8_run_begin(int all, int nwg, int w) { return (int)(((int64_t)all * w) / nwg); }
INT8_PLAN_FN int int8_run_owner(int all, int nwg, int u) { return (int)((((int64_t)u + 1) * nwg + all - 1) / all) - 1; }
#undef INT8_PLAN_FN

}  // namespace nvfp4
