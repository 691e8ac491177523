// Walks the int8 products' plans as their kernels do, on the CPU: every unit
// of every tile belongs to one workgroup, every piece of a split tile lies
// inside the partial sums, and the workgroups that a split tile waits for are
// those that bring pieces.  Prints one line per failure; "ok" and the number
// of plans at the end.
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "int8_plan.h"

using namespace nvfp4;

static int bad = 0;
#define CHECK(x, ...)              \
  do {                             \
    if (!(x)) {                    \
      if (++bad < 20) {            \
        printf("%s: ", #x);        \
        printf(__VA_ARGS__);       \
        printf("\n");              \
      }                            \
      return;                      \
    }                              \
  } while (0)

static void ring(const Int8Plan &p, int m, int n, int k, int nmat) {
  const int cols = 32 / nmat * p.slots;
  CHECK(16 * p.mt >= m && p.slots >= 1 && p.slots <= kInt8MaxSlots, "m %d mt %d slots %d", m, p.mt, p.slots);
  CHECK((int64_t)p.groups * cols >= n && (int64_t)(p.groups - 1) * cols < n, "n %d", n);
  CHECK((int64_t)p.units * kInt8UnitK >= k && (int64_t)(p.units - 1) * kInt8UnitK < k, "k %d", k);
  const int pairs = p.groups * p.parts;
  CHECK(p.parts >= 1 && p.parts <= p.units && p.nwg >= 1 && p.nwg <= kInt8MaxWG && p.nwg <= pairs, "parts %d nwg %d", p.parts, p.nwg);
  CHECK(p.parts == 1 || pairs == p.nwg, "%d pairs, nwg %d", pairs, p.nwg);
  CHECK(p.partial_bytes == (p.parts > 1 ? (size_t)pairs * int8_piece_bytes(p.mt, p.slots) : 0), "partial sums of %d pairs", pairs);
  std::vector<int> seen(p.groups, 0);
  int64_t units = 0;
  for (int w = 0; w < p.nwg; ++w)
    for (int i = w; i < pairs; i += p.nwg) {
      const int part = i / p.groups, len = p.units * (part + 1) / p.parts - p.units * part / p.parts;
      CHECK(part < p.parts && len > 0, "part %d of %d", part, p.parts);
      ++seen[i % p.groups], units += len;
    }
  CHECK(units == (int64_t)p.groups * p.units, "%lld units of %d groups", (long long)units, p.groups);
  for (int x : seen) CHECK(x == p.parts, "%d parts end, %d are waited for", x, p.parts);
}

static void tiles(const Int8TilePlan &p, int m, int n, int k, int nmat) {
  const Int8Tile t = kInt8Tiles[p.shape];
  CHECK((int64_t)p.row_blocks * t.rows >= m && (int64_t)(p.row_blocks - 1) * t.rows < m, "m %d", m);
  CHECK((int64_t)p.groups * (t.cols / nmat) >= n && (int64_t)(p.groups - 1) * (t.cols / nmat) < n, "n %d", n);
  CHECK((int64_t)p.units * kInt8TileK >= k && (int64_t)(p.units - 1) * kInt8TileK < k, "k %d", k);
  const int all = p.row_blocks * p.groups, split = all - p.whole, pairs = split * p.parts;
  CHECK(p.whole >= 0 && split >= 0 && split < kInt8MaxWG && p.nwg >= 1 && p.nwg <= kInt8MaxWG, "whole %d nwg %d", p.whole, p.nwg);
  CHECK(p.nwg <= (p.whole > pairs ? p.whole : pairs), "an idle workgroup: %d tiles, %d pairs, nwg %d", p.whole, pairs, p.nwg);
  CHECK(p.parts >= 1 && p.parts <= p.units, "%d parts of %d units", p.parts, p.units);
  CHECK((size_t)pairs * t.rows * t.cols * 4 == p.partial_bytes, "partial sums of %d pairs", pairs);
  // the workgroups' units: each of them once, and at least one to a part
  std::vector<int> seen(split, 0);
  int64_t units = 0;
  for (int w = 0; w < p.nwg; ++w) {
    int own = 0;
    for (int i = w; i < p.whole; i += p.nwg) own += p.units;
    for (int i = w; i < pairs; i += p.nwg) {
      const int part = i / split, len = p.units * (part + 1) / p.parts - p.units * part / p.parts;
      CHECK(part < p.parts && len > 0, "part %d of %d", part, p.parts);
      ++seen[i % split], own += len;
    }
    CHECK(own > 0, "nothing for workgroup %d", w);
    units += own;
  }
  CHECK(units == (int64_t)all * p.units, "%lld units of %d tiles", (long long)units, all);
  for (int x : seen) CHECK(x == p.parts, "%d parts end, %d are waited for", x, p.parts);
}

// what is planned for few rows fits what is bound for more
static void bound(int few, int many, int n, int k, int nmat) {
  if (few > many) return;
  const size_t most = int8_partial_bound(many, n, k, nmat);
  const size_t need = few <= kInt8RingRows ? int8_plan(few, n, k, nmat).partial_bytes : int8_tile_partial_bytes(int8_tile_plan(few, n, k, nmat));
  CHECK(need <= most, "m %d of %d, n %d k %d: %zu of %zu", few, many, n, k, need, most);
  CHECK(int8_partial_bound(few, n, k, nmat) <= most, "bound of m %d and %d", few, many);
}

int main(int argc, char **argv) {
  srand(argc > 1 ? atoi(argv[1]) : 1);
  int plans = 0;
  auto pick = [](int most) {  // spread over the logarithm
    int b = 1;
    while (b < most && rand() % 12) b *= 2;
    const int x = b + rand() % b;
    return x < most ? x : most;
  };
  for (int i = 0; i < 30000; ++i) {
    const int n = pick(1 << 17), k = 32 * pick(4096), nmat = 1 + rand() % 2;
    const int few = 1 + rand() % kInt8RingRows;
    ring(int8_plan(few, n, k, nmat), few, n, k, nmat);
    ring(int8_plan_of(1 + rand() % kInt8MaxSlots, 1 + rand() % kInt8RingParts, few, n, k, nmat), few, n, k, nmat);
    const int m = kInt8RingRows + 1 + pick(1 << 15);
    const Int8TilePlans two = int8_tile_plan(m, n, k, nmat);
    int columns = 0;
    for (int j = 0; j < two.count; ++j) {
      // (a second launch's first column starts 16 bytes of y, and a whole group of columns)
      if (columns % 64) ++bad, printf("column %d\n", columns);
      tiles(two.part[j], m, two.part[j].columns, k, nmat);
      columns += two.part[j].columns;
    }
    if (columns != n || two.count < 1 || two.count > 2) ++bad, printf("columns %d of %d\n", columns, n);
    const int shape = rand() % kInt8Shapes;
    tiles(int8_tile_plan_of(shape, 1 + rand() % kInt8MaxParts, m, n, k, nmat), m, n, k, nmat);
    tiles(int8_tile_plan_of(shape, 1, m, n, k, nmat), m, n, k, nmat);
    bound(1 + rand() % 600, m, n, k, nmat);
    bound(m - rand() % (m - 1), m, n, k, nmat);
    plans += 4;
  }
  if (bad) return 1;
  printf("ok %d\n", plans);
  return 0;
}
