// Walks the int8 products' plans as their kernels do, on the CPU: every unit
// of every tile belongs to one workgroup, every piece of a split tile lies
// inside the partial sums, and the workgroups that a split tile waits for are
// those that bring pieces.  Prints one line per failure; "ok" and the number
// of plans at the end.
#include <cstdio>
#include <cstdlib>
#include <map>
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

// Runs over `all` units, `units` a tile: [begin, end) of each workgroup.
static void runs(int all, int units, int nwg, size_t piece, size_t bytes) {
  CHECK(nwg >= 1 && nwg <= kInt8MaxWG && nwg <= all, "all %d nwg %d", all, nwg);
  int at = 0;
  std::map<int, int> arrivals, waits;  // by the counter a tile uses
  for (int w = 0; w < nwg; ++w) {
    const int b = int8_run_begin(all, nwg, w), e = int8_run_begin(all, nwg, w + 1);
    CHECK(b == at && e > b, "all %d nwg %d w %d", all, nwg, w);
    at = e;
    CHECK(int8_run_owner(all, nwg, b) == w && int8_run_owner(all, nwg, e - 1) == w, "owner of %d", w);
    std::vector<int> used;
    for (int tile = b / units; tile * units < e; ++tile) {
      const int u0 = tile * units, u1 = u0 + units;
      if (u0 >= b && u1 <= e) continue;  // whole
      const int which = u0 <= b ? 0 : 1;
      for (int x : used) CHECK(x != which, "slot %d twice in %d", which, w);
      used.push_back(which);
      CHECK(((size_t)w * 2 + which + 1) * piece <= bytes, "piece of %d", w);
      const int v0 = int8_run_owner(all, nwg, u0), v1 = int8_run_owner(all, nwg, u1 - 1);
      CHECK(v0 >= 0 && v1 < nwg && v1 > v0 && v0 <= w && w <= v1, "owners %d %d of tile %d", v0, v1, tile);
      CHECK(!waits.count(v0) || waits[v0] == tile + 1, "counter %d of tiles %d and %d", v0, waits[v0] - 1, tile);
      waits[v0] = tile + 1;
      ++arrivals[v0];
    }
  }
  CHECK(at == all, "ends at %d of %d", at, all);
  for (auto &a : arrivals) {
    const int u0 = (waits[a.first] - 1) * units;
    CHECK(a.second == int8_run_owner(all, nwg, u0 + units - 1) - a.first + 1, "arrivals at %d", a.first);
  }
}

static void ring(int m, int n, int k, int nmat) {
  const Int8Plan p = int8_plan(m, n, k, nmat);
  CHECK(16 * p.mt >= m, "m %d mt %d", m, p.mt);
  CHECK((int64_t)p.groups * (kInt8GroupCols / nmat) >= n && (int64_t)(p.groups - 1) * (kInt8GroupCols / nmat) < n, "n %d", n);
  CHECK((int64_t)p.units * kInt8UnitK >= k && (int64_t)(p.units - 1) * kInt8UnitK < k, "k %d", k);
  runs(p.groups * p.units, p.units, p.nwg, int8_piece_bytes(p.mt), p.partial_bytes);
}

static void tiles(const Int8TilePlan &p, int m, int n, int k, int nmat) {
  const Int8Tile t = kInt8Tiles[p.shape];
  CHECK((int64_t)p.row_blocks * t.rows >= m && (int64_t)(p.row_blocks - 1) * t.rows < m, "m %d", m);
  CHECK((int64_t)p.groups * (t.cols / nmat) >= n && (int64_t)(p.groups - 1) * (t.cols / nmat) < n, "n %d", n);
  CHECK((int64_t)p.units * kInt8TileK >= k && (int64_t)(p.units - 1) * kInt8TileK < k, "k %d", k);
  const int all = p.row_blocks * p.groups;
  CHECK(p.whole >= 0 && p.whole <= all && p.nwg >= 1 && p.nwg <= kInt8MaxWG, "whole %d nwg %d", p.whole, p.nwg);
  CHECK(p.whole == all || p.whole == 0 || p.whole % p.nwg == 0, "whole %d of %d, nwg %d", p.whole, all, p.nwg);
  CHECK(p.whole < all || p.nwg <= all, "an idle workgroup: %d tiles, nwg %d", all, p.nwg);
  if (p.whole < all)
    runs((all - p.whole) * p.units, p.units, p.nwg, (size_t)t.rows * t.cols * 4, p.partial_bytes);
  else
    CHECK(p.partial_bytes == 0, "partial sums without a split");
}

// what is planned for few rows fits what is bound for more
static void bound(int few, int many, int n, int k, int nmat) {
  if (few > many) return;
  const size_t most = int8_partial_bound(many, n, k, nmat);
  const size_t need = few <= 256 ? int8_plan(few, n, k, nmat).partial_bytes : int8_tile_partial_bytes(int8_tile_plan(few, n, k, nmat));
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
    ring(1 + rand() % 256, n, k, nmat);
    const int m = 257 + pick(1 << 15);
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
    tiles(int8_tile_plan_of(shape, true, m, n, k, nmat), m, n, k, nmat);
    tiles(int8_tile_plan_of(shape, false, m, n, k, nmat), m, n, k, nmat);
    bound(1 + rand() % 600, m, n, k, nmat);
    bound(m - rand() % (m - 1), m, n, k, nmat);
    plans += 4;
  }
  if (bad) return 1;
  printf("ok %d\n", plans);
  return 0;
}
