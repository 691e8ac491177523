// Which kernels, and which ways through them, the int8 products' plans choose
// (nvfp4_weight_dense_amd/csrc/int8_plan.h), on the CPU.
//   int8_plan_classes of < lines of "m n k nmat"   the classes of each, on a line
//   int8_plan_classes all                          every class that a sweep of sizes meets, with its smallest product
// A class: ring, rows of a tile, slots, matrices, parts or whole groups, one
// round of them or more; or tile, shape, matrices, whole tiles (none, one
// round or more), parts of others, one of two launches.
#include <cstdio>
#include <cstring>
#include <map>
#include <string>
#include <vector>

#include "int8_plan.h"

using namespace nvfp4;

static std::vector<std::string> classes(int m, int n, int k, int nmat) {
  char b[96];
  std::vector<std::string> r;
  if (m <= kInt8RingRows) {
    const Int8Plan p = int8_plan(m, n, k, nmat);
    snprintf(b, sizeof b, "ring-mt%d-slots%d-x%d-%s", p.mt, p.slots, nmat,
             p.parts > 1 ? "parts" : p.groups > p.nwg ? "rounds" : "whole");
    return {b};
  }
  const Int8TilePlans two = int8_tile_plan(m, n, k, nmat);
  for (int i = 0; i < two.count; ++i) {
    const Int8TilePlan &p = two.part[i];
    const int split = p.row_blocks * p.groups - p.whole;
    snprintf(b, sizeof b, "tile%d-x%d-%s%s", p.shape, nmat, p.whole == 0 ? "" : p.whole > p.nwg ? "rounds" : "whole",
             split ? "-parts" : "");
    r.push_back(b);
  }
  if (two.count > 1) {
    snprintf(b, sizeof b, "tile-two-launches-x%d", nmat);
    r.push_back(b);
  }
  return r;
}

int main(int argc, char **argv) {
  if (argc > 1 && !strcmp(argv[1], "of")) {
    int m, n, k, nmat;
    while (scanf("%d %d %d %d", &m, &n, &k, &nmat) == 4) {
      for (const std::string &c : classes(m, n, k, nmat)) printf("%s ", c.c_str());
      printf("\n");
    }
    return 0;
  }
  struct Size {
    double work;
    int m, n, k;
  };
  std::map<std::string, Size> least;
  const int rows[] = {5, 16, 17, 32, 33, 64, 65, 100, 128, 129, 200, 256, 257, 300, 384, 512, 513, 700, 1024, 1300, 1536, 2048, 2500, 4096};
  for (int nmat = 1; nmat <= 2; ++nmat)
    for (int m : rows)
      for (int n = 32; n <= 200000; n += n < 512 ? 32 : n < 4096 ? 96 : n < 20000 ? 352 : 10016)
        for (int k = 32; k <= (n < 20000 ? 18432 : 256); k += k < 512 ? 32 : k < 4096 ? 224 : 1024) {
          const double work = (double)m * n * k * nmat + 1e3 * (double)n * k * nmat;
          for (const std::string &c : classes(m, n, k, nmat)) {
            auto it = least.find(c);
            if (it == least.end() || work < it->second.work) least[c] = Size{work, m, n, k};
          }
        }
  for (const auto &c : least) printf("%s %d %d %d\n", c.first.c_str(), c.second.m, c.second.n, c.second.k);
  return 0;
}
