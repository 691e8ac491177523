// Sweeps the KV cache attention's plan against its workspace bound: whatever a
// call of these sizes or smaller ones plans, with any window, has to fit.
// Prints one line per call that does not, then "checked=N over=M".
#include <cstdio>
#include <cstdlib>
#include <random>

#include "kv8_plan.h"

using namespace nvfp4;

struct Sizes {
  int seqs, heads, group, dim, rows, len, window;
};

static Kv8Attn attn(const Sizes &z) {
  Kv8Attn a{};
  a.q_heads = z.heads * z.group;
  a.max_len = z.len;
  a.window = z.window;
  return a;
}
static Kv8Batch batch(const Sizes &z) { return Kv8Batch{nullptr, nullptr, nullptr, z.seqs, 1, z.rows * z.seqs, z.rows}; }

static long checked = 0, over = 0;

static void check(const Sizes &made, const Sizes &used, bool weights) {
  static float w;
  const Kv8Pool c{nullptr, nullptr, nullptr, nullptr, weights ? &w : nullptr, 1, made.heads, 4};
  const size_t bound = kv8_workspace_bound(attn(made), c, batch(made), made.dim);
  // with weights, what a call that accumulates takes, and what one that does not
  for (int accumulate = 0; accumulate <= (weights ? 1 : 0); ++accumulate) {
    Kv8Plan pl = kv8_plan(attn(used), c, batch(used), used.dim);
    if (!accumulate) pl.score_floats = 0;
    ++checked;
    if (kv8_workspace_bytes(pl) <= bound) continue;
    if (++over <= 20)
      printf("seqs=%d heads=%d group=%d dim=%d rows=%d len=%d weights=%d: %zu bytes, a call of seqs=%d rows=%d len=%d "
             "window=%d takes %zu\n",
             made.seqs, made.heads, made.group, made.dim, made.rows, made.len, weights, bound, used.seqs, used.rows,
             used.len, used.window, kv8_workspace_bytes(pl));
  }
}

int main(int argc, char **argv) {
  std::mt19937 g(7);
  auto log_of = [&](double lo, double hi) {  // whole, spread over its logarithm
    std::uniform_real_distribution<double> u(std::log(lo), std::log(hi + 1));
    return (int)std::min(std::max(std::floor(std::exp(u(g))), lo), hi);
  };
  // windows that add a step to a whole number of pieces; rounds that pieces just fill or just pass
  for (int weights = 0; weights < 2; ++weights) {
    check({64, 8, 8, 128, 16, 3968, 0}, {64, 8, 8, 128, 16, 3968, 4096}, weights);
    check({48, 8, 8, 256, 8, 7936, 0}, {48, 8, 8, 256, 8, 7936, 7936}, weights);
    check({8, 8, 4, 128, 1, 524288, 0}, {8, 8, 4, 128, 1, 524288, 454351}, weights);
    check({1, 8, 1, 256, 1, 520000, 0}, {1, 8, 1, 256, 1, 520000, 500000}, weights);
    check({8, 8, 4, 128, 1, 600000, 0}, {8, 8, 4, 128, 1, 422923, 0}, weights);
    for (int len : {507904, 507905, 1015808, 1015809}) check({2, 8, 4, 64, 8, len, 0}, {2, 8, 4, 64, 8, 507904, 0}, weights);
  }
  const int dims[] = {64, 128, 256};
  const long n = argc > 1 ? atol(argv[1]) : 20000;
  for (long i = 0; i < n; ++i) {
    Sizes z{log_of(1, 4096), 1 << (int)(g() % 6), 1 + (int)(g() % 16), dims[g() % 3], log_of(1, 8192), 0, 0};
    z.len = g() % 2 ? log_of(1, 1 << 22) : 3968 * (1 + (int)(g() % 160)) + (int)(g() % 65) - 32;
    const bool weights = g() % 2;
    for (int k = 0; k < 12; ++k) {
      Sizes u = z;
      if (k % 2) u.rows = log_of(1, z.rows);
      if (k % 3 == 1) u.len = log_of(1, z.len);
      if (k % 3 == 2) u.len = std::min(z.len, 507904);
      if (k > 8) u.seqs = log_of(1, z.seqs);
      u.window = k % 4 == 0 ? 0 : k % 4 == 1 ? log_of(1, u.len) : k % 4 == 2 ? u.len : 0x7FFFFFFF;
      check(z, u, weights);
    }
  }
  printf("checked=%ld over=%ld\n", checked, over);
  return over != 0;
}
