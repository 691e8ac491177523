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
