// k_int8_tile.hip -- the int8 projection of many rows (gfx950), bound by the
// matrix cores (the formula and why any split of K gives the same bits:
// k_int8_gemm.hip).
//
// A workgroup of eight waves computes tiles of the output.  Both operands go
// from memory straight into a ring in LDS, 128 codes of K (a unit) at a time,
// as whole lines; a wave's part of a tile is MT x 2 blocks of
// v_mfma_i32_32x32x32_i8, for which it reads MT + 2 operands of 1 KB from LDS
// for each quarter of a unit.  The quarters alternate between two sets of
// registers: the reads of the next are issued before the products of this
// one, across units too.  The barrier of a unit lies before its last quarter:
// it says that the next unit has arrived for all waves, and that this unit's
// last operands are in registers everywhere, so its place in the ring is free.
//
// A row of a unit is 128 bytes, eight chunks of 16; chunk q of row r is stored
// at q ^ (r / 2 % 8), so that the rows that are read together lie in different
// banks.  The weights are the first operand: a lane then holds four
// neighbouring columns of one row, and after a trade between lanes stores
// eight of them at once.  The scales come into LDS with a tile's first unit,
// so that a tile's end waits for no memory.
//
// 8192 x 8192 x 8192 477 to 487 us (2260 to 2305 TOP/s; a library's product of
// that size 534); 2048 rows of 17408 x 5120 in two launches 198 to 205 (186
// with one set of operands again and again, which the last cache holds), gate
// and up of the same FFN 359, down 196.  (Operands in turn; a kernel's time
// under the profiler.)  The matrix cores are 55% busy
// in tiles of 256 x 256 (48% in 256 x 128), 80% of the lines come from L2, no
// bank conflicts.  Of the products and the transfers either alone takes 80% of
// the time: they share the LDS.
#include "int8_common.h"

namespace nvfp4 {

namespace {

constexpr int kWaves = 8;

struct TileArgs {
  const int8_t *x;
  const float *xs;
  int m, k, n;
  const int8_t *w0, *w1;
  const float *s0, *s1;
  void *y;
  int ldy;             // columns of y, of which this launch's are the first n
  int *partial;        // [split tile][part][8 waves][2 MT][4][64 lanes][4]
  unsigned *counters;  // [split tile], zero between calls
  int row_blocks, groups, units, whole, parts;
};

// WM: waves along the rows (8 / WM along the columns); MT: 32-row blocks of a wave
template <int WM, int MT>
struct Cfg {
  static constexpr int kRows = WM * MT * 32, kCols = 8 / WM * 64;
  static constexpr uint32_t kXBytes = kRows * kInt8TileK, kStage = (kRows + kCols) * kInt8TileK;
  // The scales of a tile, its rows' and then its columns', come with its first
  // unit, 64 to a wave.  A unit is requested kStages ahead, which may be as many tiles.
  static constexpr uint32_t kScaleBytes = kWaves * 64 * 4;
  static constexpr int kStages = (160 * 1024 - 256) / (kStage + kScaleBytes) > 4 ? 4 : (160 * 1024 - 256) / (kStage + kScaleBytes);
  static constexpr int kScales = kStages + 1;
  static_assert(kRows + kCols <= kWaves * 64 && kRows % 64 == 0 && kCols / 2 % 64 == 0, "scales of a wave");
  static constexpr int kX = kRows / 8 / kWaves, kW = kCols / 8 / kWaves;  // transfers of a wave for a unit
  static constexpr uint32_t kWavePiece = 2u * MT * 16u * 256u;
};

template <int WM, int MT, int NMAT>
__global__ __launch_bounds__(kWaves * 64, 2) void k_int8_tile(TileArgs p) {
  typedef Cfg<WM, MT> C;
  constexpr int S = C::kStages, X = C::kX + C::kW;
  constexpr int kCols = C::kCols / NMAT;
  static_assert(kWaves * C::kWavePiece == C::kRows * C::kCols * 4, "a piece");
  __shared__ __attribute__((aligned(1024))) uint8_t ring[S * C::kStage];
  __shared__ __attribute__((aligned(256))) float scales[C::kScales][kWaves * 64];
  __shared__ unsigned last_flag;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave % WM, wn = wave / WM;
  const int c = lane & 31, h = lane >> 5;
  const uint32_t ring_at = lds_address(ring);
  // Workgroups go to the eight XCDs in turn; each XCD takes a contiguous run
  // of the workgroups' numbers, so that neighbouring tiles, which share rows
  // or columns, are read through one L2.
  const int nwg = (int)gridDim.x;
  const int me = [&] {
    const int q = nwg >> 3, rem = nwg & 7, xcd = (int)blockIdx.x & 7;
    return xcd * q + min(xcd, rem) + ((int)blockIdx.x >> 3);
  }();

  // ---- this workgroup's work: tiles me, me + nwg, .. of the whole ones, then
  // pairs me, me + nwg, .. of the others and their parts (int8_plan.h)
  const int tiles = p.row_blocks * p.groups, split = tiles - p.whole, pairs = split * p.parts;
  const int mine = me < p.whole ? (p.whole - me + nwg - 1) / nwg : 0;
  auto part_begin = [&](int part) __attribute__((always_inline)) { return p.units * part / p.parts; };
  int count = mine * p.units;  // units of this workgroup
  for (int i = me; i < pairs; i += nwg) count += part_begin(i / split + 1) - part_begin(i / split);
  // a place in its work: tile, part, unit of K and the part's end, tiles done
  struct At {
    int tile, part, unit, end, done;
  };
  auto go = [&](At &a) __attribute__((always_inline)) {
    if (a.done < mine) {
      a.tile = me + a.done * nwg, a.part = 0, a.unit = 0, a.end = p.units;
    } else {
      const int i = me + (a.done - mine) * nwg;
      if (i < pairs) {
        a.part = i / split, a.tile = p.whole + i - a.part * split;
        a.unit = part_begin(a.part), a.end = part_begin(a.part + 1);
      } else {
        a.tile = 0, a.part = 0, a.unit = 0, a.end = p.units;  // (past the work: not used)
      }
    }
  };
  // Row blocks of eight, columns within them, rows fastest: 32 tiles in a row
  // are eight row blocks of four column groups.
  auto place = [&](int tile, int &rb, int &cg) __attribute__((always_inline)) {
    const int super = tile / (8 * p.groups), in = tile - super * 8 * p.groups;
    const int high = min(8, p.row_blocks - 8 * super);
    cg = in / high;
    rb = 8 * super + in - cg * high;
  };

  // ---- requests: activation rows 8 t + lane / 8; weight rows 8 t + lane / 8
  // of the tile's columns (with two matrices 32 of gate and 32 of up in turn)
  const uint32_t line = (uint32_t)lane >> 3;
  uint32_t lk[2], voff[2];  // for even and odd t
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    lk[j] = 16u * ((lane & 7u) ^ (4u * j + (line >> 1)));
    voff[j] = line * (uint32_t)p.k + lk[j];
  }
  At la;
  la.done = 0;
  go(la);
  int requested = 0;
  bool fresh = true;  // the next request is a tile's first
  u32x4_t xr, wr[C::kW], sr;
  int scale_set = 0;
  const uint32_t scales_at = lds_address(scales) + (uint32_t)wave * 256u;
  auto ranges = [&]() __attribute__((always_inline)) {
    int rb, cg;
    place(la.tile, rb, cg);
    const int row0 = rb * C::kRows, col0 = cg * kCols;
    // this wave's scales: 64 rows', or 64 columns' of a matrix
    const int at = (wave * 64 - C::kRows) & (kCols - 1);
    const bool up = NMAT > 1 && wave * 64 >= C::kRows + kCols;
    if (wave * 64 < C::kRows)
      sr = range_of(p.xs + min(row0 + wave * 64, p.m), (size_t)max(min(64, p.m - row0 - wave * 64), 0) * 4);
    else
      sr = range_of((up ? p.s1 : p.s0) + min(col0 + at, p.n), (size_t)max(min(64, p.n - col0 - at), 0) * 4);
    xr = range_of(p.x + (size_t)row0 * p.k, (size_t)min(C::kRows, p.m - row0) * p.k);
#pragma unroll
    for (int j = 0; j < C::kW; ++j) {
      const int t = wave * C::kW + j;
      const int at = col0 + (NMAT > 1 ? (t >> 3) * 32 + (t & 3) * 8 : 8 * t);
      wr[j] = range_of((NMAT > 1 && (t & 4) ? p.w1 : p.w0) + (size_t)min(at, p.n) * p.k,
                       (size_t)max(min(8, p.n - at), 0) * p.k);
    }
  };
  ranges();
  auto request = [&](uint32_t stage) __attribute__((always_inline)) {
    const bool live = requested < count;
    // (0 past the run: an offset of its own must not pass a range that is empty there)
    const uint32_t k0 = live ? (uint32_t)la.unit * kInt8TileK : 0u;
    const uint32_t to = ring_at + stage * C::kStage;
    if (live && fresh) {
      words_to_lds(sr, scales_at + (uint32_t)scale_set * C::kScaleBytes, 4u * (uint32_t)lane);
      scale_set = scale_set == C::kScales - 1 ? 0 : scale_set + 1;
    }
    fresh = false;
#pragma unroll
    for (int j = 0; j < C::kX; ++j) {
      const uint32_t t = (uint32_t)(wave * C::kX + j);
      to_lds(xr, to + t * 1024u,
             live && k0 + lk[j & 1] < (uint32_t)p.k ? voff[j & 1] + 8u * t * (uint32_t)p.k : kOOB, k0);
    }
#pragma unroll
    for (int j = 0; j < C::kW; ++j)
      // (a range without rows takes no offset either)
      to_lds(wr[j], to + C::kXBytes + (uint32_t)(wave * C::kW + j) * 1024u, live ? voff[j & 1] : kOOB,
             wr[j][2] ? k0 : 0u);
    ++requested;
    if (++la.unit == la.end) {
      ++la.done;
      go(la);
      ranges();
      fresh = true;
    }
  };

  i32x16 acc[2][MT];
  auto clear = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[j][t][e] = 0;
  };
  struct Step {
    i32x4 a[MT], b[2];
  };
  const uint32_t swz = ((uint32_t)c >> 1) & 7u;
  auto read = [&](uint32_t stage, int kk, Step &f) __attribute__((always_inline)) {
    const uint8_t *at = ring + stage * C::kStage + (uint32_t)c * 128u + 16u * ((uint32_t)(2 * kk + h) ^ swz);
#pragma unroll
    for (int j = 0; j < 2; ++j) f.b[j] = *(const i32x4 *)(at + C::kXBytes + (uint32_t)(wn * 64 + j * 32) * 128u);
#pragma unroll
    for (int t = 0; t < MT; ++t) f.a[t] = *(const i32x4 *)(at + (uint32_t)((wm * MT + t) * 32) * 128u);
  };
  auto multiply = [&](const Step &f) __attribute__((always_inline)) {
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[j][t] = __builtin_amdgcn_mfma_i32_32x32x32_i8(f.b[j], f.a[t], acc[j][t], 0, 0, 0);
    // a read after each of the first products
#pragma unroll
    for (int i = 0; i < 2 * MT; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      if (i < MT + 2) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    }
  };

  // Element e of block (j, t): row 32 (wm MT + t) + c of the tile, column
  // 8 (e / 4) + 4 h + e % 4 of the block's 32.
  int epilogue_set = 0;
  auto epilogue = [&](int tile) __attribute__((always_inline)) {
    int rb, cg;
    place(tile, rb, cg);
    const float *set = scales[epilogue_set];
    const int row0 = rb * C::kRows + wm * MT * 32 + c;
#pragma unroll
    for (int j = 0; j < (NMAT > 1 ? 1 : 2); ++j)
#pragma unroll
      for (int q = 0; q < 2; ++q) {  // sixteen of the block's columns: elements 8 q ..
        const int col0 = cg * kCols + (NMAT > 1 ? wn * 32 : wn * 64 + j * 32) + 16 * q;
        Int8Scale s0[8], s1[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float *col = set + C::kRows + (col0 - cg * kCols) + 8 * (e >> 2) + 4 * h + (e & 3);
          s0[e] = int8_scale(col[0]);
          if (NMAT > 1) s1[e] = int8_scale(col[kCols]);
        }
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          const int r = row0 + 32 * t;
          const Int8Scale rs = int8_scale(set[wm * MT * 32 + 32 * t + c]);
          uint32_t v[4];  // two columns each
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            bf16x2 two;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float f = int8_scaled(acc[j][t][8 * q + e + i], rs, s0[e + i]);
              two[i] = NMAT > 1 ? swiglu_bf16(f, int8_scaled(acc[1][t][8 * q + e + i], rs, s1[e + i])) : (__bf16)f;
            }
            v[e >> 1] = __builtin_bit_cast(uint32_t, two);
          }
          __bf16 *to = (__bf16 *)p.y + (size_t)r * p.ldy + col0;
          // Lane (c, 0) holds columns 0..3 of either eight and lane (c, 1)
          // columns 4..7: they trade halves, and each has a whole eight.
          const auto lo = __builtin_amdgcn_permlane32_swap(v[0], v[2], false, false);
          const auto hi = __builtin_amdgcn_permlane32_swap(v[1], v[3], false, false);
          const u32x4_at2 eight{lo[0], hi[0], lo[1], hi[1]};
          const int left = p.n - (col0 + 8 * h);
          if (r < p.m && left >= 8) {
            *(u32x4_at2 *)(to + 8 * h) = eight;
          } else if (r < p.m) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (e < left) to[8 * h + e] = __builtin_bit_cast(__bf16, (uint16_t)(e & 1 ? eight[e >> 1] >> 16 : eight[e >> 1]));
          }
        }
      }
  };
  auto piece = [&](int tile, int part) __attribute__((always_inline)) {
    const size_t at = ((size_t)(tile - p.whole) * p.parts + part) * kWaves + wave;
    return rsrc_uniform((const uint8_t *)p.partial + at * C::kWavePiece, C::kWavePiece);
  };
  auto each_part = [&](auto &&f) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int q = 0; q < 4; ++q) f(acc[j][t], q, (uint32_t)((j * MT + t) * 4 + q) * 1024u + 16u * (uint32_t)lane);
  };
  // the end of a tile, or of a part of one
  auto flush = [&](int tile, int part) __attribute__((always_inline)) {
    bool finish = true;
    if (tile >= p.whole) {
      const __amdgpu_buffer_rsrc_t out = piece(tile, part);
      each_part([&](const i32x16 &v, int q, uint32_t off) __attribute__((always_inline)) {
        st16_coherent(out, off, i32x4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]});
      });
      wait_all_memory();
      __syncthreads();
      if (tid == 0)
        last_flag = __hip_atomic_fetch_add(&p.counters[tile - p.whole], 1u, __ATOMIC_RELAXED,
                                           __HIP_MEMORY_SCOPE_AGENT) == (unsigned)(p.parts - 1);
      __syncthreads();
      finish = last_flag != 0;
      if (finish) {
        for (int v = 0; v < p.parts; ++v) {
          if (v == part) continue;  // (still in registers)
          const __amdgpu_buffer_rsrc_t r = piece(tile, v);
          each_part([&](i32x16 &s, int q, uint32_t off) __attribute__((always_inline)) {
            const i32x4 w = ld16_coherent(r, off);
#pragma unroll
            for (int e = 0; e < 4; ++e) s[4 * q + e] += w[e];
          });
        }
        if (tid == 0)
          __hip_atomic_store(&p.counters[tile - p.whole], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
    }
    if (finish) epilogue(tile);
    epilogue_set = epilogue_set == C::kScales - 1 ? 0 : epilogue_set + 1;
    clear();
    // (Memory operations end in order, so with stores among the youngest the
    // waits of the unit loop cover more transfers than they ask for, never fewer.)
  };

#pragma unroll
  for (int i = 0; i < S; ++i) request((uint32_t)i);
  clear();
  At at;
  at.done = 0;
  go(at);
  uint32_t stage = 0;
  Step f0, f1;
  wait_transfers<(S - 1) * X>();
  ring_barrier();
  read(0, 0, f0);
  for (int i = 0; i < count; ++i) {
    read(stage, 1, f1);
    multiply(f0);
    read(stage, 2, f0);
    multiply(f1);
    read(stage, 3, f1);
    multiply(f0);
    wait_transfers<(S - 2) * X>();
    ring_barrier();
    request(stage);
    stage = stage == S - 1 ? 0 : stage + 1;
    const bool ends = ++at.unit == at.end;
    if (!ends) read(stage, 0, f0);
    multiply(f1);
    if (ends) {  // (the next operands only behind it: it has no registers to spare)
      flush(at.tile, at.part);
      ++at.done;
      go(at);
      read(stage, 0, f0);
    }
  }
  wait_all_memory();
}

template <int WM, int MT>
hipError_t launch_shape(const TileArgs &p, int shape, int nmat, int nwg, hipStream_t s) {
  static_assert(Cfg<WM, MT>::kStages >= 2, "a ring of two units at least");
  if (Cfg<WM, MT>::kRows != kInt8Tiles[shape].rows || Cfg<WM, MT>::kCols != kInt8Tiles[shape].cols)
    return hipErrorInvalidValue;
  if (nmat == 1)
    hipLaunchKernelGGL((k_int8_tile<WM, MT, 1>), dim3(nwg), dim3(kWaves * 64), 0, s, p);
  else
    hipLaunchKernelGGL((k_int8_tile<WM, MT, 2>), dim3(nwg), dim3(kWaves * 64), 0, s, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_int8_tile(const Int8ActRef &a, int m, int k, int n, int nmat, const Int8MatRef *w, void *y,
                            const Int8TilePlans &pl, unsigned *counters, int *partial, hipStream_t s) {
  int col0 = 0;
  for (int i = 0; i < pl.count; ++i) {
    const Int8TilePlan &q = pl.part[i];
    auto codes = [&](int j) { return w[j].codes + (size_t)col0 * k; };
    const TileArgs p{a.codes, a.row_scale, m, k, q.columns, codes(0), nmat > 1 ? codes(1) : nullptr, w[0].scales + col0,
                     nmat > 1 ? w[1].scales + col0 : nullptr, (__bf16 *)y + col0, n, partial, counters, q.row_blocks,
                     q.groups, q.units, q.whole, q.parts};
    hipError_t e;
    switch (q.shape) {
      case 0: e = launch_shape<2, 4>(p, 0, nmat, q.nwg, s); break;
      case 1: e = launch_shape<4, 2>(p, 1, nmat, q.nwg, s); break;
      case 2: e = launch_shape<2, 2>(p, 2, nmat, q.nwg, s); break;
      default: e = launch_shape<4, 1>(p, 3, nmat, q.nwg, s); break;
    }
    if (e != hipSuccess) return e;
    col0 += q.columns;
  }
  return hipSuccess;
}

}  // namespace nvfp4
