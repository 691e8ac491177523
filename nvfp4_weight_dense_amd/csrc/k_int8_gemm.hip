// k_int8_gemm.hip -- the int8 projection (gfx950) up to 256 rows a pass,
// bound by reading the weight once:
//
//   y[r][c] = bf16( s_row[r] * s_col[c] * sum_k x[r][k] * w[c][k] )
//
// The sum is of whole numbers, |x| <= 127 and |w| <= 128, below 2^31 for the
// k that are allowed: every order of summation gives the same bits, so a
// row's result does not depend on the rows beside it or on how K is split,
// and K is split wherever that fills the CUs.
//
// One workgroup of eight waves per CU walks an equal run of (column group,
// K unit) pairs (int8_plan.h).  A unit is 128 codes of 128 weight rows and of
// every activation row: whole 128-byte lines, moved from memory straight into
// a ring in LDS by 16-byte lanes, as many units ahead as LDS holds (two
// thirds of it are weights under way; registers hold none).  One barrier a
// unit: it says that a unit has arrived for all waves and that the one before
// it has been read by all, so its place is free for the unit that is
// requested next.
//
// Wave (s, h) = (wave % 4, wave / 4) owns columns 32 s .. of the group -- or
// gate and up columns 16 s .. -- for half of the rows, or with one row tile
// for half of each unit's K.  Operands are read from LDS in 16-byte lanes
// (v_mfma_i32_16x16x64_i8: lane (c, g) holds row c, K 16 g ..); the eight
// chunks of a line are stored at chunk ^ (row / 2 % 8), so that the sixteen
// rows of a read lie in different banks.
#include "int8_common.h"

namespace nvfp4 {

namespace {

constexpr int kWaves = 8;
constexpr uint32_t kWeightBytes = kInt8GroupCols * kInt8UnitK;

struct Int8Args {
  const int8_t *x;  // [m][k]
  const float *xs;  // [m]
  int m, k, n;
  const int8_t *w0, *w1;  // gate and up, or the matrix and null
  const float *s0, *s1;
  void *y;
  int *partial;        // [nwg][2][waves with sums][2 kTiles][64 lanes][4]
  unsigned *counters;  // [nwg], zero between calls
  int units, all, nwg; // units of a group, pairs in all, workgroups
};

// MT: 16-row tiles of the workgroup
template <int MT>
struct Cfg {
  static constexpr uint32_t kStage = kWeightBytes + 2048u * MT;
  static constexpr int kStages = MT == 1 ? 8 : MT == 2 ? 7 : MT == 4 ? 6 : MT == 8 ? 4 : 3;
  static constexpr bool kSplitK = MT == 1;          // the wave halves: of K, else of the rows
  static constexpr int kTiles = kSplitK ? 1 : MT / 2;  // row tiles of a wave
  // transfers of a wave for a unit: two of weights, and of the 2 MT of
  // activations that many, for waves below kXWaves
  static constexpr int kX = MT >= 4 ? MT / 4 : 1;
  static constexpr int kXWaves = MT >= 4 ? kWaves : 2 * MT;
  // a piece of a split group: what each wave (of a split K: of half 0) holds
  static constexpr uint32_t kWavePiece = 2u * kTiles * 1024u;
  static constexpr int kPieceWaves = kSplitK ? 4 : kWaves;
};

template <int MT, int NMAT>
__global__ __launch_bounds__(kWaves * 64, 2) void k_int8_gemm(Int8Args p) {
  typedef Cfg<MT> C;
  constexpr int T = C::kTiles, S = C::kStages;
  constexpr int kCols = kInt8GroupCols / NMAT;
  static_assert(C::kPieceWaves * C::kWavePiece == kInt8GroupCols * 16 * MT * 4, "int8_piece_bytes");
  __shared__ __attribute__((aligned(1024))) uint8_t ring[S * C::kStage];
  __shared__ i32x4 halves[C::kSplitK ? 4 * 2 * 64 : 1];
  __shared__ unsigned last_flag;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int slot = wave & 3, half = wave >> 2;
  const int c = lane & 15, g = lane >> 4;
  const int me = (int)blockIdx.x;
  const int begin = int8_run_begin(p.all, p.nwg, me), count = int8_run_begin(p.all, p.nwg, me + 1) - begin;
  const uint32_t ring_at = lds_address(ring);

  // ---- requests: weight rows 16 wave + 8 j + lane / 8 of the group (gate for
  // waves 0..3 and up for the others, with two matrices), activation rows
  // 8 t + lane / 8
  const uint32_t line = (uint32_t)lane >> 3;
  uint32_t wvoff[2], xvoff[C::kX], xk[C::kX];
  const uint32_t wrow = NMAT > 1 ? 16u * (uint32_t)(wave & 3) : 16u * (uint32_t)wave;
#pragma unroll
  for (int j = 0; j < 2; ++j)
    wvoff[j] = (wrow + 8u * j + line) * (uint32_t)p.k + 16u * ((lane & 7u) ^ (4u * j + (line >> 1)));
#pragma unroll
  for (int j = 0; j < C::kX; ++j) {
    const uint32_t t = (uint32_t)(wave * C::kX + j);
    xk[j] = 16u * ((lane & 7u) ^ (4u * (t & 1u) + (line >> 1)));
    xvoff[j] = (8u * t + line) * (uint32_t)p.k + xk[j];
  }
  const u32x4_t xr = range_of(p.x, (size_t)p.m * p.k);
  const int8_t *wmat = NMAT > 1 && wave >= 4 ? p.w1 : p.w0;
  int lgroup = begin / p.units, lunit = begin - lgroup * p.units, requested = 0;
  u32x4_t wr;
  auto group_range = [&]() __attribute__((always_inline)) {
    const int at = lgroup * kCols;
    wr = range_of(wmat + (size_t)at * p.k, (size_t)max(min(kCols, p.n - at), 0) * p.k);
  };
  group_range();
  auto request = [&](uint32_t stage) __attribute__((always_inline)) {
    const bool live = requested < count;
    // (0 past the run: an offset of its own must not pass a range that is empty there)
    const uint32_t k0 = live ? (uint32_t)lunit * kInt8UnitK : 0u;
    const uint32_t to = ring_at + stage * C::kStage;
#pragma unroll
    for (int j = 0; j < 2; ++j) to_lds(wr, to + (uint32_t)(wave * 2 + j) * 1024u, live ? wvoff[j] : kOOB, k0);
    if (wave < C::kXWaves) {
#pragma unroll
      for (int j = 0; j < C::kX; ++j)
        to_lds(xr, to + kWeightBytes + (uint32_t)(wave * C::kX + j) * 1024u,
               live && k0 + xk[j] < (uint32_t)p.k ? xvoff[j] : kOOB, k0);
    }
    ++requested;
    if (++lunit == p.units) {
      lunit = 0, ++lgroup;
      group_range();
    }
  };

  i32x4 acc[2][T] = {};
  // operands of a unit: column tile j at weight rows 64 j + 16 slot or
  // 32 slot + 16 j, K chunk 4 kk + g
  const uint32_t swz = ((uint32_t)c >> 1) & 7u;
  auto compute = [&](uint32_t stage) __attribute__((always_inline)) {
    const uint8_t *at = ring + stage * C::kStage;
    constexpr int kSteps = C::kSplitK ? 1 : 2;
#pragma unroll
    for (int kk = 0; kk < kSteps; ++kk) {
      const uint32_t chunk = 16u * (((uint32_t)((C::kSplitK ? half : kk) * 4 + g)) ^ swz);
      i32x4 b[2];
#pragma unroll
      for (int j = 0; j < 2; ++j)
        b[j] = *(const i32x4 *)(at + (uint32_t)((NMAT > 1 ? 64 * j + 16 * slot : 32 * slot + 16 * j) + c) * 128u + chunk);
#pragma unroll
      for (int t = 0; t < T; ++t) {
        const int row = 16 * ((C::kSplitK ? 0 : half * T) + t) + c;
        const i32x4 a = *(const i32x4 *)(at + kWeightBytes + (uint32_t)row * 128u + chunk);
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[j][t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b[j], acc[j][t], 0, 0, 0);
      }
    }
  };

  // element e of row tile t: row 16 (half T + t) + 4 g + e
  auto epilogue = [&](int group) __attribute__((always_inline)) {
    const int row0 = C::kSplitK ? 0 : 16 * half * T;
    if (C::kSplitK && half) return;
#pragma unroll
    for (int j = 0; j < (NMAT > 1 ? 1 : 2); ++j) {
      const int col = group * kCols + (NMAT > 1 ? 16 * slot : 32 * slot + 16 * j) + c;
      const bool in = col < p.n;
      const Int8Scale s0 = int8_scale(in ? p.s0[col] : 0.0f);
      const Int8Scale s1 = NMAT > 1 ? int8_scale(in ? p.s1[col] : 0.0f) : s0;
#pragma unroll
      for (int t = 0; t < T; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = row0 + 16 * t + 4 * g + e;
          if (r >= p.m || !in) continue;
          const Int8Scale rs = int8_scale(p.xs[r]);
          const float v = int8_scaled(acc[j][t][e], rs, s0);
          ((__bf16 *)p.y)[(size_t)r * p.n + col] =
              NMAT > 1 ? swiglu_bf16(v, int8_scaled(acc[1][t][e], rs, s1)) : (__bf16)v;
        }
    }
  };
  auto piece = [&](int wg, int which) __attribute__((always_inline)) {
    const size_t at = (size_t)(wg * 2 + which) * C::kPieceWaves + (C::kSplitK ? slot : wave);
    return rsrc_uniform((const uint8_t *)p.partial + at * C::kWavePiece, C::kWavePiece);
  };
  // the end of this run's part of a group
  auto flush = [&](int group, bool whole) __attribute__((always_inline)) {
    if constexpr (C::kSplitK) {
      if (half) {
#pragma unroll
        for (int j = 0; j < 2; ++j) halves[(slot * 2 + j) * 64 + lane] = acc[j][0];
      }
      lds_barrier();
      if (!half) {
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[j][0] += halves[(slot * 2 + j) * 64 + lane];
      }
    }
    if (whole) {
      epilogue(group);
    } else {
      const int v0 = int8_run_owner(p.all, p.nwg, group * p.units);
      const int v1 = int8_run_owner(p.all, p.nwg, group * p.units + p.units - 1);
      const __amdgpu_buffer_rsrc_t mine = piece(me, group == begin / p.units ? 0 : 1);
      if (!C::kSplitK || !half) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int t = 0; t < T; ++t) st16_coherent(mine, (uint32_t)(j * T + t) * 1024u + 16u * lane, acc[j][t]);
      }
      wait_all_memory();
      __syncthreads();
      if (tid == 0)
        last_flag = __hip_atomic_fetch_add(&p.counters[v0], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
                    (unsigned)(v1 - v0);
      __syncthreads();
      if (last_flag) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int t = 0; t < T; ++t) acc[j][t] = i32x4{0, 0, 0, 0};
        for (int v = v0; v <= v1; ++v) {
          const __amdgpu_buffer_rsrc_t r = piece(v, group == int8_run_begin(p.all, p.nwg, v) / p.units ? 0 : 1);
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int t = 0; t < T; ++t) acc[j][t] += ld16_coherent(r, (uint32_t)(j * T + t) * 1024u + 16u * lane);
        }
        epilogue(group);
        if (tid == 0) __hip_atomic_store(&p.counters[v0], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int t = 0; t < T; ++t) acc[j][t] = i32x4{0, 0, 0, 0};
    // (the waits of the unit loop count transfers alone again)
    wait_all_memory();
  };

#pragma unroll
  for (int i = 0; i < S - 1; ++i) request((uint32_t)i);
  int group = begin / p.units, unit = begin - group * p.units, from = unit;
  uint32_t stage = 0;
  for (int i = 0; i < count; ++i) {
    // the S - 2 units behind this one may be under way
    if (wave < C::kXWaves)
      wait_transfers<(S - 2) * (2 + C::kX)>();
    else
      wait_transfers<(S - 2) * 2>();
    ring_barrier();
    request(stage == 0 ? S - 1 : stage - 1);
    compute(stage);
    stage = stage == S - 1 ? 0 : stage + 1;
    if (++unit == p.units || i == count - 1) {
      flush(group, from == 0 && unit == p.units);
      unit = 0, from = 0, ++group;
    }
  }
}

template <int MT>
hipError_t launch_mt(const Int8Args &p, int nmat, hipStream_t s) {
  if (nmat == 1)
    hipLaunchKernelGGL((k_int8_gemm<MT, 1>), dim3(p.nwg), dim3(kWaves * 64), 0, s, p);
  else
    hipLaunchKernelGGL((k_int8_gemm<MT, 2>), dim3(p.nwg), dim3(kWaves * 64), 0, s, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_int8_gemm(const Int8ActRef &a, int m, int k, int n, int nmat, const Int8MatRef *w, void *y,
                            const Int8Plan &pl, unsigned *counters, int *partial, hipStream_t s) {
  for (int r0 = 0; r0 < m; r0 += 256) {
    const Int8Args p{a.codes + (size_t)r0 * k, a.row_scale + r0, m - r0 < 256 ? m - r0 : 256, k, n, w[0].codes,
                     nmat > 1 ? w[1].codes : nullptr, w[0].scales, nmat > 1 ? w[1].scales : nullptr,
                     (__bf16 *)y + (size_t)r0 * n, partial, counters, pl.units, pl.groups * pl.units, pl.nwg};
    hipError_t e;
    switch (pl.mt) {
      case 1: e = launch_mt<1>(p, nmat, s); break;
      case 2: e = launch_mt<2>(p, nmat, s); break;
      case 4: e = launch_mt<4>(p, nmat, s); break;
      case 8: e = launch_mt<8>(p, nmat, s); break;
      default: e = launch_mt<16>(p, nmat, s); break;
    }
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace nvfp4
