// k_int8_gemm.hip -- the int8 projection of up to 64 rows (gfx950), bound by
// reading the weight once:
//
//   y[r][c] = bf16( s_row[r] * s_col[c] * sum_k x[r][k] * w[c][k] )
//
// The sum is of whole numbers, |x| <= 127 and |w| <= 128, below 2^31 for the
// k that are allowed: every order of summation gives the same bits, so a
// row's result does not depend on the rows beside it or on how K is split.
//
// A workgroup of eight waves computes groups of P slots of columns (32 of one
// matrix, or 16 of gate and the same 16 of up), or a part of K of one group; P
// and the parts are chosen so that the CUs have equal work (int8_plan.h).  K
// goes by units of 128, each workgroup from a unit of its own around to it, so
// that the rows' lines that are read at one time, a row's length apart, do not
// all lie in the same few channels of memory.  The weight
// rows and all activation rows of a unit, whole lines, are moved from memory
// straight into a ring in LDS that holds as many units as fit, all but the
// one in work under way.  One barrier a unit: it says that the next unit has
// arrived for all waves and that the last operands of this one are in
// registers everywhere, so its place in the ring is free.  Half a unit's
// operands are read while the half before is multiplied: read, multiplied and
// only then waited for, a unit took 0.5 us whatever its bytes.
//
// Wave s < P multiplies slot s with all rows (v_mfma_i32_16x16x64_i8, operands
// from LDS in 16-byte lanes: lane (c, g) reads row c, K 16 g ..); it is idle
// most of the time.  Chunk q of a line of row r is stored at q ^ (r / 2 % 8),
// so that the sixteen rows of a read lie in different banks.  The weights are
// the first operand: a lane then holds four neighbouring columns of one row.
//
// 64 rows of 5120, 17408: gate and up 40.0 us (4.5 TB/s of weights), down 23
// to 25 us (3.6 to 3.9; its columns alone do not fill the CUs: 40 groups of
// four slots in six parts of K, whose sums go through memory; twice the pieces
// of them in flight gain nothing).  The matrix cores are 10 and 7% busy; no
// bank conflicts.
#include "int8_common.h"

namespace nvfp4 {

namespace {

constexpr int kWaves = 8;

struct Int8Args {
  const int8_t *x;  // [m][k]
  const float *xs;  // [m]
  int m, k, n;
  const int8_t *w0, *w1;  // gate and up, or the matrix and null
  const float *s0, *s1;
  void *y;
  int *partial;        // [group][part][P waves][2 MT][64 lanes][4]
  unsigned *counters;  // [group], zero between calls
  int groups, units, parts;
};

// MT: 16-row tiles; P: slots
template <int MT, int P>
struct Cfg {
  static constexpr uint32_t kWeights = 32u * P * kInt8UnitK;  // bytes of a unit
  static constexpr uint32_t kStage = kWeights + 16u * MT * kInt8UnitK;
  // transfers of a wave for a unit: of weights, eight rows each, wave, wave +
  // 8, .. of 4 P, and one of the 2 MT of activations (those past the last go
  // nowhere: all waves count alike)
  static constexpr int kW = (P + 1) / 2, kX = kW + 1;
  // The scales of a group come with its first unit, 64 to a wave: rows,
  // columns.  A unit is requested kStages ahead, which may be as many groups.
  static constexpr uint32_t kScaleBytes = 5 * 64 * 4;
  static constexpr int kFit = (160 * 1024 - 1024 - 256 - kScaleBytes) / (kStage + kScaleBytes);
  static constexpr int kStages = kFit > 16 ? 16 : kFit;
  static constexpr int kScales = kStages + 1;
  static constexpr uint32_t kWavePiece = 2u * MT * 1024u;
  static_assert(kStages >= 3, "a ring of three units at least");
};

template <int MT, int P, int NMAT>
__global__ __launch_bounds__(kWaves * 64, 2) void k_int8_gemm(Int8Args p) {
  typedef Cfg<MT, P> C;
  constexpr int S = C::kStages, kCols = 32 * P / NMAT;
  static_assert(P * C::kWavePiece == int8_piece_bytes(MT, P), "a piece");
  __shared__ __attribute__((aligned(1024))) uint8_t ring[S * C::kStage];
  __shared__ __attribute__((aligned(1024))) uint8_t nowhere[1024];
  __shared__ __attribute__((aligned(256))) float scales[C::kScales][C::kScaleBytes / 4];
  __shared__ unsigned last_flag;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = lane & 15, g = lane >> 4;
  const uint32_t ring_at = lds_address(ring), nowhere_at = lds_address(nowhere);

  // ---- this workgroup's work: groups me, me + nwg, .. , or with parts the
  // pair `me` of the groups and their parts, numbered part by part
  const int me = (int)blockIdx.x, nwg = (int)gridDim.x;
  const int part = p.parts > 1 ? me / p.groups : 0, first = me - part * p.groups;
  const int begin = p.units * part / p.parts, len = p.units * (part + 1) / p.parts - begin;
  const int items = p.parts > 1 ? 1 : (p.groups - me + nwg - 1) / nwg;
  const int count = items * len;
  const int turn = ((me >> 3) + 32 * (me & 7)) % len;  // (workgroups go to the eight XCDs in turn)

  // ---- requests: row 8 t + lane / 8 of transfer t, of the group's weights
  // (with two matrices the gate's rows first) and of the activations
  const uint32_t line = (uint32_t)lane >> 3;
  // (t is wave + 8 j: its row's swizzle goes by wave alone)
  const uint32_t lk = 16u * ((lane & 7u) ^ (4u * (wave & 1u) + (line >> 1)));
  const uint32_t voff = line * (uint32_t)p.k + lk;
  int lgroup = first, lunit = 0, lset = 0, requested = 0;
  bool fresh = true;  // the next request is a group's first
  u32x4_t wr[C::kW], sr;
  const u32x4_t xr = range_of(p.x + (size_t)min(8 * wave, p.m) * p.k, (size_t)max(min(8, p.m - 8 * wave), 0) * p.k);
  const uint32_t scales_at = wave < 5 ? lds_address(scales) + (uint32_t)wave * 256u : nowhere_at;
  auto ranges = [&]() __attribute__((always_inline)) {
    const int col0 = min(lgroup, p.groups - 1) * kCols;
#pragma unroll
    for (int j = 0; j < C::kW; ++j) {
      const int row = 8 * (wave + 8 * j);
      const bool up = NMAT > 1 && row >= kCols;
      const int at = col0 + (up ? row - kCols : row);
      wr[j] = range_of((up ? p.w1 : p.w0) + (size_t)min(at, p.n) * p.k,
                       (size_t)(row < 32 * P ? max(min(8, p.n - at), 0) : 0) * p.k);
    }
    // wave 0: the rows' scales; waves 1 .. 4: 64 columns' each, or with two
    // matrices waves 1 and 2 the gate's and 3 and 4 the up's
    const int at = col0 + 64 * (NMAT > 1 ? (wave - 1) & 1 : wave - 1);
    if (wave == 0) sr = range_of(p.xs, (size_t)p.m * 4);
    else
      sr = range_of((NMAT > 1 && wave > 2 ? p.s1 : p.s0) + min(at, p.n),
                    (size_t)(wave < 5 ? max(min(64, p.n - at), 0) : 0) * 4);
  };
  ranges();
  auto request = [&](uint32_t stage) __attribute__((always_inline)) {
    const bool live = requested < count;
    const int unit = lunit + turn < len ? lunit + turn : lunit + turn - len;
    const uint32_t k0 = live ? (uint32_t)(begin + unit) * kInt8UnitK : 0u;
    const uint32_t to = ring_at + stage * C::kStage;
    if (live && fresh) {
      words_to_lds(sr, scales_at + (wave < 5 ? (uint32_t)lset * C::kScaleBytes : 0u), 4u * (uint32_t)lane);
      lset = lset == C::kScales - 1 ? 0 : lset + 1;
    }
    fresh = false;
#pragma unroll
    for (int j = 0; j < C::kW; ++j) {
      const int t = wave + 8 * j;
      // (a range without rows takes no offset either)
      to_lds(wr[j], t < 4 * P ? to + (uint32_t)t * 1024u : nowhere_at, live ? voff : kOOB, wr[j][2] ? k0 : 0u);
    }
    to_lds(xr, wave < 2 * MT ? to + C::kWeights + (uint32_t)wave * 1024u : nowhere_at,
           live && wave < 2 * MT && k0 + lk < (uint32_t)p.k ? voff : kOOB, xr[2] ? k0 : 0u);
    ++requested;
    if (++lunit == len) {
      lunit = 0, lgroup += nwg;
      ranges();
      fresh = true;
    }
  };

  i32x4 acc[2][MT];
  auto clear = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int t = 0; t < MT; ++t) acc[j][t] = i32x4{0, 0, 0, 0};
  };
  clear();
  // Operands of half a unit; column tile j of slot `wave` is weight rows
  // 32 wave + 16 j, or of gate and of up 16 wave.
  struct Half {
    i32x4 a[MT], b[2];
  };
  const uint32_t swz = ((uint32_t)c >> 1) & 7u;
  auto read = [&](uint32_t stage, int kk, Half &f) __attribute__((always_inline)) {
    const uint8_t *at = ring + stage * C::kStage + (uint32_t)c * 128u + 16u * ((uint32_t)(kk * 4 + g) ^ swz);
#pragma unroll
    for (int j = 0; j < 2; ++j)
      f.b[j] = *(const i32x4 *)(at + (uint32_t)(NMAT > 1 ? kCols * j + 16 * wave : 32 * wave + 16 * j) * 128u);
#pragma unroll
    for (int t = 0; t < MT; ++t) f.a[t] = *(const i32x4 *)(at + C::kWeights + (uint32_t)(16 * t) * 128u);
  };
  auto multiply = [&](const Half &f) __attribute__((always_inline)) {
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[j][t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(f.b[j], f.a[t], acc[j][t], 0, 0, 0);
  };

  // element e of tile (j, t): row 16 t + c, column 4 g + e of the tile
  auto epilogue = [&](int group, int scale_set) __attribute__((always_inline)) {
    const float *set = scales[scale_set];
#pragma unroll
    for (int j = 0; j < (NMAT > 1 ? 1 : 2); ++j) {
      const int in = (NMAT > 1 ? 16 * wave : 32 * wave + 16 * j) + 4 * g, col = group * kCols + in;
      Int8Scale s0[4], s1[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s0[e] = int8_scale(set[64 + in + e]);
        if (NMAT > 1) s1[e] = int8_scale(set[192 + in + e]);
      }
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        const int r = 16 * t + c;
        const Int8Scale rs = int8_scale(set[r]);
        __bf16 v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float f = int8_scaled(acc[j][t][e], rs, s0[e]);
          v[e] = NMAT > 1 ? swiglu_bf16(f, int8_scaled(acc[1][t][e], rs, s1[e])) : (__bf16)f;
        }
        __bf16 *to = (__bf16 *)p.y + (size_t)r * p.n + col;
        if (r >= p.m) continue;
        if (col + 4 <= p.n) {
          *(u32x2_at2 *)to = u32x2_at2{__builtin_bit_cast(uint32_t, bf16x2{v[0], v[1]}),
                                       __builtin_bit_cast(uint32_t, bf16x2{v[2], v[3]})};
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (col + e < p.n) to[e] = v[e];
        }
      }
    }
  };
  auto piece = [&](int v) __attribute__((always_inline)) {
    const size_t at = ((size_t)first * p.parts + v) * P + wave;
    return rsrc_uniform((const uint8_t *)p.partial + at * C::kWavePiece, C::kWavePiece);
  };

#pragma unroll
  for (int i = 0; i < S; ++i) request((uint32_t)i);
  int group = first, unit = 0, set = 0;
  uint32_t stage = 0;
  Half f0, f1;
  wait_transfers<(S - 1) * C::kX>();
  ring_barrier();
  if (wave < P) read(0, 0, f0);
  for (int i = 0; i < count; ++i) {
    if (wave < P) {
      read(stage, 1, f1);
      multiply(f0);
    }
    // the S - 2 units behind the next may be under way
    wait_transfers<(S - 2) * C::kX>();
    ring_barrier();
    request(stage);
    stage = stage == S - 1 ? 0 : stage + 1;
    if (wave < P) {
      read(stage, 0, f0);
      multiply(f1);
    }
    if (p.parts == 1 && ++unit == len) {
      // (Memory operations end in order, so with stores among the youngest the
      // waits above cover more transfers than they ask for, never fewer.)
      if (wave < P) epilogue(group, set);
      clear();
      unit = 0, group += nwg;
      set = set == C::kScales - 1 ? 0 : set + 1;
    }
  }
  if (p.parts == 1) {
    wait_all_memory();
    return;
  }

  // ---- a part: its sums to memory; the last of the group's to arrive joins them
  if (wave < P) {
    const __amdgpu_buffer_rsrc_t out = piece(part);
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int t = 0; t < MT; ++t) st16_coherent(out, (uint32_t)(j * MT + t) * 1024u + 16u * lane, acc[j][t]);
  }
  wait_all_memory();
  __syncthreads();
  if (tid == 0)
    last_flag = __hip_atomic_fetch_add(&p.counters[first], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
                (unsigned)(p.parts - 1);
  __syncthreads();
  if (!last_flag) return;
  if (tid == 0) __hip_atomic_store(&p.counters[first], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  if (wave >= P) return;
  constexpr int kAtOnce = 8 / MT;  // pieces in flight
  for (int v = 0; v < p.parts; v += kAtOnce) {
    i32x4 w[kAtOnce][2][MT];
#pragma unroll
    for (int d = 0; d < kAtOnce; ++d) {
      // (this part's sums are still in registers)
      const bool other = v + d < p.parts && v + d != part;
      const __amdgpu_buffer_rsrc_t r = piece(min(v + d, p.parts - 1));
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int t = 0; t < MT; ++t)
          w[d][j][t] = ld16_coherent(r, other ? (uint32_t)(j * MT + t) * 1024u + 16u * lane : kOOB);
    }
#pragma unroll
    for (int d = 0; d < kAtOnce; ++d)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int t = 0; t < MT; ++t) acc[j][t] += w[d][j][t];
  }
  epilogue(first, 0);
}

template <int MT, int P>
hipError_t launch_p(const Int8Args &p, int nmat, int nwg, hipStream_t s) {
  if (nmat == 1)
    hipLaunchKernelGGL((k_int8_gemm<MT, P, 1>), dim3(nwg), dim3(kWaves * 64), 0, s, p);
  else
    hipLaunchKernelGGL((k_int8_gemm<MT, P, 2>), dim3(nwg), dim3(kWaves * 64), 0, s, p);
  return hipGetLastError();
}
template <int MT>
hipError_t launch_mt(const Int8Args &p, int slots, int nmat, int nwg, hipStream_t s) {
  static_assert(kInt8MaxSlots == 6, "the slots below");
  switch (slots) {
    case 1: return launch_p<MT, 1>(p, nmat, nwg, s);
    case 2: return launch_p<MT, 2>(p, nmat, nwg, s);
    case 3: return launch_p<MT, 3>(p, nmat, nwg, s);
    case 4: return launch_p<MT, 4>(p, nmat, nwg, s);
    case 5: return launch_p<MT, 5>(p, nmat, nwg, s);
    case 6: return launch_p<MT, 6>(p, nmat, nwg, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

hipError_t launch_int8_gemm(const Int8ActRef &a, int m, int k, int n, int nmat, const Int8MatRef *w, void *y,
                            const Int8Plan &pl, unsigned *counters, int *partial, hipStream_t s) {
  const Int8Args p{a.codes, a.row_scale, m, k, n, w[0].codes, nmat > 1 ? w[1].codes : nullptr, w[0].scales,
                   nmat > 1 ? w[1].scales : nullptr, y, partial, counters, pl.groups, pl.units, pl.parts};
  if (m > 16 * pl.mt) return hipErrorInvalidValue;
  switch (pl.mt) {
    case 1: return launch_mt<1>(p, pl.slots, nmat, pl.nwg, s);
    case 2: return launch_mt<2>(p, pl.slots, nmat, pl.nwg, s);
    case 4: return launch_mt<4>(p, pl.slots, nmat, pl.nwg, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace nvfp4
