// k_kv8_attn.hip -- attention over the 8-bit paged KV cache.
//
// Row i of a sequence of n tokens with r rows sits at position n - r + i and
// sees the tokens j up to its own position, with a window the last `window`
// of them.  s_ij = scale * q_i . k_j, o_i = sum_j e^(s_ij - m) v_j / sum_j
// e^(s_ij - m), lse_i = m + log sum_j e^(s_ij - m); a row that sees nothing
// gives zeros and -inf.  Sums and the softmax's statistics are fp32, powers
// are of two (log2 e is folded into the scale).
#include <algorithm>
#include <type_traits>

#include "kv8_common.h"
#include "launchers.h"

namespace nvfp4 {

namespace {

constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.693147180559945309f;

// The tokens of a sequence that some row sees: [lo, hi); its rows and the first.
struct Kv8Seen {
  int r0, rows, lo, hi;
};
__device__ __forceinline__ Kv8Seen kv8_seen(const Kv8Attn &a, const Kv8Batch &s, int shift, int b) {
  const Kv8Span sp = kv8_span(s, shift, b);
  const int rows = min(sp.rows, s.max_rows), first = sp.len - sp.rows;
  if (rows <= 0) return {0, 0, 0, 0};
  return {sp.r0, rows, a.window ? max(first - a.window + 1, 0) : 0, min(first + rows, min(sp.len, a.max_len))};
}
// Chains block `col` of sequence b to its page's list, where some row sees it.
__device__ __forceinline__ void kv8_chain(const Kv8Links &links, const Kv8Pool &c, const Kv8Batch &s,
                                          const Kv8Seen &q, int b, int col) {
  if (q.hi <= q.lo || col < q.lo >> c.shift || col > (q.hi - 1) >> c.shift) return;
  const int id = kv8_page(s, c, b, col);
  if (id < 0) return;
  const unsigned groups = 1u << links.bits, e = (unsigned)b * (unsigned)links.blocks + (unsigned)col;
  const unsigned at = ((unsigned)id & (groups - 1u)) + ((((unsigned)id >> links.bits) & (kKv8Chains - 1u)) << links.bits);
  links.next[e] = uint2{atomicExch(&links.head[at], e + 1u), (unsigned)id};
}

// ---- few rows: one pass over the cache, split along the tokens ---------------------
//
// What bounds it: the bytes of the codes.  A step is 32 tokens of one KV
// head, 64 * D bytes of codes that a wave loads as contiguous 1 KB pieces
// straight into matrix operands.  S^T = K Q^T (rows: tokens, columns: the
// group's query heads of up to 16 * CT (row, head) pairs) leaves lane
// (g, n) with tokens 4 g .. 4 g + 3 of each 16-token unit for column n, which
// is the operand layout that O^T = V^T P^T wants, so P goes from the
// accumulators to the next product without LDS or shuffles.  No maximum is
// looked for: the running one stays until a step's sum of powers passes
// kRaise (the sums are fp32 and P is a floating type, so a factor of some
// hundred costs nothing; overflow to infinity passes it too), and only then
// is it found and the powers taken again.
//
// A workgroup's four waves take its steps in turn; their results are joined
// in LDS, those of a sequence's workgroups by the last of them to arrive, in
// the order of the tokens.
//
// Measured (32 query heads on 8 KV heads of 128 but where said): 48 sequences
// of up to 8191 tokens 78 us, 5400 GB/s of codes; 2 of 131000 (40 heads) 93 us,
// 5750 GB/s of the 5990 that reading alone reaches; 24 of 4099 with four rows, a
// window of 2048 and heads of 64 16 us (40 MB: start, look-ups and join are
// most of it); one of 521 9.3 us in a graph, where the call's own 12 us do not
// hide it.

constexpr float kRaise = 1024.0f;  // a step's sum of powers that has the running maximum found anew
constexpr float kLowest = -3.4028234663852886e38f;  // below every finite score

struct DecodeParams {
  Kv8Attn a;
  Kv8Pool c;
  Kv8Batch s;
  int group, blocks;  // query heads per KV head; column blocks
  int spw, rounds;    // a wave's steps at a time, and times
  int splits;         // workgroups per item at most
  float *part;        // [item]: o [split][column][D], then m and l [split][column]
  unsigned *counters;
  float *scores;      // [seq][head][column][len_pad], or null: not wanted
  int len_pad, score_cols;
  Kv8Links links;     // where scores are wanted
};

__device__ __forceinline__ bf16x8 fp8x8_to_bf16(uint32_t lo, uint32_t hi, float scale) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}
__device__ __forceinline__ void st16_coherent(__amdgpu_buffer_rsrc_t r, uint32_t off, f32x4 v) {
  __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), r, off, 0, kCoherent);
}
__device__ __forceinline__ f32x4 ld16_coherent(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, kCoherent));
}
// 0x80 in each byte that is a NaN code
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
  return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
}

template <int D, int CT>
__global__ __launch_bounds__(64 * kDecodeWaves, decode_waves(D, CT)) void k_kv8_decode(DecodeParams p) {
  constexpr int kCols = 16 * CT, kPad = D + 4;
  constexpr bool kRest = CT < 4;  // P's second part
  __shared__ __align__(16) float osum[kDecodeWaves][16][kPad];
  __shared__ float stat[2][kDecodeWaves][kCols];
  __shared__ bool last_flag;
  __shared__ float wsplit[kMaxSplits][16];
  // Consecutive workgroups go to the 8 XCDs in turn.  The items (sequence, KV
  // head, column block) are side by side, a step further for each split: with
  // the splits side by side, an even number of them would leave the XCDs of
  // the later ones idle where sequences are short.
  const int items = p.s.seqs * p.c.heads * p.blocks;
  const int split = (int)blockIdx.x / items, item = ((int)blockIdx.x % items + split) % items;
  const int cb = item % p.blocks, h = item / p.blocks % p.c.heads, b = item / p.blocks / p.c.heads;
  const int tid = (int)threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n = lane & 15, g = lane >> 4, shift = p.c.shift;
  const Kv8Span sp = kv8_span(p.s, shift, b);
  const int c0 = cb * kCols, cols = min(min(sp.rows, p.s.max_rows) * p.group - c0, kCols);
  if (cols <= 0) return;

  // the tokens that the block's first and last rows see: [lo, hi] of each
  const int first = sp.len - sp.rows + c0 / p.group, final = sp.len - sp.rows + (c0 + cols - 1) / p.group;
  const int end = min(sp.len, p.a.max_len);
  auto low = [&](int pos) { return p.a.window ? max(pos - p.a.window + 1, 0) : 0; };
  const int step0 = low(first) >> 5, step1 = (min(final + 1, end) + 31) >> 5;
  const int per = p.spw * kDecodeWaves, whole_per = per * p.rounds;
  const int nsplit = max((step1 - step0 + whole_per - 1) / whole_per, 1);
  if (split >= nsplit) return;
  const int full_lo = low(final), full_hi = min(first, end - 1);  // every row sees these
  if constexpr (CT == 1) {
    if (p.scores) {  // a block for a thread of the sequence's workgroups
      const Kv8Seen seen = kv8_seen(p.a, p.s, shift, b);
      for (int col = (seen.lo >> shift) + (split * p.c.heads + h) * 64 * kDecodeWaves + tid;
           col <= (seen.hi - 1) >> shift; col += nsplit * p.c.heads * 64 * kDecodeWaves)
        kv8_chain(p.links, p.c, p.s, seen, b, col);
    }
  }

  // columns of this lane
  const float cs = fmaxf(fabsf(p.a.scale) * kLog2e, 1.1754944e-38f);  // its sign goes to q
  const uint32_t flip = p.a.scale < 0.f ? 0x80008000u : 0u;
  bf16x8 q[CT][D / 32];
  int lo[CT], hi[CT];
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) {
    const int c = ct * 16 + n, i = (c0 + c) / p.group;
    const bool in = c < cols;
    const __bf16 *qr = (const __bf16 *)p.a.q.ptr + (int64_t)(sp.r0 + (in ? i : 0)) * p.a.q.row_stride +
                       (int64_t)(h * p.group + (in ? (c0 + c) % p.group : 0)) * p.a.q.head_stride;
#pragma unroll
    for (int t = 0; t < D / 64; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint4 w = *(const uint4 *)(qr + 64 * t + 16 * g + 8 * e);
        q[ct][2 * t + e] = as_bf16x8(in ? uint4{w.x ^ flip, w.y ^ flip, w.z ^ flip, w.w ^ flip} : uint4{0, 0, 0, 0});
      }
    const int pos = sp.len - sp.rows + i;
    lo[ct] = low(pos);
    hi[ct] = min(pos, end - 1);
  }

  // this wave's steps of a round: base + 4 s; lane 2 s + u: unit u of step s
  int base = 0, count = 0, at = -1;
  float ksc = 1.f, vsc = 1.f;
  auto look_up = [&](int round) {
    base = step0 + split * whole_per + round * per + wave;
    count = min(max((step1 - base + kDecodeWaves - 1) / kDecodeWaves, 0), p.spw);
    at = -1;
    ksc = vsc = 1.f;
    const int t0 = (base + kDecodeWaves * (lane >> 1)) * 32 + (lane & 1) * 16;
    if ((lane >> 1) < count && t0 < end) {
      const int id = kv8_page(p.s, p.c, b, t0 >> shift);
      if (id >= 0) {
        const size_t ph = (size_t)id * p.c.heads + h;
        at = (int)((ph << (shift - 4)) + ((t0 >> 4) & ((1 << (shift - 4)) - 1)));
        ksc = fmaxf(cs * kv8_scale(p.c.ks[ph]), 1.1754944e-38f);
        vsc = kv8_scale(p.c.vs[ph]);
      }
    }
  };
  uint4 kx[2][D / 64];  // K of a step [unit][t]: token lane % 16, channels 64 t + 16 g ..
  // V [unit][a], this step's and the next's: tokens 4 g .., channels 64 a + 16 c + lane % 16
  uint4 vx[2][D / 64], vy[2][D / 64];
  auto load = [&](const uint8_t *codes, uint4 (&x)[2][D / 64], int s) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint32_t unit = (uint32_t)__builtin_amdgcn_readlane(at, min(2 * s, 62) + u);
      // (a unit that no page holds reads the pool's first; its scores are masked)
      const uint4 *src = (const uint4 *)(codes + (size_t)(unit == 0xFFFFFFFFu ? 0u : unit) * (16 * D)) + lane;
#pragma unroll
      for (int t = 0; t < D / 64; ++t) x[u][t] = load_once(src + 64 * t);
    }
  };

  f32x4 o[CT][D / 16] = {};
  float m[CT], l[CT] = {};
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) m[ct] = kLowest;

  const size_t score_bytes = (size_t)p.score_cols * p.len_pad * 4;  // of an item, below 2^31
  const __amdgpu_buffer_rsrc_t left =
      rsrc_uniform((const char *)p.scores + ((size_t)b * p.c.heads + h) * score_bytes, score_bytes);
  const uint32_t score_at = n < cols ? (uint32_t)(n * p.len_pad + 4 * g) * 4u : kOOB;

  f32x4 sc[CT][2];
  bf16x8 pr[CT], rest[CT];
  float sum[CT];
  auto of_unit = [&](float x, int s, int u) {
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), 2 * s + u));
  };
  auto has_page = [&](int s, int u) { return __builtin_amdgcn_readlane(at, 2 * s + u) != -1; };
  auto scores = [&]() {
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int t = 0; t < D / 64; ++t) {
        const bf16x8 k0 = fp8x8_to_bf16(kx[u][t].x, kx[u][t].y, 1.0f);
        const bf16x8 k1 = fp8x8_to_bf16(kx[u][t].z, kx[u][t].w, 1.0f);
        const f32x4 zero = {};
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
          sc[ct][u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k0, q[ct][2 * t], t ? sc[ct][u] : zero, 0, 0, 0);
          sc[ct][u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k1, q[ct][2 * t + 1], sc[ct][u], 0, 0, 0);
        }
      }
  };
  auto sees = [&](int ct, int t0, int s) {  // bit e: accumulator e's token is one that the lane's column sees
    uint32_t bits = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int j = t0 + 16 * (e >> 2) + 4 * g + (e & 3);
      bits |= (((j >= lo[ct]) & (j <= hi[ct])) ? 1u : 0u) << e;
    }
    return bits & ((has_page(s, 0) ? 0xFu : 0u) | (has_page(s, 1) ? 0xF0u : 0u));
  };
  // P and its sum (fp32); the product with V takes P as the sum of two bf16, off
  // by 2^-16 of itself, but where there are four column tiles: with one, off by
  // 2^-8, their 16 sequences of 8000 tokens take 44 us, with two 52 us
  auto powers = [&](int s) {
    const float f0 = of_unit(ksc, s, 0), f1 = of_unit(ksc, s, 1);
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
      float e[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) e[i] = __builtin_amdgcn_exp2f(fmaf(sc[ct][i >> 2][i & 3], i < 4 ? f0 : f1, -m[ct]));
      sum[ct] = ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        pr[ct][i] = (__bf16)e[i];
        if constexpr (kRest) rest[ct][i] = (__bf16)(e[i] - (float)pr[ct][i]);
      }
    }
  };
  // V of channels 64 a + 16 c + n of the lane's eight tokens, as an operand
  auto widen = [&](uint32_t w0, uint32_t w1, float v0, float v1) {
    const bf16x2 x0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, v0, false);
    const bf16x2 x1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, v0, true);
    const bf16x2 y0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, v1, false);
    const bf16x2 y1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, v1, true);
    return bf16x8{x0[0], x0[1], x1[0], x1[1], y0[0], y0[1], y1[0], y1[1]};
  };
  auto take = [&]() {
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int a = 0; a < D / 64; ++a) vx[u][a] = vy[u][a];
  };
  auto word = [](const uint4 &v, int c) { return c == 0 ? v.x : c == 1 ? v.y : c == 2 ? v.z : v.w; };

  // The next step's codes are loaded when this one's scores are done, K into
  // the registers that held K.  The loads are not conditional; a step past the
  // last is the pool's first unit.  The loop proper has no rare work in it,
  // which keeps the accumulators in place: a step that raises the maximum, or
  // where a NaN code of V must not reach a row that does not see its token, is
  // finished below from its scores.
  for (int round = 0; round < p.rounds; ++round) {
    look_up(round);
    load(p.c.k, kx, 0);
    load(p.c.v, vx, 0);
    int s = 0;
    while (s < count) {
      bool leave;
      do {
        const int t0 = (base + kDecodeWaves * s) * 32;
        scores();
        load(p.c.k, kx, s + 1);
        load(p.c.v, vy, s + 1);
        uint32_t odd = 0;
        if (t0 < full_lo || t0 + 31 > full_hi || !has_page(s, 0) || !has_page(s, 1)) {
#pragma unroll
          for (int ct = 0; ct < CT; ++ct) {
            const uint32_t bits = sees(ct, t0, s);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              sc[ct][e >> 2][e & 3] = bits >> e & 1u ? sc[ct][e >> 2][e & 3] : -__builtin_inff();
          }
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int a = 0; a < D / 64; ++a)
              odd |= nan_bytes(vx[u][a].x) | nan_bytes(vx[u][a].y) | nan_bytes(vx[u][a].z) | nan_bytes(vx[u][a].w);
        }
        if constexpr (CT == 1) {
          if (p.scores) {  // (lanes past the columns store out of range, that is nowhere)
#pragma unroll
            for (int u = 0; u < 2; ++u)
              __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, sc[0][u] * of_unit(ksc, s, u)), left,
                                                     score_at + (uint32_t)(t0 + 16 * u) * 4u, 0, 0);
          }
        }
        powers(s);
        bool raise = odd != 0;
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) raise |= sum[ct] > kRaise;
        leave = __any(raise);
        if (leave) break;
        const float v0 = of_unit(vsc, s, 0), v1 = of_unit(vsc, s, 1);
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) l[ct] += sum[ct];
#pragma unroll
        for (int a = 0; a < D / 64; ++a)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const bf16x8 vt = widen(word(vx[0][a], c), word(vx[1][a], c), v0, v1);
#pragma unroll
            for (int ct = 0; ct < CT; ++ct)
              o[ct][4 * a + c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vt, pr[ct], o[ct][4 * a + c], 0, 0, 0);
            if constexpr (kRest) {
#pragma unroll
              for (int ct = 0; ct < CT; ++ct)
                o[ct][4 * a + c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vt, rest[ct], o[ct][4 * a + c], 0, 0, 0);
            }
          }
        take();
      } while (++s < count);
      if (!leave) break;

      const int t0 = (base + kDecodeWaves * s) * 32;
      const float f0 = of_unit(ksc, s, 0), f1 = of_unit(ksc, s, 1);
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        float x = kLowest;
#pragma unroll
        for (int e = 0; e < 8; ++e) x = fmaxf(x, sc[ct][e >> 2][e & 3] * (e < 4 ? f0 : f1));
        x = fmaxf(x, __shfl_xor(x, 16));
        x = fmaxf(x, __shfl_xor(x, 32));
        const float mn = fmaxf(m[ct], x), down = __builtin_amdgcn_exp2f(m[ct] - mn);
        m[ct] = mn;
        l[ct] *= down;
#pragma unroll
        for (int d = 0; d < D / 16; ++d) o[ct][d] *= down;
      }
      powers(s);
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) l[ct] += sum[ct];
      const float v0 = of_unit(vsc, s, 0), v1 = of_unit(vsc, s, 1);
#pragma unroll
      for (int a = 0; a < D / 64; ++a)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t w0 = word(vx[0][a], c), w1 = word(vx[1][a], c);
          const uint32_t b0 = nan_bytes(w0) >> 7, b1 = nan_bytes(w1) >> 7;
          if (__any((b0 | b1) != 0)) {  // ones where a code is NaN, against ones where a row sees the token
            w0 &= ~(b0 * 0xFFu);
            w1 &= ~(b1 * 0xFFu);
            bf16x8 here;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              here[i] = (__bf16)(float)((b0 >> (8 * i)) & 1u);
              here[4 + i] = (__bf16)(float)((b1 >> (8 * i)) & 1u);
            }
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
              const uint32_t bits = sees(ct, t0, s);
              bf16x8 yes;
#pragma unroll
              for (int i = 0; i < 8; ++i) yes[i] = (__bf16)(float)((bits >> i) & 1u);
              f32x4 hit = {};
              hit = __builtin_amdgcn_mfma_f32_16x16x32_bf16(here, yes, hit, 0, 0, 0);
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (hit[i] > 0.f) o[ct][4 * a + c][i] = __builtin_nanf("");
            }
          }
          const bf16x8 vt = widen(w0, w1, v0, v1);
#pragma unroll
          for (int ct = 0; ct < CT; ++ct) {
            o[ct][4 * a + c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vt, pr[ct], o[ct][4 * a + c], 0, 0, 0);
            if constexpr (kRest)
              o[ct][4 * a + c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vt, rest[ct], o[ct][4 * a + c], 0, 0, 0);
          }
          __builtin_amdgcn_sched_barrier(0);  // one at a time: rare work need not set the registers' number
        }
      take();
      ++s;
    }
  }

  // ---- join the waves
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) {
    l[ct] += __shfl_xor(l[ct], 16);
    l[ct] += __shfl_xor(l[ct], 32);
    if (g == 0) {
      stat[0][wave][ct * 16 + n] = m[ct];
      stat[1][wave][ct * 16 + n] = l[ct];
    }
  }
  __syncthreads();
  const __amdgpu_buffer_rsrc_t parts =  // (not touched when there is one split)
      rsrc_uniform(p.part + (size_t)item * p.splits * kCols * (D + 2), (size_t)p.splits * kCols * (D + 2) * 4);
  const uint32_t stats = (uint32_t)p.splits * kCols * D * 4u;  // m and l of (split, column)
  const int64_t row0 = (int64_t)sp.r0 * p.a.q_heads + (int64_t)h * p.group;
  auto put = [&](int c, int d, f32x4 x, float ll) {  // four channels of column c, done
    const float inv = ll > 0.f || ll != ll ? 1.0f / ll : 0.f;
    const int64_t r = row0 + (int64_t)((c0 + c) / p.group) * p.a.q_heads + (c0 + c) % p.group;
    bf16x2 y[2] = {{(__bf16)(x[0] * inv), (__bf16)(x[1] * inv)}, {(__bf16)(x[2] * inv), (__bf16)(x[3] * inv)}};
    *(uint2 *)((__bf16 *)p.a.out + r * D + d) =
        uint2{__builtin_bit_cast(uint32_t, y[0]), __builtin_bit_cast(uint32_t, y[1])};
  };
  auto put_lse = [&](int c, float mm, float ll) {
    const int64_t r = row0 + (int64_t)((c0 + c) / p.group) * p.a.q_heads + (c0 + c) % p.group;
    p.a.lse[r] = ll > 0.f || ll != ll ? (mm + log2f(ll)) * kLn2 : -__builtin_inff();
  };
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) {
    if (ct * 16 >= cols) break;
    float top = kLowest;
#pragma unroll
    for (int w = 0; w < kDecodeWaves; ++w) top = fmaxf(top, stat[0][w][ct * 16 + n]);
    const float f = __builtin_amdgcn_exp2f(m[ct] - top);
    if (ct) __syncthreads();
#pragma unroll
    for (int d = 0; d < D / 16; ++d) *(f32x4 *)&osum[wave][n][16 * d + 4 * g] = o[ct][d] * f;
    __syncthreads();
    for (int i = tid; i < 16 * (D / 4); i += 64 * kDecodeWaves) {
      const int col = i / (D / 4), d = i % (D / 4) * 4, c = ct * 16 + col;
      if (c >= cols) break;
      float mm = kLowest, ll = 0.f;
#pragma unroll
      for (int w = 0; w < kDecodeWaves; ++w) mm = fmaxf(mm, stat[0][w][c]);
#pragma unroll
      for (int w = 0; w < kDecodeWaves; ++w) ll += stat[1][w][c] * __builtin_amdgcn_exp2f(stat[0][w][c] - mm);
      f32x4 x = *(const f32x4 *)&osum[0][col][d];
#pragma unroll
      for (int w = 1; w < kDecodeWaves; ++w) x += *(const f32x4 *)&osum[w][col][d];
      if (nsplit == 1) {
        put(c, d, x, ll);
        if (d == 0 && p.a.lse) put_lse(c, mm, ll);
      } else {
        const uint32_t off = (uint32_t)(split * kCols + c);
        st16_coherent(parts, (off * D + d) * 4u, x);
        if (d == 0) {
          st_coherent(parts, stats + off * 8u, mm);
          st_coherent(parts, stats + off * 8u + 4u, ll);
        }
      }
    }
  }
  if (nsplit == 1) return;

  // ---- join the splits: the last workgroup of the item to arrive
  wait_all_memory();
  __syncthreads();
  if (tid == 0)
    last_flag = __hip_atomic_fetch_add(&p.counters[item], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
                (unsigned)(nsplit - 1);
  __syncthreads();
  if (!last_flag) return;
  // 16 columns at a time: the statistics first, then the sums, the splits of a
  // column dealt over as many threads as there are and added in order
  constexpr int kThreads = 64 * kDecodeWaves;
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) {
    const int here = min(cols - ct * 16, 16);
    if (here <= 0) break;
    if (ct) __syncthreads();
    for (int i = tid; i < nsplit * here; i += kThreads)
      wsplit[i / here][i % here] = ld_coherent(parts, stats + (uint32_t)(i / here * kCols + ct * 16 + i % here) * 8u);
    __syncthreads();
    float *top = stat[0][0], *total = stat[1][0];  // (done with)
    for (int c = tid >> 4; c < here; c += kThreads / 16) {
      float x = kLowest;
      for (int t = tid & 15; t < nsplit; t += 16) x = fmaxf(x, wsplit[t][c]);
#pragma unroll
      for (int k = 8; k > 0; k >>= 1) x = fmaxf(x, __shfl_xor(x, k));
      float y = 0.f;
      for (int t = tid & 15; t < nsplit; t += 16) {
        const float f = __builtin_amdgcn_exp2f(wsplit[t][c] - x);
        wsplit[t][c] = f;
        y = fmaf(f, ld_coherent(parts, stats + (uint32_t)(t * kCols + ct * 16 + c) * 8u + 4u), y);
      }
#pragma unroll
      for (int k = 8; k > 0; k >>= 1) y += __shfl_xor(y, k);
      if ((tid & 15) == 0) {
        top[c] = x;
        total[c] = y;
      }
    }
    __syncthreads();
    const int items = here * (D / 4);
    int deal = 1;  // threads of one item
    while (deal < 8 && items * deal * 2 <= kThreads) deal *= 2;
    float *sums = &osum[0][0][0];  // [deal][items] of four
    for (int i = tid; i < items * deal; i += kThreads) {
      const int k = i / items, c = i % items / (D / 4), d = i % items % (D / 4) * 4;
      f32x4 x = {};
#pragma unroll 8
      for (int t = k; t < nsplit; t += deal)
        x += ld16_coherent(parts, (uint32_t)((t * kCols + ct * 16 + c) * D + d) * 4u) * wsplit[t][c];
      if (deal == 1) {
        put(ct * 16 + c, d, x, total[c]);
        if (d == 0 && p.a.lse) put_lse(ct * 16 + c, top[c], total[c]);
      } else {
        *(f32x4 *)(sums + 4 * i) = x;
      }
    }
    if (deal > 1) {
      __syncthreads();
      for (int i = tid; i < items; i += kThreads) {
        const int c = i / (D / 4), d = i % (D / 4) * 4;
        f32x4 x = *(const f32x4 *)(sums + 4 * i);
        for (int k = 1; k < deal; ++k) x += *(const f32x4 *)(sums + 4 * (i + k * items));
        put(ct * 16 + c, d, x, total[c]);
        if (d == 0 && p.a.lse) put_lse(ct * 16 + c, top[c], total[c]);
      }
    }
  }
  if (tid == 0) __hip_atomic_store(&p.counters[item], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// ---- many rows ------------------------------------------------------------------------
//
// What bounds it: the matrix instructions (4 D operations for each score
// against about 5 vector instructions of the softmax).  A workgroup takes
// 32 * CT * NW columns ((row, head) pairs of one KV head, so the heads of a
// group share its codes) and walks the tokens in tiles of 32 * ST: the codes are
// read one tile ahead into registers, widened to bf16 once by the workgroup
// (K and V times their scales, exact) and written to LDS as the operands of
// the 32x32x16 instructions, two tiles in turn, one barrier a tile.  As in
// the kernel for few rows S^T = K Q^T leaves each lane the probabilities of
// its column as the next product's operand: accumulator row
// (r % 4) + 8 (r / 4) + 4 half of a 32-token step is token 16 ks + 8 (e / 4)
// + 4 half + e % 4 for r = 8 ks + e, so V's operand takes, of unit ks, the
// token groups `half` and 2 + half.  No maximum is looked for either: the
// running one stays until a tile's sum of powers passes kRaise (overflow to
// infinity does), and only then is it found and the powers taken again.
//
// An item is a block of columns over all its tokens.  Where there are many, a
// workgroup takes one.  Where there are few (DEALT) the tiles of all items
// stand in a row, one KV head after the other, and are dealt in equal runs
// over one workgroup per CU, whatever the lengths: a run's first and last item
// may be parts, whose sums and statistics go to memory (two places a
// workgroup) for a second kernel to join in the order of the tokens.
//
// Measured: a prompt of 8192 tokens, 32 heads on 8 of 128, 520 to 540 us from
// card to card, 1020 to 1060 TFLOP/s; 3 pieces of up to 1023 rows, 16 heads on 4 of 256, a window of 3000,
// 171 us, 710 TFLOP/s (its 32-token tiles and one wave's 128 accumulators leave
// the softmax less to hide behind).
struct PrefillParams {
  Kv8Attn a;
  Kv8Pool c;
  Kv8Batch s;
  int group, blocks;
  float *part;  // [workgroup][2]: o as the kernel holds it, then m and l
  int2 *parts;  // [item]: the workgroup with its first part, how many parts (0: whole)
};
template <int D, int CT, int NW, int ST, bool DEALT>
__global__ __launch_bounds__(64 * NW, NW / 4) void k_kv8_prefill(PrefillParams p) {
  constexpr int kCols = 32 * CT * NW;
  constexpr int KT = D / 16, VT = D / 32;   // operands of a step: K's and (of each 16 tokens) V's
  constexpr int kUnits = 2 * ST, kShift = ST == 2 ? 6 : 5, kTile = 32 * ST;
  // a wave reads and widens its share of one unit: 64-channel parts of both K
  // and V, or (with one part) K or V
  constexpr int kShare = NW / kUnits, kParts = D / 64 >= kShare ? D / 64 / kShare : 1;
  constexpr bool kBoth = D / 64 >= kShare;
  __shared__ uint4 kbuf[2][ST][KT][64];     // [tile][step][channels 16 t ..][lane]
  __shared__ uint4 vbuf[2][ST][2][VT][64];  // [tile][step][unit][channels 32 t ..][lane]
  __shared__ int bad[2][kUnits];            // a unit without a page
  __shared__ int odd[2][NW];                // whether a wave met a NaN code of V
  constexpr int kPairs = 64 * NW;
  __shared__ int before[DEALT ? kPairs + 1 : 1], wave_sum[NW];  // tiles of one head before each (sequence, block)
  static_assert(kCols == kManyCols && kPairs >= kManyItems && (kPairs & (kPairs - 1)) == 0, "");
  const int tid = (int)threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n = lane & 31, half = lane >> 5, shift = p.c.shift;
  auto low = [&](int pos) { return p.a.window ? max(pos - p.a.window + 1, 0) : 0; };
  // the tiles of an item: [x, y)
  auto tiles_of = [&](const Kv8Span &sp, int c0) {
    const int all = min(sp.rows, p.s.max_rows) * p.group, pos0 = sp.len - sp.rows;
    const int wg_first = pos0 + c0 / p.group, wg_final = pos0 + (min(c0 + kCols, all) - 1) / p.group;
    return int2{low(wg_first) >> kShift, (min(min(wg_final + 1, sp.len), p.a.max_len) + kTile - 1) >> kShift};
  };
  // heads side by side, so that those of one XCD's workgroups share its L2; the longest first
  int h = (int)blockIdx.x % p.c.heads, cb = p.blocks - 1 - (int)blockIdx.x / p.c.heads, b = (int)blockIdx.y;
  // a run [run0, run1) of the tiles of all heads, `row` of them a head's
  int run0 = 0, run1 = 1, row = 1, per = 1, rank = 0;
  const int pairs = p.s.seqs * p.blocks;
  if constexpr (DEALT) {
    const int seq = min(tid / p.blocks, p.s.seqs - 1), first = (tid - seq * p.blocks) * kCols;
    const Kv8Span one = kv8_span(p.s, shift, seq);
    const int2 x = tiles_of(one, first);
    // (one at least where there are columns: they may see nothing, and have results all the same)
    const int sum =
        tid < pairs && first < min(one.rows, p.s.max_rows) * p.group ? kStart + max(x.y - x.x, 1) : 0;
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int x = __shfl_up(incl, o);
      if (lane >= o) incl += x;
    }
    if (lane == 63) wave_sum[wave] = incl;
    __syncthreads();
    for (int i = 0; i < wave; ++i) incl += wave_sum[i];
    before[tid + 1] = incl;
    if (tid == 0) before[0] = 0;
    __syncthreads();
    row = __builtin_amdgcn_readfirstlane(before[pairs]);
    const int total = row * p.c.heads, groups = (int)gridDim.x;
    per = max((total + groups - 1) / groups, kStart + 512 / kTile);
    // neighbouring runs on one XCD (a workgroup's is its number modulo 8): they read the same codes
    rank = groups % 8 ? (int)blockIdx.x : (int)blockIdx.x % 8 * (groups / 8) + (int)blockIdx.x / 8;
    run0 = min(rank * per, total);
    run1 = min(run0 + per, total);
  }
  while (run0 < run1) {
    int part_at = -1, skip = 0, most = 0x7FFFFFFF;  // where a part goes; its first tile and how many
    if constexpr (DEALT) {
      h = run0 / row;
      const int x = run0 - h * row;
      int pair = 0;  // the last with before[pair] <= x, found bit by bit (equal ones: the last has tiles)
#pragma unroll
      for (int bit = kPairs / 2; bit > 0; bit >>= 1)
        if (pair + bit < pairs && __builtin_amdgcn_readfirstlane(before[pair + bit]) <= x) pair += bit;
      b = pair / p.blocks;
      cb = pair - b * p.blocks;
      const int from = __builtin_amdgcn_readfirstlane(before[pair]);
      const int size = __builtin_amdgcn_readfirstlane(before[pair + 1]) - from;
      skip = x - from;
      most = min(size - skip, run1 - run0);
      const bool whole = most == size;
      if (!whole) part_at = 2 * rank + (skip == 0 ? 1 : 0);
      if (skip == 0 && tid == 0) {
        const int w0 = run0 / per, w1 = (run0 + size - 1) / per;
        p.parts[((size_t)b * p.c.heads + h) * p.blocks + cb] = int2{w0, whole ? 0 : w1 - w0 + 1};
      }
      run0 += most;
    } else {
      run0 = run1;
    }
    const Kv8Span sp = kv8_span(p.s, shift, b);
    const int all = min(sp.rows, p.s.max_rows) * p.group, c0 = cb * kCols;
    if (c0 >= all) return;
    const int end = min(sp.len, p.a.max_len), pos0 = sp.len - sp.rows;
    const int2 span = tiles_of(sp, c0);
    const int tile0 = span.x + max(skip - kStart, 0);
    const int tile1 = most == 0x7FFFFFFF ? span.y : min(span.x + max(skip + most - kStart, 0), span.y);
    // the wave's columns and the tokens that its first and last row see
    const int w0 = c0 + wave * 32 * CT, cols = min(all - w0, 32 * CT);
    const int first = pos0 + w0 / p.group, final = pos0 + (w0 + max(cols, 1) - 1) / p.group;
    const int full_lo = low(final), full_hi = min(first, end - 1);
    const int any_lo = low(first), any_hi = cols > 0 ? min(final, end - 1) : -1;

    const float cs = fmaxf(fabsf(p.a.scale) * kLog2e, 1.1754944e-38f);  // its sign goes to q
    const uint32_t flip = p.a.scale < 0.f ? 0x80008000u : 0u;
    bf16x8 q[CT][KT];
    int lo[CT], hi[CT];
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
      const int c = w0 + ct * 32 + n, i = c / p.group;
      const bool in = c < all;
      const __bf16 *qr = (const __bf16 *)p.a.q.ptr + (int64_t)(sp.r0 + (in ? i : 0)) * p.a.q.row_stride +
                         (int64_t)(h * p.group + (in ? c % p.group : 0)) * p.a.q.head_stride;
#pragma unroll
      for (int t = 0; t < KT; ++t) {
        const uint4 w = *(const uint4 *)(qr + 16 * t + 8 * half);
        q[ct][t] = as_bf16x8(in ? uint4{w.x ^ flip, w.y ^ flip, w.z ^ flip, w.w ^ flip} : uint4{0, 0, 0, 0});
      }
      lo[ct] = low(pos0 + i);
      hi[ct] = min(pos0 + i, end - 1);
    }

    // lane i: the wave's unit of tile `meta + i`
    int meta = tile0 - 64, at = -1;
    float ksc = 1.f, vsc = 1.f;
    const int unit = wave % kUnits, share = wave / kUnits;
    const int part0 = kBoth ? share * kParts : 0;
    const bool does_k = kBoth || share == 0, does_v = kBoth || share == 1;
    uint4 kr[kParts], vr[kParts];
    int a_next = -1;  // of the tile in kr and vr
    float k_next = 1.f, v_next = 1.f;
    auto look_up = [&](int tile) {  // pages and scales of 64 tiles from here
      meta = tile;
      const int t = (tile + lane) * kTile + unit * 16;
      at = -1;
      ksc = vsc = 1.f;
      if (t < end && tile + lane < tile1) {
        const int id = kv8_page(p.s, p.c, b, t >> shift);
        if (id >= 0) {
          const size_t ph = (size_t)id * p.c.heads + h;
          at = (int)((ph << (shift - 4)) + ((t >> 4) & ((1 << (shift - 4)) - 1)));
          ksc = kv8_scale(p.c.ks[ph]);
          vsc = kv8_scale(p.c.vs[ph]);
        }
      }
    };
    auto load = [&](int tile) {
      if (tile - meta >= 64) look_up(tile);
      a_next = __builtin_amdgcn_readlane(at, tile - meta);
      k_next = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, ksc), tile - meta));
      v_next = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, vsc), tile - meta));
      // (a unit that no page holds reads the pool's first; its scores are masked)
      const size_t off = (size_t)(a_next == -1 ? 0u : (uint32_t)a_next) * (16 * D);
      if (does_k) {
        const uint4 *k = (const uint4 *)(p.c.k + off) + 64 * part0 + lane;
#pragma unroll
        for (int t = 0; t < kParts; ++t) kr[t] = k[64 * t];
      }
      if (does_v) {
        const uint4 *v = (const uint4 *)(p.c.v + off) + 64 * part0 + lane;
#pragma unroll
        for (int t = 0; t < kParts; ++t) vr[t] = v[64 * t];
      }
    };
    auto widen = [&](int buf) {
      const int r = lane & 15, g = lane >> 4, step = unit >> 1;
      if (does_k) {
#pragma unroll
        for (int t = 0; t < kParts; ++t) {  // token r, channels 16 (4 (part0 + t) + g) ..
          uint4 *to = &kbuf[buf][step][4 * (part0 + t) + g][16 * (unit & 1) + r];
          to[0] = __builtin_bit_cast(uint4, fp8x8_to_bf16(kr[t].x, kr[t].y, k_next));
          to[32] = __builtin_bit_cast(uint4, fp8x8_to_bf16(kr[t].z, kr[t].w, k_next));
        }
        if (lane == 0) bad[buf][unit] = a_next == -1;
      }
      if (does_v) {
        uint32_t any = 0;
#pragma unroll
        for (int t = 0; t < kParts; ++t) {  // tokens 4 g .., channels 64 (part0 + t) + 16 c + r
          const uint32_t w[4] = {vr[t].x, vr[t].y, vr[t].z, vr[t].w};
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            any |= nan_bytes(w[c]);
            const bf16x2 x0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[c], v_next, false);
            const bf16x2 x1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[c], v_next, true);
            uint2 *to = (uint2 *)&vbuf[buf][step][unit & 1][2 * (part0 + t) + (c >> 1)]
                                      [32 * (g & 1) + 16 * (c & 1) + r];
            to[g >> 1] = uint2{__builtin_bit_cast(uint32_t, x0), __builtin_bit_cast(uint32_t, x1)};
          }
        }
        const bool some = __any(any != 0);
        if (lane == 0) odd[buf][wave] = some;
      } else if (lane == 0) {
        odd[buf][wave] = 0;
      }
    };

    f32x16 o[CT][VT] = {};
    float m[CT], l[CT] = {};
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) m[ct] = kLowest;

    if (tile0 < tile1) {
      load(tile0);
      widen(0);
      load(min(tile0 + 1, tile1 - 1));
    }
    lds_barrier();

    f32x16 s[CT][ST];
    bf16x8 pr[CT][kUnits];
    float sum[CT];
    auto scores = [&](int buf) {
      const f32x16 zero = {};
#pragma unroll
      for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int j = 0; j < ST; ++j) {
          const bf16x8 k = as_bf16x8(kbuf[buf][j][t][lane]);
#pragma unroll
          for (int ct = 0; ct < CT; ++ct)
            s[ct][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k, q[ct][t], t ? s[ct][j] : zero, 0, 0, 0);
        }
      __builtin_amdgcn_sched_group_barrier(0x100, 6, 0);
#pragma unroll
      for (int i = 0; i < ST * KT - 6; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x8, CT, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      }
      __builtin_amdgcn_sched_group_barrier(0x8, 6 * CT, 0);
    };
    // P and its sum (fp32).  P itself is rounded to bf16, off by 2^-8: a second
    // bf16 for the rest, as the kernel for few rows takes it, makes the prompt
    // 716 us instead of 524 and the wide chunk 206 instead of 170.
    auto powers = [&]() {
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        float part[kUnits];
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
          float e[8];
#pragma unroll
          for (int i = 0; i < 8; ++i)
            e[i] = __builtin_amdgcn_exp2f(fmaf(s[ct][u >> 1][8 * (u & 1) + i], cs, -m[ct]));
          part[u] = ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
#pragma unroll
          for (int i = 0; i < 8; ++i) pr[ct][u][i] = (__bf16)e[i];
        }
        sum[ct] = part[0] + part[1];
        if constexpr (ST == 2) sum[ct] += part[2] + part[3];
      }
    };
    auto any_of = [](const int *flags, int n) {
      int x = 0;
#pragma unroll
      for (int i = 0; i < n; ++i) x |= flags[i];
      return __builtin_amdgcn_readfirstlane(x) != 0;
    };
    // whether every row of the wave sees every token of the tile
    auto is_whole = [&](int t0, int buf) {
      return t0 >= full_lo && t0 + kTile - 1 <= full_hi && !any_of(bad[buf], kUnits);
    };
    // bit r of step j: accumulator row r's token is one that the lane's column sees
    auto sees = [&](int ct, int j, int t0, int buf) {
      uint32_t bits = 0;
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int k = t0 + 32 * j + (r & 3) + 8 * (r >> 2) + 4 * half;
        bits |= (((k >= lo[ct]) & (k <= hi[ct])) ? 1u : 0u) << r;
      }
      return bits & ((bad[buf][2 * j] ? 0u : 0xFFu) | (bad[buf][2 * j + 1] ? 0u : 0xFF00u));
    };
    auto mask = [&](int t0, int buf) {
#pragma unroll
      for (int ct = 0; ct < CT; ++ct)
#pragma unroll
        for (int j = 0; j < ST; ++j) {
          const uint32_t bits = sees(ct, j, t0, buf);
#pragma unroll
          for (int r = 0; r < 16; ++r) s[ct][j][r] = bits >> r & 1u ? s[ct][j][r] : -__builtin_inff();
        }
    };
    auto fetch = [&](int tile, int buf) {  // the next tile to LDS, the one after it to registers
      widen(buf ^ 1);
      load(min(tile + 2, tile1 - 1));
    };

    // tiles that some row of the wave sees: [mine0, mine1)
    const int mine0 = min(max(any_lo >> kShift, tile0), tile1);
    const int mine1 = max(min((any_hi >> kShift) + 1, tile1), mine0);
    int tile = tile0;
    for (; tile < mine0; ++tile) {
      fetch(tile, (tile - tile0) & 1);
      lds_barrier();
    }
    // The loop proper has no rare work in it: it leaves for a tile that raises
    // the maximum, or where a NaN code of V must not reach a row that does not
    // see its token, and such a tile is done again from its scores below.
    while (true) {
      bool again = false;
      for (; tile < mine1; ++tile) {
        const int buf = (tile - tile0) & 1, t0 = tile * kTile;
        scores(buf);
        if (!is_whole(t0, buf)) {
          mask(t0, buf);
          again = any_of(odd[buf], NW);
        }
        powers();
        bool raise = again;
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) raise |= sum[ct] > kRaise;
        again = __any(raise);
        if (again) break;
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) l[ct] += sum[ct];
#pragma unroll
        for (int u = 0; u < kUnits; ++u)
#pragma unroll
          for (int t = 0; t < VT; ++t) {
            const bf16x8 v = as_bf16x8(vbuf[buf][u >> 1][u & 1][t][lane]);
#pragma unroll
            for (int ct = 0; ct < CT; ++ct)
              o[ct][t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v, pr[ct][u], o[ct][t], 0, 0, 0);
          }
        __builtin_amdgcn_sched_group_barrier(0x100, 6, 1);
#pragma unroll
        for (int i = 0; i < kUnits * VT - 6; ++i) {
          __builtin_amdgcn_sched_group_barrier(0x8, CT, 1);
          __builtin_amdgcn_sched_group_barrier(0x100, 1, 1);
        }
        __builtin_amdgcn_sched_group_barrier(0x8, 6 * CT, 1);
        fetch(tile, buf);
        lds_barrier();
      }
      if (!again) break;

      const int buf = (tile - tile0) & 1, t0 = tile * kTile;
      scores(buf);
      mask(t0, buf);
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        float x = kLowest;
#pragma unroll
        for (int j = 0; j < ST; ++j)
#pragma unroll
          for (int r = 0; r < 16; ++r) x = fmaxf(x, s[ct][j][r]);
        x *= cs;
        x = fmaxf(x, __shfl_xor(x, 32));
        const float mn = fmaxf(m[ct], x), down = __builtin_amdgcn_exp2f(m[ct] - mn);
        m[ct] = mn;
        l[ct] *= down;
#pragma unroll
        for (int t = 0; t < VT; ++t) o[ct][t] *= down;
      }
      powers();
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) l[ct] += sum[ct];
      fetch(tile, buf);
#pragma unroll
      for (int u = 0; u < kUnits; ++u)
#pragma unroll
        for (int t = 0; t < VT; ++t) {
          bf16x8 v = as_bf16x8(vbuf[buf][u >> 1][u & 1][t][lane]), here;
          bool some = false;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float x = (float)v[i];
            here[i] = (__bf16)(x != x ? 1.0f : 0.0f);
            v[i] = x != x ? (__bf16)0.0f : v[i];
            some |= x != x;
          }
          if (__any(some)) {  // ones where a code is NaN, against ones where a row sees the token
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
              const uint32_t bits = sees(ct, u >> 1, t0, buf) >> (8 * (u & 1));
              bf16x8 yes;
#pragma unroll
              for (int i = 0; i < 8; ++i) yes[i] = (__bf16)(float)((bits >> i) & 1u);
              f32x16 hit = {};
              hit = __builtin_amdgcn_mfma_f32_32x32x16_bf16(here, yes, hit, 0, 0, 0);
#pragma unroll
              for (int r = 0; r < 16; ++r)
                if (hit[r] > 0.f) o[ct][t][r] = __builtin_nanf("");
            }
          }
#pragma unroll
          for (int ct = 0; ct < CT; ++ct)
            o[ct][t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v, pr[ct][u], o[ct][t], 0, 0, 0);
          __builtin_amdgcn_sched_barrier(0);
        }
      lds_barrier();
      ++tile;
    }
    for (; tile < tile1; ++tile) {
      fetch(tile, (tile - tile0) & 1);
      lds_barrier();
    }

#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
      const int c = w0 + ct * 32 + n;
      const float ll = l[ct] + __shfl_xor(l[ct], 32);
      if (DEALT && part_at >= 0) {  // [wave][32 channels][4 of 8][lane]
        float *to = p.part + (size_t)part_at * many_floats(D);
#pragma unroll
        for (int t = 0; t < VT; ++t)
#pragma unroll
          for (int r = 0; r < 16; r += 4)
            *(f32x4 *)(to + (((wave * VT + t) * 4 + r / 4) * 64 + lane) * 4) =
                f32x4{o[ct][t][r], o[ct][t][r + 1], o[ct][t][r + 2], o[ct][t][r + 3]};
        *(float2 *)(to + kManyCols * D + (wave * 64 + lane) * 2) = float2{m[ct], ll};
        continue;
      }
      if (c >= all) continue;
      const int64_t out_row = (int64_t)(sp.r0 + c / p.group) * p.a.q_heads + h * p.group + c % p.group;
      const float inv = ll > 0.f || ll != ll ? 1.0f / ll : 0.f;
      __bf16 *to = (__bf16 *)p.a.out + out_row * D;
#pragma unroll
      for (int t = 0; t < VT; ++t)
#pragma unroll
        for (int r = 0; r < 16; r += 4) {
          const bf16x2 x = {(__bf16)(o[ct][t][r] * inv), (__bf16)(o[ct][t][r + 1] * inv)};
          const bf16x2 y = {(__bf16)(o[ct][t][r + 2] * inv), (__bf16)(o[ct][t][r + 3] * inv)};
          *(uint2 *)(to + 32 * t + 2 * r + 4 * half) =
              uint2{__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, y)};
        }
      if (half == 0 && p.a.lse)
        p.a.lse[out_row] = ll > 0.f || ll != ll ? (m[ct] + log2f(ll)) * kLn2 : -__builtin_inff();
    }
  }
}

// Joins the parts of the kernel above, in the order of the tokens: a workgroup
// for 32 columns and T times 32 channels, a wave for 8 of each 32.
template <int D, int T>
__global__ __launch_bounds__(256) void k_kv8_prefill_join(PrefillParams p) {
  constexpr int VT = D / 32, NW = kManyCols / 32;
  const int cb = (int)blockIdx.x / NW, w = (int)blockIdx.x % NW, h = (int)blockIdx.y;
  const int b = (int)blockIdx.z / (VT / T), t0 = (int)blockIdx.z % (VT / T) * T;
  const int lane = (int)threadIdx.x & 63, r4 = (int)threadIdx.x >> 6, n = lane & 31, half = lane >> 5;
  const Kv8Span sp = kv8_span(p.s, p.c.shift, b);
  const int all = min(sp.rows, p.s.max_rows) * p.group, c = cb * kManyCols + 32 * w + n;
  if (c - n >= all) return;
  const int2 at = p.parts[((size_t)b * p.c.heads + h) * p.blocks + cb];
  if (at.y == 0 || c >= all) return;
  // the first part is its workgroup's last item, the others their workgroups' first
  auto place = [&](int k) { return p.part + (size_t)(2 * (at.x + k) + (k == 0 ? 1 : 0)) * many_floats(D); };
  float m = kLowest, l = 0.f;
  f32x4 o[T] = {};
#pragma unroll 2
  for (int k = 0; k < at.y; ++k) {
    const float *from = place(k);
    const float2 x = *(const float2 *)(from + kManyCols * D + (w * 64 + lane) * 2);
    f32x4 y[T];
#pragma unroll
    for (int t = 0; t < T; ++t) y[t] = *(const f32x4 *)(from + (((w * VT + t0 + t) * 4 + r4) * 64 + lane) * 4);
    const float mn = fmaxf(m, x.x), f = __builtin_amdgcn_exp2f(x.x - mn), g = __builtin_amdgcn_exp2f(m - mn);
    m = mn;
    l = l * g + x.y * f;
#pragma unroll
    for (int t = 0; t < T; ++t) o[t] = o[t] * g + y[t] * f;
  }
  const int64_t row = (int64_t)(sp.r0 + c / p.group) * p.a.q_heads + h * p.group + c % p.group;
  const float inv = l > 0.f || l != l ? 1.0f / l : 0.f;
  __bf16 *to = (__bf16 *)p.a.out + row * D + 32 * t0 + 8 * r4 + 4 * half;
#pragma unroll
  for (int t = 0; t < T; ++t) {
    const bf16x2 y[2] = {{(__bf16)(o[t][0] * inv), (__bf16)(o[t][1] * inv)},
                         {(__bf16)(o[t][2] * inv), (__bf16)(o[t][3] * inv)}};
    *(uint2 *)(to + 32 * t) = uint2{__builtin_bit_cast(uint32_t, y[0]), __builtin_bit_cast(uint32_t, y[1])};
  }
  if (t0 == 0 && r4 == 0 && half == 0 && p.a.lse)
    p.a.lse[row] = l > 0.f || l != l ? (m + log2f(l)) * kLn2 : -__builtin_inff();
}

// ---- accumulated attention weight -----------------------------------------------------
//
// A token's sum over rows and heads needs the finished log-sums, so it is a
// second pass.  With one tile of columns the attention leaves its scores
// behind (fp32, 4 bytes for each of at most 16 columns against the D bytes
// of K's codes), and k_kv8_weights_add turns them into weights.  With more,
// k_kv8_weights_many takes K Q^T again: a wave keeps 64 tokens of one KV
// head as matrix operands, the workgroup's columns pass through LDS 64 at a
// time, a lane adds up its tokens over its column of every tile, and the 32
// columns are joined at the end; where there are few tokens the columns are
// dealt over workgroups (parts).  A token's sum has one order, and so have
// those that k_kv8_weights_add adds to a page.
//
// Measured with the attention: 16 sequences of up to 6007 tokens, one row,
// 42 us (the weights 7 of them); 2 of up to 4093 with 1531 rows of 40 heads
// 326 us (K Q^T again 157, 500 TFLOP/s: a power for each score, 256 matrix
// operations, and two turns of workgroups that each first widen their tokens).

struct WeightParams {
  Kv8Attn a;
  Kv8Pool c;
  Kv8Batch s;
  int group, parts, len_pad;
  const float *scores;  // few: [seq][head][column][len_pad]
  int cols;
  float *part;          // many: [part][seq][head][len_pad]
  Kv8Links links;
};

// Adds x[i] of the lanes n and n ^ O, and leaves them the halves of the sums.
template <int O>
__device__ __forceinline__ void fold(float (&x)[32], int n) {
  const bool up = (n & O) != 0;
#pragma unroll
  for (int i = 0; i < O; ++i) {
    const float lo = x[i], hi = x[i + O];
    x[i] = (up ? hi : lo) + __shfl_xor(up ? lo : hi, O);
  }
}

template <int D>
__global__ __launch_bounds__(64 * kWeightWaves, 2) void k_kv8_weights_many(WeightParams p) {
  constexpr int KT = D / 16, kOps = 2 * KT;                        // operands of 32 columns, of 64
  constexpr int kMine = (kOps + kWeightWaves - 1) / kWeightWaves;  // brought by a wave
  __shared__ uint4 qbuf[2][kOps][64];
  const int h = (int)blockIdx.y, b = (int)blockIdx.z / p.parts, piece = (int)blockIdx.z % p.parts;
  const int tid = (int)threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n = lane & 31, half = lane >> 5, shift = p.c.shift;
  const Kv8Span sp = kv8_span(p.s, shift, b);
  const int end = min(sp.len, p.a.max_len), wg0 = (int)blockIdx.x * kWeightTokens;
  if (wg0 >= end) return;
  const int rows = min(sp.rows, p.s.max_rows), all = rows * p.group, pos0 = sp.len - sp.rows;
  const int t0 = wg0 + wave * 64;
  if (h == 0 && piece == 0 && tid < kWeightTokens >> shift)
    kv8_chain(p.links, p.c, p.s, kv8_seen(p.a, p.s, shift, b), b, (wg0 >> shift) + tid);

  // this wave's tokens as operands: row m of step u is token t0 + 32 u + m
  const float cs = fmaxf(fabsf(p.a.scale) * kLog2e, 1.1754944e-38f);  // its sign goes to q
  const uint32_t flip = p.a.scale < 0.f ? 0x80008000u : 0u;
  bf16x8 k[2][KT];
  uint32_t valid = 0;  // bit i: unit i has a page
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = t0 + 16 * i;
    const int id = t < end ? kv8_page(p.s, p.c, b, t >> shift) : -1;
    valid |= (id >= 0 ? 1u : 0u) << i;
  }
  valid = __builtin_amdgcn_readfirstlane(valid);
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int t = t0 + 32 * u + (n & 16);
    const int id = t < end ? max(kv8_page(p.s, p.c, b, t >> shift), 0) : 0;
    const size_t ph = (size_t)id * p.c.heads + h;
    const float f = kv8_scale(p.c.ks[ph]);
    const uint8_t *src = p.c.k + ((ph << (shift - 4)) + ((t >> 4) & ((1 << (shift - 4)) - 1))) * (16 * D) +
                         (n & 15) * 16 + half * 8;
#pragma unroll
    for (int c = 0; c < KT; ++c) {
      const uint2 w = *(const uint2 *)(src + c * 256);
      k[u][c] = fp8x8_to_bf16(w.x, w.y, f);
    }
  }

  // the workgroup's columns, in tiles of 64: those of rows that see a token of it
  const int wg_last = min(wg0 + kWeightTokens, end) - 1;
  const int row0 = min(max(wg0 - pos0, 0), rows);
  const int row1 = p.a.window ? max(min(rows, wg_last + p.a.window - pos0), row0) : rows;
  int tile0 = row0 * p.group >> 6, tile1 = (row1 * p.group + 63) >> 6;
  const int per = (tile1 - tile0 + p.parts - 1) / p.parts;
  tile0 += piece * per;
  tile1 = min(tile1, tile0 + per);

  // the lane's columns of the next tile to load, 64 tile + n and 32 on: row and
  // head, kept by steps (a division of each would cost more than the products)
  int row_at = (tile0 * 64 + n) / p.group, head_at = (tile0 * 64 + n) % p.group;
  const int row64 = 64 / p.group, head64 = 64 % p.group, row32 = 32 / p.group, head32 = 32 % p.group;
  uint4 qr[kMine];
  float z[2], z_next[2];
  int row[2], row_next[2];
  auto load = [&]() {
    const __bf16 *src[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      int i = row_at + (u ? row32 : 0), g = head_at + (u ? head32 : 0);
      if (g >= p.group) {
        g -= p.group;
        ++i;
      }
      // (a column past the last stands for one of the last row, before every token)
      row_next[u] = i < rows ? i : -(1 << 29);
      const int64_t r = sp.r0 + min(i, rows - 1), head = h * p.group + g;
      src[u] = (const __bf16 *)p.a.q.ptr + r * p.a.q.row_stride + head * p.a.q.head_stride + 8 * half;
      // (a row whose scores are all -inf gives 0 to each of its tokens)
      const float lse = p.a.lse[r * p.a.q_heads + head];
      z_next[u] = lse == -__builtin_inff() ? 0.f : lse * kLog2e;
    }
#pragma unroll
    for (int e = 0; e < kMine; ++e) {
      const int op = wave * kMine + e;  // column 32 (op / KT) + n, channels 16 (op % KT) + 8 half
      if (op < kOps) qr[e] = *(const uint4 *)((op / KT ? src[1] : src[0]) + op % KT * 16);
    }
    row_at += row64;
    head_at += head64;
    if (head_at >= p.group) {
      head_at -= p.group;
      ++row_at;
    }
  };
  auto store = [&](int buf) {
#pragma unroll
    for (int e = 0; e < kMine; ++e) {
      const int op = wave * kMine + e;
      if (op < kOps) qbuf[buf][op][lane] = uint4{qr[e].x ^ flip, qr[e].y ^ flip, qr[e].z ^ flip, qr[e].w ^ flip};
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      z[u] = z_next[u];
      row[u] = row_next[u];
    }
  };

  float sum[2][16] = {};
  if (tile0 < tile1) {
    load();
    store(0);
  }
  lds_barrier();
  for (int tile = tile0; tile < tile1; ++tile) {
    const int buf = (tile - tile0) & 1;
    if (tile + 1 < tile1) load();
    const int first = pos0 + tile * 64 / p.group, final = pos0 + min(tile * 64 + 63, all - 1) / p.group;
    // some column sees a token of the wave; every column sees all of them
    const bool some = t0 < end && final >= t0 && (!p.a.window || first - p.a.window < t0 + 63);
    const bool whole = valid == 15u && first >= t0 + 63 && t0 + 64 <= end && tile * 64 + 64 <= all &&
                       (!p.a.window || final - p.a.window < t0);
    if (some) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {  // 32 columns
        f32x16 s[2];
        const f32x16 zero = {};
#pragma unroll
        for (int t = 0; t < KT; ++t) {
          const bf16x8 q = as_bf16x8(qbuf[buf][c * KT + t][lane]);
#pragma unroll
          for (int u = 0; u < 2; ++u)
            s[u] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k[u][t], q, t ? s[u] : zero, 0, 0, 0);
        }
        if (whole) {
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int r = 0; r < 16; ++r) sum[u][r] += __builtin_amdgcn_exp2f(fmaf(s[u][r], cs, -z[c]));
        } else {
          const int pos = pos0 + row[c], hi = min(pos, end - 1), lo = p.a.window ? pos - p.a.window + 1 : 0;
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
              const int j = t0 + 32 * u + (r & 3) + 8 * (r >> 2) + 4 * half;
              const bool yes = ((valid >> (2 * u + (r >> 3)) & 1u) != 0) & (j >= lo) & (j <= hi);
              sum[u][r] += yes ? __builtin_amdgcn_exp2f(fmaf(s[u][r], cs, -z[c])) : 0.f;
            }
        }
      }
    }
    if (tile + 1 < tile1) store(buf ^ 1);
    lds_barrier();
  }
  // The 32 columns' sums of each of a lane's 32 tokens: every exchange halves
  // the tokens a lane holds, until lane n of each half has the whole sum of one.
  float x[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) x[i] = sum[i >> 4][i & 15];
  fold<16>(x, n);
  fold<8>(x, n);
  fold<4>(x, n);
  fold<2>(x, n);
  fold<1>(x, n);
  const int r = n & 15;
  float *out = p.part + (((size_t)piece * p.s.seqs + b) * p.c.heads + h) * p.len_pad;
  out[t0 + 32 * (n >> 4) + (r & 3) + 8 * (r >> 2) + 4 * half] = x[0];
}

// A token's sum of the weights pass for one sequence: from the scores that the
// attention left (FEW), or from the parts of k_kv8_weights_many.
template <bool FEW>
__device__ __forceinline__ float token_sum(const WeightParams &p, int b, int r0, int rows, int j) {
  float sum = 0.f;
  if constexpr (FEW) {
    const float *x = p.scores + (size_t)b * p.c.heads * p.cols * p.len_pad + j;
    const float *z = p.a.lse + (size_t)r0 * p.a.q_heads;
    // Columns of all heads in turn, kStep scores and log-sums in flight together
    // (columns beyond a sequence's own rows are not written; ones past the last
    // head read its own again).
    constexpr int kStep = 16;
    const int cols = rows * p.group, total = p.c.heads * cols;
    int h = 0, c = 0, i = 0, u = 0;  // head, its column (row i, query head u of the group)
    for (int e0 = 0; e0 < total; e0 += kStep) {
      float y[kStep], lse[kStep];
#pragma unroll
      for (int k = 0; k < kStep; ++k) {
        const int hh = min(h, p.c.heads - 1);
        y[k] = x[(size_t)(hh * p.cols + c) * p.len_pad];
        lse[k] = z[(size_t)i * p.a.q_heads + hh * p.group + u];
        if (++u == p.group) u = 0, ++i;
        if (++c == cols) c = i = u = 0, ++h;
      }
#pragma unroll
      for (int k = 0; k < kStep; ++k) {
        // (a row that sees nothing has -inf there and -inf scores)
        const float add = y[k] == -__builtin_inff() ? 0.f : __builtin_amdgcn_exp2f(y[k] - lse[k] * kLog2e);
        sum += e0 + k < total ? add : 0.f;
      }
    }
  } else {
    for (int i = 0; i < p.parts; ++i) {
      const float *x = p.part + ((size_t)i * p.s.seqs + b) * p.c.heads * p.len_pad + j;
#pragma unroll 8
      for (int h = 0; h < p.c.heads; ++h) sum += x[(size_t)h * p.len_pad];
    }
  }
  return sum;
}

// Adds the sums to the pages' weights.  Sequences may share pages (a common
// prefix) and a table may name one twice, so a page's sums are added by one
// workgroup, in the order of the tables' blocks: the attention (or the kernel
// above) has chained each block that some row sees to its page's list, one of
// kKv8Chains of its workgroup; the workgroup's threads follow them, the blocks
// are put in order, and as many as the threads hold are taken at a time.
// Where a list is longer than a look through the tables takes (a page that
// very many share), or all together longer than kBlocks, it does that instead.
//
// Bound by latency: list, lengths, scores, one after the other.  With the
// attention, 16 sequences of 6007 tokens (94 blocks) 54 us, and 64 us where they
// share 40 blocks; 256 of 1000 (16 blocks) 124 us, and 325 us where they share
// 10, each of them one workgroup's, four uses at a time.
constexpr int kBlocks = 1024, kLook = 4;

template <bool FEW>
__global__ __launch_bounds__(256) void k_kv8_weights_add(WeightParams p) {
  constexpr int T = 256;
  static_assert(T * kLook >= kBlocks, "");
  __shared__ int2 found[kBlocks], list[T * kLook];  // (block's number, page)
  __shared__ int count, part[kLook][T / 64];
  __shared__ float sums[T];
  const int tid = (int)threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int shift = p.c.shift, page = 1 << shift, deal = T >> shift;
  const unsigned all = (unsigned)p.s.seqs * (unsigned)p.links.blocks;
  const unsigned mine = blockIdx.x;
  // this thread's word of the page that is added to (threads of the first `page`)
  int open = -1;
  float acc = 0.f;
  float *const word = p.c.w + (tid & (page - 1));
  auto close = [&]() {
    if (open >= 0) word[(size_t)open << shift] = acc;
  };
  auto take = [&](int n) {  // the first n of the list
    // a thread's block: sequence, token, and what is seen of it (looked up a step ahead)
    unsigned b = 0;
    int j = 0;
    Kv8Seen q = {0, 0, 0, 0};
    auto look_up = [&](int i) {
      const unsigned e = (unsigned)list[min(i, n - 1)].x;
      b = e / (unsigned)p.links.blocks;
      j = (int)((e - b * (unsigned)p.links.blocks) << shift) + (tid & (page - 1));
      q = kv8_seen(p.a, p.s, shift, (int)b);
      if (i >= n) q.hi = 0;
    };
    if (n > 0) look_up(tid >> shift);
    for (int i0 = 0; i0 < n; i0 += deal) {
      const unsigned bb = b;
      const int jj = j;
      const Kv8Seen now = q;
      if (i0 + deal < n) look_up(i0 + deal + (tid >> shift));
      float x = 0.f;
      if (jj >= now.lo && jj < now.hi) x = token_sum<FEW>(p, (int)bb, now.r0, now.rows, jj);
      sums[tid] = x;
      __syncthreads();
      if (tid < page) {
        for (int k = 0; k < deal && i0 + k < n; ++k) {
          const int id = list[i0 + k].y;
          if (id != open) {
            close();
            open = id;
            acc = word[(size_t)id << shift];
          }
          acc += sums[(k << shift) + tid];
        }
      }
      __syncthreads();
    }
  };

  if (tid == 0) count = 0;
  __syncthreads();
  if (tid < kKv8Chains) {
    unsigned *head = p.links.head + ((unsigned)tid << p.links.bits) + mine;
    unsigned e = *head;
    if (e) *head = 0;
    // (a link costs half of what T * kLook numbers do)
    for (unsigned most = max(all / (T * kLook) * 2u, 16u); e; --most) {
      const int at = atomicAdd(&count, most ? 1 : kBlocks + 1);
      if (at >= kBlocks || !most) break;
      const uint2 link = p.links.next[e - 1];
      found[at] = int2{(int)(e - 1), (int)link.y};
      e = link.x;
    }
  }
  __syncthreads();
  const int n = count;
  if (n == 0) return;
  if (n <= kBlocks) {
    for (int i = tid; i < n; i += T) {
      const int2 x = found[i];
      int rank = 0;
      for (int k = 0; k < n; ++k) rank += (unsigned)found[k].x < (unsigned)x.x ? 1 : 0;
      list[rank] = x;
    }
    __syncthreads();
    take(n);
  } else {
    for (unsigned e0 = 0; e0 < all; e0 += T * kLook) {
      uint64_t hit[kLook];
      int id[kLook];
#pragma unroll
      for (int u = 0; u < kLook; ++u) {
        const unsigned e = e0 + T * u + tid, b = e / (unsigned)p.links.blocks;
        id[u] = -1;
        if (e < all) {
          const Kv8Seen q = kv8_seen(p.a, p.s, shift, (int)b);
          const int col = (int)(e - b * (unsigned)p.links.blocks);
          if (q.hi > q.lo && col >= q.lo >> shift && col <= (q.hi - 1) >> shift) id[u] = kv8_page(p.s, p.c, (int)b, col);
        }
        hit[u] = __ballot(id[u] >= 0 && ((unsigned)id[u] & ((1u << p.links.bits) - 1u)) == mine);
        if (lane == 0) part[u][wave] = __popcll(hit[u]);
      }
      __syncthreads();
      int m = 0;
#pragma unroll
      for (int u = 0; u < kLook; ++u) {
        int to = m;
        for (int w = 0; w < T / 64; ++w) {
          if (w < wave) to += part[u][w];
          m += part[u][w];
        }
        if (hit[u] >> lane & 1u)
          list[to + __popcll(hit[u] & ((1ull << lane) - 1ull))] = int2{(int)(e0 + T * u + tid), id[u]};
      }
      __syncthreads();
      take(m);
    }
  }
  close();
}

}  // namespace

hipError_t launch_kv8_attention(const Kv8Attn &a, const Kv8Pool &c, const Kv8Batch &s, int dim,
                                const Kv8Plan &pl, unsigned *counters, float *part, float *scores,
                                const Kv8Links &links, hipStream_t stream) {
  if (pl.few) {
    const DecodeParams p{a, c, s, pl.group, pl.blocks, pl.spw, pl.rounds, pl.splits, part, counters,
                         pl.score_cols ? scores : nullptr, pl.len_pad, pl.score_cols, links};
    const dim3 grid((unsigned)pl.splits * (unsigned)(s.seqs * c.heads * pl.blocks));
    auto k = dim == 64    ? (pl.ct == 1   ? k_kv8_decode<64, 1>
                             : pl.ct == 2 ? k_kv8_decode<64, 2>
                                          : k_kv8_decode<64, 4>)
             : dim == 128 ? (pl.ct == 1 ? k_kv8_decode<128, 1> : k_kv8_decode<128, 2>)
                          : k_kv8_decode<256, 1>;
    k<<<grid, dim3(64 * kDecodeWaves), 0, stream>>>(p);
    return hipGetLastError();
  }
  const PrefillParams p{a, c, s, pl.group, pl.blocks, part,
                        (int2 *)(part + 2 * kManyGroups * (size_t)many_floats(dim))};
  const dim3 grid = pl.dealt ? dim3(kManyGroups) : dim3((unsigned)c.heads * (unsigned)pl.blocks, (unsigned)s.seqs);
  auto pick = [&](auto dealt) {
    constexpr bool kDealt = decltype(dealt)::value;
    return dim == 64    ? k_kv8_prefill<64, 1, 8, 2, kDealt>
           : dim == 128 ? k_kv8_prefill<128, 1, 8, 2, kDealt>
                        : k_kv8_prefill<256, 1, 8, 1, kDealt>;
  };
  auto k = pl.dealt ? pick(std::true_type{}) : pick(std::false_type{});
  k<<<grid, dim3(512), 0, stream>>>(p);
  if (hipError_t e = hipGetLastError()) return e;
  if (!pl.dealt) return hipSuccess;
  // All channels of 32 columns for a workgroup, unless there are few items of
  // many parts (8 items of 32 parts: 32 channels at a time 66 us with the
  // attention, all 256 100 us; 192 items of up to 3 177 and 173 us).
  const bool wide = (int64_t)s.seqs * c.heads * pl.blocks >= 64;
  const dim3 jgrid((unsigned)pl.blocks * (kManyCols / 32), (unsigned)c.heads,
                   (unsigned)(s.seqs * (wide ? 1 : dim / 32)));
  auto kj = dim == 64    ? (wide ? k_kv8_prefill_join<64, 2> : k_kv8_prefill_join<64, 1>)
            : dim == 128 ? (wide ? k_kv8_prefill_join<128, 4> : k_kv8_prefill_join<128, 1>)
                         : (wide ? k_kv8_prefill_join<256, 8> : k_kv8_prefill_join<256, 1>);
  kj<<<jgrid, dim3(256), 0, stream>>>(p);
  return hipGetLastError();
}

hipError_t launch_kv8_weights(const Kv8Attn &a, const Kv8Pool &c, const Kv8Batch &s, int dim,
                              const Kv8Plan &pl, float *scores, const Kv8Links &links, hipStream_t stream) {
  if (a.max_len <= 0) return hipSuccess;
  const WeightParams p{a, c, s, pl.group, pl.parts, pl.len_pad, scores, pl.score_cols, scores, links};
  const unsigned groups = 1u << links.bits;
  if (pl.score_cols) {
    k_kv8_weights_add<true><<<dim3(groups), dim3(256), 0, stream>>>(p);
    return hipGetLastError();
  }
  const dim3 grid((unsigned)(pl.len_pad / kWeightTokens), (unsigned)c.heads, (unsigned)(s.seqs * pl.parts));
  auto k = dim == 64 ? k_kv8_weights_many<64> : dim == 128 ? k_kv8_weights_many<128> : k_kv8_weights_many<256>;
  k<<<grid, dim3(64 * kWeightWaves), 0, stream>>>(p);
  if (hipError_t e = hipGetLastError()) return e;
  k_kv8_weights_add<false><<<dim3(groups), dim3(256), 0, stream>>>(p);
  return hipGetLastError();
}

}  // namespace nvfp4
