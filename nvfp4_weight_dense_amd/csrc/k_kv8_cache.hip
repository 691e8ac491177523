// k_kv8_cache.hip -- writing the 8-bit paged KV cache: new tokens into it
// (k_kv8_append) and the tokens that an eviction keeps into fresh pages
// (k_kv8_select, k_kv8_move).
//
// A page's scale of one head is 2^E with the smallest E that holds the
// page's largest finite magnitude (amax <= 448 * 2^E).  E4M3 is a floating
// code, so a power of two loses no precision against an exact quotient
// except in the lowest, subnormal codes, and it lets a later token raise
// the page's scale without a second rounding of the codes that are there
// (kv8_rescale4).
#include <algorithm>
#include <type_traits>

#include "kv8_common.h"
#include "launchers.h"

namespace nvfp4 {

namespace {

struct AppendParams {
  const __bf16 *x[2];  // K and V rows
  int64_t row_stride[2], head_stride[2];
  Kv8Pool c;
  Kv8Batch s;
};

typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

// the larger of two packed pairs of bf16 magnitudes (as bits, NaN above infinity)
__device__ __forceinline__ uint32_t max_bits(uint32_t m, uint32_t v) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, m),
                                                                __builtin_bit_cast(u16x2, v & 0x7FFF7FFFu)));
}
// four bf16 (two packed pairs) over a power of two -> E4M3 bytes, nearest-even, for magnitudes up to 448 scales
__device__ __forceinline__ uint32_t encode_pairs(uint32_t a, uint32_t b, float scale) {
  s16x2 w = {0, 0};
  w = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(w, __builtin_bit_cast(bf16x2, a), scale, false);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(w, __builtin_bit_cast(bf16x2, b), scale, true);
  return __builtin_bit_cast(uint32_t, w);
}
// eight bf16 as fp32
__device__ __forceinline__ void widen8(uint4 v, float *f) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_bits_to_f32(u[i] & 0xFFFFu);
    f[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}

// One workgroup of T threads: one page that a sequence's new tokens touch,
// one KV head, K or V.  Bound by the bytes (4 read for each element of K and
// V, 2 written): a thread takes all its pieces into registers at once -- of K
// 2 NU times 16 channels of a token, of V NU times 8 channels of a group of
// four tokens, whose codes of a channel are one dword -- finds the largest
// magnitude with the workgroup, and writes codes.  V's codes are put in order
// in LDS; its 16-byte pieces that also hold older tokens, or places not yet
// used, take those bytes from the page.
//
// Measured (8 heads of 128): 5 prompts of up to 2741 tokens 15.9 us, 4250 GB/s
// of the 4750 that a copy reaches; a token of each of 64 sequences 4.9 us,
// a start and three dependent look-ups.
template <int D, int NU, int T>
__global__ __launch_bounds__(T) void k_kv8_append(AppendParams p) {
  extern __shared__ __align__(16) uint8_t image[];
  __shared__ unsigned part[4];
  const int b = (int)blockIdx.z, h = (int)blockIdx.y >> 1, isv = (int)blockIdx.y & 1;
  const int tid = (int)threadIdx.x;
  const int shift = p.c.shift, page = 1 << shift;
  const Kv8Span sp = kv8_span(p.s, shift, b);
  const int pos0 = sp.len - sp.rows;  // position of row 0 (rows before position 0 are dropped)
  const int col = (max(pos0, 0) >> shift) + (int)blockIdx.x;
  const int s0 = max(max(pos0, 0) - (col << shift), 0);
  // (of more rows than max_rows, for which the grid and the pieces are too few, the first are written)
  const int s1 = min(pos0 + min(sp.rows, p.s.max_rows) - (col << shift), page);
  if (s1 <= s0) return;

  const int64_t xs = p.row_stride[isv];
  const __bf16 *x = p.x[isv] + (int64_t)h * p.head_stride[isv] +
                    (int64_t)(sp.r0 + (col << shift) - pos0) * xs;  // slot 0's row
  // K: piece i is channels 16 (i % (D/16)) .. of slot s0 + i / (D/16), two
  // loads; V: channels 8 (i % (D/8)) .. of slots 4 (q0 + i / (D/8)) .., four
  const int q0 = s0 >> 2, q1 = (s1 + 3) >> 2;
  uint4 r[NU][4];
  if (!isv) {
#pragma unroll
    for (int u = 0; u < 2 * NU; ++u) {
      const int i = tid + T * u, slot = s0 + i / (D / 16);
      const uint4 *src = (const uint4 *)(x + slot * xs + i % (D / 16) * 16);
      const bool in = slot < s1;
      r[u >> 1][2 * (u & 1)] = in ? load_once(src) : uint4{0, 0, 0, 0};
      r[u >> 1][2 * (u & 1) + 1] = in ? load_once(src + 1) : uint4{0, 0, 0, 0};
    }
  } else {
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      const int i = tid + T * u, slot = 4 * (q0 + i / (D / 8));
#pragma unroll
      for (int k = 0; k < 4; ++k)
        r[u][k] = slot + k >= s0 && slot + k < s1 ? load_once((const uint4 *)(x + (slot + k) * xs + i % (D / 8) * 8))
                                                  : uint4{0, 0, 0, 0};
    }
  }
  const int id = kv8_page(p.s, p.c, b, col);  // (while the rows are on their way)
  if (id < 0) return;
  const size_t ph = (size_t)id * p.c.heads + h;
  uint8_t *codes = (isv ? p.c.v : p.c.k) + (ph << shift) * D;
  uint8_t *scale = (isv ? p.c.vs : p.c.ks) + ph;
  const int was = s0 > 0 ? min((int)*scale - 127, kKv8MaxExp) : kKv8MinExp;

  uint32_t bits = 0;
#pragma unroll
  for (int u = 0; u < NU; ++u)
#pragma unroll
    for (int k = 0; k < 4; ++k)
      bits = max_bits(max_bits(max_bits(max_bits(bits, r[u][k].x), r[u][k].y), r[u][k].z), r[u][k].w);
  bits = kv8_block_max_u(max(bits & 0xFFFFu, bits >> 16), part);
  float amax = bf16_bits_to_f32(bits);
  if (bits >= 0x7F80u) {  // infinities and NaN count for no scale
    amax = 0.f;
#pragma unroll
    for (int u = 0; u < NU; ++u)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float f[8];
        widen8(r[u][k], f);
#pragma unroll
        for (int j = 0; j < 8; ++j) amax = kv8_max_finite(amax, f[j]);
      }
    __syncthreads();
    amax = __uint_as_float(kv8_block_max_u(__float_as_uint(amax), part));
  }
  const int e = max(kv8_exponent(amax), was);
  // 2^(was - e): below 2^-126 every code goes to zero either way
  const float move = e > was ? kv8_two(max(was - e, -126)) : 1.0f;
  // every magnitude is at most 448 scales, and none is NaN: the conversion needs no clamp
  const bool plain = bits < 0x7F80u && amax <= 448.0f * kv8_two(kKv8MaxExp);
  const float sc = kv8_two(e);
  const float inv = kv8_two(-e);

  if (!isv) {
    if (e > was && s0 > 0)
      for (int i = tid; i < s0 * (D / 16); i += T) {
        uint4 *q = (uint4 *)(codes + kv8_k_at(i % s0, i / s0 * 16, D));
        uint4 v = *q;
        v.x = kv8_rescale4(v.x, move);
        v.y = kv8_rescale4(v.y, move);
        v.z = kv8_rescale4(v.z, move);
        v.w = kv8_rescale4(v.w, move);
        *q = v;
      }
#pragma unroll
    for (int u = 0; u < 2 * NU; ++u) {
      const int i = tid + T * u, slot = s0 + i / (D / 16);
      if (slot >= s1) continue;
      uint4 *to = (uint4 *)(codes + kv8_k_at(slot, i % (D / 16) * 16, D));
      if (plain) {
        const uint4 lo = r[u >> 1][2 * (u & 1)], hi = r[u >> 1][2 * (u & 1) + 1];
        *to = uint4{encode_pairs(lo.x, lo.y, sc), encode_pairs(lo.z, lo.w, sc), encode_pairs(hi.x, hi.y, sc),
                    encode_pairs(hi.z, hi.w, sc)};
        continue;
      }
      float f[16];
      widen8(r[u >> 1][2 * (u & 1)], f);
      widen8(r[u >> 1][2 * (u & 1) + 1], f + 8);
#pragma unroll
      for (int j = 0; j < 16; ++j) f[j] *= inv;
      *to = uint4{kv8_encode4(f), kv8_encode4(f + 4), kv8_encode4(f + 8), kv8_encode4(f + 12)};
    }
    if (h == 0 && p.c.w)
      for (int i = s0 + tid; i < s1; i += T) p.c.w[((size_t)id << shift) + i] = 0.f;
  } else {
    // 16-byte piece i of the groups from `from` on: slots 4 q .., channels 64 a + 16 c + r
    const int from = e > was ? 0 : q0, np = (q1 - from) * (D / 4);
    auto piece = [&](int i) {
      const int q = from + i / (D / 4), ar = i % (D / 4);
      return kv8_v_at(4 * q, (ar >> 4) * 64 + (ar & 15), D);
    };
    for (int i = tid; i < np; i += T) {
      const int q = from + i / (D / 4);
      if (4 * q >= s0 && 4 * q + 3 < s1) continue;  // all new
      const int at = piece(i);
      uint4 v = *(const uint4 *)(codes + at);
      if (e > was && 4 * q < s0) {
        const int keep = s0 - 4 * q;  // this many of its tokens are older
        const uint32_t mask = keep >= 4 ? 0xFFFFFFFFu : (1u << (8 * keep)) - 1u;
        v.x = (kv8_rescale4(v.x, move) & mask) | (v.x & ~mask);
        v.y = (kv8_rescale4(v.y, move) & mask) | (v.y & ~mask);
        v.z = (kv8_rescale4(v.z, move) & mask) | (v.z & ~mask);
        v.w = (kv8_rescale4(v.w, move) & mask) | (v.w & ~mask);
      }
      *(uint4 *)(image + at) = v;
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      const int i = tid + T * u, slot = 4 * (q0 + i / (D / 8)), d = i % (D / 8) * 8;
      if (slot >= s1) continue;
      const uint32_t lo = (uint32_t)max(s0 - slot, 0), hi = (uint32_t)min(s1 - slot, 4);  // its new tokens
      const uint32_t mask = (hi == 4 ? 0xFFFFFFFFu : (1u << (8 * hi)) - 1u) & (0xFFFFFFFFu << (8 * lo));
      uint32_t w[8];  // a channel's four tokens
      if (plain) {
        const uint32_t t[4][4] = {{r[u][0].x, r[u][0].y, r[u][0].z, r[u][0].w},
                                  {r[u][1].x, r[u][1].y, r[u][1].z, r[u][1].w},
                                  {r[u][2].x, r[u][2].y, r[u][2].z, r[u][2].w},
                                  {r[u][3].x, r[u][3].y, r[u][3].z, r[u][3].w}};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t sel = j & 1 ? 0x07060302u : 0x05040100u;
          w[j] = encode_pairs(__builtin_amdgcn_perm(t[1][j >> 1], t[0][j >> 1], sel),
                              __builtin_amdgcn_perm(t[3][j >> 1], t[2][j >> 1], sel), sc);
        }
      } else {
        float f[4][8];
#pragma unroll
        for (int k = 0; k < 4; ++k) widen8(r[u][k], f[k]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float y[4] = {f[0][j] * inv, f[1][j] * inv, f[2][j] * inv, f[3][j] * inv};
          w[j] = kv8_encode4(y);
        }
      }
      const int at = kv8_v_at(slot, d, D);  // channels d .. d + 7 are 16 bytes apart
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t *to = (uint32_t *)(image + at + 16 * j);
        *to = mask == 0xFFFFFFFFu ? w[j] : (w[j] & mask) | (*to & ~mask);
      }
    }
    __syncthreads();
    for (int i = tid; i < np; i += T) {
      const int at = piece(i);
      *(uint4 *)(codes + at) = *(const uint4 *)(image + at);
    }
  }
  if (tid == 0) *scale = (uint8_t)(e + 127);
}

// ---- eviction ---------------------------------------------------------------------
//
// Which tokens stay: the first `sink`, the last `recent` and of those between
// them the `need` = keep - sink - recent with the largest weights.  Weights
// become words of the same order, and the smallest word that stays is found
// by three digits (11, 11, 10 bits) with a histogram each; of the tokens
// that share it the first stay.  Counts are whole numbers, so the order of
// their atomic additions does not show.
//
// Bound by latency: 12 sequences of up to 6143 tokens 11.7 us (one workgroup
// each: look-ups, three scans, the list), one of 130001 tokens 27 us in five
// launches of 4.4 to 7.1 us (72 us with the move; one workgroup for it all: 430).

struct SelectParams {
  Kv8Pool c;
  Kv8Batch s;
  int keep, recent, sink, max_len;
  int *new_lens;     // [seqs]
  int *kept;         // [seqs][keep]
  // where a sequence is dealt over workgroups:
  int chunks;
  uint32_t *words;   // [seqs][chunks * kChunk]
  unsigned *hist;    // [seqs][3][kBins], zero on entry, left zero
  int *counts;       // [seqs][chunks][2]: tokens that stay, tokens with the last word
  unsigned *limit;   // [seqs][2]: the last word, how many of its tokens stay
};

constexpr int kBins = 2048, kDealt = 256, kChunk = 4 * kDealt;
__device__ __forceinline__ int digit_shift(int i) { return i == 0 ? 21 : i == 1 ? 10 : 0; }
__device__ __forceinline__ uint32_t digit(uint32_t w, int i) { return w >> digit_shift(i) & (i == 2 ? 1023u : 2047u); }

// A weight as an unsigned word with the same order (-0 as +0, NaN above all).
__device__ __forceinline__ uint32_t order_word(float w) {
  if (w != w) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(w == 0.f ? 0.f : w);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

struct Span {  // the tokens that compete: [lo, hi)
  int len, lo, hi, need;
};
__device__ __forceinline__ Span select_span(const SelectParams &p, int b) {
  Span s;
  s.len = min(kv8_span(p.s, p.c.shift, b).len, p.max_len);
  s.lo = p.sink;
  s.hi = s.len - p.recent;
  s.need = p.keep - p.sink - p.recent;
  return s;
}
// The words of the tokens j + k * step below hi (all loads in flight together;
// hi > 0, and places beyond it read its last token).
template <int N>
__device__ __forceinline__ void token_words(const SelectParams &p, int b, int j, int step, int hi, uint32_t (&u)[N]) {
  int id[N];
#pragma unroll
  for (int k = 0; k < N; ++k) id[k] = kv8_page(p.s, p.c, b, min(j + k * step, hi - 1) >> p.c.shift);
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const int slot = min(j + k * step, hi - 1) & ((1 << p.c.shift) - 1);
    u[k] = __float_as_uint(p.c.w[((size_t)max(id[k], 0) << p.c.shift) + slot]);
  }
#pragma unroll
  for (int k = 0; k < N; ++k) u[k] = id[k] < 0 ? 0u : order_word(__uint_as_float(u[k]));
}

// The digit of the `left`-th largest word from a histogram (1 <= left <= its
// sum), and which of that digit's words it is.  A thread owns neighbouring
// bins, the first thread the highest; scratch: LDS of NT / 64 + 2 words.
template <int NT>
__device__ __forceinline__ void find_digit(const unsigned *hist, unsigned &left, uint32_t &dig, unsigned *scratch) {
  constexpr int kPer = kBins / NT;
  const int tid = (int)threadIdx.x, lane = tid & 63, wave = tid >> 6;
  unsigned c[kPer], sum = 0;
#pragma unroll
  for (int k = 0; k < kPer; ++k) c[k] = hist[kBins - 1 - tid * kPer - k];
#pragma unroll
  for (int k = 0; k < kPer; ++k) sum += c[k];
  unsigned incl = sum;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const unsigned x = __shfl_up(incl, o);
    if (lane >= o) incl += x;
  }
  if (lane == 63) scratch[2 + wave] = incl;
  __syncthreads();
  for (int i = 0; i < wave; ++i) incl += scratch[2 + i];
  unsigned run = incl - sum;
  if (run < left && left <= incl) {
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      if (run < left && left <= run + c[k]) {
        scratch[0] = (unsigned)(kBins - 1 - tid * kPer - k);
        scratch[1] = left - run;
      }
      run += c[k];
    }
  }
  __syncthreads();
  dig = scratch[0];
  left = scratch[1];
  __syncthreads();
}

// Writes the positions that stay of [j0, j1) from kept[at]; `seen` tokens
// with the last word lie before j0.  Each wave owns one run of positions, so
// the order needs one exchange of counts.
template <int NT, typename F>
__device__ __forceinline__ void emit(const Span &sp, int j0, int j1, uint32_t last, int left, int at, int seen,
                                     int *kept, int (*part)[2], F word) {
  const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
  const int run = (((j1 - j0 + NT / 64 - 1) / (NT / 64)) + 63) & ~63;
  const int a = min(j0 + wave * run, j1), z = min(a + run, j1);
  auto kind = [&](int j) {  // 0 goes, 1 stays, 2 stays if among the first with the last word
    if (j >= z) return 0;
    if (j < sp.lo || j >= sp.hi) return 1;
    if (sp.need == 0) return 0;
    const uint32_t u = word(j);
    return u > last ? 1 : u == last ? 2 : 0;
  };
  int na = 0, ne = 0;
  for (int j = a; j < z; j += 64) {
    const int k = kind(j + lane);
    na += __popcll(__ballot(k == 1));
    ne += __popcll(__ballot(k == 2));
  }
  if (lane == 0) {
    part[wave][0] = na;
    part[wave][1] = ne;
  }
  __syncthreads();
  for (int i = 0; i < wave; ++i) {
    at += part[i][0] + min(max(left - seen, 0), part[i][1]);
    seen += part[i][1];
  }
  const uint64_t before = (1ull << lane) - 1ull;
  for (int j = a; j < z; j += 64) {
    const int k = kind(j + lane);
    const uint64_t eq = __ballot(k == 2);
    const bool in = k == 1 || (k == 2 && seen + __popcll(eq & before) < left);
    const uint64_t yes = __ballot(in);
    if (in) kept[at + __popcll(yes & before)] = j + lane;
    at += __popcll(yes);
    seen += __popcll(eq);
  }
}

// Up to kWhole tokens: one workgroup per sequence, the words in LDS.
constexpr int kWhole = 32768, kWholeThreads = 1024;

__global__ __launch_bounds__(kWholeThreads) void k_kv8_select(SelectParams p) {
  __shared__ uint32_t words[kWhole];
  __shared__ unsigned hist[kBins], scratch[2 + kWholeThreads / 64];
  __shared__ int part[kWholeThreads / 64][2];
  const int b = (int)blockIdx.x, tid = (int)threadIdx.x;
  const Span sp = select_span(p, b);
  int *kept = p.kept + (size_t)b * p.keep;
  if (tid == 0) p.new_lens[b] = min(sp.len, p.keep);
  if (sp.len <= p.keep) {
    for (int i = tid; i < p.keep; i += kWholeThreads) kept[i] = i < sp.len ? i : -1;
    return;
  }
  uint32_t prefix = 0;
  unsigned left = (unsigned)sp.need;
  if (sp.need > 0) {
    for (int i = tid; i < kBins; i += kWholeThreads) hist[i] = 0;
    __syncthreads();
    for (int j0 = sp.lo + tid; j0 < sp.hi; j0 += 8 * kWholeThreads) {
      uint32_t u[8];
      token_words(p, b, j0, kWholeThreads, sp.hi, u);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int j = j0 + k * kWholeThreads;
        if (j >= sp.hi) break;
        words[j] = u[k];
        atomicAdd(&hist[digit(u[k], 0)], 1u);
      }
    }
    __syncthreads();
    for (int i = 0; i < 3; ++i) {
      uint32_t d;
      find_digit<kWholeThreads>(hist, left, d, scratch);
      prefix |= d << digit_shift(i);
      if (i == 2) break;
      for (int k = tid; k < kBins; k += kWholeThreads) hist[k] = 0;
      __syncthreads();
      for (int j = sp.lo + tid; j < sp.hi; j += kWholeThreads)
        if (words[j] >> digit_shift(i) == prefix >> digit_shift(i)) atomicAdd(&hist[digit(words[j], i + 1)], 1u);
      __syncthreads();
    }
  }
  emit<kWholeThreads>(sp, 0, sp.len, prefix, (int)left, 0, 0, kept, part, [&](int j) { return words[j]; });
}

// More tokens: chunks of them, a launch for each digit, one for the counts of
// each chunk and one that writes.
template <int STAGE>  // 0: words and the first histogram; 1, 2: the next digit's; 3: counts
__global__ __launch_bounds__(kDealt) void k_kv8_select_stage(SelectParams p) {
  __shared__ unsigned local[kBins], scratch[2 + kDealt / 64];
  __shared__ int part[2];
  const int b = (int)blockIdx.y, tid = (int)threadIdx.x;
  const Span sp = select_span(p, b);
  const int j0 = (int)blockIdx.x * kChunk, j1 = min(j0 + kChunk, sp.len);
  if (sp.len <= p.keep || j0 >= sp.len) return;
  uint32_t *words = p.words + (size_t)b * p.chunks * kChunk;
  unsigned *hist = p.hist + (size_t)b * 3 * kBins;
  uint32_t prefix = 0;
  unsigned left = (unsigned)sp.need;
  if (sp.need > 0) {
#pragma unroll
    for (int i = 0; i < STAGE; ++i) {
      uint32_t d;
      find_digit<kDealt>(hist + i * kBins, left, d, scratch);
      prefix |= d << digit_shift(i);
    }
  }
  // a thread's four tokens: whether they compete, and their words
  bool in[4];
  uint32_t u[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int j = j0 + tid + k * kDealt;
    in[k] = j < j1 && j >= sp.lo && j < sp.hi && sp.need > 0;
    if constexpr (STAGE > 0) u[k] = words[min(max(j, sp.lo), max(sp.hi - 1, sp.lo))];
  }
  if constexpr (STAGE == 0) token_words(p, b, j0 + tid, kDealt, sp.len, u);
  if constexpr (STAGE < 3) {
    if (sp.need == 0) return;
    for (int i = tid; i < kBins; i += kDealt) local[i] = 0;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (!in[k]) continue;
      if constexpr (STAGE == 0) {
        words[j0 + tid + k * kDealt] = u[k];
      } else {
        if (u[k] >> digit_shift(STAGE - 1) != prefix >> digit_shift(STAGE - 1)) continue;
      }
      atomicAdd(&local[digit(u[k], STAGE)], 1u);
    }
    __syncthreads();
    for (int i = tid; i < kBins; i += kDealt)
      if (local[i]) atomicAdd(&hist[STAGE * kBins + i], local[i]);
  } else {
    if (tid < 2) part[tid] = 0;
    __syncthreads();
    int above = 0, equal = 0;  // of the wave
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int j = j0 + tid + k * kDealt;
      const bool always = j < j1 && (j < sp.lo || j >= sp.hi);
      above += __popcll(__ballot(always || (in[k] && u[k] > prefix)));
      equal += __popcll(__ballot(in[k] && u[k] == prefix));
    }
    if ((tid & 63) == 0) {
      atomicAdd(&part[0], above);
      atomicAdd(&part[1], equal);
    }
    __syncthreads();
    if (tid < 2) p.counts[((size_t)b * p.chunks + blockIdx.x) * 2 + tid] = part[tid];
    if (blockIdx.x == 0 && tid == 0) {
      p.limit[2 * b] = prefix;
      p.limit[2 * b + 1] = left;
    }
  }
}

__global__ __launch_bounds__(kDealt) void k_kv8_select_emit(SelectParams p) {
  __shared__ int part[kDealt / 64][2];
  const int b = (int)blockIdx.y, tid = (int)threadIdx.x, chunk = (int)blockIdx.x;
  const Span sp = select_span(p, b);
  int *kept = p.kept + (size_t)b * p.keep;
  if (chunk == 0 && tid == 0) p.new_lens[b] = min(sp.len, p.keep);
  if (sp.len <= p.keep) {
    for (int i = chunk * kDealt + tid; i < p.keep; i += p.chunks * kDealt) kept[i] = i < sp.len ? i : -1;
    return;
  }
  if (chunk == 0)  // (the histograms' last reader has ended)
    for (int i = tid; i < 3 * kBins; i += kDealt) p.hist[(size_t)b * 3 * kBins + i] = 0;
  const int j0 = chunk * kChunk, j1 = min(j0 + kChunk, sp.len);
  if (j0 >= sp.len) return;
  const int left = (int)p.limit[2 * b + 1];
  const int *counts = p.counts + (size_t)b * p.chunks * 2;
  __shared__ int before[2];
  if (tid < 2) before[tid] = 0;
  __syncthreads();
  int stays = 0, same = 0;
  for (int i = tid; i < chunk; i += kDealt) {
    stays += counts[2 * i];
    same += counts[2 * i + 1];
  }
  if (stays) atomicAdd(&before[0], stays);
  if (same) atomicAdd(&before[1], same);
  __syncthreads();
  const int seen = before[1], at = before[0] + min(seen, left);
  const uint32_t *words = p.words + (size_t)b * p.chunks * kChunk;
  emit<kDealt>(sp, j0, j1, p.limit[2 * b], left, at, seen, kept, part, [&](int j) { return words[j]; });
}

struct MoveParams {
  Kv8Pool c;
  Kv8Batch s;
  const int *new_table;  // [seqs][new_cols]
  int new_cols, keep, max_len;
  const int *kept;
};

// One workgroup: one fresh page of one sequence, one KV head, K or V.  A
// thread gathers NP 16-byte pieces of the new page (of K one token's 16
// channels, of V four tokens of four channels: a byte of each dword of four
// source pieces), the largest magnitude gives the new scale, and the codes
// move to it in registers.
//
// Bound by the reads: a token's 16 channels lie beside those of its 15
// neighbours, so most lines of the old pages are read where a quarter of
// their tokens stay.  1500 of up to 6143 tokens of each of 12 sequences 27 us
// (36 MB of codes kept, 84 MB fetched for them); 16411 of 130001 tokens 36 us
// (34 MB; a 128-byte line holds a part of eight tokens of K: two in three are read).
template <int D, int NP>
__global__ __launch_bounds__(256) void k_kv8_move(MoveParams p) {
  __shared__ unsigned part[4];
  __shared__ int src[128];  // unit of each token's codes, -1: none
  __shared__ int src_slot[128];
  __shared__ float src_scale[128];
  const int b = (int)blockIdx.z, h = (int)blockIdx.y >> 1, isv = (int)blockIdx.y & 1;
  const int tid = (int)threadIdx.x, nt = (int)blockDim.x;
  const int shift = p.c.shift, page = 1 << shift, col = (int)blockIdx.x;
  const int len = min(min(kv8_span(p.s, shift, b).len, p.max_len), p.keep);
  const int n = min(len - (col << shift), page);  // tokens of this page
  if (n <= 0) return;
  const int to = p.new_table[(size_t)b * p.new_cols + col];
  if ((unsigned)to >= (unsigned)p.c.pages) return;
  uint8_t *codes = isv ? p.c.v : p.c.k;
  uint8_t *scales = isv ? p.c.vs : p.c.ks;
  if (tid < n) {
    const int j = p.kept[(size_t)b * p.keep + (col << shift) + tid];
    const int id = kv8_page(p.s, p.c, b, j >> shift), slot = j & (page - 1);
    const size_t ph = (size_t)max(id, 0) * p.c.heads + h;
    src[tid] = id < 0 ? -1 : (int)((ph << (shift - 4)) + (slot >> 4));
    src_slot[tid] = slot & 15;
    src_scale[tid] = id < 0 ? 1.0f : kv8_scale(scales[ph]);
    if (h == 0 && !isv && p.c.w) p.c.w[((size_t)to << shift) + tid] = id < 0 ? 0.f : p.c.w[((size_t)id << shift) + slot];
  }
  __syncthreads();
  uint8_t *out = codes + (((size_t)to * p.c.heads + h) << shift) * D;
  // (a piece of tokens that no page names is zero)
  auto from = [&](int t, int at) {
    const int u = src[t];
    return u < 0 ? uint4{0, 0, 0, 0} : *(const uint4 *)(codes + (size_t)(uint32_t)u * (16 * D) + at);
  };
  uint32_t w[NP][4];
  float amax = 0.f;
  if (!isv) {
#pragma unroll
    for (int k = 0; k < NP; ++k) {  // piece: channels 16 ch of token t, tokens side by side
      const int i = tid + nt * k, t = i % page, ch = i / page;
      uint4 v = uint4{0, 0, 0, 0};
      if (ch < D / 16 && t < n) v = from(t, ch * 256 + src_slot[t] * 16);
      w[k][0] = v.x, w[k][1] = v.y, w[k][2] = v.z, w[k][3] = v.w;
    }
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      const float s = src_scale[min((tid + nt * k) % page, n - 1)];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        float f[4];
        kv8_decode4(w[k][c], f);
#pragma unroll
        for (int e = 0; e < 4; ++e) amax = fmaxf(amax, fabsf(f[e]) * s);
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < NP; ++k) {  // piece: group of four tokens q, channels 64 a + 16 c + r
      const int i = tid + nt * k, q = i / (D / 4), ar = i % (D / 4);
      uint4 v[4];
      uint32_t sel[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int t = 4 * q + e;
        v[e] = uint4{0, 0, 0, 0};
        sel[e] = 0;
        if (t < n) {
          v[e] = from(t, (ar >> 4) * 1024 + (src_slot[t] >> 2) * 256 + (ar & 15) * 16);
          sel[e] = (uint32_t)src_slot[t] & 3u;
        }
      }
      // bytes sel[0] of v[0], sel[1] of v[1] and so on, of each dword
      const uint32_t p01 = (4u + sel[0]) | sel[1] << 8, p23 = (4u + sel[2]) | sel[3] << 8;
      const uint32_t a0[4] = {v[0].x, v[0].y, v[0].z, v[0].w}, a1[4] = {v[1].x, v[1].y, v[1].z, v[1].w};
      const uint32_t a2[4] = {v[2].x, v[2].y, v[2].z, v[2].w}, a3[4] = {v[3].x, v[3].y, v[3].z, v[3].w};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint32_t lo = __builtin_amdgcn_perm(a0[c], a1[c], p01), hi = __builtin_amdgcn_perm(a2[c], a3[c], p23);
        w[k][c] = (lo & 0xFFFFu) | hi << 16;
      }
    }
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      const int q = (tid + nt * k) / (D / 4);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        float f[4];
        kv8_decode4(w[k][c], f);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (4 * q + e < n) amax = fmaxf(amax, fabsf(f[e]) * src_scale[4 * q + e]);
      }
    }
  }
  amax = __uint_as_float(kv8_block_max_u(__float_as_uint(amax), part));
  const int e = kv8_exponent(amax);
  const float inv = kv8_two(-e);
  // a code that is not zero is below 448 * 2^e and at least 2^-9 scales: its
  // factor is under 2^18 (the bound keeps a zero under a huge scale a zero)
  auto factor = [&](int t) { return fminf(src_scale[t] * inv, 0x1p18f); };
  if (!isv) {
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      const int i = tid + nt * k, t = i % page, ch = i / page;
      if (ch >= D / 16 || t >= n) continue;
      const float f = factor(t);
      *(uint4 *)(out + kv8_k_at(t, 16 * ch, D)) = uint4{kv8_rescale4(w[k][0], f), kv8_rescale4(w[k][1], f),
                                                        kv8_rescale4(w[k][2], f), kv8_rescale4(w[k][3], f)};
    }
  } else {
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      const int i = tid + nt * k, q = i / (D / 4), ar = i % (D / 4);
      if (4 * q >= n) continue;
      uint4 *at = (uint4 *)(out + kv8_v_at(4 * q, (ar >> 4) * 64 + (ar & 15), D));
      float f[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) f[x] = 4 * q + x < n ? factor(4 * q + x) : 1.0f;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        float y[4];
        kv8_decode4(w[k][c], y);
#pragma unroll
        for (int x = 0; x < 4; ++x) y[x] *= f[x];
        w[k][c] = kv8_encode4(y);
      }
      if (4 * q + 3 >= n) {  // places that stay unused keep their bytes
        const uint4 old = *at;
        const uint32_t keep = 0xFFFFFFFFu << (8 * (n - 4 * q));
        w[k][0] = (w[k][0] & ~keep) | (old.x & keep);
        w[k][1] = (w[k][1] & ~keep) | (old.y & keep);
        w[k][2] = (w[k][2] & ~keep) | (old.z & keep);
        w[k][3] = (w[k][3] & ~keep) | (old.w & keep);
      }
      *at = uint4{w[k][0], w[k][1], w[k][2], w[k][3]};
    }
  }
  if (tid == 0) scales[(size_t)to * p.c.heads + h] = (uint8_t)(e + 127);
}

}  // namespace

hipError_t launch_kv8_append(const Kv8Rows &k, const Kv8Rows &v, const Kv8Pool &c, const Kv8Batch &s,
                             int dim, hipStream_t stream) {
  AppendParams p;
  p.x[0] = (const __bf16 *)k.ptr;
  p.x[1] = (const __bf16 *)v.ptr;
  p.row_stride[0] = k.row_stride;
  p.row_stride[1] = v.row_stride;
  p.head_stride[0] = k.head_stride;
  p.head_stride[1] = v.head_stride;
  p.c = c;
  p.s = s;
  const int page = 1 << c.shift;
  // pages that max_rows tokens can touch, wherever they start
  const int64_t most = ((int64_t)s.max_rows + 2 * page - 2) >> c.shift;
  const int touched = (int)(most < s.cols ? most : s.cols);
  const dim3 grid((unsigned)touched, (unsigned)(2 * c.heads), (unsigned)s.seqs);
  // A few tokens are one wave's work, and each page's part one load for a
  // thread; otherwise a page is 8192 elements for each unit of 256 threads.
  const bool few = s.max_rows * dim <= 1024;
  const int units = page * dim / 8192;
  auto pick = [&](auto d) {
    constexpr int D = decltype(d)::value, kMost = 128 * D / 8192;
    return few ? k_kv8_append<D, 1, 64>
               : units <= 1 ? k_kv8_append<D, 1, 256> : units == 2 ? k_kv8_append<D, kMost < 2 ? kMost : 2, 256>
                                                                   : k_kv8_append<D, kMost, 256>;
  };
  auto k_append = dim == 64 ? pick(std::integral_constant<int, 64>{})
                            : dim == 128 ? pick(std::integral_constant<int, 128>{})
                                         : pick(std::integral_constant<int, 256>{});
  k_append<<<grid, dim3(few ? 64 : 256), (size_t)page * dim, stream>>>(p);
  return hipGetLastError();
}

Kv8EvictPlan kv8_evict_plan(const Kv8Batch &s, int max_len) {
  Kv8EvictPlan pl = {};
  if (max_len <= kWhole) return pl;  // in LDS
  pl.chunks = (max_len + kChunk - 1) / kChunk;
  pl.hist_words = (size_t)s.seqs * 3 * kBins;
  pl.words = (size_t)s.seqs * pl.chunks * (kChunk + 2) + (size_t)s.seqs * 2;
  return pl;
}

hipError_t launch_kv8_evict(const Kv8Pool &c, const Kv8Batch &s, int dim, int max_len, const int *new_table,
                            int new_cols, int keep, int recent, int sink, int *new_lens, int *kept,
                            const Kv8EvictPlan &pl, unsigned *hist, uint32_t *words, hipStream_t stream) {
  SelectParams sel{c, s, keep, recent, sink, max_len, new_lens, kept, pl.chunks, words, hist, nullptr, nullptr};
  if (pl.chunks == 0) {
    k_kv8_select<<<dim3((unsigned)s.seqs), dim3(kWholeThreads), 0, stream>>>(sel);
    if (hipError_t e = hipGetLastError()) return e;
  } else {
    sel.counts = (int *)(words + (size_t)s.seqs * pl.chunks * kChunk);
    sel.limit = (unsigned *)(sel.counts + (size_t)s.seqs * pl.chunks * 2);
    const dim3 grid((unsigned)pl.chunks, (unsigned)s.seqs), block(kDealt);
    for (auto k : {k_kv8_select_stage<0>, k_kv8_select_stage<1>, k_kv8_select_stage<2>, k_kv8_select_stage<3>,
                   k_kv8_select_emit}) {
      k<<<grid, block, 0, stream>>>(sel);
      if (hipError_t e = hipGetLastError()) return e;
    }
  }
  const MoveParams p{c, s, new_table, new_cols, keep, max_len, kept};
  const int page = 1 << c.shift, np = page * dim / 4096;  // 16-byte pieces of a thread
  const dim3 grid((unsigned)((keep + page - 1) >> c.shift), (unsigned)(2 * c.heads), (unsigned)s.seqs);
  auto pick = [&](auto d) {
    constexpr int D = decltype(d)::value;
    return np <= 1 ? k_kv8_move<D, 1> : np == 2 ? k_kv8_move<D, 2> : np == 4 ? k_kv8_move<D, D / 32 < 4 ? D / 32 : 4>
                                                                              : k_kv8_move<D, D / 32>;
  };
  auto k = dim == 64 ? pick(std::integral_constant<int, 64>{})
                     : dim == 128 ? pick(std::integral_constant<int, 128>{}) : pick(std::integral_constant<int, 256>{});
  k<<<grid, dim3((unsigned)std::min(page * dim / 16, 256)), 0, stream>>>(p);  // a small page: a thread a piece
  return hipGetLastError();
}

}  // namespace nvfp4
