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

__device__ __forceinline__ void load8(const __bf16 *p, float *f) {
  const uint4 v = *(const uint4 *)p;
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_bits_to_f32(u[i] & 0xFFFFu);
    f[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}

// One workgroup: one page that a sequence's new tokens touch, one KV head,
// K or V.  Reads the new tokens twice (amax, then codes; the second time
// from the caches).  V's codes are put together in LDS, since one 16-byte
// piece holds four tokens; its pieces that also hold older tokens, or
// places not yet used, take those bytes from the page.
template <int D>
__global__ void k_kv8_append(AppendParams p) {
  extern __shared__ __align__(16) uint8_t image[];
  __shared__ float part[4];
  const int b = (int)blockIdx.z, h = (int)blockIdx.y >> 1, isv = (int)blockIdx.y & 1;
  const int tid = (int)threadIdx.x, nt = (int)blockDim.x;
  const int shift = p.c.shift, page = 1 << shift;
  const Kv8Span sp = kv8_span(p.s, shift, b);
  const int pos0 = sp.len - sp.rows;  // position of row 0 (rows before position 0 are dropped)
  const int col = (max(pos0, 0) >> shift) + (int)blockIdx.x;
  const int s0 = max(max(pos0, 0) - (col << shift), 0);
  const int s1 = min(sp.len - (col << shift), page);
  if (s1 <= s0) return;
  const int id = kv8_page(p.s, p.c, b, col);
  if (id < 0) return;

  const __bf16 *x = p.x[isv] + (int64_t)h * p.head_stride[isv] +
                    (int64_t)(sp.r0 + (col << shift) - pos0) * p.row_stride[isv];  // slot 0's row
  const int64_t xs = p.row_stride[isv];
  const size_t ph = (size_t)id * p.c.heads + h;
  uint8_t *codes = (isv ? p.c.v : p.c.k) + (ph << shift) * D;
  uint8_t *scale = (isv ? p.c.vs : p.c.ks) + ph;

  float amax = 0.f;
  for (int i = tid; i < (s1 - s0) * (D / 8); i += nt) {
    float f[8];
    load8(x + (s0 + i / (D / 8)) * xs + i % (D / 8) * 8, f);
#pragma unroll
    for (int j = 0; j < 8; ++j) amax = kv8_max_finite(amax, f[j]);
  }
  amax = kv8_block_max(amax, part);
  const int was = s0 > 0 ? (int)*scale - 127 : kKv8MinExp;
  const int e = max(kv8_exponent(amax), was);
  // 2^(was - e): below 2^-126 every code goes to zero either way
  const float move = e > was ? kv8_two(max(was - e, -126)) : 1.0f;
  const float inv = kv8_two(-e);

  if (!isv) {
    if (e > was && s0 > 0)
      for (int i = tid; i < s0 * (D / 16); i += nt) {
        uint4 *q = (uint4 *)(codes + kv8_k_at(i % s0, i / s0 * 16, D));
        uint4 v = *q;
        v.x = kv8_rescale4(v.x, move);
        v.y = kv8_rescale4(v.y, move);
        v.z = kv8_rescale4(v.z, move);
        v.w = kv8_rescale4(v.w, move);
        *q = v;
      }
    for (int i = tid; i < (s1 - s0) * (D / 16); i += nt) {
      const int slot = s0 + i / (D / 16), d = i % (D / 16) * 16;
      float f[16];
      load8(x + slot * xs + d, f);
      load8(x + slot * xs + d + 8, f + 8);
#pragma unroll
      for (int j = 0; j < 16; ++j) f[j] *= inv;
      *(uint4 *)(codes + kv8_k_at(slot, d, D)) =
          uint4{kv8_encode4(f), kv8_encode4(f + 4), kv8_encode4(f + 8), kv8_encode4(f + 12)};
    }
    if (h == 0 && p.c.w)
      for (int i = s0 + tid; i < s1; i += nt) p.c.w[((size_t)id << shift) + i] = 0.f;
  } else {
    // pieces of 16 bytes: piece (group of 4 tokens q, a, b) at
    // 16 * (unit * D + 64 a + 16 g + b); groups from the first that is
    // written to the last
    const int q0 = e > was ? 0 : s0 >> 2, q1 = (s1 + 3) >> 2;
    auto piece = [&](int i) {  // i-th piece of the range -> its byte offset
      const int q = q0 + i / (D / 4), r = i % (D / 4);
      return kv8_v_at(4 * q, (r >> 4) * 64 + (r & 15), D);
    };
    const int np = (q1 - q0) * (D / 4);
    for (int i = tid; i < np; i += nt) {
      const int q = q0 + i / (D / 4);
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
    for (int i = tid; i < (s1 - s0) * (D / 8); i += nt) {
      const int slot = s0 + i / (D / 8), d = i % (D / 8) * 8;
      float f[8];
      load8(x + slot * xs + d, f);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] *= inv;
      const uint32_t c0 = kv8_encode4(f), c1 = kv8_encode4(f + 4);
      const int at = kv8_v_at(slot, d, D);  // channels d..d+7 are 16 bytes apart
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        image[at + 16 * j] = (uint8_t)(c0 >> (8 * j));
        image[at + 16 * (4 + j)] = (uint8_t)(c1 >> (8 * j));
      }
    }
    __syncthreads();
    for (int i = tid; i < np; i += nt) {
      const int at = piece(i);
      *(uint4 *)(codes + at) = *(const uint4 *)(image + at);
    }
  }
  if (tid == 0) *scale = (uint8_t)(e + 127);
}

// ---- eviction ---------------------------------------------------------------------

struct SelectParams {
  Kv8Pool c;
  Kv8Batch s;
  int keep, recent, sink;
  int *new_lens;  // [seqs]
  int *kept;      // [seqs][keep]
};

// A weight as an unsigned word with the same order (-0 as +0, NaN above all).
__device__ __forceinline__ uint32_t order_word(float w) {
  if (w != w) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(w == 0.f ? 0.f : w);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// One workgroup per sequence.  The tokens between the first `sink` and the
// last `recent` compete for the remaining places: the smallest word that
// stays is found digit by digit (8 bits, a histogram each), then the kept
// positions are written in order; of the tokens that share that word the
// first stay.  Each wave owns one run of positions, so the order needs one
// exchange of counts.
constexpr int kSelThreads = 1024, kSelWaves = kSelThreads / 64;

__global__ __launch_bounds__(kSelThreads) void k_kv8_select(SelectParams p) {
  __shared__ unsigned hist[256];
  __shared__ unsigned pick[2];  // digit, places left below it
  __shared__ int above[kSelWaves], equal[kSelWaves];
  const int b = (int)blockIdx.x, tid = (int)threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int shift = p.c.shift;
  const int len = kv8_span(p.s, shift, b).len;
  int *kept = p.kept + (size_t)b * p.keep;
  const int stay = min(len, p.keep);
  if (tid == 0) p.new_lens[b] = stay;
  if (len <= p.keep) {
    for (int i = tid; i < p.keep; i += kSelThreads) kept[i] = i < len ? i : -1;
    return;
  }
  const int lo = p.sink, hi = len - p.recent, need = p.keep - p.sink - p.recent;
  auto word = [&](int j) {
    const int id = kv8_page(p.s, p.c, b, j >> shift);
    return id < 0 ? 0u : order_word(p.c.w[((size_t)id << shift) + (j & ((1 << shift) - 1))]);
  };
  uint32_t prefix = 0, mask = 0;
  int left = need;  // places among the words that match the prefix
  for (int sh = 24; sh >= 0 && need > 0; sh -= 8) {
    if (tid < 256) hist[tid] = 0;
    __syncthreads();
    for (int j = lo + tid; j < hi; j += kSelThreads) {
      const uint32_t u = word(j);
      if ((u & mask) == prefix) atomicAdd(&hist[(u >> sh) & 255], 1u);
    }
    __syncthreads();
    if (tid == 0) {
      int d = 255;
      unsigned sum = 0;
      while (d > 0 && sum + hist[d] < (unsigned)left) sum += hist[d--];
      pick[0] = (unsigned)d;
      pick[1] = (unsigned)left - sum;
    }
    __syncthreads();
    prefix |= pick[0] << sh;
    mask |= 255u << sh;
    left = (int)pick[1];
    __syncthreads();
  }
  // stays: protected, word > prefix, or one of the first `left` equal ones
  const int run = (((len + kSelWaves - 1) / kSelWaves) + 63) & ~63;
  const int j0 = wave * run, j1 = min(j0 + run, len);
  auto kind = [&](int j) {  // 0 goes, 1 stays, 2 stays if among the first equal ones
    if (j >= j1) return 0;
    if (j < lo || j >= hi) return 1;
    if (need == 0) return 0;
    const uint32_t u = word(j);
    return u > prefix ? 1 : u == prefix ? 2 : 0;
  };
  int na = 0, ne = 0;
  for (int j = j0; j < j1; j += 64) {
    const int k = kind(j + lane);
    na += __popcll(__ballot(k == 1));
    ne += __popcll(__ballot(k == 2));
  }
  if (lane == 0) {
    above[wave] = na;
    equal[wave] = ne;
  }
  __syncthreads();
  int at = 0, seen = 0;
  for (int i = 0; i < wave; ++i) {
    at += above[i] + min(max(left - seen, 0), equal[i]);
    seen += equal[i];
  }
  const uint64_t before = (1ull << lane) - 1ull;
  for (int j = j0; j < j1; j += 64) {
    const int k = kind(j + lane);
    const uint64_t eq = __ballot(k == 2);
    const bool in = k == 1 || (k == 2 && seen + __popcll(eq & before) < left);
    const uint64_t yes = __ballot(in);
    if (in) kept[at + __popcll(yes & before)] = j + lane;
    at += __popcll(yes);
    seen += __popcll(eq);
  }
}

struct MoveParams {
  Kv8Pool c;
  Kv8Batch s;
  const int *new_table;  // [seqs][new_cols]
  int new_cols, keep;
  const int *kept;
};

// One workgroup: one fresh page of one sequence, one KV head, K or V.  The
// kept tokens' codes are gathered into LDS in the page's order, their
// largest magnitude gives the new scale, and the codes move to it.
template <int D>
__global__ __launch_bounds__(256) void k_kv8_move(MoveParams p) {
  extern __shared__ __align__(16) uint8_t image[];
  __shared__ float part[4];
  __shared__ int src[128];      // page id of each token, -1: none
  __shared__ int src_slot[128];
  __shared__ float src_scale[128];
  const int b = (int)blockIdx.z, h = (int)blockIdx.y >> 1, isv = (int)blockIdx.y & 1;
  const int tid = (int)threadIdx.x, nt = (int)blockDim.x;
  const int shift = p.c.shift, page = 1 << shift, col = (int)blockIdx.x;
  const int len = min(kv8_span(p.s, shift, b).len, p.keep);
  const int n = min(len - (col << shift), page);  // tokens of this page
  if (n <= 0) return;
  const int to = p.new_table[(size_t)b * p.new_cols + col];
  if ((unsigned)to >= (unsigned)p.c.pages) return;
  const uint8_t *codes = isv ? p.c.v : p.c.k;
  const uint8_t *scales = isv ? p.c.vs : p.c.ks;
  for (int i = tid; i < n; i += nt) {
    const int j = p.kept[(size_t)b * p.keep + (col << shift) + i];
    const int id = kv8_page(p.s, p.c, b, j >> shift);
    src[i] = id;
    src_slot[i] = j & (page - 1);
    src_scale[i] = id < 0 ? 1.0f : kv8_scale(scales[(size_t)id * p.c.heads + h]);
    if (h == 0 && !isv && p.c.w)
      p.c.w[((size_t)to << shift) + i] = id < 0 ? 0.f : p.c.w[((size_t)id << shift) + (j & (page - 1))];
  }
  __syncthreads();
  uint8_t *out = (uint8_t *)codes + (((size_t)to * p.c.heads + h) << shift) * D;
  auto from = [&](int i) { return codes + (((size_t)src[i] * p.c.heads + h) << shift) * D; };
  float amax = 0.f;
  if (!isv) {
    for (int i = tid; i < n * (D / 16); i += nt) {
      const int t = i % n, d = i / n * 16;
      uint4 v = uint4{0, 0, 0, 0};
      if (src[t] >= 0) v = *(const uint4 *)(from(t) + kv8_k_at(src_slot[t], d, D));
      *(uint4 *)(image + kv8_k_at(t, d, D)) = v;
      const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float f[4];
        kv8_decode4(u[q], f);
#pragma unroll
        for (int k = 0; k < 4; ++k) amax = fmaxf(amax, fabsf(f[k]) * src_scale[t]);
      }
    }
  } else {
    // a dword holds one channel's four tokens: one source byte each
    const int nw = ((n + 3) >> 2) * D;
    for (int i = tid; i < nw; i += nt) {
      const int q = i / D, r = i % D;
      const int d = (r >> 6) * 64 + (r & 3) * 16 + ((r >> 2) & 15);  // neighbours: the dwords of a piece
      const int at = kv8_v_at(4 * q, d, D);
      uint32_t w = 0;
      if (4 * q + 3 >= n) w = *(const uint32_t *)(out + at);  // places that stay unused keep their bytes
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int t = 4 * q + k;
        if (t >= n) break;
        uint32_t c = 0;
        if (src[t] >= 0) c = from(t)[kv8_v_at(src_slot[t], d, D)];
        w = (w & ~(0xFFu << (8 * k))) | (c << (8 * k));
        float f[4];
        kv8_decode4(c, f);
        amax = fmaxf(amax, fabsf(f[0]) * src_scale[t]);
      }
      *(uint32_t *)(image + at) = w;
    }
  }
  amax = kv8_block_max(amax, part);
  __syncthreads();
  const int e = kv8_exponent(amax);
  const float inv = kv8_two(-e);
  // a code that is not zero is below 448 * 2^e and at least 2^-9 scales: its
  // factor is under 2^18 (the bound keeps a zero under a huge scale a zero)
  auto factor = [&](int t) { return fminf(src_scale[t] * inv, 0x1p18f); };
  if (!isv) {
    for (int i = tid; i < n * (D / 16); i += nt) {
      const int t = i % n, at = kv8_k_at(t, i / n * 16, D);
      const float f = factor(t);
      uint4 v = *(const uint4 *)(image + at);
      v.x = kv8_rescale4(v.x, f);
      v.y = kv8_rescale4(v.y, f);
      v.z = kv8_rescale4(v.z, f);
      v.w = kv8_rescale4(v.w, f);
      *(uint4 *)(out + at) = v;
    }
  } else {
    const int nw = ((n + 3) >> 2) * (D / 4);
    for (int i = tid; i < nw; i += nt) {
      const int q = i / (D / 4), r = i % (D / 4);
      const int at = kv8_v_at(4 * q, (r >> 4) * 64 + (r & 15), D);
      uint4 v = *(const uint4 *)(image + at);
      uint32_t u[4] = {v.x, v.y, v.z, v.w};
      float f[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) f[k] = 4 * q + k < n ? factor(4 * q + k) : 1.0f;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        float y[4];
        kv8_decode4(u[c], y);
#pragma unroll
        for (int k = 0; k < 4; ++k) y[k] *= f[k];
        u[c] = kv8_encode4(y);
      }
      *(uint4 *)(out + at) = uint4{u[0], u[1], u[2], u[3]};
    }
  }
  if (tid == 0) ((uint8_t *)scales)[(size_t)to * p.c.heads + h] = (uint8_t)(e + 127);
}

template <typename P>
hipError_t by_dim(int dim, void (*k64)(P), void (*k128)(P), void (*k256)(P), const P &p, dim3 grid,
                  int threads, size_t lds, hipStream_t stream) {
  auto k = dim == 64 ? k64 : dim == 128 ? k128 : k256;
  k<<<grid, dim3((unsigned)threads), lds, stream>>>(p);
  return hipGetLastError();
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
  // a few tokens are one wave's work
  const int threads = s.max_rows * dim <= 1024 ? 64 : 256;
  return by_dim(dim, k_kv8_append<64>, k_kv8_append<128>, k_kv8_append<256>, p, grid, threads,
                (size_t)page * dim, stream);
}

hipError_t launch_kv8_evict(const Kv8Pool &c, const Kv8Batch &s, int dim, const int *new_table,
                            int new_cols, int keep, int recent, int sink, int *new_lens, int *kept,
                            hipStream_t stream) {
  k_kv8_select<<<dim3((unsigned)s.seqs), dim3(kSelThreads), 0, stream>>>(
      SelectParams{c, s, keep, recent, sink, new_lens, kept});
  if (hipError_t e = hipGetLastError()) return e;
  const MoveParams p{c, s, new_table, new_cols, keep, kept};
  const int page = 1 << c.shift;
  const dim3 grid((unsigned)((keep + page - 1) >> c.shift), (unsigned)(2 * c.heads), (unsigned)s.seqs);
  return by_dim(dim, k_kv8_move<64>, k_kv8_move<128>, k_kv8_move<256>, p, grid, 256,
                (size_t)page * dim, stream);
}

}  // namespace nvfp4
