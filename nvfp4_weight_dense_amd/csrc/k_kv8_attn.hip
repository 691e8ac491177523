// k_kv8_attn.hip -- attention over the 8-bit paged KV cache.
//
// Row i of a sequence of n tokens with r rows sits at position n - r + i and
// sees the tokens j up to its own position, with a window the last `window`
// of them.  s_ij = scale * q_i . k_j, o_i = sum_j e^(s_ij - m) v_j / sum_j
// e^(s_ij - m), lse_i = m + log sum_j e^(s_ij - m); a row that sees nothing
// gives zeros and -inf.  Sums and the softmax's statistics are fp32, powers
// are of two (log2 e is folded into the scale).
#include "kv8_common.h"
#include "launchers.h"

namespace nvfp4 {

namespace {

constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.693147180559945309f;

struct AttnParams {
  Kv8Attn a;
  Kv8Pool c;
  Kv8Batch s;
};

// scale * log2(e) * q . k of one token, from fp32 q in LDS
template <int D>
__device__ __forceinline__ float dot_token(const float *q, const uint8_t *codes, int slot) {
  float acc = 0.f;
  for (int d = 0; d < D; d += 16) {
    const uint4 v = *(const uint4 *)(codes + kv8_k_at(slot, d, D));
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      float f[4];
      kv8_decode4(u[w], f);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc = fmaf(q[d + 4 * w + i], f[i], acc);
    }
  }
  return acc;
}

// One wave: one row and query head; 64 tokens at a time, a lane each for the
// products with K, a lane per channel for those with V.
template <int D>
__global__ __launch_bounds__(64) void k_kv8_attn_row(AttnParams p) {
  __shared__ float q[D], prob[64];
  const int i = (int)blockIdx.x, hq = (int)blockIdx.y, b = (int)blockIdx.z, lane = (int)threadIdx.x;
  const Kv8Span sp = kv8_span(p.s, p.c.shift, b);
  if (i >= sp.rows) return;
  const int h = hq / (p.a.q_heads / p.c.heads), page = 1 << p.c.shift;
  const __bf16 *qr = (const __bf16 *)p.a.q.ptr + (int64_t)(sp.r0 + i) * p.a.q.row_stride +
                     (int64_t)hq * p.a.q.head_stride;
  for (int d = lane; d < D; d += 64) q[d] = (float)qr[d];
  __syncthreads();
  const int pos = sp.len - sp.rows + i;
  const int j0 = p.a.window ? max(pos - p.a.window + 1, 0) : 0;
  float m = -__builtin_inff(), l = 0.f, o[D / 64] = {};
  const int last = min(pos, p.a.max_len - 1);
  for (int j = j0 & ~63; j <= last; j += 64) {
    const int mine = j + lane;
    float s = -__builtin_inff();
    if (mine >= j0 && mine <= last) {
      const int id = kv8_page(p.s, p.c, b, mine >> p.c.shift);
      if (id >= 0) {
        const size_t ph = (size_t)id * p.c.heads + h;
        s = dot_token<D>(q, p.c.k + (ph << p.c.shift) * D, mine & (page - 1)) *
            (p.a.scale * kLog2e * kv8_scale(p.c.ks[ph]));
      }
    }
    float top = s;
#pragma unroll
    for (int x = 32; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor(top, x));
    const float mn = fmaxf(m, top), base = mn == -__builtin_inff() ? 0.f : mn;
    const float keep = __builtin_amdgcn_exp2f(m - base), e = __builtin_amdgcn_exp2f(s - base);
    m = mn;
    l = l * keep + e;
    prob[lane] = e;
    __syncthreads();
#pragma unroll
    for (int a = 0; a < D / 64; ++a) o[a] *= keep;
    for (int t = 0; t < 64 && j + t <= last; ++t) {
      const int id = kv8_page(p.s, p.c, b, (j + t) >> p.c.shift);
      if (id < 0 || j + t < j0) continue;
      const size_t ph = (size_t)id * p.c.heads + h;
      const uint8_t *codes = p.c.v + (ph << p.c.shift) * D;
      const float w = prob[t] * kv8_scale(p.c.vs[ph]);
#pragma unroll
      for (int a = 0; a < D / 64; ++a)
        o[a] = fmaf(w, e4m3_to_f32(codes[kv8_v_at((j + t) & (page - 1), 64 * a + lane, D)]), o[a]);
    }
    __syncthreads();
  }
#pragma unroll
  for (int x = 32; x > 0; x >>= 1) l += __shfl_xor(l, x);
  const size_t at = (size_t)(sp.r0 + i) * p.a.q_heads + hq;
  const float inv = l > 0.f || l != l ? 1.0f / l : 0.f;
#pragma unroll
  for (int a = 0; a < D / 64; ++a) ((__bf16 *)p.a.out)[at * D + 64 * a + lane] = (__bf16)(o[a] * inv);
  if (lane == 0 && p.a.lse) p.a.lse[at] = l > 0.f || l != l ? (m + log2f(l)) * kLn2 : -__builtin_inff();
}

// One wave: 64 tokens of one sequence, a lane each; every row and query head
// in order, so a token's sum has one order.
template <int D>
__global__ __launch_bounds__(64) void k_kv8_weights_token(AttnParams p) {
  __shared__ float q[D];
  const int b = (int)blockIdx.y, lane = (int)threadIdx.x, j = (int)blockIdx.x * 64 + lane;
  const Kv8Span sp = kv8_span(p.s, p.c.shift, b);
  if ((int)blockIdx.x * 64 >= sp.len) return;
  const int page = 1 << p.c.shift, group = p.a.q_heads / p.c.heads;
  const int id = j < min(sp.len, p.a.max_len) ? kv8_page(p.s, p.c, b, j >> p.c.shift) : -1;
  float sum = 0.f;
  for (int i = 0; i < sp.rows; ++i) {
    const int pos = sp.len - sp.rows + i;
    if (pos < (int)blockIdx.x * 64) continue;
    for (int hq = 0; hq < p.a.q_heads; ++hq) {
      const __bf16 *qr = (const __bf16 *)p.a.q.ptr + (int64_t)(sp.r0 + i) * p.a.q.row_stride +
                         (int64_t)hq * p.a.q.head_stride;
      __syncthreads();
      for (int d = lane; d < D; d += 64) q[d] = (float)qr[d];
      __syncthreads();
      if (id < 0 || j > pos || (p.a.window && j <= pos - p.a.window)) continue;
      const size_t ph = (size_t)id * p.c.heads + hq / group;
      const float s = dot_token<D>(q, p.c.k + (ph << p.c.shift) * D, j & (page - 1)) *
                      (p.a.scale * kLog2e * kv8_scale(p.c.ks[ph]));
      sum += __builtin_amdgcn_exp2f(s - p.a.lse[(size_t)(sp.r0 + i) * p.a.q_heads + hq] * kLog2e);
    }
  }
  if (id >= 0) p.c.w[((size_t)id << p.c.shift) + (j & (page - 1))] += sum;
}

}  // namespace

hipError_t launch_kv8_attention(const Kv8Attn &a, const Kv8Pool &c, const Kv8Batch &s, int dim,
                                hipStream_t stream) {
  const AttnParams p{a, c, s};
  const dim3 grid((unsigned)s.max_rows, (unsigned)a.q_heads, (unsigned)s.seqs);
  auto k = dim == 64 ? k_kv8_attn_row<64> : dim == 128 ? k_kv8_attn_row<128> : k_kv8_attn_row<256>;
  k<<<grid, dim3(64), 0, stream>>>(p);
  return hipGetLastError();
}

hipError_t launch_kv8_weights(const Kv8Attn &a, const Kv8Pool &c, const Kv8Batch &s, int dim,
                              hipStream_t stream) {
  const AttnParams p{a, c, s};
  const dim3 grid((unsigned)((a.max_len + 63) / 64), (unsigned)s.seqs);
  auto k = dim == 64 ? k_kv8_weights_token<64> : dim == 128 ? k_kv8_weights_token<128> : k_kv8_weights_token<256>;
  k<<<grid, dim3(64), 0, stream>>>(p);
  return hipGetLastError();
}

}  // namespace nvfp4
