// kv8_common.h -- device helpers of the 8-bit paged KV cache kernels.
//
// A cache is a pool of pages of 2^shift tokens (16..128).  Per page and KV
// head it holds the E4M3 codes of K and of V and one E8M0 scale byte for
// each: value = e4m3(code) * 2^(byte - 127).  A page's codes of one head are
// units of 16 tokens, 16 * D bytes each, in the operand order of the 16-row
// matrix instructions, so that a wave reads an operand as contiguous 16-byte
// lanes with no shuffle and no LDS:
//   K unit: [D/16][16 tokens][16 d]         lane (g, r) of a QK operand reads
//     token r, channels 64 t + 16 g .. + 15, at 1024 t + 16 (16 g + r);
//   V unit: [D/64][4 g][16 b][4 c][4 i]     token 4 g + i, channel
//     64 a + 16 c + b: lane (g, b) of a PV operand reads the four tokens of
//     four channel tiles at 1024 a + 16 (16 g + b).
#pragma once

#include "encode_hw.h"
#include "launchers.h"
#include "nvfp4_common.h"

namespace nvfp4 {

constexpr int kKv8MinExp = -117, kKv8MaxExp = 119;  // exponents of a scale

// One sequence's rows and length, held inside the arrays whatever the
// device buffers say.
struct Kv8Span {
  int r0, rows, len;
};
__device__ __forceinline__ Kv8Span kv8_span(const Kv8Batch &s, int shift, int b) {
  Kv8Span o;
  if (s.starts) {
    o.r0 = min(max(s.starts[b], 0), s.rows);
    o.rows = min(max(s.starts[b + 1], o.r0), s.rows) - o.r0;
  } else {
    o.rows = s.rows / s.seqs;
    o.r0 = b * o.rows;
  }
  o.len = min(max(s.lens[b], 0), s.cols << shift);
  return o;
}

// page of block `col` of sequence b; -1 where the table names none
__device__ __forceinline__ int kv8_page(const Kv8Batch &s, const Kv8Pool &c, int b, int col) {
  const int id = s.table[(size_t)b * s.cols + col];
  return (unsigned)id < (unsigned)c.pages ? id : -1;
}

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
// 16 bytes that this call reads once: kept from displacing reused lines in the caches
__device__ __forceinline__ uint4 load_once(const uint4 *p) {
  return __builtin_bit_cast(uint4, __builtin_nontemporal_load((const u32x4 *)p));
}

__device__ __forceinline__ float kv8_two(int e) {  // 2^e, e >= -126
  return __uint_as_float((uint32_t)(e + 127) << 23);
}
// The scale of a byte.  One above 246 (2^119, the largest that append and
// eviction write) acts as 246: 448 * 2^120 is no bf16 number, and an infinite
// operand times the probability 0 of a row that does not see it would be NaN.
__device__ __forceinline__ float kv8_scale(uint32_t byte) {
  return __uint_as_float(min(max(byte, 1u), (uint32_t)(kKv8MaxExp + 127)) << 23);
}

// Smallest E in the scales' range with amax <= 448 * 2^E (448 = 1.75 * 2^8).
__device__ __forceinline__ int kv8_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return min(max(e, kKv8MinExp), kKv8MaxExp);
}

// byte offset of (slot, channel) in a page's codes of one head
__device__ __forceinline__ int kv8_k_at(int slot, int d, int dim) {
  return (slot >> 4) * 16 * dim + (d >> 4) * 256 + (slot & 15) * 16 + (d & 15);
}
__device__ __forceinline__ int kv8_v_at(int slot, int d, int dim) {
  return (slot >> 4) * 16 * dim + (d >> 6) * 1024 + ((slot & 15) >> 2) * 256 + (d & 15) * 16 +
         ((d & 63) >> 4) * 4 + (slot & 3);
}

// Four fp32 -> E4M3 bytes, nearest-even, saturating at 448; NaN gives 0x7F
// (the clamp inside e4m3x4_hw does not keep it).
__device__ __forceinline__ uint32_t kv8_encode4(const float *q) {
  uint32_t w = e4m3x4_hw(q);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (q[i] != q[i]) w |= 0x7Fu << (8 * i);
  return w;
}

// Four E4M3 bytes -> fp32, exact.
__device__ __forceinline__ void kv8_decode4(uint32_t w, float *x) {
  const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
  const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
  x[0] = lo[0];
  x[1] = lo[1];
  x[2] = hi[0];
  x[3] = hi[1];
}

// The codes of the same values under a scale `f` = 2^(old - new) times as
// fine: whole exponents move, so only results below 2^-6 (subnormal codes)
// are rounded.
__device__ __forceinline__ uint32_t kv8_rescale4(uint32_t w, float f) {
  float x[4];
  kv8_decode4(w, x);
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] *= f;
  return kv8_encode4(x);
}

__device__ __forceinline__ float kv8_max_finite(float m, float x) {
  const float a = fabsf(x);
  return a < __builtin_inff() ? fmaxf(m, a) : m;
}

// maximum over a workgroup of whole waves; `part` is LDS of one word per wave
// (magnitudes as fp32 bits have their order)
__device__ __forceinline__ uint32_t kv8_block_max_u(uint32_t m, unsigned *part) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o));
  const int waves = (int)blockDim.x >> 6;
  if (waves > 1) {
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
    __syncthreads();
    m = part[0];
    for (int i = 1; i < waves; ++i) m = max(m, part[i]);
  }
  return m;
}

}  // namespace nvfp4
