// int8_common.h -- device helpers of the 8-bit integer kernels: the row
// quantizer's steps and the scaling of a product's sum.
//
// A row in int8: s = amax / 127 rounded to fp32 (1 for a row of zeros; NaN,
// with codes of 0, for one that holds an infinity or a NaN), code = x / s
// rounded to fp32 and then to the nearest whole number, ties to even.
#pragma once

#include "encode_hw.h"
#include "launchers.h"
#include "nvfp4_common.h"

namespace nvfp4 {

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

// Magnitudes of bf16 values compare as their bits do, infinities above the
// finite ones and NaN above those, so a row's largest is found on the bits,
// two at a time: `top` holds the largest so far in each half.
__device__ __forceinline__ uint32_t amax_bits(uint32_t top, uint32_t w) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, top),
                                                                __builtin_bit_cast(u16x2, w & 0x7FFF7FFFu)));
}
__device__ __forceinline__ uint32_t amax_bits(uint32_t top, const uint4 &v) {
  return amax_bits(amax_bits(amax_bits(amax_bits(top, v.x), v.y), v.z), v.w);
}
__device__ __forceinline__ uint32_t amax_fold(uint32_t top) { return max(top & 0xFFFFu, top >> 16); }

// How a row's values become codes.
struct Int8Row {
  float s, y;  // scale; its reciprocal, rounded
  bool fast;   // the quotients may be formed from y (encode_hw.h)
  bool fine;   // no infinity and no NaN in the row
};
__device__ __forceinline__ Int8Row int8_row(uint32_t bits) {
#pragma clang fp contract(off)
  Int8Row r;
  r.fine = bits < 0x7F80u;
  r.s = bits == 0 ? 1.0f : bf16_bits_to_f32(bits) / 127.0f;
  r.y = 1.0f / r.s;
  r.fast = recip_div_ok(r.s);
  if (!r.fine) r.s = __builtin_nanf("");
  return r;
}

// The code of x in the low byte.  |x / s| stays below 127.5 (s is off by at
// most 2^-10 of itself, where it is subnormal), so adding 1.5 * 2^23 rounds
// the quotient to a whole number, half to even, and leaves its two's
// complement in the low bits.
__device__ __forceinline__ uint32_t int8_code(float x, const Int8Row &r) {
#pragma clang fp contract(off)
  const float q = r.fast ? div_by_recip(x, r.s, r.y) : x / r.s;
  return __float_as_uint(q + 12582912.0f);
}
// Eight bf16 values -> eight codes.
__device__ __forceinline__ uint2 int8_codes(const uint4 &v, const Int8Row &r) {
  if (!r.fine) return uint2{0u, 0u};
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t p[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    p[i] = __builtin_amdgcn_perm(int8_code(bf16_bits_to_f32(w[i] >> 16), r),
                                 int8_code(bf16_bits_to_f32(w[i] & 0xFFFFu), r), 0x0C0C0400u);
  return uint2{__builtin_amdgcn_perm(p[1], p[0], 0x05040100u), __builtin_amdgcn_perm(p[3], p[2], 0x05040100u)};
}

// s_row * s_col * sum, rounded to fp32 a few times and never out of range in
// between: the scales' fractions are multiplied and the sum of their
// exponents comes last.  (Two tiny or two large scales whose product alone
// leaves fp32's range still give a result inside it.)
struct Int8Scale {
  float f;
  int e;
};
__device__ __forceinline__ Int8Scale int8_scale(float s) {
  return Int8Scale{__builtin_amdgcn_frexp_mantf(s), __builtin_amdgcn_frexp_expf(s)};
}
__device__ __forceinline__ float int8_scaled(int sum, const Int8Scale &row, const Int8Scale &col) {
  return __builtin_ldexpf((float)sum * row.f * col.f, row.e + col.e);
}

// Results of neighbouring columns, stored together wherever a row begins: rows
// of an odd number of columns begin at two bytes, which wide stores take (6839
// rows of 2047 x 992 60 -> 37 us over stores of two bytes; 2048 columns 28).
typedef uint32_t u32x4_at2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2_at2 __attribute__((ext_vector_type(2), aligned(2)));

// ---- rings in LDS --------------------------------------------------------------
// 16 bytes a lane from memory to LDS at `lds` + 16 lane; lanes out of the
// range write zeros.  The compiler does not see the transfer, so it places no
// waits for it: the kernel's own waits count it, and every transfer has to be
// complete before its workgroup ends.
__device__ __forceinline__ void to_lds(u32x4_t r, uint32_t lds, uint32_t voff, uint32_t soff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               :
               : "s"(lds), "v"(voff), "s"(r), "s"(soff)
               : "memory");
}
// Likewise 4 bytes a lane.
__device__ __forceinline__ void words_to_lds(u32x4_t r, uint32_t lds, uint32_t voff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds"
               :
               : "s"(lds), "v"(voff), "s"(r)
               : "memory");
}
__device__ __forceinline__ u32x4_t range_of(const void *base, size_t bytes) {
  const uint64_t a = (uint64_t)base;
  return u32x4_t{(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)a),
                 (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(a >> 32)),
                 (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)bytes), 0x00020000u};
}
__device__ __forceinline__ uint32_t lds_address(const void *p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void *)p;
}
// This wave's transfers but the youngest N are complete, and its LDS reads.
template <int N>
__device__ __forceinline__ void wait_transfers() {
  static_assert(N < 64, "the counter has six bits");
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_s_waitcnt(0x0070 | (N & 15) | ((N >> 4) << 14));
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
}
__device__ __forceinline__ void ring_barrier() {
  __builtin_amdgcn_s_barrier();
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

// Pieces of sums handed from workgroup to workgroup, past the caches
// (kCoherent in nvfp4_common.h).
__device__ __forceinline__ void st16_coherent(__amdgpu_buffer_rsrc_t r, uint32_t off, i32x4 v) {
  __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, v), r, off, 0, kCoherent);
}
__device__ __forceinline__ i32x4 ld16_coherent(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, kCoherent));
}

}  // namespace nvfp4
