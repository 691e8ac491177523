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
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

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

}  // namespace nvfp4
