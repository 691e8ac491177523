// k_int8_gemm.hip -- the projection in 8-bit integers (gfx950):
//
//   y[r][c] = bf16( s_row[r] * s_col[c] * sum_k x[r][k] * w[c][k] )
//
// The sum is of whole numbers, |x| <= 127 and |w| <= 128, below 2^31 for the
// k that are allowed: every order of summation gives the same bits, so a
// row's result does not depend on the rows beside it or on how K is split.
//
// A wave owns 16 rows x 16 columns and takes K 64 at a time, its operands
// straight from memory: lane (c, g) = (lane % 16, lane / 16) holds the 16
// codes of row c at K 16 g of the step.
#include "int8_common.h"

namespace nvfp4 {

namespace {

struct Int8Args {
  const int8_t *x;
  const float *xs;
  int m, k, n;
  const int8_t *w0, *w1;
  const float *s0, *s1;
  void *y;
};

template <int NMAT>
__global__ __launch_bounds__(256) void k_int8_gemm(Int8Args p) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = lane & 15, g = lane >> 4;
  const int row0 = (int)blockIdx.x * 16, col0 = ((int)blockIdx.y * 4 + wave) * 16;
  if (col0 >= p.n) return;
  const size_t k = (size_t)p.k;
  const __amdgpu_buffer_rsrc_t xr = rsrc(p.x + row0 * k, min(16, p.m - row0) * k);
  const size_t cols = min(16, p.n - col0) * k;
  const __amdgpu_buffer_rsrc_t wr[2] = {rsrc(p.w0 + col0 * k, cols), rsrc((NMAT > 1 ? p.w1 : p.w0) + col0 * k, cols)};
  i32x4 acc[NMAT] = {};
  for (int k0 = 16 * g; k0 < p.k + 16 * g; k0 += 64) {
    const uint32_t off = k0 < p.k ? (uint32_t)(c * p.k + k0) : kOOB;
    const i32x4 a = __builtin_bit_cast(i32x4, ld16(xr, off));
#pragma unroll
    for (int i = 0; i < NMAT; ++i)
      acc[i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a, __builtin_bit_cast(i32x4, ld16(wr[i], off)), acc[i], 0, 0, 0);
  }
  if (col0 + c >= p.n) return;
  const Int8Scale s0 = int8_scale(p.s0[col0 + c]), s1 = int8_scale((NMAT > 1 ? p.s1 : p.s0)[col0 + c]);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int r = row0 + 4 * g + e;
    if (r >= p.m) break;
    const Int8Scale row = int8_scale(p.xs[r]);
    const float v = int8_scaled(acc[0][e], row, s0);
    ((__bf16 *)p.y)[(size_t)r * p.n + col0 + c] =
        NMAT > 1 ? swiglu_bf16(v, int8_scaled(acc[NMAT - 1][e], row, s1)) : (__bf16)v;
  }
}

}  // namespace

hipError_t launch_int8_gemm(const Int8ActRef &a, int m, int k, int n, int nmat, const Int8MatRef *w, void *y,
                            hipStream_t s) {
  const Int8Args p{a.codes, a.row_scale, m, k, n, w[0].codes, nmat > 1 ? w[1].codes : nullptr, w[0].scales,
                   nmat > 1 ? w[1].scales : nullptr, y};
  const dim3 grid(cdiv(m, 16), cdiv(n, 64));
  if (nmat == 1)
    hipLaunchKernelGGL(k_int8_gemm<1>, grid, dim3(256), 0, s, p);
  else
    hipLaunchKernelGGL(k_int8_gemm<2>, grid, dim3(256), 0, s, p);
  return hipGetLastError();
}

}  // namespace nvfp4
