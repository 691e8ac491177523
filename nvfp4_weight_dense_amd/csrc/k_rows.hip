// k_rows.hip -- passes over bf16 rows around a block (gfx950): the norm
// before it, the norm, gate, scale and residual after it with the next
// block's norm, and the int8 row quantizer, which the norms can end in.
//
//   norm(x)  = x / sqrt(mean(x^2) + eps) * (offset + weight)
//   residual: h = bf16(residual + scale * gate * norm(y)), then norm(h)
//   int8:    s = amax / 127, code = x / s (int8_common.h)
//
// All are bound by memory: one workgroup takes a row, each thread keeps its
// pieces of eight values in registers from the one read of the row to the
// one write, and what the row needs as a whole (a sum of squares, a largest
// magnitude) is exchanged once each.  Statistics are fp32.  The norm's
// result is rounded to bf16 before it is quantized, and h before it is
// normed, so that the fused calls give the bits of the calls one by one.
#include <algorithm>

#include "int8_common.h"

namespace nvfp4 {

namespace {

constexpr int kMaxThreads = 1024;

__device__ __forceinline__ void unpack8(const uint4 &v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_bits_to_f32(w[i] & 0xFFFFu);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = __builtin_bit_cast(uint32_t, bf16x2{(__bf16)f[2 * i], (__bf16)f[2 * i + 1]});
  return uint4{w[0], w[1], w[2], w[3]};
}

// One value of every thread combined over the workgroup.  `slots`: 16 words
// of LDS that no other exchange of the kernel uses.
template <class T, class Op>
__device__ __forceinline__ T over_row(T v, T *slots, Op op) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v = op(v, __shfl_xor(v, off));
  const int waves = (int)blockDim.x >> 6;
  if (waves == 1) return v;
  if ((threadIdx.x & 63) == 0) slots[threadIdx.x >> 6] = v;
  __syncthreads();
  T r = slots[0];
  for (int w = 1; w < waves; ++w) r = op(r, slots[w]);
  return r;
}

// 1 / sqrt(mean of squares + eps) of the row in v.  A row whose squares leave
// fp32's range (values past 2^50) is summed again with its values times
// 2^-80.
template <int P>
__device__ __forceinline__ float row_rstd(const uint4 (&v)[P], int k, float eps, float (*slots)[16]) {
  auto squares = [&](float by, float *at) {
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      float f[8];
      unpack8(v[i], f);
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(f[j] * by, f[j] * by, ss);
    }
    return over_row(ss, at, [](float a, float b) { return a + b; });
  };
  const float ss = squares(1.0f, slots[0]);
  if (ss < 0x1p100f) return __builtin_amdgcn_rsqf(ss / (float)k + eps);
  return __builtin_amdgcn_rsqf(squares(0x1p-80f, slots[1]) / (float)k) * 0x1p-80f;  // (eps is far below)
}

// v = bf16(v * rstd * (offset + weight)), or without a weight bf16(v * rstd)
template <int P>
__device__ __forceinline__ void scale_row(uint4 (&v)[P], const uint4 *weight, float offset, float rstd, int pieces) {
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int p = (int)threadIdx.x + i * (int)blockDim.x;
    if (p >= pieces) break;
    float f[8];
    unpack8(v[i], f);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] *= rstd;
    if (weight) {
      float w[8];
      unpack8(weight[p], w);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] *= offset + w[j];
    }
    v[i] = pack8(f);
  }
}

// The row in v, to out or as codes and a scale.
template <int P>
__device__ __forceinline__ void write_row(const uint4 (&v)[P], const RowsOut &o, int row, int pieces, uint32_t *slots) {
  if (o.out) {
    uint4 *to = (uint4 *)o.out + (size_t)row * pieces;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int p = (int)threadIdx.x + i * (int)blockDim.x;
      if (p < pieces) to[p] = v[i];
    }
    return;
  }
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < P; ++i) top = amax_bits(top, v[i]);
  const Int8Row r =
      int8_row(over_row(amax_fold(top), slots, [](uint32_t a, uint32_t b) { return max(a, b); }));
  if (threadIdx.x == 0) o.row_scale[row] = r.s;
  uint2 *to = (uint2 *)o.codes + (size_t)row * pieces;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int p = (int)threadIdx.x + i * (int)blockDim.x;
    if (p < pieces) to[p] = int8_codes(v[i], r);
  }
}

template <int P>
__device__ __forceinline__ void read_row(const void *x, int row, int pieces, uint4 (&v)[P]) {
  const uint4 *at = (const uint4 *)x + (size_t)row * pieces;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int p = (int)threadIdx.x + i * (int)blockDim.x;
    v[i] = p < pieces ? at[p] : uint4{0u, 0u, 0u, 0u};
  }
}

template <int P>
__global__ __launch_bounds__(kMaxThreads) void k_int8_rows(const void *x, int k, RowsOut o) {
  __shared__ uint32_t top[16];
  uint4 v[P];
  read_row(x, (int)blockIdx.x, k >> 3, v);
  write_row(v, o, (int)blockIdx.x, k >> 3, top);
}

template <int P>
__global__ __launch_bounds__(kMaxThreads) void k_rms_norm(const void *x, int k, NormRef n, float eps, RowsOut o) {
  __shared__ float sums[2][16];
  __shared__ uint32_t top[16];
  const int row = (int)blockIdx.x, pieces = k >> 3;
  uint4 v[P];
  read_row(x, row, pieces, v);
  const float rstd = row_rstd(v, k, eps, sums);
  scale_row(v, (const uint4 *)n.weight, n.offset, rstd, pieces);
  write_row(v, o, row, pieces, top);
}

template <int P>
__global__ __launch_bounds__(kMaxThreads) void k_rms_norm_residual(ResidualArgs a, int k, float eps, RowsOut o) {
  __shared__ float sums[4][16];
  __shared__ uint32_t top[16];
  const int row = (int)blockIdx.x, pieces = k >> 3;
  uint4 v[P], r[P];
  read_row(a.y, row, pieces, v);
  read_row(a.residual, row, pieces, r);
  const float rstd = a.post.on ? row_rstd(v, k, eps, sums) : 1.0f;
  const uint4 *post = a.post.on ? (const uint4 *)a.post.weight : nullptr;
  const uint4 *gate = a.gate ? (const uint4 *)a.gate + (size_t)(row / a.rows_per_gate) * pieces : nullptr;
  uint4 *h = (uint4 *)a.h + (size_t)row * pieces;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int p = (int)threadIdx.x + i * (int)blockDim.x;
    if (p >= pieces) break;
    float f[8], g[8];
    unpack8(v[i], f);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] *= rstd;
    if (post) {
      unpack8(post[p], g);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] *= a.post.offset + g[j];
    }
    if (gate) {
      unpack8(gate[p], g);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] *= g[j];
    }
    unpack8(r[i], g);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = fmaf(a.scale, f[j], g[j]);
    v[i] = pack8(f);
    h[p] = v[i];
  }
  if (!a.next.on) return;
  const float next = row_rstd(v, k, eps, sums + 2);
  scale_row(v, (const uint4 *)a.next.weight, a.next.offset, next, pieces);
  write_row(v, o, row, pieces, top);
}

// Threads that hold a row of k values in P pieces each.
struct RowShape {
  int p, threads;
};
RowShape row_shape(int k) {
  const int pieces = k >> 3;
  int p = 1;
  while (cdiv(pieces, p) > kMaxThreads) p *= 2;
  return RowShape{p, cdiv(cdiv(pieces, p), 64) * 64};
}

template <class F>
hipError_t with_pieces(int p, F &&f) {
  switch (p) {
    case 1: f(std::integral_constant<int, 1>()); break;
    case 2: f(std::integral_constant<int, 2>()); break;
    case 4: f(std::integral_constant<int, 4>()); break;
    case 8: f(std::integral_constant<int, 8>()); break;
    case 16: f(std::integral_constant<int, 16>()); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_int8_rows(const void *x, int m, int k, int8_t *codes, float *row_scale, hipStream_t s) {
  const RowShape r = row_shape(k);
  return with_pieces(r.p, [&](auto p) {
    hipLaunchKernelGGL((k_int8_rows<decltype(p)::value>), dim3(m), dim3(r.threads), 0, s, x, k,
                       (RowsOut{nullptr, codes, row_scale}));
  });
}

hipError_t launch_rms_norm(const void *x, int m, int k, const NormRef &n, float eps, const RowsOut &o, hipStream_t s) {
  const RowShape r = row_shape(k);
  return with_pieces(r.p, [&](auto p) {
    hipLaunchKernelGGL((k_rms_norm<decltype(p)::value>), dim3(m), dim3(r.threads), 0, s, x, k, n, eps, o);
  });
}

hipError_t launch_rms_norm_residual(const ResidualArgs &a, int m, int k, float eps, const RowsOut &o, hipStream_t s) {
  const RowShape r = row_shape(k);
  return with_pieces(r.p, [&](auto p) {
    hipLaunchKernelGGL((k_rms_norm_residual<decltype(p)::value>), dim3(m), dim3(r.threads), 0, s, a, k, eps, o);
  });
}

}  // namespace nvfp4
