// k_rows.hip -- passes over bf16 rows around a block (gfx950): the norm
// before it, the norm, gate, scale and residual after it with the next
// block's norm, and the int8 row quantizer, which the norms can end in.
//
//   norm(x)  = x / sqrt(mean(x^2) + eps) * (offset + weight)
//   residual: h = bf16(residual + scale * gate * norm(y)), then norm(h)
//   int8:    s = amax / 127, code = x / s (int8_common.h)
//
// All are bound by memory: norm of 8192 rows of 5120 28.7 us (5.8 TB/s), to
// int8 35 (3.6: its divisions count), end of a block with post norm, int8 and
// no gate 56 to 65 us (4.5 to 5.3), quantizer of 17408 rows of 5120 45 us
// (5.9); a large copy makes 4.8.  With few rows what counts
// is the way of one row through memory and the exchanges: 64 rows of 5120
// 4.6, 6.3 and 4 us.  A workgroup takes a row -- for the quantizer, where
// there are many rows that are not too long, a wave --, each thread keeps its
// pieces of eight values in registers from the one read of the row to the one
// write, and what the row needs as a whole (a sum of squares, a largest
// magnitude) is exchanged once each.  Of rows past 65536, sixteen pieces a
// thread, the norms hold some fifty registers in scratch memory (norm of 512
// rows of 131072 89 us, 3.0 TB/s; of 65536 32 us, 4.1).  Rows of 512 and less
// fill a wave or less of a workgroup (norm of 131072 rows of 256 36 us, 3.8
// TB/s; of 65536 of 512 22 us, 6.1).  Statistics are fp32.  The norm's
// result is rounded to bf16 before it is quantized, and h before it is
// normed, so that the fused calls give the bits of the calls one by one.
#include <algorithm>
#include <type_traits>

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

// The pieces stay packed: without this the compiler keeps the values that a
// pass over them unpacked for the next one, twice the registers.
template <int P>
__device__ __forceinline__ void stay_packed(uint4 (&v)[P]) {
#pragma unroll
  for (int i = 0; i < P; ++i) asm volatile("" : "+v"(v[i].x), "+v"(v[i].y), "+v"(v[i].z), "+v"(v[i].w));
}

// A row's threads: a wave's (WAVE), or the workgroup's.
template <bool WAVE>
__device__ __forceinline__ int row_thread() {
  return WAVE ? (int)threadIdx.x & 63 : (int)threadIdx.x;
}
template <bool WAVE>
__device__ __forceinline__ int row_threads() {
  return WAVE ? 64 : (int)blockDim.x;
}

template <bool WAVE, int P>
__device__ __forceinline__ void read_row(const void *x, int row, int pieces, uint4 (&v)[P]) {
  const uint4 *at = (const uint4 *)x + (size_t)row * pieces;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int p = row_thread<WAVE>() + i * row_threads<WAVE>();
    v[i] = p < pieces ? at[p] : uint4{0u, 0u, 0u, 0u};
  }
}

// One value of every thread combined over the row's.  `slots`: 16 words of
// LDS that no other exchange of the kernel uses.
template <bool WAVE, class T, class Op>
__device__ __forceinline__ T over_row(T v, T *slots, Op op) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v = op(v, __shfl_xor(v, off));
  const int waves = (int)blockDim.x >> 6;
  if (WAVE || waves == 1) return v;
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
__device__ __forceinline__ float row_rstd(uint4 (&v)[P], int k, float eps, float (*slots)[16]) {
  auto squares = [&](float by, float *at) {
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      float f[8];
      unpack8(v[i], f);
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(f[j] * by, f[j] * by, ss);
    }
    return over_row<false>(ss, at, [](float a, float b) { return a + b; });
  };
  const float ss = squares(1.0f, slots[0]);
  stay_packed(v);
  if (ss < 0x1p100f) return __builtin_amdgcn_rsqf(ss / (float)k + eps);
  return __builtin_amdgcn_rsqf(squares(0x1p-80f, slots[1]) / (float)k) * 0x1p-80f;  // (eps is far below)
}

// A row beside the one that is normed (weights, gate, residual).  It is
// requested with it, so that nothing waits for memory behind a sum (64 rows of
// 5120, end of a block with all of them: 8.1 -> 6.2 us; 4099 rows of 4096 with
// a gate to a row: 31.4 -> 27.9); rows too long for the registers are read
// where they are used.
template <int P>
struct Beside {
  static constexpr bool kHeld = P <= 4;
  const uint4 *at;  // null: there is none
  uint4 v[kHeld ? P : 1];
  __device__ __forceinline__ Beside(const void *base, int row, int pieces)
      : at(base ? (const uint4 *)base + (size_t)row * pieces : nullptr) {
    if constexpr (kHeld) {
      if (at) read_row<false>(base, row, pieces, v);
    }
  }
  __device__ __forceinline__ void get(int i, int p, int pieces, float (&f)[8]) const {
    if constexpr (kHeld) unpack8(v[i], f);
    else unpack8(p < pieces ? at[p] : uint4{0u, 0u, 0u, 0u}, f);
  }
};

// v = bf16(v * rstd * (offset + weight)), or without a weight bf16(v * rstd)
template <int P>
__device__ __forceinline__ void scale_row(uint4 (&v)[P], const Beside<P> &weight, float offset, float rstd, int pieces) {
#pragma unroll
  for (int i = 0; i < P; ++i) {
    float f[8], w[8];
    unpack8(v[i], f);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] *= rstd;
    if (weight.at) {
      weight.get(i, (int)threadIdx.x + i * (int)blockDim.x, pieces, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] *= offset + w[j];
    }
    v[i] = pack8(f);
  }
}

// The row in v, to out or as codes and a scale.
template <bool WAVE, int P>
__device__ __forceinline__ void write_row(const uint4 (&v)[P], const RowsOut &o, int row, int pieces, uint32_t *slots) {
  if (o.out) {
    uint4 *to = (uint4 *)o.out + (size_t)row * pieces;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int p = row_thread<WAVE>() + i * row_threads<WAVE>();
      if (p < pieces) to[p] = v[i];
    }
    return;
  }
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < P; ++i) top = amax_bits(top, v[i]);
  const Int8Row r =
      int8_row(over_row<WAVE>(amax_fold(top), slots, [](uint32_t a, uint32_t b) { return max(a, b); }));
  if (row_thread<WAVE>() == 0) o.row_scale[row] = r.s;
  uint2 *to = (uint2 *)o.codes + (size_t)row * pieces;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int p = row_thread<WAVE>() + i * row_threads<WAVE>();
    if (p < pieces) to[p] = int8_codes(v[i], r);
  }
}

// The row of this wave or workgroup; past the last: -1.
constexpr int kWaveRows = 4;  // rows of a workgroup whose waves take one each
template <bool WAVE>
__device__ __forceinline__ int own_row(int m) {
  if (!WAVE) return (int)blockIdx.x;
  const int row = (int)blockIdx.x * kWaveRows + __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  return row < m ? row : -1;
}
template <bool WAVE>
constexpr int most_threads() { return WAVE ? 64 * kWaveRows : kMaxThreads; }

// With gridDim.y > 1 (few rows) each slice of a row is a workgroup: it looks
// for the largest magnitude in all of the row and encodes every gridDim.y-th of
// its threads' pieces, so that the divisions of a row spread over several CUs.
template <bool WAVE, int P>
__global__ __launch_bounds__(most_threads<WAVE>()) void k_int8_rows(const void *x, int m, int k, RowsOut o) {
  __shared__ uint32_t top[16];
  const int row = own_row<WAVE>(m), pieces = k >> 3;
  if (row < 0) return;
  uint4 v[P];
  read_row<WAVE>(x, row, pieces, v);
  if (WAVE || gridDim.y == 1) {
    write_row<WAVE>(v, o, row, pieces, top);
    return;
  }
  uint32_t bits = 0;
#pragma unroll
  for (int i = 0; i < P; ++i) bits = amax_bits(bits, v[i]);
  const Int8Row r =
      int8_row(over_row<WAVE>(amax_fold(bits), top, [](uint32_t a, uint32_t b) { return max(a, b); }));
  if (threadIdx.x == 0 && blockIdx.y == 0) o.row_scale[row] = r.s;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int p = (int)threadIdx.x + i * (int)blockDim.x;
    if (i % (int)gridDim.y == (int)blockIdx.y && p < pieces)
      ((uint2 *)o.codes)[(size_t)row * pieces + p] = int8_codes(v[i], r);
  }
}

template <int P>
__global__ __launch_bounds__(kMaxThreads) void k_rms_norm(const void *x, int k, NormRef n, float eps, RowsOut o) {
  __shared__ float sums[2][16];
  __shared__ uint32_t top[16];
  const int row = (int)blockIdx.x, pieces = k >> 3;
  uint4 v[P];
  read_row<false>(x, row, pieces, v);
  const Beside<P> weight(n.weight, 0, pieces);
  const float rstd = row_rstd(v, k, eps, sums);
  scale_row(v, weight, n.offset, rstd, pieces);
  write_row<false>(v, o, row, pieces, top);
}

template <int P>
__global__ __launch_bounds__(kMaxThreads) void k_rms_norm_residual(ResidualArgs a, int k, float eps, RowsOut o) {
  __shared__ float sums[4][16];
  __shared__ uint32_t top[16];
  const int row = (int)blockIdx.x, pieces = k >> 3;
  uint4 v[P];
  read_row<false>(a.y, row, pieces, v);
  const Beside<P> residual(a.residual, row, pieces), gate(a.gate, row / a.rows_per_gate, pieces),
      post(a.post.on ? a.post.weight : nullptr, 0, pieces), next(a.next.on ? a.next.weight : nullptr, 0, pieces);
  const float rstd = a.post.on ? row_rstd(v, k, eps, sums) : 1.0f;
  uint4 *h = (uint4 *)a.h + (size_t)row * pieces;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int p = (int)threadIdx.x + i * (int)blockDim.x;
    float f[8], g[8];
    unpack8(v[i], f);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] *= rstd;
    if (post.at) {
      post.get(i, p, pieces, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] *= a.post.offset + g[j];
    }
    if (gate.at) {
      gate.get(i, p, pieces, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] *= g[j];
    }
    residual.get(i, p, pieces, g);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = fmaf(a.scale, f[j], g[j]);
    v[i] = p < pieces ? pack8(f) : uint4{0u, 0u, 0u, 0u};
    if (p < pieces) h[p] = v[i];
  }
  if (!a.next.on) return;
  const float again = row_rstd(v, k, eps, sums + 2);
  scale_row(v, next, a.next.offset, again, pieces);
  write_row<false>(v, o, row, pieces, top);
}

// Pieces of a thread, for a workgroup to a row: two (8192 rows of 5120, norm
// 28 and end of a block 64 us; with one 36 and 87, with four 32 and 68), and
// more where 1024 threads do not hold a row so.  Not by the number of rows: a
// row's sums then have one order and its results the same bits in any batch
// (with one piece 64 rows would take 4.4 and 5.9 us in place of 4.6 and 6.2).
int row_pieces(int k) {
  const int pieces = k >> 3;
  int p = pieces > 256 ? 2 : 1;
  while (cdiv(pieces, p) > kMaxThreads) p *= 2;
  return p;
}
int row_block(int k, int p) { return cdiv(cdiv(k >> 3, p), 64) * 64; }

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

// The quantizer's rows go to a wave each where there are many: short ones (of
// up to four pieces a lane, 2048 values) from 2048 rows on, where a workgroup
// has little to exchange (17408 rows of 2048: 17.9 us, with a workgroup to a
// row 21.2; 4096 rows 6.8 and 7.2; 2048 rows 4.9 and 4.8), longer ones up to
// 12 pieces from 16384 on (17408 rows of 2560 22.6 and 23.1, of 4096 35.0 and
// 33.8, of 4608 40.0 and 42.7, of 5120 44.4 and 46.4, of 6144 59.5 and 57.7;
// but 4096 rows of 4096 11.9 and 11.0, 17408 rows of 7168 73.2 and 65.8).
constexpr int kWaveMaxPieces = 12;
bool rows_to_waves(int m, int lane_pieces) {
  return lane_pieces <= kWaveMaxPieces && m >= (lane_pieces <= 4 ? 2048 : 16384);
}

// The smallest even number of pieces that holds `pieces` of a lane.
template <int P, class F>
hipError_t with_wave_pieces(int pieces, F &&f) {
  if (pieces <= P) {
    f(std::integral_constant<int, P>());
    return hipGetLastError();
  }
  if constexpr (P + 2 <= kWaveMaxPieces) return with_wave_pieces<P + 2>(pieces, f);
  else return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_int8_rows(const void *x, int m, int k, int8_t *codes, float *row_scale, hipStream_t s) {
  const RowsOut o{nullptr, codes, row_scale};
  const int pieces = k >> 3, lane_pieces = cdiv(pieces, 64);
  if (rows_to_waves(m, lane_pieces)) {
    return with_wave_pieces<2>(lane_pieces, [&](auto p) {
      hipLaunchKernelGGL((k_int8_rows<true, decltype(p)::value>), dim3(cdiv(m, kWaveRows)), dim3(64 * kWaveRows), 0, s, x,
                         m, k, o);
    });
  }
  // few rows: up to eight slices, for about as many workgroups as CUs (64 rows
  // of 17408: 8.4 us a call, 9.6 without), and a piece of a thread for each
  int slices = 1;
  while (slices < 8 && slices * 2 * m <= 256 && slices * 2 * 64 <= pieces) slices *= 2;
  return with_pieces(std::max(row_pieces(k), slices), [&](auto p) {
    hipLaunchKernelGGL((k_int8_rows<false, decltype(p)::value>), dim3(m, slices), dim3(row_block(k, p)), 0, s, x, m, k, o);
  });
}

hipError_t launch_rms_norm(const void *x, int m, int k, const NormRef &n, float eps, const RowsOut &o, hipStream_t s) {
  return with_pieces(row_pieces(k), [&](auto p) {
    hipLaunchKernelGGL((k_rms_norm<decltype(p)::value>), dim3(m), dim3(row_block(k, p)), 0, s, x, k, n, eps, o);
  });
}

hipError_t launch_rms_norm_residual(const ResidualArgs &a, int m, int k, float eps, const RowsOut &o, hipStream_t s) {
  return with_pieces(row_pieces(k), [&](auto p) {
    hipLaunchKernelGGL((k_rms_norm_residual<decltype(p)::value>), dim3(m), dim3(row_block(k, p)), 0, s, a, k, eps, o);
  });
}

}  // namespace nvfp4
