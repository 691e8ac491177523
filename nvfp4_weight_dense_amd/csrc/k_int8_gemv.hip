// k_int8_gemv.hip -- the int8 projection of 1 to 4 rows (gfx950), bound by
// reading the weight once.
//
// A workgroup of 16 waves owns a run of output columns (n / 256 of them, one
// workgroup per CU) of one or, for gate and up, both weights.  Its weight
// rows are cut into pieces of 1024 codes, which a wave reads as one
// contiguous kilobyte, and the pieces, row after row, are dealt to the waves
// in equal runs whatever the number of columns: sums of whole numbers may be
// joined in any order, so a row that several waves share is summed with LDS
// atomics.  Eight pieces are requested while eight are summed (128 to 256 KB
// in flight for a CU).  One row of 4096, 12288: gate and up with the row
// quantized 21.6 us (4.7 TB/s), down 12.5 us (4.0); a product of 6144 x 4096
// of quantized rows 9.0 us (8.7 with one weight again and again), of which
// start, the first way through memory and the end are some 5.  Four rows are
// bound by the products: 29.0, 17.3 and 11.3 us.
//
// The activation rows lie in LDS as codes; lane l multiplies codes 16 l .. of
// a piece with dot products of four.  bf16 rows are quantized here, in every
// workgroup, while its first weights are under way: a launch less.
#include <algorithm>

#include "int8_common.h"

namespace nvfp4 {

namespace {

constexpr int kThreads = 1024, kWaves = 16;
constexpr int kBatch = 8;     // pieces requested together by a wave
constexpr int kMaxCols = 512; // columns of a workgroup
// Pieces of eight bf16 values that a thread quantizes: one or two rows of any
// length that LDS takes, three or four up to 16384.  Each workgroup encodes
// all rows, so longer ones of three or four go faster through the quantizer
// and the kernel for up to 64 rows: 4 rows of 5120 x 12288 19.8 us here and
// 20.2 there, 5120 x 17408 26.3 and 24.7, 8192 x 16384 35.6 and 31.4 (5120 x
// 16384 24.6 and 27.1); 2 rows of 5120 x 17408 21.6 and 24.7.
constexpr int kXPieces = 8;

struct GemvArgs {
  const void *x;        // bf16 [m][k], or int8 [m][k] with
  const float *xs;      // [m]
  int m, k, n, cols;
  const int8_t *w0, *w1;
  const float *s0, *s1;
  void *y;
};

// bytes of LDS for the rows
constexpr int x_bytes(int m) { return m * 32768; }

// M: rows as laid out (1, 2 or 4, not less than m)
template <int M, int NMAT, bool QUANT>
__global__ __launch_bounds__(kThreads) void k_int8_gemv(GemvArgs p) {
  __shared__ __attribute__((aligned(16))) uint8_t xq[M][x_bytes(1)];
  __shared__ int sums[NMAT * kMaxCols * M];
  __shared__ Int8Scale row_scale[M];
  __shared__ uint32_t tops[kWaves];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int k = p.k;
  const int col0 = (int)blockIdx.x * p.cols, cols = min(p.cols, p.n - col0);

  // the activation rows are requested first, then the first weights
  constexpr int kRowThreads = kThreads / M;
  const int xrow = tid / kRowThreads, xt = tid % kRowThreads;
  uint4 xv[kXPieces];
  if constexpr (QUANT) {
    const uint4 *from = (const uint4 *)p.x + (size_t)xrow * (k >> 3);
#pragma unroll
    for (int i = 0; i < kXPieces; ++i) {
      const int at = xt + i * kRowThreads;
      xv[i] = xrow < p.m && at < (k >> 3) ? from[at] : uint4{0u, 0u, 0u, 0u};
    }
  }

  // this wave's run of (weight row, piece): rows 0 .. cols - 1 of w0, then of w1
  const int per_row = (k + 1023) >> 10;
  const int items = NMAT * cols * per_row;
  const int first = (int)((int64_t)items * wave / kWaves), last = (int)((int64_t)items * (wave + 1) / kWaves);
  const __amdgpu_buffer_rsrc_t w0 = rsrc_uniform(p.w0 + (size_t)col0 * k, (size_t)cols * k);
  const __amdgpu_buffer_rsrc_t w1 = rsrc_uniform((NMAT > 1 ? p.w1 : p.w0) + (size_t)col0 * k, (size_t)cols * k);
  int lrow = first / per_row, lpiece = first - lrow * per_row;  // of the next request
  int left = last - first;
  auto request = [&](uint4 (&v)[kBatch]) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const uint32_t at = (uint32_t)lpiece * 1024u + 16u * (uint32_t)lane;
      const bool up = NMAT > 1 && lrow >= cols;
      const uint32_t off = left > 0 && at < (uint32_t)k ? (uint32_t)(up ? lrow - cols : lrow) * (uint32_t)k + at : kOOB;
      v[i] = ld16(up ? w1 : w0, off);
      --left;
      if (++lpiece == per_row) lpiece = 0, ++lrow;
    }
  };
  uint4 va[kBatch], vb[kBatch];
  request(va);

  for (int i = tid; i < NMAT * cols * M; i += kThreads) sums[i] = 0;
  if constexpr (QUANT) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kXPieces; ++i) {
      top = amax_bits(top, xv[i]);
    }
    top = amax_fold(top);
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, off));
    if (lane == 0) tops[wave] = top;
    lds_barrier();
    constexpr int kRowWaves = kWaves / M;
    top = tops[xrow * kRowWaves];
#pragma unroll
    for (int i = 1; i < kRowWaves; ++i) top = max(top, tops[xrow * kRowWaves + i]);
    const Int8Row r = int8_row(top);
    if (xt == 0) row_scale[xrow] = int8_scale(r.s);
#pragma unroll
    for (int i = 0; i < kXPieces; ++i) {
      const int at = xt + i * kRowThreads;
      if (at < (k >> 3)) *(uint2 *)&xq[xrow][8 * at] = int8_codes(xv[i], r);
    }
  } else {
    const uint4 *from = (const uint4 *)p.x;
    for (int i = tid; i < p.m * (k >> 4); i += kThreads) {
      const int r = i / (k >> 4);
      *(uint4 *)&xq[r][16 * (i - r * (k >> 4))] = from[i];
    }
    if (tid < p.m) row_scale[tid] = int8_scale(p.xs[tid]);
  }
  lds_barrier();

  int row = first / per_row, piece = first - row * per_row;
  int todo = last - first;
  int acc[M] = {};
  auto add = [&](const uint4 (&v)[kBatch]) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (todo <= 0) break;
#pragma unroll
      for (int r = 0; r < M; ++r) {
        // (past k the weights read as 0)
        const uint4 x = *(const uint4 *)&xq[r][piece * 1024 + 16 * lane];
        acc[r] = __builtin_amdgcn_sdot4((int)v[i].x, (int)x.x, acc[r], false);
        acc[r] = __builtin_amdgcn_sdot4((int)v[i].y, (int)x.y, acc[r], false);
        acc[r] = __builtin_amdgcn_sdot4((int)v[i].z, (int)x.z, acc[r], false);
        acc[r] = __builtin_amdgcn_sdot4((int)v[i].w, (int)x.w, acc[r], false);
      }
      --todo;
      const bool ends = ++piece == per_row;
      if (ends || todo == 0) {
        // sixteen lanes join by rotations, the four sixteens in LDS
#pragma unroll
        for (int r = 0; r < M; ++r) {
          int s = acc[r];
          s += __builtin_amdgcn_update_dpp(0, s, 0x128, 0xf, 0xf, false);
          s += __builtin_amdgcn_update_dpp(0, s, 0x124, 0xf, 0xf, false);
          s += __builtin_amdgcn_update_dpp(0, s, 0x122, 0xf, 0xf, false);
          s += __builtin_amdgcn_update_dpp(0, s, 0x121, 0xf, 0xf, false);
          if ((lane & 15) == 0) atomicAdd(&sums[row * M + r], s);
          acc[r] = 0;
        }
      }
      if (ends) piece = 0, ++row;
    }
  };
  while (todo > 0) {
    request(vb);
    add(va);
    request(va);
    add(vb);
  }
  __syncthreads();

  for (int i = tid; i < cols * p.m; i += kThreads) {
    const int r = i / cols, c = i - r * cols;
    const float v = int8_scaled(sums[c * M + r], row_scale[r], int8_scale(p.s0[col0 + c]));
    __bf16 out = (__bf16)v;
    if constexpr (NMAT > 1)
      out = swiglu_bf16(v, int8_scaled(sums[(cols + c) * M + r], row_scale[r], int8_scale(p.s1[col0 + c])));
    ((__bf16 *)p.y)[(size_t)r * p.n + col0 + c] = out;
  }
}

// rows as a kernel takes them
int gemv_rows(int m) { return m == 3 ? 4 : m; }

}  // namespace

bool int8_gemv_eligible(int m, int k) { return m <= 4 && k <= x_bytes(1); }

bool int8_gemv_quantizes(int m, int k) {
  return int8_gemv_eligible(m, k) && cdiv(k >> 3, kThreads / gemv_rows(m)) <= kXPieces;
}

hipError_t launch_int8_gemv(const void *x, const float *row_scale, int m, int k, int n, int nmat, const Int8MatRef *w,
                            void *y, hipStream_t s) {
  const int cols = std::min(kMaxCols, cdiv(n, 256));
  const GemvArgs p{x, row_scale, m, k, n, cols, w[0].codes, nmat > 1 ? w[1].codes : nullptr, w[0].scales,
                   nmat > 1 ? w[1].scales : nullptr, y};
  auto run = [&](auto rows) {
    constexpr int M = decltype(rows)::value;
    const dim3 grid(cdiv(n, cols)), block(kThreads);
    if (nmat == 1) {
      if (row_scale) hipLaunchKernelGGL((k_int8_gemv<M, 1, false>), grid, block, 0, s, p);
      else hipLaunchKernelGGL((k_int8_gemv<M, 1, true>), grid, block, 0, s, p);
    } else {
      if (row_scale) hipLaunchKernelGGL((k_int8_gemv<M, 2, false>), grid, block, 0, s, p);
      else hipLaunchKernelGGL((k_int8_gemv<M, 2, true>), grid, block, 0, s, p);
    }
  };
  if (m == 1) run(std::integral_constant<int, 1>());
  else if (m == 2) run(std::integral_constant<int, 2>());
  else run(std::integral_constant<int, 4>());
  return hipGetLastError();
}

}  // namespace nvfp4
