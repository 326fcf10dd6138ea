// Block-scaled E4M3 quantization: activations by pieces of 128 columns of a
// row, weights by blocks of 128 x 128.
//
// Per block: a = max |x| over its finite elements, scale s = fl32(a / 448) or
// the least power of two with a <= 448 s, codes = E4M3 nearest to the exact
// x / s (e4m3.h).  Elements that are not finite become the NaN code and do not
// count in a, so one bad element spoils neither the scale nor its neighbours.
//
// fl32(a / 448) without a division: a / 448 = (a / 7) 2^-6, and with y the
// float32 nearest to 1/7, q = fl(a y), r = a - 7 q (exact in an fma), fl(q +
// r y) is the correctly rounded a / 7 (Markstein's theorem: y correctly
// rounded, q within one ulp).  Below 2^-80 the division is done in float64.
//
// Bound: HBM (one read, one byte written per element, 4 bytes per 128).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_util.h"
#include "e4m3.h"
#include "internal.h"
#include "layer_ops.h"

namespace nvfp4 {

namespace {

using namespace dev;

constexpr int kLanes = 16;  // lanes of a row piece, 8 elements each

__device__ inline float block_scale(float a, bool pow2) {
  if (pow2) {
    // bits + 0x1FFFFF carries into the exponent exactly when the mantissa is above 1.75
    const int b = (int)((__float_as_uint(a) + 0x1FFFFFu) >> 23) - 8;
    return __uint_as_float((uint32_t)max(b, 1) << 23);
  }
  if (a < 0x1p-80f) return (float)((double)a / 448.0);
  const float y = 0.14285714924335479736328125f;  // float32 nearest to 1/7
  const float q = a * y;
  return fmaf(fmaf(-7.0f, q, a), y, q) * 0.015625f;
}

// Elements of v that are not finite, one bit each; they are replaced by a zero of their sign.
__device__ inline uint32_t take_nonfinite(float v[8]) {
  uint32_t top = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(v[e]) & 0x7FFFFFFFu);
  uint32_t bad = 0;
  if (top >= 0x7F800000u) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if ((__float_as_uint(v[e]) & 0x7FFFFFFFu) >= 0x7F800000u) {
        bad |= 1u << e;
        v[e] = __uint_as_float(__float_as_uint(v[e]) & 0x80000000u);
      }
  }
  return bad;
}

__device__ inline float max8(const float v[8]) {
  float m = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(v[e]));
  return m;
}

// The 8 code bytes of v / s, s a block's scale; `bad` from take_nonfinite.
__device__ inline uint2 codes_of(const float v[8], const E4m3Scale& s, uint32_t bad) {
  uint2 w;
  if (s.sf == 0.0f) {
    uint32_t h[2] = {0u, 0u};
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e >> 2] |= (__float_as_uint(v[e]) >> 31) << (8 * (e & 3) + 7);
    w = make_uint2(h[0], h[1]);
  } else {
    w = s.encode8(v);
  }
  if (bad != 0) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (bad >> e & 1u) (e < 4 ? w.x : w.y) |= 0x7Fu << (8 * (e & 3));
  }
  return w;
}

// 16 lanes per piece; pieces are dealt to lane groups in a linear walk, two per
// iteration so that a second one's load is in flight.
template <int DT>
__global__ __launch_bounds__(kElemThreads) void fp8_quantize_rows_kernel(const uint8_t* __restrict__ x, int64_t ld_bytes,
                                                                         int64_t rows, int64_t cols, int64_t pieces,
                                                                         const Fp8Mat q, bool pow2) {
  constexpr int kChunkBytes = DT == NVFP4_DTYPE_BF16 ? 16 : 32;
  const int part = threadIdx.x & (kLanes - 1);
  const int64_t step = (int64_t)gridDim.x * (kElemThreads / kLanes);
  const int64_t first = (int64_t)blockIdx.x * (kElemThreads / kLanes) + threadIdx.x / kLanes;
  const int64_t dr = step / pieces, db = step - dr * pieces;
  int64_t r = first / pieces, b = first - r * pieces;
  while (r < rows) {
    int64_t rr[2], bb[2];
    float v[2][8];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      rr[u] = r;
      bb[u] = b;
      const int64_t c = b * 128 + part * 8;
      if (r < rows && c < cols) {
        load8<DT>(x + r * ld_bytes + (c / 8) * kChunkBytes, v[u]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[u][e] = 0.0f;
      }
      r += dr;
      b += db;
      if (b >= pieces) {
        b -= pieces;
        ++r;
      }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint32_t bad = take_nonfinite(v[u]);
      float a = max8(v[u]);
#pragma unroll
      for (int off = kLanes / 2; off > 0; off >>= 1) a = fmaxf(a, __shfl_xor(a, off));
      const E4m3Scale s(block_scale(a, pow2));
      const uint2 w = codes_of(v[u], s, bad);
      const int64_t c = bb[u] * 128 + part * 8;
      if (rr[u] < rows && c < cols) {
        store_stream8(q.codes + rr[u] * q.ld_codes + c, w.x, w.y);
        if (part == 0) q.scales[rr[u] * q.scale_row + bb[u] * q.scale_block] = s.sf;
      }
    }
  }
}

// One workgroup per block of 128 x 128: thread t holds 8 columns of the rows
// t / 16 + 16 i.
template <int DT>
__global__ __launch_bounds__(kElemThreads) void fp8_quantize_blocks_kernel(const uint8_t* __restrict__ x, int64_t ld_bytes,
                                                                           int64_t rows, int64_t cols, int pieces,
                                                                           const Fp8Mat q, bool pow2) {
  constexpr int kChunkBytes = DT == NVFP4_DTYPE_BF16 ? 16 : 32;
  __shared__ float red[kElemThreads / 64];
  const int64_t br = blockIdx.x / pieces, bc = blockIdx.x - br * pieces;
  const int64_t c = bc * 128 + (threadIdx.x & 15) * 8, r0 = br * 128 + threadIdx.x / 16;
  float v[8][8];
  uint32_t bad[8];
  float a = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (c < cols && r0 + 16 * i < rows) {
      load8<DT>(x + (r0 + 16 * i) * ld_bytes + (c / 8) * kChunkBytes, v[i]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = 0.0f;
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    bad[i] = take_nonfinite(v[i]);
    a = fmaxf(a, max8(v[i]));
  }
  a = wave_max(a);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = a;
  __syncthreads();
  a = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  const E4m3Scale s(block_scale(a, pow2));
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint2 w = codes_of(v[i], s, bad[i]);
    if (c < cols && r0 + 16 * i < rows) store_stream8(q.codes + (r0 + 16 * i) * q.ld_codes + c, w.x, w.y);
  }
  if (threadIdx.x == 0) q.scales[br * q.scale_row + bc * q.scale_block] = s.sf;
}

}  // namespace

hipError_t launch_fp8_quantize_rows(const void* x, int dtype, int64_t rows, int64_t cols, int64_t ld_x, const Fp8Mat& q,
                                    bool pow2, hipStream_t s) {
  const int64_t pieces = (cols + 127) / 128;
  const int64_t groups = (rows * pieces + kElemThreads / kLanes - 1) / (kElemThreads / kLanes);
  const int grid = (int)(groups < 2048 ? groups : 2048);
  if (dtype == NVFP4_DTYPE_BF16)
    fp8_quantize_rows_kernel<NVFP4_DTYPE_BF16><<<grid, kElemThreads, 0, s>>>((const uint8_t*)x, ld_x * 2, rows, cols, pieces, q, pow2);
  else
    fp8_quantize_rows_kernel<NVFP4_DTYPE_F32><<<grid, kElemThreads, 0, s>>>((const uint8_t*)x, ld_x * 4, rows, cols, pieces, q, pow2);
  return hipGetLastError();
}

hipError_t launch_fp8_quantize_blocks(const void* x, int dtype, int64_t rows, int64_t cols, int64_t ld_x, const Fp8Mat& q,
                                      bool pow2, hipStream_t s) {
  const int64_t pieces = (cols + 127) / 128;
  const unsigned grid = (unsigned)((rows + 127) / 128 * pieces);
  if (dtype == NVFP4_DTYPE_BF16)
    fp8_quantize_blocks_kernel<NVFP4_DTYPE_BF16><<<grid, kElemThreads, 0, s>>>((const uint8_t*)x, ld_x * 2, rows, cols, (int)pieces, q, pow2);
  else
    fp8_quantize_blocks_kernel<NVFP4_DTYPE_F32><<<grid, kElemThreads, 0, s>>>((const uint8_t*)x, ld_x * 4, rows, cols, (int)pieces, q, pow2);
  return hipGetLastError();
}

}  // namespace nvfp4
