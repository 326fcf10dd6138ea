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

#include <type_traits>

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

// 8 neighbouring elements as they lie in memory, and the bits of their largest
// magnitude as a float32's (for bf16 two at a time as 16-bit integers: the order of
// magnitudes is that of their bits).
template <int DT>
struct Chunk;
template <>
struct Chunk<NVFP4_DTYPE_BF16> {
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  static constexpr int kBytes = 16;
  u32x4 w;
  __device__ void load(const uint8_t* p) { w = *reinterpret_cast<const u32x4*>(p); }
  __device__ void clear() { w = u32x4{0u, 0u, 0u, 0u}; }
  __device__ uint32_t top() const {
    u16x2 m = __builtin_bit_cast(u16x2, w[0] & 0x7FFF7FFFu);
#pragma unroll
    for (int i = 1; i < 4; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, w[i] & 0x7FFF7FFFu));
    return (uint32_t)max(m[0], m[1]) << 16;
  }
  __device__ void floats(float v[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
};
template <>
struct Chunk<NVFP4_DTYPE_F32> {
  static constexpr int kBytes = 32;
  u32x4 w, h;
  __device__ void load(const uint8_t* p) {
    w = *reinterpret_cast<const u32x4*>(p);
    h = *reinterpret_cast<const u32x4*>(p + 16);
  }
  __device__ void clear() { w = h = u32x4{0u, 0u, 0u, 0u}; }
  __device__ uint32_t top() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max(max(m, w[i] & 0x7FFFFFFFu), h[i] & 0x7FFFFFFFu);
    return m;
  }
  __device__ void floats(float v[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = __uint_as_float(w[i]);
      v[4 + i] = __uint_as_float(h[i]);
    }
  }
};

constexpr uint32_t kInf = 0x7F800000u;

// The bits of the largest magnitude among v's finite elements.
__device__ inline uint32_t finite_top(const float v[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t b = __float_as_uint(v[e]) & 0x7FFFFFFFu;
    m = max(m, b < kInf ? b : 0u);
  }
  return m;
}

// A block's scale, with what its codes need.
struct Divider {
  float s, r_lo, r_hi;
  __device__ Divider(float a, bool pow2) : s(block_scale(a, pow2)) {
    // the hardware reciprocal is within an ulp; the bracket of 2^-18 holds that too
    const float r = __builtin_amdgcn_rcpf(s);
    r_lo = r * (1.0f - 0x1p-18f);
    r_hi = r * (1.0f + 0x1p-18f);
  }
  // The 8 code bytes of v / s, no element beyond 448 s (1 + 2^-23): 448 times the bracket still converts to 448.
  __device__ uint2 codes(const float v[8]) const {
    if (s >= 0x1p-90f) return make_uint2(e4m3_quad_in_range(v, r_lo, r_hi, s), e4m3_quad_in_range(v + 4, r_lo, r_hi, s));
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int e = 0; e < 8; ++e) {  // scales near the subnormal range: in float64; a scale of 0 leaves the signs
      const uint32_t m = s == 0.0f ? 0u : e4m3_rne((double)fabsf(v[e]) / (double)s);
      w[e >> 2] |= (m | ((__float_as_uint(v[e]) >> 31) << 7)) << (8 * (e & 3));
    }
    return make_uint2(w[0], w[1]);
  }
  // With elements that are not finite among them: these become the NaN code.
  __device__ uint2 codes_any(const float v[8]) const {
    float f[8];
    uint32_t bad[2] = {0u, 0u};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t b = __float_as_uint(v[e]);
      const bool out = (b & 0x7FFFFFFFu) >= kInf;
      f[e] = out ? __uint_as_float(b & 0x80000000u) : v[e];
      bad[e >> 2] |= (out ? 0x7Fu : 0u) << (8 * (e & 3));
    }
    const uint2 c = codes(f);
    return make_uint2(c.x | bad[0], c.y | bad[1]);
  }
};

// The largest of the 16 lanes of a row piece, in all of them.
__device__ inline uint32_t max16(uint32_t v) {
  auto with = [&](auto ctrl) {
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, decltype(ctrl)::value, 0xF, 0xF, true));
  };
  with(std::integral_constant<int, 0xB1>{});   // lane ^ 1
  with(std::integral_constant<int, 0x4E>{});   // lane ^ 2
  with(std::integral_constant<int, 0x141>{});  // 7 - lane of 8
  with(std::integral_constant<int, 0x140>{});  // 15 - lane of 16
  return v;
}

// 16 lanes per piece; pieces are dealt to lane groups in a linear walk, kAhead per
// iteration so that the others' loads are in flight.
template <int DT>
__global__ __launch_bounds__(kElemThreads) void fp8_quantize_rows_kernel(const uint8_t* __restrict__ x, int64_t ld_bytes,
                                                                         int64_t rows, int64_t cols, int64_t pieces,
                                                                         const Fp8Mat q, bool pow2) {
  constexpr int kBytes = Chunk<DT>::kBytes, kAhead = 2;
  const int part = threadIdx.x & (kLanes - 1);
  const int64_t step = (int64_t)gridDim.x * (kElemThreads / kLanes);
  const int64_t first = (int64_t)blockIdx.x * (kElemThreads / kLanes) + threadIdx.x / kLanes;
  const int64_t dr = step / pieces, db = step - dr * pieces;
  int64_t r = first / pieces, b = first - r * pieces;
  while (r < rows) {
    int64_t rr[kAhead], bb[kAhead];
    bool there[kAhead];
    Chunk<DT> c[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      rr[u] = r;
      bb[u] = b;
      there[u] = r < rows && b * 128 + part * 8 < cols;
      c[u].clear();
      if (there[u]) c[u].load(x + r * ld_bytes + (b * 16 + part) * kBytes);
      r += dr;
      b += db;
      if (b >= pieces) {
        b -= pieces;
        ++r;
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      float v[8];
      c[u].floats(v);
      uint32_t top = max16(c[u].top());
      const bool any = top >= kInf;  // the same in the piece's 16 lanes
      if (any) top = max16(finite_top(v));
      const Divider d(__uint_as_float(top), pow2);
      const uint2 w = any ? d.codes_any(v) : d.codes(v);
      if (there[u]) {
        store_stream8(q.codes + rr[u] * q.ld_codes + bb[u] * q.code_block + part * 8, w.x, w.y);
        if (part == 0) q.scales[rr[u] * q.scale_row + bb[u] * q.scale_block] = d.s;
      }
    }
  }
}

// One workgroup of 1024 threads per block of 128 x 128: a thread holds 8 columns of two rows.  1000 x 2064 float32: 5.0 us.
template <int DT>
__global__ __launch_bounds__(1024) void fp8_quantize_blocks_kernel(const uint8_t* __restrict__ x, int64_t ld_bytes,
                                                                   int64_t rows, int64_t cols, int pieces, const Fp8Mat q,
                                                                   bool pow2) {
  __shared__ uint32_t red[2][16];
  const int64_t br = blockIdx.x / pieces, bc = blockIdx.x - br * pieces;
  const int64_t c = bc * 128 + (threadIdx.x & 15) * 8, r0 = br * 128 + threadIdx.x / 16;
  Chunk<DT> chunk[2];
  float v[2][8];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    chunk[i].clear();
    if (c < cols && r0 + 64 * i < rows) chunk[i].load(x + (r0 + 64 * i) * ld_bytes + c / 8 * Chunk<DT>::kBytes);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) chunk[i].floats(v[i]);
  auto over_all = [&](uint32_t top, uint32_t* at) {
    top = max16(top);
    top = max(top, (uint32_t)__shfl_xor((int)top, 16));
    top = max(top, (uint32_t)__shfl_xor((int)top, 32));
    if ((threadIdx.x & 63) == 0) at[threadIdx.x >> 6] = top;
    __syncthreads();
    return max16(at[threadIdx.x & 15]);
  };
  uint32_t top = over_all(max(chunk[0].top(), chunk[1].top()), red[0]);
  const bool any = top >= kInf;  // the same in all threads
  if (any) top = over_all(max(finite_top(v[0]), finite_top(v[1])), red[1]);
  const Divider d(__uint_as_float(top), pow2);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint2 w = any ? d.codes_any(v[i]) : d.codes(v[i]);
    if (c < cols && r0 + 64 * i < rows) store_stream8(q.codes + (r0 + 64 * i) * q.ld_codes + c, w.x, w.y);
  }
  if (threadIdx.x == 0) q.scales[br * q.scale_row + bc * q.scale_block] = d.s;
}

}  // namespace

hipError_t launch_fp8_quantize_rows(const void* x, int dtype, int64_t rows, int64_t cols, int64_t ld_x, const Fp8Mat& q,
                                    bool pow2, hipStream_t s) {
  const int64_t pieces = (cols + 127) / 128;
  const int64_t groups = (rows * pieces + kElemThreads / kLanes - 1) / (kElemThreads / kLanes);
  // Measured, us, with at most 2048, 8192, 16384, 32768 workgroups: 8192 x 17408 100, 85, 84 (5.1 TB/s, a copy's rate), 90;
  // 8192 x 5120 27.6, 26.4, 33, 38; 2048 x 5120 9.6, 12.2, 11.9, 12.1.
  const int64_t most = groups / 4 < 2048 ? 2048 : groups / 4 < 16384 ? groups / 4 : 16384;
  const int grid = (int)(groups < most ? groups : most);
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
    fp8_quantize_blocks_kernel<NVFP4_DTYPE_BF16><<<grid, 1024, 0, s>>>((const uint8_t*)x, ld_x * 2, rows, cols, (int)pieces, q, pow2);
  else
    fp8_quantize_blocks_kernel<NVFP4_DTYPE_F32><<<grid, 1024, 0, s>>>((const uint8_t*)x, ld_x * 4, rows, cols, (int)pieces, q, pow2);
  return hipGetLastError();
}

}  // namespace nvfp4
