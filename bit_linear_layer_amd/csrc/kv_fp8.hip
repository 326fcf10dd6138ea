// FP8 (E4M3) KV cache with a calibrated per-tensor scale (evolve.pub review
// of arXiv 2609.04098, "Key claims under review", fifth claim; chatpaper.ai
// English abstract): calibration s = fl32(amax / 448); write: the E4M3 byte
// nearest to the exact real x / s (ties to even code, saturating at 448,
// IEEE sign), scattered to cache rows by an optional slot index; read:
// fl32(e4m3 * s), optionally rounded to bf16.  s = 1 is the uncalibrated
// cache, so calibrated and uncalibrated caches run the same code.
//
// The write divides without a division per element (e4m3.h); the read
// decodes with the hardware conversion (exact for every byte) and rounds to
// bf16 with the hardware conversion (nearest even).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_util.h"
#include "e4m3.h"
#include "internal.h"

namespace nvfp4 {

namespace {

using namespace dev;

// Walk over the 8-element chunks of a [rows, cpr] matrix from chunk `start`
// in steps of `stride` chunks, keeping (row, chunk-in-row) without a division
// per step.
struct ChunkWalk {
  int64_t r, c, cpr, rows, dr, dc;
  __device__ ChunkWalk(int64_t rows_, int64_t cpr_, int64_t start, int64_t stride) : cpr(cpr_), rows(rows_) {
    r = start / cpr;
    c = start - r * cpr;
    dr = stride / cpr;
    dc = stride - dr * cpr;
  }
  __device__ bool valid() const { return r < rows; }
  __device__ void next() {
    r += dr;
    c += dc;
    if (c >= cpr) {
      c -= cpr;
      ++r;
    }
  }
};

// Each thread takes two chunks per iteration, one grid-width apart (so every
// load instruction of a wavefront still reads contiguous bytes), and the
// cache and output bytes go out as streaming stores.  A write of contiguous
// rows without slots runs a kernel that walks one linear chunk index
// instead of (row, chunk) pairs and 64-bit row products, and issues both
// loads before the first wait.  Measured on 32768 x 1024 bf16 with 16
// rotating buffers (none left in the last-level cache), against one chunk
// per iteration with plain stores: calibrated write 25.7 -> 21.4 us (the
// linear walk and the skipped clamps -2.9 us of it), unit-scale write
// 21.7 -> 20.3 us, bf16 read unchanged at 20.5-20.9 us; four chunks per
// iteration, or fewer workgroups, were slower.
constexpr int kChunksPerIter = 2;

// Contiguous x and cache rows, no slots: chunk i at byte i * chunk of x and
// i * 8 of the cache.
template <int DT>
__global__ __launch_bounds__(kElemThreads) void kv_quant_linear_kernel(const uint8_t* __restrict__ x, int64_t total,
                                                                       uint8_t* __restrict__ cache,
                                                                       const float* __restrict__ scale) {
  constexpr int kChunkBytes = DT == NVFP4_DTYPE_BF16 ? 16 : 32;
  const E4m3Scale ks(*scale);
  const int64_t T = (int64_t)gridDim.x * blockDim.x;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += 2 * T) {
    const int64_t i1 = i + T;
    const bool ok1 = i1 < total;
    float v0[8], v1[8];
    load8<DT>(x + i * kChunkBytes, v0);
    load8<DT>(x + (ok1 ? i1 : i) * kChunkBytes, v1);
    const uint2 w0 = ks.encode8(v0);
    store_stream8(cache + i * 8, w0.x, w0.y);
    const uint2 w1 = ks.encode8(v1);
    if (ok1) store_stream8(cache + i1 * 8, w1.x, w1.y);
  }
}

template <int DT>
__global__ __launch_bounds__(kElemThreads) void kv_quant_kernel(
    const uint8_t* __restrict__ x, int64_t ld_bytes, int64_t rows, int64_t cpr,
    const int64_t* __restrict__ slots, int64_t cache_rows, uint8_t* __restrict__ cache,
    int64_t ld_cache, const float* __restrict__ scale) {
  constexpr int kChunkBytes = DT == NVFP4_DTYPE_BF16 ? 16 : 32;
  const E4m3Scale ks(*scale);
  constexpr int U = kChunksPerIter;
  static_assert(U == 2, "the walkers below are listed one by one");
  const int64_t T = (int64_t)gridDim.x * blockDim.x;
  const int64_t start = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  ChunkWalk it[U] = {ChunkWalk(rows, cpr, start, U * T), ChunkWalk(rows, cpr, start + T, U * T)};
  while (it[0].valid()) {
    float v[U][8];
    int64_t dst[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const bool ok = it[j].valid();
      dst[j] = ok ? (slots != nullptr ? slots[it[j].r] : it[j].r) : -1;
      if (ok) load8<DT>(x + it[j].r * ld_bytes + it[j].c * kChunkBytes, v[j]);
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      if (dst[j] < 0 || dst[j] >= cache_rows) continue;  // documented: such rows are not written
      const uint2 wv = ks.encode8(v[j]);
      store_stream8(cache + dst[j] * ld_cache + it[j].c * 8, wv.x, wv.y);
    }
#pragma unroll
    for (int j = 0; j < U; ++j) it[j].next();
  }
}

template <int OUT>
__global__ __launch_bounds__(kElemThreads) void kv_dequant_kernel(
    const uint8_t* __restrict__ cache, int64_t ld_cache, int64_t rows, int64_t cpr,
    const float* __restrict__ scale, uint8_t* __restrict__ out, int64_t ld_out_bytes) {
  const float s = *scale;
  constexpr int U = kChunksPerIter;
  static_assert(U == 2, "the walkers below are listed one by one");
  const int64_t T = (int64_t)gridDim.x * blockDim.x;
  const int64_t start = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  ChunkWalk it[U] = {ChunkWalk(rows, cpr, start, U * T), ChunkWalk(rows, cpr, start + T, U * T)};
  while (it[0].valid()) {
    uint2 q[U];
#pragma unroll
    for (int j = 0; j < U; ++j)
      if (it[j].valid()) q[j] = *reinterpret_cast<const uint2*>(cache + it[j].r * ld_cache + it[j].c * 8);
#pragma unroll
    for (int j = 0; j < U; ++j) {
      if (!it[j].valid()) continue;
      float f[8];
      const f32x2_t d0 = __builtin_amdgcn_cvt_pk_f32_fp8((int)q[j].x, false), d1 = __builtin_amdgcn_cvt_pk_f32_fp8((int)q[j].x, true);
      const f32x2_t d2 = __builtin_amdgcn_cvt_pk_f32_fp8((int)q[j].y, false), d3 = __builtin_amdgcn_cvt_pk_f32_fp8((int)q[j].y, true);
      f[0] = d0.x * s; f[1] = d0.y * s; f[2] = d1.x * s; f[3] = d1.y * s;
      f[4] = d2.x * s; f[5] = d2.y * s; f[6] = d3.x * s; f[7] = d3.y * s;
      if constexpr (OUT == NVFP4_DTYPE_BF16) {
        store_stream16(out + it[j].r * ld_out_bytes + it[j].c * 16, pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                       pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
      } else {
        uint8_t* o = out + it[j].r * ld_out_bytes + it[j].c * 32;
        store_stream16(o, __float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
        store_stream16(o + 16, __float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7]));
      }
    }
#pragma unroll
    for (int j = 0; j < U; ++j) it[j].next();
  }
}

// s = fl32(max(partials) / 448): one correctly rounded division (53 >= 2*24+2).
__global__ __launch_bounds__(kElemThreads) void kv_scale_kernel(const float* __restrict__ partials,
                                                                int n, float* __restrict__ scale) {
  __shared__ float red[kElemThreads / 64];
  float m = 0.0f;
  for (int i = threadIdx.x; i < n; i += blockDim.x) m = fmaxf(m, partials[i]);
  m = wave_max(m);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
  __syncthreads();
  if (threadIdx.x == 0) {
    float v = red[0];
    for (int i = 1; i < kElemThreads / 64; ++i) v = fmaxf(v, red[i]);
    *scale = (float)((double)v / 448.0);
  }
}

// At most 2048 workgroups (8 per CU on 256 CUs, all resident at once),
// each thread walking several chunks: measured faster than 8192 or 32768
// workgroups with fewer chunks each (32768 x 1024 bf16: write 27.3 -> 25.9
// us calibrated, read 22.9 -> 20.6 us), and than 1024 or 1536.
int chunk_grid(int64_t chunks) {
  int64_t wg = (chunks + kElemThreads - 1) / kElemThreads;
  if (wg > 2048) wg = 2048;
  if (wg < 1) wg = 1;
  return (int)wg;
}

}  // namespace

hipError_t launch_kv_quantize(const void* x, int dtype, int64_t rows, int64_t cols, int64_t ld_x,
                              const int64_t* slots, int64_t cache_rows, uint8_t* cache,
                              int64_t ld_cache, const float* scale, hipStream_t s) {
  const int64_t cpr = cols / 8;
  const int grid = chunk_grid(rows * cpr);
  if (slots == nullptr && ld_x == cols && ld_cache == cols) {
    if (dtype == NVFP4_DTYPE_BF16)
      kv_quant_linear_kernel<NVFP4_DTYPE_BF16><<<grid, kElemThreads, 0, s>>>((const uint8_t*)x, rows * cpr, cache, scale);
    else
      kv_quant_linear_kernel<NVFP4_DTYPE_F32><<<grid, kElemThreads, 0, s>>>((const uint8_t*)x, rows * cpr, cache, scale);
    return hipGetLastError();
  }
  if (dtype == NVFP4_DTYPE_BF16)
    kv_quant_kernel<NVFP4_DTYPE_BF16><<<grid, kElemThreads, 0, s>>>(
        (const uint8_t*)x, ld_x * 2, rows, cpr, slots, cache_rows, cache, ld_cache, scale);
  else
    kv_quant_kernel<NVFP4_DTYPE_F32><<<grid, kElemThreads, 0, s>>>(
        (const uint8_t*)x, ld_x * 4, rows, cpr, slots, cache_rows, cache, ld_cache, scale);
  return hipGetLastError();
}

hipError_t launch_kv_dequantize(const uint8_t* cache, int64_t rows, int64_t cols, int64_t ld_cache,
                                const float* scale, void* out, int out_dtype, int64_t ld_out,
                                hipStream_t s) {
  const int64_t cpr = cols / 8;
  const int grid = chunk_grid(rows * cpr);
  if (out_dtype == NVFP4_DTYPE_BF16)
    kv_dequant_kernel<NVFP4_DTYPE_BF16><<<grid, kElemThreads, 0, s>>>(cache, ld_cache, rows, cpr, scale,
                                                                      (uint8_t*)out, ld_out * 2);
  else
    kv_dequant_kernel<NVFP4_DTYPE_F32><<<grid, kElemThreads, 0, s>>>(cache, ld_cache, rows, cpr, scale,
                                                                     (uint8_t*)out, ld_out * 4);
  return hipGetLastError();
}

hipError_t launch_kv_scale(const float* partials, int n, float* scale, hipStream_t s) {
  kv_scale_kernel<<<1, kElemThreads, 0, s>>>(partials, n, scale);
  return hipGetLastError();
}

}  // namespace nvfp4
