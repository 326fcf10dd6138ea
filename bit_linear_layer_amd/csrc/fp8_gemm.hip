// Matrix product of E4M3 operands with a float32 scale per block of 128 columns
// (activations: per row, weights: per 128 rows):
//     out[m, n] = sum_b sa[m, b] sw[n / 128, b] sum_{k in b} a[m, k] w[n, k].
// One block of 128 is the depth of one 16x16x128 matrix instruction, so a tile's
// sum over a block comes out of the matrix unit by itself and enters the
// running sum with one fma per output: out += (sa sw) tmp.
//
// The weight is the instruction's first operand, the activations its second:
// a lane then holds one token (lane % 16) and four consecutive columns, needs
// one activation scale per 16-token tile and stores its columns side by side.
//
// Two products (block_product):
//   bf16 output     v_mfma_scale_f32_16x16x128_f8f6f4 with unit scales.  The
//                   instruction cuts the products of 8 neighbouring k to
//                   multiples of 2^-13 of the largest's power of two before it
//                   adds them (measured); 1.5e-5 of a normally distributed result,
//                   against 1.7e-3 for the output's own rounding.
//   float32 output  codes converted to fp16 (exact), four 16x16x32 fp16
//                   instructions, exact products and float32 sums.
// Which k meets which inside a block is free as long as both operands agree: lane
// group g = lane / 16 takes the 16-byte pieces g and g + 4 of its row.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_util.h"
#include "layer_ops.h"

namespace nvfp4 {

namespace {

using namespace dev;
typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x8 __attribute__((ext_vector_type(8)));

// 8 E4M3 codes -> fp16, exact.
__device__ inline half8 half_of(uint32_t lo, uint32_t hi) {
  const half2v a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false);
  const half2v b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true);
  const half2v c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false);
  const half2v d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true);
  return half8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// A lane's 32 codes of one row and block.
struct Frag {
  u32x4 p[2];
};

// The 16 x 16 sums over one block of 128.
template <bool EXACT>
__device__ inline floatx4 block_product(const Frag& w, const Frag& x) {
  floatx4 c = {0.0f, 0.0f, 0.0f, 0.0f};
  if constexpr (EXACT) {
#pragma unroll
    for (int s = 0; s < 4; ++s)
      c = __builtin_amdgcn_mfma_f32_16x16x32_f16(half_of(w.p[s >> 1][2 * (s & 1)], w.p[s >> 1][2 * (s & 1) + 1]),
                                                 half_of(x.p[s >> 1][2 * (s & 1)], x.p[s >> 1][2 * (s & 1) + 1]), c, 0, 0, 0);
  } else {
    const i32x8 a = {(int)w.p[0][0], (int)w.p[0][1], (int)w.p[0][2], (int)w.p[0][3],
                     (int)w.p[1][0], (int)w.p[1][1], (int)w.p[1][2], (int)w.p[1][3]};
    const i32x8 b = {(int)x.p[0][0], (int)x.p[0][1], (int)x.p[0][2], (int)x.p[0][3],
                     (int)x.p[1][0], (int)x.p[1][1], (int)x.p[1][2], (int)x.p[1][3]};
    c = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, 127, 0, 127);
  }
  return c;
}

// Four consecutive columns of one row; vec: the row's address allows one store.
template <int OUT>
__device__ inline void store4(void* out, int64_t at, const floatx4& v, int left, bool vec) {
  if constexpr (OUT == NVFP4_DTYPE_BF16) {
    uint16_t* o = reinterpret_cast<uint16_t*>(out) + at;
    if (vec && left >= 4) {
      *reinterpret_cast<u32x2*>(o) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (r < left) o[r] = (uint16_t)f32_to_bf16_bits(v[r]);
    }
  } else {
    float* o = reinterpret_cast<float*>(out) + at;
    if (vec && left >= 4) {
      *reinterpret_cast<floatx4*>(o) = v;
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (r < left) o[r] = v[r];
    }
  }
}

// Tiles of FN * WN * 16 columns x FM * WM * 16 tokens, WN x WM waves; a block of
// 128 columns per step through registers into one of two LDS stages, rows of
// 128 bytes with their 16-byte pieces XOR-swizzled by the row so that the 8
// rows a quarter-wave reads fall into distinct banks.  Takes any sizes: rows
// behind the last are read as the last (their outputs are not stored), pieces
// behind K as zeros.
template <int FN, int FM, int WN, int WM, bool EXACT, int OUT>
__global__ __launch_bounds__(WN * WM * 64) void fp8_tile_kernel(const Fp8GemmArgs p, int tiles_m, int tiles_n) {
  constexpr int kThreads = WN * WM * 64, TN = FN * WN * 16, TM = FM * WM * 16;
  constexpr int kPieces = (TN + TM) * 8 / kThreads;
  static_assert((TN + TM) * 8 % kThreads == 0 && 128 % TN == 0, "whole pieces per thread, a tile in one weight block");
  __shared__ __attribute__((aligned(16))) uint8_t smem[2][(TN + TM) * 128];

  int tm, tn;
  tile_of(blockIdx.x, tiles_m * tiles_n, tiles_m, tiles_n, tm, tn);
  const int n0 = tn * TN, m0 = tm * TM;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wn = wave / WM, wm = wave % WM, li = lane & 15, lg = lane >> 4;
  const int blocks = (p.K + 127) / 128;

  const uint8_t* src[kPieces];
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int row = (tid + i * kThreads) >> 3, piece = tid & 7;
    src[i] = (row < TN ? p.w.codes + (int64_t)min(n0 + row, p.N - 1) * p.w.ld_codes
                       : p.a.codes + (int64_t)min(m0 + row - TN, p.M - 1) * p.a.ld_codes) + piece * 16;
  }
  u32x4 hold[kPieces];
  auto load = [&](int b) {
    const bool there = b * 128 + (tid & 7) * 16 < p.K;
#pragma unroll
    for (int i = 0; i < kPieces; ++i)
      hold[i] = there ? *reinterpret_cast<const u32x4*>(src[i] + b * 128) : u32x4{0u, 0u, 0u, 0u};
  };
  auto put = [&](int st) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int row = (tid + i * kThreads) >> 3, piece = tid & 7;
      *reinterpret_cast<u32x4*>(&smem[st][row * 128 + ((piece ^ (row & 7)) << 4)]) = hold[i];
    }
  };
  auto frag = [&](int st, int row) {
    Frag f;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      f.p[h] = *reinterpret_cast<const u32x4*>(&smem[st][row * 128 + (((lg + 4 * h) ^ (row & 7)) << 4)]);
    return f;
  };
  const float* sa[FM];
#pragma unroll
  for (int j = 0; j < FM; ++j)
    sa[j] = p.a.scales + (int64_t)min(m0 + (wm * FM + j) * 16 + li, p.M - 1) * p.a.scale_row;
  const float* sw = p.w.scales + (int64_t)(n0 / 128) * p.w.scale_row;

  floatx4 acc[FN][FM];
#pragma unroll
  for (int i = 0; i < FN; ++i)
#pragma unroll
    for (int j = 0; j < FM; ++j) acc[i][j] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};

  load(0);
  put(0);
  __syncthreads();
  for (int b = 0; b < blocks; ++b) {
    if (b + 1 < blocks) load(b + 1);
    float sc[FM];
    const float s = sw[b * p.w.scale_block];
#pragma unroll
    for (int j = 0; j < FM; ++j) sc[j] = sa[j][b * p.a.scale_block] * s;
    Frag w[FN];
#pragma unroll
    for (int i = 0; i < FN; ++i) w[i] = frag(b & 1, (wn * FN + i) * 16 + li);
#pragma unroll
    for (int j = 0; j < FM; ++j) {
      const Frag x = frag(b & 1, TN + (wm * FM + j) * 16 + li);
#pragma unroll
      for (int i = 0; i < FN; ++i) {
        const floatx4 t = block_product<EXACT>(w[i], x);
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[i][j][r] = fmaf(t[r], sc[j], acc[i][j][r]);
      }
    }
    if (b + 1 < blocks) put((b + 1) & 1);
    __syncthreads();
  }
  const bool vec = p.ld_out % 4 == 0 && (uintptr_t)p.out % (OUT == NVFP4_DTYPE_BF16 ? 8 : 16) == 0;
#pragma unroll
  for (int j = 0; j < FM; ++j) {
    const int m = m0 + (wm * FM + j) * 16 + li;
    if (m >= p.M) continue;
#pragma unroll
    for (int i = 0; i < FN; ++i) {
      const int n = n0 + (wn * FN + i) * 16 + 4 * lg;
      store4<OUT>(p.out, (int64_t)m * p.ld_out + n, acc[i][j], p.N - n, vec);
    }
  }
}

template <int FN, int FM, int WN, int WM>
hipError_t launch_tiles(const Fp8GemmArgs& g, hipStream_t s) {
  constexpr int TN = FN * WN * 16, TM = FM * WM * 16;
  const int tiles_m = (g.M + TM - 1) / TM, tiles_n = (g.N + TN - 1) / TN;
  const dim3 grid((unsigned)tiles_m * (unsigned)tiles_n), block(WN * WM * 64);
  if (g.out_dtype == NVFP4_DTYPE_BF16)
    fp8_tile_kernel<FN, FM, WN, WM, false, NVFP4_DTYPE_BF16><<<grid, block, 0, s>>>(g, tiles_m, tiles_n);
  else
    fp8_tile_kernel<FN, FM, WN, WM, true, NVFP4_DTYPE_F32><<<grid, block, 0, s>>>(g, tiles_m, tiles_n);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_fp8_gemm(const Fp8GemmArgs& g, hipStream_t s) {
  if (g.M <= 16) return launch_tiles<1, 1, 2, 1>(g, s);
  if (g.M <= 64) return launch_tiles<2, 2, 2, 2>(g, s);
  return launch_tiles<4, 4, 2, 2>(g, s);
}

}  // namespace nvfp4
