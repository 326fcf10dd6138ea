// E4M3 bytes nearest to the exact quotients x / s of float32 numbers, shared by
// the calibrated KV cache and the block-scaled quantizer, without a division
// per element.  With R = 1/s and the bracket
// R_lo = R (1 - 2^-18), R_hi = R (1 + 2^-18), the float32 products x R_lo and
// x R_hi lie on either side of the exact quotient x / s (the margin exceeds
// the roundings of R and of the products); clamped to +-448, both go through
// gfx950's E4M3 conversion, which rounds to nearest with ties to even (and
// keeps the sign of zero) but does not saturate -- hence the clamp, which is
// the saturating rule's own answer (when every product of a wavefront's
// chunks lies within +-448 already, the clamps are skipped: they would change
// nothing).  Where both bytes agree that byte is
// exact (the map is monotone).  Where they differ (codes m and m + 1, the
// bracket being far narrower than a grid step) the quotient sits next to the
// midpoint mu between the two values; mu has <= 5 significant bits, so
// fma(mu, s, -|x|) rounds the exact difference once and its sign decides
// (zero on a tie, which goes to the even code).  Scales outside [2^-90,
// 2^126] -- where that difference could leave float32's normal range --
// divide in float64 instead (e4m3_rne, exact by the bit counts).  A power-of-
// two scale (the unit scale among them) needs no bracket: x / s is then an
// exact float32 product and one conversion is the answer.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_util.h"
#include "nvfp4.h"
#include "quant_block.h"

namespace nvfp4 {
namespace dev {

// 8 consecutive elements as floats from a 16-byte (bf16) or 32-byte (f32) run.
template <int DT>
__device__ inline void load8(const uint8_t* p, float v[8]) {
  if constexpr (DT == NVFP4_DTYPE_BF16) {
    const uint4 q = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
    const float4 a = *reinterpret_cast<const float4*>(p);
    const float4 b = *reinterpret_cast<const float4*>(p + 16);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
}

// Magnitude of the E4M3 byte P of `src`, decoded by the hardware conversion (exact).
template <int P>
__device__ inline float e4m3_byte_mag(uint32_t src) {
  return fabsf(__builtin_amdgcn_cvt_f32_fp8((int)src, P));
}

// Bracket repair of byte P: lo and hi differ there (magnitudes m, m + 1).
template <int P>
__device__ inline void repair_byte(uint32_t& word, uint32_t lo, uint32_t hi, float x, float s) {
  constexpr int sh = 8 * P;
  if (((lo ^ hi) >> sh) & 0xFFu) {
    const float mid = 0.5f * (e4m3_byte_mag<P>(lo) + e4m3_byte_mag<P>(hi));  // exact, <= 5 bits
    const float d = fmaf(mid, s, -fabsf(x));
    const bool up = d < 0.0f || (d == 0.0f && ((lo >> sh) & 1u));
    if (up) word = (word & ~(0xFFu << sh)) | (hi & (0xFFu << sh));
  }
}

// Four E4M3 bytes (element 0 in the low byte) of x[0..3] * r with r = 1/s a
// power of two: the products are exact (or far below the first midpoint, or
// clamped), so one conversion is the exact answer.
__device__ inline uint32_t e4m3_quad_exact(const float* x, float r) {
  const float y0 = __builtin_amdgcn_fmed3f(x[0] * r, -448.0f, 448.0f);
  const float y1 = __builtin_amdgcn_fmed3f(x[1] * r, -448.0f, 448.0f);
  const float y2 = __builtin_amdgcn_fmed3f(x[2] * r, -448.0f, 448.0f);
  const float y3 = __builtin_amdgcn_fmed3f(x[3] * r, -448.0f, 448.0f);
  const uint32_t w = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y0, y1, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y2, y3, (int)w, true);
}

// Four E4M3 bytes (element 0 in the low byte) of x[0..3] / s, exactly rounded.
__device__ inline uint32_t e4m3_quad(const float* x, float r_lo, float r_hi, float s) {
  const float l0 = __builtin_amdgcn_fmed3f(x[0] * r_lo, -448.0f, 448.0f);
  const float l1 = __builtin_amdgcn_fmed3f(x[1] * r_lo, -448.0f, 448.0f);
  const float l2 = __builtin_amdgcn_fmed3f(x[2] * r_lo, -448.0f, 448.0f);
  const float l3 = __builtin_amdgcn_fmed3f(x[3] * r_lo, -448.0f, 448.0f);
  const float h0 = __builtin_amdgcn_fmed3f(x[0] * r_hi, -448.0f, 448.0f);
  const float h1 = __builtin_amdgcn_fmed3f(x[1] * r_hi, -448.0f, 448.0f);
  const float h2 = __builtin_amdgcn_fmed3f(x[2] * r_hi, -448.0f, 448.0f);
  const float h3 = __builtin_amdgcn_fmed3f(x[3] * r_hi, -448.0f, 448.0f);
  uint32_t lo = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(l0, l1, 0, false);
  lo = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(l2, l3, (int)lo, true);
  uint32_t hi = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(h0, h1, 0, false);
  hi = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(h2, h3, (int)hi, true);
  uint32_t word = lo;
  if (lo != hi) {
    repair_byte<0>(word, lo, hi, x[0], s);
    repair_byte<1>(word, lo, hi, x[1], s);
    repair_byte<2>(word, lo, hi, x[2], s);
    repair_byte<3>(word, lo, hi, x[3], s);
  }
  return word;
}

// e4m3_quad without the clamps, for inputs whose bracket products are all
// within +-448 (then the clamps change nothing).
__device__ inline uint32_t e4m3_quad_in_range(const float* x, float r_lo, float r_hi, float s) {
  uint32_t lo = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(x[0] * r_lo, x[1] * r_lo, 0, false);
  lo = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(x[2] * r_lo, x[3] * r_lo, (int)lo, true);
  uint32_t hi = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(x[0] * r_hi, x[1] * r_hi, 0, false);
  hi = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(x[2] * r_hi, x[3] * r_hi, (int)hi, true);
  uint32_t word = lo;
  if (lo != hi) {
    repair_byte<0>(word, lo, hi, x[0], s);
    repair_byte<1>(word, lo, hi, x[1], s);
    repair_byte<2>(word, lo, hi, x[2], s);
    repair_byte<3>(word, lo, hi, x[3], s);
  }
  return word;
}

// Division by the float32 scale sf of a group of elements, with E4M3 bytes as
// its exactly rounded result.
struct E4m3Scale {
  float sf, R, r_lo, r_hi;
  double s;
  bool fast, pow2;
  __device__ explicit E4m3Scale(float sf_) : sf(sf_) {
    fast = sf >= 0x1p-90f && sf <= 0x1p126f;
    pow2 = fast && (__float_as_uint(sf) & 0x7FFFFFu) == 0u;  // 1/s exact (s = 1 among them)
    R = 1.0f / sf;
    r_lo = R * (1.0f - 0x1p-18f);
    r_hi = R * (1.0f + 0x1p-18f);
    s = (double)sf;
  }
  // The 8 E4M3 bytes of v[0..7] / s.
  __device__ uint2 encode8(const float v[8]) const {
    uint32_t w[2] = {0u, 0u};
    if (pow2) {
      w[0] = e4m3_quad_exact(v, R);
      w[1] = e4m3_quad_exact(v + 4, R);
    } else if (fast) {
      float mx = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) mx = fmaxf(mx, fabsf(v[e]));
      if (__all(mx * r_hi <= 448.0f)) {  // the clamps would change nothing
        w[0] = e4m3_quad_in_range(v, r_lo, r_hi, sf);
        w[1] = e4m3_quad_in_range(v + 4, r_lo, r_hi, sf);
      } else {
        w[0] = e4m3_quad(v, r_lo, r_hi, sf);
        w[1] = e4m3_quad(v + 4, r_lo, r_hi, sf);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t m = e4m3_rne((double)fabsf(v[e]) / s);
        w[e >> 2] |= (m | ((__float_as_uint(v[e]) >> 31) << 7)) << (8 * (e & 3));
      }
    }
    return make_uint2(w[0], w[1]);
  }
};

}  // namespace dev
}  // namespace nvfp4
