// The gated delta rule for the next tokens of many sequences, each with its
// float32 states (128 x 128 per value head) in a pool:
//     S <- exp(g) S (I - beta k k^T) + beta v k^T,   o = S q.
// Bound: HBM -- a state is 64 KB, read and written once, whatever else is done.
//
// Row i of S (a value dimension) evolves by itself: with d = S_i . k and e = S_i . q of the old row,
//     u = beta (v_i - exp(g) d),  S_i <- exp(g) S_i + u k,  o_i = exp(g) e + u (k . q),
// so both products are taken of the old row at once.  8 lanes hold a row, 16
// floats each (4 pieces of 16 bytes, so that a load instruction reads 128
// neighbouring bytes of 8 rows), and sum over themselves.  A state stays in
// registers over the call's tokens.  k, q and their norms are worked out by every
// wave for itself: 1 KB from the cache against 4 KB of state.
//
// A wave has 8 rows, so that a single sequence's 48 heads are 192 workgroups.  Measured, us, 8 | 16 | 32 rows a wave, 16 key
// and 48 value heads, one token of 1, 4, 16, 64 sequences: 4.8, 9.0, 24.0, 74.5 (403 MB: 5.4 TB/s) | 5.3, 9.9, 24.6, 77.6 |
// 6.5, 10.4, 23.5, 79.7.  A copy of as many bytes reaches 5.1 TB/s.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_util.h"
#include "internal.h"
#include "layer_ops.h"

namespace nvfp4 {

namespace {

using namespace dev;
typedef float floatx4 __attribute__((ext_vector_type(4)));

constexpr int kD = 128;

__device__ inline float sum8(float v) {
  v += __shfl_xor(v, 1);
  v += __shfl_xor(v, 2);
  v += __shfl_xor(v, 4);
  return v;
}

// The lane's 16 of a head's 128 elements: 4 each at 32 j + 4 l.
template <int DT>
__device__ inline void load_row(const void* base, int64_t at, int l, floatx4 v[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (DT == NVFP4_DTYPE_BF16) {
      const u32x2 w = *reinterpret_cast<const u32x2*>(reinterpret_cast<const uint16_t*>(base) + at + 32 * j + 4 * l);
      v[j] = floatx4{__uint_as_float(w[0] << 16), __uint_as_float(w[0] & 0xFFFF0000u), __uint_as_float(w[1] << 16),
                     __uint_as_float(w[1] & 0xFFFF0000u)};
    } else {
      v[j] = *reinterpret_cast<const floatx4*>(reinterpret_cast<const float*>(base) + at + 32 * j + 4 * l);
    }
  }
}

template <int DT>
__device__ inline float load_one(const void* base, int64_t at) {
  if constexpr (DT == NVFP4_DTYPE_BF16) return bf16_bits_to_f32(reinterpret_cast<const uint16_t*>(base)[at]);
  else return reinterpret_cast<const float*>(base)[at];
}

__device__ inline float dot(const floatx4 a[4], const floatx4 b[4]) {
  float s = 0.0f;
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) s = fmaf(a[j][e], b[j][e], s);
  return s;
}

// One wave per 8 rows of a state, 4 waves a workgroup.
template <int DT>
__global__ __launch_bounds__(256) void gdn_step_kernel(const GdnStepArgs p) {
  constexpr int kShare = 4 * 8;  // rows of a workgroup
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l = lane & 7;
  const int h = blockIdx.x / (kD / kShare);
  const int row = blockIdx.x % (kD / kShare) * kShare + wave * 8 + lane / 8;
  for (int b = blockIdx.y; b < p.batch; b += gridDim.y) {
    const int64_t slot = p.slots != nullptr ? (int64_t)p.slots[b] : b;
    if (slot < 0 || slot >= p.n_states) continue;
    float* st = p.states + slot * p.ld_states + (int64_t)h * kD * kD;
    const bool fresh = p.fresh != nullptr && p.fresh[b] != 0;
    floatx4 s[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      s[j] = fresh ? floatx4{0.0f, 0.0f, 0.0f, 0.0f} : *reinterpret_cast<const floatx4*>(st + row * kD + 32 * j + 4 * l);
    const int hk = h / (p.hv / p.hk);
    for (int t = 0; t < p.q_len; ++t) {
      const int64_t at = (int64_t)b * p.q_len + t;
      floatx4 k[4], q[4];
      load_row<DT>(p.in.k, at * p.in.ld_k + hk * kD, l, k);
      load_row<DT>(p.in.q, at * p.in.ld_q + hk * kD, l, q);
      const float beta = load_one<DT>(p.in.beta, at * p.in.ld_beta + h);
      const float decay = expf(load_one<DT>(p.in.g, at * p.in.ld_g + h));
      if (p.normalize) {
        const float fk = 1.0f / fmaxf(sqrtf(sum8(dot(k, k))), 1e-30f);
        const float fq = 0.08838834764831845f / fmaxf(sqrtf(sum8(dot(q, q))), 1e-30f);  // 128^-1/2 / |q|
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            k[j][e] *= fk;
            q[j][e] *= fq;
          }
      }
      const float kq = sum8(dot(k, q));
      const float d = sum8(dot(s, k)), e = sum8(dot(s, q));
      const float v = load_one<DT>(p.in.v, at * p.in.ld_v + h * kD + row);
      const float u = beta * (v - decay * d);
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[j][i] = fmaf(u, k[j][i], decay * s[j][i]);
      const float o = fmaf(u, kq, decay * e);
      if (l == 0) {
        const int64_t to = at * p.ld_o + h * kD + row;
        if (p.o_dtype == NVFP4_DTYPE_BF16) reinterpret_cast<uint16_t*>(p.o)[to] = (uint16_t)f32_to_bf16_bits(o);
        else reinterpret_cast<float*>(p.o)[to] = o;
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) *reinterpret_cast<floatx4*>(st + row * kD + 32 * j + 4 * l) = s[j];
  }
}

}  // namespace

hipError_t launch_gdn_step(const GdnStepArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)(a.hv * (kD / 32)), (unsigned)(a.batch < 65535 ? a.batch : 65535));
  if (a.in_dtype == NVFP4_DTYPE_BF16) gdn_step_kernel<NVFP4_DTYPE_BF16><<<grid, 256, 0, s>>>(a);
  else gdn_step_kernel<NVFP4_DTYPE_F32><<<grid, 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace nvfp4
