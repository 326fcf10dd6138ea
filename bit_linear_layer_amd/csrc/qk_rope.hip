// Query and key heads: RMS norm per head and the position rotation, one pass.
//     z = x / sqrt(mean x^2 + eps) (w + offset);
//     (z_i, z_j) -> (z_i cos - z_j sin, z_j cos + z_i sin) for the pairs (i, j),
// each result rounded once.  Bound: HBM (every element read and written once).
//
// A workgroup takes one token and a share of its heads.  A head's elements lie
// in head_dim / 8 neighbouring lanes, 16 bytes (bf16) each: the sum of squares
// stays in those lanes, and the partner of a pair i, i + rotary_dim / 2 is
// the same element of the lane rotary_dim / 16 away.  The token's sines and
// cosines (at most 128 pairs) are computed once per workgroup, while the rows' loads
// are in flight: angle / 2 pi in float64, its distance to the nearest integer,
// and sincospi of that in float32 -- a float32 product of a far position would be
// off by whole turns.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_util.h"
#include "e4m3.h"
#include "internal.h"
#include "layer_ops.h"

namespace nvfp4 {

namespace {

using namespace dev;

template <int DT>
__device__ inline void store8(uint8_t* p, const float v[8]) {
  if constexpr (DT == NVFP4_DTYPE_BF16) {
    store_stream16(p, pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  } else {
    store_stream16(p, __float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    store_stream16(p + 16, __float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7]));
  }
}

// Rows (token, head) of queries and keys in one line: heads 0 .. hq - 1 are
// queries, the rest keys.  share: head slots of one workgroup.
template <int DT, int D>
__global__ __launch_bounds__(kElemThreads) void qk_norm_rope_kernel(const RopeArgs a, int share) {
  constexpr int kLanes = D / 8, kSlots = kElemThreads / kLanes, kSize = DT == NVFP4_DTYPE_BF16 ? 2 : 4;
  __shared__ float cs[D / 2], sn[D / 2];
  const int64_t t = blockIdx.x;
  const int part = threadIdx.x & (kLanes - 1), slot = threadIdx.x / kLanes;
  const int heads = a.rows[0].heads + a.rows[1].heads;
  const int h_end = min(heads, (int)(blockIdx.y + 1) * share);
  const int half = a.rope.rotary_dim / 2;

  int h = blockIdx.y * share + slot;
  float v[8];
  auto load = [&]() {
    const bool key = h >= a.rows[0].heads;
    const nvfp4_head_rows& r = a.rows[key];
    load8<DT>((const uint8_t*)r.x + (t * r.ld_x + (int64_t)(h - (key ? a.rows[0].heads : 0)) * r.head_x + part * 8) * kSize, v);
  };
  if (h < h_end) load();
  if ((int)threadIdx.x < half) {
    const int i = threadIdx.x;
    const int axis = a.rope.axis != nullptr ? min((int)a.rope.axis[i], a.rope.axes - 1) : 0;
    const double turn = (double)a.rope.positions[axis * a.rope.ld_positions + t] * (double)a.rope.inv_freq[i] * 0.15915494309189533577;
    float sine, cosine;
    sincospif(2.0f * (float)(turn - rint(turn)), &sine, &cosine);
    cs[i] = cosine;
    sn[i] = sine;
  }
  __syncthreads();
  for (; h < h_end; h += kSlots) {
    const bool key = h >= a.rows[0].heads;
    const nvfp4_head_rows& r = a.rows[key];
    if (r.weight != nullptr) {
      float sum = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) sum = fmaf(v[e], v[e], sum);
#pragma unroll
      for (int off = kLanes / 2; off > 0; off >>= 1) sum += __shfl_xor(sum, off);
      const float f = 1.0f / sqrtf(sum * (1.0f / D) + a.eps);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = v[e] * f * (r.weight[part * 8 + e] + a.weight_offset);
    }
    if (a.rope.interleaved) {
      if (part * 8 < 2 * half) {
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const float c = cs[part * 4 + e / 2], s = sn[part * 4 + e / 2], x = v[e], y = v[e + 1];
          v[e] = x * c - y * s;
          v[e + 1] = y * c + x * s;
        }
      }
    } else if (half > 0) {
      const bool first = part * 8 < half, second = !first && part * 8 < 2 * half;
      const int from = first ? part + half / 8 : second ? part - half / 8 : part;
      const int at = first ? part * 8 : second ? part * 8 - half : 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float other = __shfl(v[e], (threadIdx.x & (63 & ~(kLanes - 1))) + from);
        const float c = cs[at + e], s = first ? -sn[at + e] : sn[at + e];
        if (first || second) v[e] = v[e] * c + other * s;
      }
    }
    store8<DT>((uint8_t*)r.out + (t * r.ld_out + (int64_t)(h - (key ? a.rows[0].heads : 0)) * r.head_out + part * 8) * kSize, v);
    const int keep = h;
    h += kSlots;
    if (h < h_end) load();
    h = keep;
  }
}

template <int DT>
void launch(const RopeArgs& a, hipStream_t s) {
  const int heads = a.rows[0].heads + a.rows[1].heads;
  const dim3 grid((unsigned)a.tokens, 1);
  if (a.head_dim == 64) qk_norm_rope_kernel<DT, 64><<<grid, kElemThreads, 0, s>>>(a, heads);
  else if (a.head_dim == 128) qk_norm_rope_kernel<DT, 128><<<grid, kElemThreads, 0, s>>>(a, heads);
  else qk_norm_rope_kernel<DT, 256><<<grid, kElemThreads, 0, s>>>(a, heads);
}

}  // namespace

hipError_t launch_qk_norm_rope(const RopeArgs& a, hipStream_t s) {
  if (a.dtype == NVFP4_DTYPE_BF16) launch<NVFP4_DTYPE_BF16>(a, s);
  else launch<NVFP4_DTYPE_F32>(a, s);
  return hipGetLastError();
}

}  // namespace nvfp4
