// Query and key heads: RMS norm per head and the position rotation, one pass.
//     z = x / sqrt(mean x^2 + eps) (w + offset);
//     (z_i, z_j) -> (z_i cos - z_j sin, z_j cos + z_i sin) for the pairs (i, j),
// each result rounded once.  Bound: HBM (every element read and written once).
//
// A workgroup takes a few tokens, all of their heads or a share of them.  A head's
// elements lie in head_dim / 8 neighbouring lanes, 16 bytes (bf16) each: the sum of
// squares stays in those lanes, and the partner of a pair i, i + rotary_dim / 2 is
// the same element of the lane rotary_dim / 16 away.  The tokens' sines and
// cosines are computed first, one a thread, while the first rows' loads are in
// flight: angle / 2 pi in float64, its distance to the nearest integer, and
// sincospi of that -- a float32 product of a far position would be off by
// whole turns.  For float32 rows the sine is taken in float64 too and rounded once; a float32 fraction puts it off by
// up to 1.9 * 2^-24, which bf16's half step of 2^-9 to 2^-8 hides, and is 4 % faster (16384 x 40 heads of 128: 73 us, 76).  They are kept in LDS for each element, the sine with the sign of
// its place in the pair, so that a result is z c + partner s without a choice.
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
typedef float floatx4 __attribute__((ext_vector_type(4)));

template <int DT>
__device__ inline void store8(uint8_t* p, const float v[8]) {
  if constexpr (DT == NVFP4_DTYPE_BF16) {
    store_stream16(p, pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  } else {
    store_stream16(p, __float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    store_stream16(p + 16, __float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7]));
  }
}

// The sum over the L lanes of a head, in all of them.
template <int L>
__device__ inline float head_sum(float v) {
  auto add = [&](auto ctrl) {
    v += __uint_as_float(__builtin_amdgcn_mov_dpp(__float_as_uint(v), decltype(ctrl)::value, 0xF, 0xF, true));
  };
  add(std::integral_constant<int, 0xB1>{});   // lane ^ 1
  add(std::integral_constant<int, 0x4E>{});   // lane ^ 2
  add(std::integral_constant<int, 0x141>{});  // 7 - lane of 8: the other four
  if constexpr (L >= 16) add(std::integral_constant<int, 0x140>{});  // 15 - lane of 16: the other eight
  if constexpr (L >= 32) v += __shfl_xor(v, 16);
  return v;
}

constexpr int kTable = 1024;  // entries of the sines' and of the cosines' table: tokens * rotary_dim

// Rows are (token, head), queries' heads first, then keys'.  A workgroup has `tokens`
// tokens and of their rows `passes` times as many as it holds at once.
template <int DT, int D>
__global__ __launch_bounds__(kElemThreads) void qk_norm_rope_kernel(const RopeArgs a, int tokens, int passes) {
  constexpr int kLanes = D / 8, kSlots = kElemThreads / kLanes, kSize = DT == NVFP4_DTYPE_BF16 ? 2 : 4;
  __shared__ __attribute__((aligned(16))) float cs[kTable], sn[kTable], weights[2][D];
  const int64_t t0 = (int64_t)blockIdx.x * tokens;
  const int part = threadIdx.x & (kLanes - 1), slot = threadIdx.x / kLanes;
  const int hq = a.rows[0].heads, heads = hq + a.rows[1].heads;
  const int n = (int)min((int64_t)tokens, a.tokens - t0) * heads;  // rows of these tokens
  const int dim = a.rope.rotary_dim, half = dim / 2;

  float v[8], next[8] = {};
  struct Row {
    int token, head;
    bool key, there;
  };
  auto row_of = [&](int pass) {
    const int row = pass * kSlots + slot;
    Row r;
    r.there = row < n;
    r.token = r.there ? row / heads : 0;  // its place in the tables
    const int h = r.there ? row - r.token * heads : 0;
    r.key = h >= hq;
    r.head = r.key ? h - hq : h;
    return r;
  };
  auto load = [&](const Row& r) {
    const uint8_t* x = (const uint8_t*)(r.key ? a.rows[1].x : a.rows[0].x);
    const int64_t ld = r.key ? a.rows[1].ld_x : a.rows[0].ld_x, hd = r.key ? a.rows[1].head_x : a.rows[0].head_x;
    if (r.there) load8<DT>(x + ((t0 + r.token) * ld + r.head * hd + part * 8) * kSize, next);
  };
  const int first = blockIdx.y * passes, last = min(first + passes, (n + kSlots - 1) / kSlots);
  Row row = row_of(first);
  load(row);
  const bool norm_q = a.rows[0].weight != nullptr, norm_k = a.rows[1].weight != nullptr;
  for (int i = threadIdx.x; i < D; i += kElemThreads) {
    if (norm_q) weights[0][i] = a.rows[0].weight[i] + a.weight_offset;
    if (norm_k) weights[1][i] = a.rows[1].weight[i] + a.weight_offset;
  }
  for (int e = threadIdx.x; e < tokens * half; e += kElemThreads) {
    const int k = e / half, i = e - k * half;
    const int64_t t = min(t0 + k, a.tokens - 1);
    const int axis = a.rope.axis != nullptr ? min((int)a.rope.axis[i], a.rope.axes - 1) : 0;
    const double turn = (double)a.rope.positions[axis * a.rope.ld_positions + t] * (double)a.rope.inv_freq[i] * 0.15915494309189533577;
    float sine, cosine;
    if constexpr (DT == NVFP4_DTYPE_F32) {
      double s, c;
      sincospi(2.0 * (turn - rint(turn)), &s, &c);
      sine = (float)s;
      cosine = (float)c;
    } else {
      sincospif(2.0f * (float)(turn - rint(turn)), &sine, &cosine);
    }
    const int p = k * dim + (a.rope.interleaved ? 2 * i : i), q = a.rope.interleaved ? p + 1 : p + half;
    cs[p] = cs[q] = cosine;
    sn[p] = -sine;
    sn[q] = sine;
  }
  __syncthreads();
  const bool turned = part * 8 < dim;
  const int partner = (threadIdx.x & (63 & ~(kLanes - 1))) + (!turned ? part : part * 8 < half ? part + half / 8 : part - half / 8);
  for (int pass = first; pass < last; ++pass) {
    const Row now = row;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = next[e];
    if (pass + 1 < last) {
      row = row_of(pass + 1);
      load(row);
    }
    if (now.key ? norm_k : norm_q) {
      float sum = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) sum = fmaf(v[e], v[e], sum);
      // within one ulp; the sum is at least eps, a normal number
      const float f = __builtin_amdgcn_rsqf(head_sum<kLanes>(sum) * (1.0f / D) + a.eps);
      const floatx4* w = reinterpret_cast<const floatx4*>(&weights[now.key][part * 8]);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= f * w[e / 4][e % 4];
    }
    if (dim > 0) {
      const floatx4* c = reinterpret_cast<const floatx4*>(&cs[turned ? now.token * dim + part * 8 : 0]);
      const floatx4* s = reinterpret_cast<const floatx4*>(&sn[turned ? now.token * dim + part * 8 : 0]);
      float other[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) other[e] = a.rope.interleaved ? v[e ^ 1] : __shfl(v[e], partner);
      if (turned) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = fmaf(v[e], c[e / 4][e % 4], other[e] * s[e / 4][e % 4]);
      }
    }
    if (now.there) {
      uint8_t* out = (uint8_t*)(now.key ? a.rows[1].out : a.rows[0].out);
      const int64_t ld = now.key ? a.rows[1].ld_out : a.rows[0].ld_out, hd = now.key ? a.rows[1].head_out : a.rows[0].head_out;
      store8<DT>(out + ((t0 + now.token) * ld + now.head * hd + part * 8) * kSize, v);
    }
  }
}

template <int DT, int D>
void launch(const RopeArgs& a, hipStream_t s) {
  constexpr int kSlots = kElemThreads / (D / 8);
  const int heads = a.rows[0].heads + a.rows[1].heads, dim = a.rope.rotary_dim;
  // Passes of a workgroup: few calls' worth of rows keep all CUs busy one by one; many share the tables' work and the
  // start.  Measured, us, one token and one pass | 1, 2, 4, 8 tokens a workgroup: bf16, 32 + 8 heads of 128, 256 tokens 4.5 |
  // 5.4, 7.1, 10.9; 2048 tokens 14.5 | 12.7, 11.9, 14.1; 16384 tokens 118 | 89, 76, 73.5, 73.4 (4.6 TB/s); 24 + 4 of 256 153 |
  // 110, 95.5, 103, 121; 16 + 4 of 64 31 | 32, 25, 20, 19; float32, 8192 tokens of 32 + 8 of 128 83 | 68, 71, 78.
  const int64_t total = a.tokens * heads / kSlots;
  const int want = total < 1024 ? 1 : DT == NVFP4_DTYPE_F32 ? 3 : total < 16384 ? 5 : 8;
  const int tokens = max(1, min(want * kSlots / heads, dim > 0 ? kTable / dim : 8));
  const int all = (tokens * heads + kSlots - 1) / kSlots;
  const int passes = min(all, max(want, 1 + (all - 1) / 60000));  // the grid's second size stays below 2^16
  const dim3 grid((unsigned)((a.tokens + tokens - 1) / tokens), (unsigned)((all + passes - 1) / passes));
  qk_norm_rope_kernel<DT, D><<<grid, kElemThreads, 0, s>>>(a, tokens, passes);
}

template <int DT>
void launch_dim(const RopeArgs& a, hipStream_t s) {
  if (a.head_dim == 64) launch<DT, 64>(a, s);
  else if (a.head_dim == 128) launch<DT, 128>(a, s);
  else launch<DT, 256>(a, s);
}

}  // namespace

hipError_t launch_qk_norm_rope(const RopeArgs& a, hipStream_t s) {
  if (a.dtype == NVFP4_DTYPE_BF16) launch_dim<NVFP4_DTYPE_BF16>(a, s);
  else launch_dim<NVFP4_DTYPE_F32>(a, s);
  return hipGetLastError();
}

}  // namespace nvfp4
