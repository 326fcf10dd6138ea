// The short causal convolution along the tokens of each channel:
//     y[t] = act(bias + sum_{j < W} w[j] in[t - W + 1 + j]),  W = 2, 3 or 4,
// over a batch of sequences; the last W - 1 inputs of each are kept in a state.
// Bound: HBM (every element read and written once; W fmas per element).
//
// A thread takes 8 channels (16 bytes of bf16) and a run of neighbouring tokens,
// the last W - 1 inputs in registers, so that an input is read once per run
// (and W - 1 more at its start, from the cache).  Neighbouring threads take
// neighbouring channels.
//
// The state is read and written in one launch without a race: what needs a
// sequence's old state -- its first W - 1 tokens and the new state of a
// sequence shorter than W - 1 -- is done by one thread per channel group, the
// one whose run holds the sequence's first token.  It goes past the end of
// its run for that where it has to, and the run that such tokens lie in leaves
// them out.  The new state comes from x, which nobody writes.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_util.h"
#include "e4m3.h"
#include "internal.h"
#include "layer_ops.h"

namespace nvfp4 {

namespace {

using namespace dev;

// 8 elements of type DT as they lie in memory.
template <int DT>
struct Eight;
template <>
struct Eight<NVFP4_DTYPE_BF16> {
  u32x4 w;
  __device__ static Eight load(const uint8_t* p) { return {*reinterpret_cast<const u32x4*>(p)}; }
  __device__ void store(uint8_t* p) const { *reinterpret_cast<u32x4*>(p) = w; }
  __device__ void floats(float v[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  __device__ static Eight of(const float v[8]) {
    return {u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])}};
  }
  __device__ void stream(uint8_t* p) const { store_stream16(p, w[0], w[1], w[2], w[3]); }
};
template <>
struct Eight<NVFP4_DTYPE_F32> {
  u32x4 w, h;
  __device__ static Eight load(const uint8_t* p) {
    return {*reinterpret_cast<const u32x4*>(p), *reinterpret_cast<const u32x4*>(p + 16)};
  }
  __device__ void store(uint8_t* p) const {
    *reinterpret_cast<u32x4*>(p) = w;
    *reinterpret_cast<u32x4*>(p + 16) = h;
  }
  __device__ void floats(float v[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = __uint_as_float(w[i]);
      v[4 + i] = __uint_as_float(h[i]);
    }
  }
  __device__ static Eight of(const float v[8]) {
    Eight r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r.w[i] = __float_as_uint(v[i]);
      r.h[i] = __float_as_uint(v[4 + i]);
    }
    return r;
  }
  __device__ void stream(uint8_t* p) const {
    store_stream16(p, w[0], w[1], w[2], w[3]);
    store_stream16(p + 16, h[0], h[1], h[2], h[3]);
  }
};

// u * sigmoid(u).  For bf16 the shared silu: its error, up to 30 * 2^-24 of the result at u = -30, since the exponent's product
// is rounded, stays far below half a step of 2^-8.  For float32 the exponent keeps its remainder, and a quotient below
// 2^-126 meets u before it is rounded: a few 2^-24 everywhere.
template <int DT>
__device__ inline float activation(float u) {
  if constexpr (DT == NVFP4_DTYPE_BF16) {
    return silu(u);
  } else {
    const ExpNeg e = exp_neg(fminf(fabsf(u), 200.0f));  // beyond 200 the result is u or 0, and infinities stay out
    if (e.tiny) return u >= 0.0f ? u : u * e.es * 0x1p-64f;
    return u * div_small(u >= 0.0f ? 1.0f : e.es, 1.0f + e.es);
  }
}

// First row of sequence b (b = batch: the end of the last).
__device__ inline int64_t start_of(const nvfp4_conv& c, int64_t each, int64_t b) {
  if (c.starts == nullptr) return b * each;
  return min(max((int64_t)c.starts[b], (int64_t)0), c.tokens);
}

template <int DT, int W>
__global__ __launch_bounds__(kElemThreads) void causal_conv_kernel(const nvfp4_conv c, int64_t each, int run, int64_t threads) {
  constexpr int kBytes = DT == NVFP4_DTYPE_BF16 ? 16 : 32, kOld = W - 1, kAhead = 4;
  const int64_t id = (int64_t)blockIdx.x * kElemThreads + threadIdx.x;
  if (id >= threads) return;
  const int64_t chunks = c.channels / 8, chunk = id % chunks;
  const int64_t r0 = id / chunks * run, r1 = min(r0 + run, c.tokens);
  const uint8_t* x = (const uint8_t*)c.x + chunk * kBytes;
  uint8_t* y = (uint8_t*)c.y + chunk * kBytes;
  const int64_t ldx = c.ld_x * (kBytes / 8), ldy = c.ld_y * (kBytes / 8);

  float w[8][W], bias[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
#pragma unroll
    for (int j = 0; j < W; ++j) w[e][j] = c.weight[(chunk * 8 + e) * W + j];
    bias[e] = c.bias != nullptr ? c.bias[chunk * 8 + e] : 0.0f;
  }

  // the last sequence that begins at r0 or before
  int64_t b = 0;
  for (int64_t lo = 0, hi = c.batch - 1; lo <= hi;) {
    const int64_t mid = (lo + hi) / 2;
    if (start_of(c, each, mid) <= r0) {
      b = mid;
      lo = mid + 1;
    } else {
      hi = mid - 1;
    }
  }
  for (; b < c.batch; ++b) {
    const int64_t first = start_of(c, each, b), last = start_of(c, each, b + 1);
    if (first >= r1) break;
    if (last <= first || last <= r0) continue;
    // this thread's tokens of the sequence: its first kOld ones belong to the run that holds the first
    const bool whole = first >= r0;
    int64_t t = whole ? first : max(r0, min(first + kOld, last));
    const int64_t end = whole ? min(max(r1, first + kOld), last) : min(r1, last);
    if (t >= end) continue;
    float in[W][8];  // in[j]: the input W - 1 - j tokens ago
    if (whole) {
      Eight<DT> old[kOld] = {};
      const int64_t slot = c.state == nullptr ? -1 : c.slots != nullptr ? (int64_t)c.slots[b] : b;
      uint8_t* st = (uint8_t*)c.state + slot * c.ld_state * (kBytes / 8) + chunk * kBytes;
      if (slot >= 0 && slot < c.n_states) {
        if (c.fresh == nullptr || c.fresh[b] == 0) {
#pragma unroll
          for (int j = 0; j < kOld; ++j) old[j] = Eight<DT>::load(st + j * chunks * kBytes);
        }
#pragma unroll
        for (int j = 0; j < kOld; ++j) {
          const int64_t at = last - first - kOld + j;  // token of the sequence, negative: an old input
          Eight<DT> keep = {};
          if (at >= 0) {
            keep = Eight<DT>::load(x + (first + at) * ldx);
          } else {
#pragma unroll
            for (int i = 0; i < kOld; ++i)
              if (i == at + kOld) keep = old[i];
          }
          keep.store(st + j * chunks * kBytes);
        }
      }
#pragma unroll
      for (int j = 0; j < kOld; ++j) old[j].floats(in[j]);
    } else {
#pragma unroll
      for (int j = 0; j < kOld; ++j) Eight<DT>::load(x + (t - kOld + j) * ldx).floats(in[j]);
    }
    auto token = [&](const Eight<DT>& now, int64_t at) {
      now.floats(in[W - 1]);
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float u = bias[e];
#pragma unroll
        for (int j = 0; j < W; ++j) u = fmaf(w[e][j], in[j][e], u);
        v[e] = c.silu ? activation<DT>(u) : u;
      }
      Eight<DT>::of(v).stream(y + at * ldy);
#pragma unroll
      for (int j = 0; j < kOld; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) in[j][e] = in[j + 1][e];
    };
    for (; t + kAhead <= end; t += kAhead) {
      Eight<DT> now[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) now[u] = Eight<DT>::load(x + (t + u) * ldx);
#pragma unroll
      for (int u = 0; u < kAhead; ++u) token(now[u], t + u);
    }
    for (; t < end; ++t) token(Eight<DT>::load(x + t * ldx), t);
  }
}

// One token of each sequence: a thread per sequence and 8 channels.  Nothing
// waits for the slot but the state itself.  64 sequences of 10240 channels: 5.8 us, the general kernel 8.3.
template <int DT, int W>
__global__ __launch_bounds__(kElemThreads) void causal_conv_step_kernel(const nvfp4_conv c) {
  constexpr int kBytes = DT == NVFP4_DTYPE_BF16 ? 16 : 32, kOld = W - 1;
  const int64_t id = (int64_t)blockIdx.x * kElemThreads + threadIdx.x;
  const int64_t chunks = c.channels / 8, b = id / chunks, chunk = id - b * chunks;
  if (b >= c.batch) return;
  const int64_t slot = c.state == nullptr ? -1 : c.slots != nullptr ? (int64_t)c.slots[b] : b;
  const bool fresh = c.fresh != nullptr && c.fresh[b] != 0;
  const Eight<DT> now = Eight<DT>::load((const uint8_t*)c.x + b * c.ld_x * (kBytes / 8) + chunk * kBytes);
  float w[8 * W], bias[8];
#pragma unroll
  for (int i = 0; i < 8 * W; i += 4) {
    const float4 f = reinterpret_cast<const float4*>(c.weight + chunk * 8 * W)[i / 4];
    w[i] = f.x; w[i + 1] = f.y; w[i + 2] = f.z; w[i + 3] = f.w;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) bias[e] = c.bias != nullptr ? c.bias[chunk * 8 + e] : 0.0f;
  const bool kept = slot >= 0 && slot < c.n_states;
  uint8_t* st = (uint8_t*)c.state + slot * c.ld_state * (kBytes / 8) + chunk * kBytes;
  Eight<DT> old[kOld] = {};
  if (kept && !fresh) {
#pragma unroll
    for (int j = 0; j < kOld; ++j) old[j] = Eight<DT>::load(st + j * chunks * kBytes);
  }
  float in[W][8], v[8];
#pragma unroll
  for (int j = 0; j < kOld; ++j) old[j].floats(in[j]);
  now.floats(in[kOld]);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float u = bias[e];
#pragma unroll
    for (int j = 0; j < W; ++j) u = fmaf(w[e * W + j], in[j][e], u);
    v[e] = c.silu ? activation<DT>(u) : u;
  }
  Eight<DT>::of(v).stream((uint8_t*)c.y + b * c.ld_y * (kBytes / 8) + chunk * kBytes);
  if (kept) {
#pragma unroll
    for (int j = 0; j < kOld; ++j) (j + 1 < kOld ? old[j + 1] : now).store(st + j * chunks * kBytes);
  }
}

template <int DT, int W>
void launch(const nvfp4_conv& c, hipStream_t s) {
  const int64_t each = c.tokens / c.batch, chunks = c.channels / 8;
  // Longer runs read fewer inputs twice, shorter ones keep more threads busy.  Measured, bf16, us with runs of 4, 8, 16, 32
  // (C = 10240 unless said): 64 rows 8.3, 8.7, 11.9, 18.5; 512 rows 11.3, 11.0, 13.5, 19.9; 2048 rows 28.2, 24.7, 22.7,
  // 26.3; 31500 rows of 1024 37.3, 33.0, 32.7, 33.3; 8192 rows 110, 88, 79, 81; 31500 rows 417, 332, 293, 269 (4.8 TB/s).
  const int64_t places = c.tokens * chunks;
  const bool step = c.starts == nullptr && each == 1 && places < (int64_t)1 << 31;  // its threads fit a grid
  const int run = places >= (int64_t)1 << 25 ? 32 : places >= 1 << 21 ? 16 : places >= 1 << 19 ? 8 : 4;
  const int64_t threads = step ? places : (c.tokens + run - 1) / run * chunks;
  const unsigned grid = (unsigned)((threads + kElemThreads - 1) / kElemThreads);
  if (step) causal_conv_step_kernel<DT, W><<<grid, kElemThreads, 0, s>>>(c);
  else causal_conv_kernel<DT, W><<<grid, kElemThreads, 0, s>>>(c, each, run, threads);
}

template <int DT>
void launch_width(const nvfp4_conv& c, hipStream_t s) {
  if (c.width == 2) launch<DT, 2>(c, s);
  else if (c.width == 3) launch<DT, 3>(c, s);
  else launch<DT, 4>(c, s);
}

}  // namespace

hipError_t launch_causal_conv(const nvfp4_conv& c, int dtype, hipStream_t s) {
  if (dtype == NVFP4_DTYPE_BF16) launch_width<NVFP4_DTYPE_BF16>(c, s);
  else launch_width<NVFP4_DTYPE_F32>(c, s);
  return hipGetLastError();
}

}  // namespace nvfp4
