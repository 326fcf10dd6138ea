// Paged FP8 KV cache: the write (quantization on the way) and the read.
//
// Per row x of D values (one token, one kv head): the scale is the power of
// two 2^e with the least e >= -126 such that max|x| <= 448 * 2^e, and a code
// is the E4M3 byte nearest to x / 2^e.  With a power of two that quotient is
// an exact float32 product (or far below the first midpoint), so one hardware
// conversion -- nearest, ties to even, sign of zero kept -- is the exactly
// rounded answer, and it never has to saturate.  448 = 1.75 * 2^8, so e is
// the exponent of max|x| less 8, and one more when its mantissa exceeds 1.75:
// both come out of one integer addition on the float's bits (scale_byte).
//
// Bound: HBM.  Per token 2 * H * D elements read (written, on a read-back)
// and as many bytes plus 2 H scales written.
//
// The value blocks hold 16 tokens of one dimension in 16 bytes (that is how
// the attention's matrix instructions want them), so a single token's values
// are D bytes 16 apart.  A workgroup takes 16 consecutive rows of one head
// and looks at their slots: a run of 16 rows that fill an aligned block goes
// out as whole 16-byte pieces, transposed through LDS; rows outside such runs
// go out byte by byte.  A run starts anywhere in the rows, so the workgroup
// looks 15 rows to both sides of its own: the run belongs to the workgroup
// that holds its first row.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "device_util.h"
#include "kv_pages.h"

namespace nvfp4 {

namespace {

using namespace dev;

constexpr int kRows = 16;  // rows of one workgroup = tokens of one block

// The exponent byte of the scale for a row whose largest magnitude is a.
// bits + 0x1FFFFF carries into the exponent exactly when the mantissa is
// above 0x600000, i.e. 1.75.
__device__ inline uint32_t scale_byte(float a) {
  const int b = (int)((__float_as_uint(a) + 0x1FFFFFu) >> 23) - 8;
  return (uint32_t)max(b, 1);
}
__device__ inline float scale_value(uint32_t byte) { return __uint_as_float(byte << 23); }

// Which of the 16 rows from t0 on belong to whole blocks.  Lane i of every
// wave looks at row t0 - 15 + i; all lanes get the same answer.
struct Runs {
  int64_t first;     // slot of the run's first row, or -1
  int64_t first_row; // that row
  uint32_t single;   // rows of the window (bit i: t0 + i) to handle one by one
  __device__ Runs(const int64_t* slots, int64_t rows, int64_t t0, int64_t n_slots) {
    const int lane = threadIdx.x & 63;
    const int64_t t = t0 - (kRows - 1) + lane;
    const bool there = t >= 0 && t < rows && lane < 3 * kRows - 1;
    const int64_t s = there ? slots[t] : -1;
    const bool ok = s >= 0 && s < n_slots;
    const int64_t before = __shfl_up(s, 1);
    const uint64_t follows = __ballot(ok && lane > 0 && s == before + 1);
    const bool leads = ok && (s & (kRows - 1)) == 0 && lane < 2 * kRows - 1 &&
                       ((follows >> lane) >> 1 & 0x7FFFu) == 0x7FFFu;
    const uint64_t leaders = __ballot(leads);
    const int o = (int)(s & (kRows - 1));
    const bool covered = ok && lane >= o && ((leaders >> (lane - o)) & 1u);
    single = (uint32_t)(__ballot(ok && !covered) >> (kRows - 1)) & 0xFFFFu;
    // leaders are 16 rows apart at least, so the window holds one at most
    const uint32_t mine = (uint32_t)(leaders >> (kRows - 1)) & 0xFFFFu;
    first = -1;
    first_row = 0;
    if (mine != 0) {
      const int at = __builtin_ctz(mine);
      first = __shfl(s, kRows - 1 + at);
      first_row = t0 + at;
    }
  }
};

// E consecutive elements as floats (E * size a multiple of 8 bytes).
template <int DT, int E>
__device__ inline void load_elems(const uint8_t* p, float v[E]) {
  if constexpr (DT == NVFP4_DTYPE_F32) {
#pragma unroll
    for (int i = 0; i < E; i += 4) {
      const float4 a = *reinterpret_cast<const float4*>(p + 4 * i);
      v[i] = a.x; v[i + 1] = a.y; v[i + 2] = a.z; v[i + 3] = a.w;
    }
  } else {
    uint32_t w[E / 2];
    if constexpr (E == 4) {
      const uint2 a = *reinterpret_cast<const uint2*>(p);
      w[0] = a.x; w[1] = a.y;
    } else {
#pragma unroll
      for (int i = 0; i < E / 2; i += 4) {
        const uint4 a = *reinterpret_cast<const uint4*>(p + 4 * i);
        w[i] = a.x; w[i + 1] = a.y; w[i + 2] = a.z; w[i + 3] = a.w;
      }
    }
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
}

template <int DT, int E>
__device__ inline void store_elems(uint8_t* p, const float v[E]) {
  if constexpr (DT == NVFP4_DTYPE_F32) {
#pragma unroll
    for (int i = 0; i < E; i += 4)
      store_stream16(p + 4 * i, __float_as_uint(v[i]), __float_as_uint(v[i + 1]), __float_as_uint(v[i + 2]),
                     __float_as_uint(v[i + 3]));
  } else if constexpr (E == 4) {
    store_stream8(p, pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
  } else {
#pragma unroll
    for (int i = 0; i < E; i += 8)
      store_stream16(p + 2 * i, pack_bf16x2(v[i], v[i + 1]), pack_bf16x2(v[i + 2], v[i + 3]), pack_bf16x2(v[i + 4], v[i + 5]),
                     pack_bf16x2(v[i + 6], v[i + 7]));
  }
}

// N / 4 dwords from or to consecutive bytes.
template <int W>
__device__ inline void copy_words(uint32_t* to, const uint32_t* from) {
  if constexpr (W == 1) {
    *to = *from;
  } else if constexpr (W == 2) {
    *reinterpret_cast<uint2*>(to) = *reinterpret_cast<const uint2*>(from);
  } else {
    *reinterpret_cast<uint4*>(to) = *reinterpret_cast<const uint4*>(from);
  }
}

// Byte offset of dimensions d.. (d within one 16-group) of token o in a key block.
template <int D>
__device__ inline int key_offset(int o, int d) {
  return (o >> 2) * (4 * D) + (d >> 4) * 64 + (o & 3) * 16 + (d & 15);
}

struct Place {
  uint8_t *codes, *scale;  // of the slot's 16-token block; of the slot
  int o;
  __device__ Place(const KvPages& c, uint8_t* codes_, uint8_t* scales_, int head, int64_t slot) {
    const int ps = 1 << c.page_shift;
    const int64_t page = slot >> c.page_shift;
    const int i = (int)(slot & (ps - 1));
    o = i & (kRows - 1);
    codes = codes_ + page * c.ld_codes + (int64_t)(head * ps + (i - o)) * c.dim;
    scale = scales_ + page * c.ld_scales + (head * ps + i);
  }
};

// One thread: E = D / 16 elements of one of 16 rows; 16 threads a row.
template <int DT, int D>
__global__ __launch_bounds__(256) void kv_pages_write_kernel(KvPages c, const uint8_t* __restrict__ k, int64_t ldk,
                                                             const uint8_t* __restrict__ v, int64_t ldv, int64_t rows,
                                                             const int64_t* __restrict__ slots) {
  constexpr int E = D / 16, W = E / 4, kEsz = DT == NVFP4_DTYPE_BF16 ? 2 : 4;
  __shared__ __attribute__((aligned(16))) uint8_t tile[16 * D];
  const int tid = threadIdx.x, r = tid >> 4, p = tid & 15, head = blockIdx.y;
  const bool values = blockIdx.z != 0;
  const int64_t t0 = (int64_t)blockIdx.x * kRows;
  const uint8_t* const x = (values ? v + (int64_t)head * D * kEsz : k + (int64_t)head * D * kEsz) + p * E * kEsz;
  const int64_t ld = values ? ldv : ldk;
  uint8_t* const codes = values ? c.vc : c.kc;
  uint8_t* const scales = values ? c.vs : c.ks;

  const Runs runs(slots, rows, t0, (int64_t)c.n_pages << c.page_shift);

  // This thread's codes and the row's scale byte.
  auto encode = [&](int64_t row, uint32_t w[W]) {
    float f[E];
    load_elems<DT, E>(x + row * ld, f);
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < E; ++i) a = fmaxf(a, fabsf(f[i]));
#pragma unroll
    for (int off = 8; off > 0; off >>= 1) a = fmaxf(a, __shfl_xor(a, off));
    const uint32_t b = scale_byte(a);
    const float inv = scale_value(254u - b);
#pragma unroll
    for (int i = 0; i < W; ++i) {
      uint32_t q = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(f[4 * i] * inv, f[4 * i + 1] * inv, 0, false);
      w[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(f[4 * i + 2] * inv, f[4 * i + 3] * inv, (int)q, true);
    }
    return b;
  };

  if (runs.first >= 0) {
    uint32_t w[W];
    const uint32_t b = encode(runs.first_row + r, w);
    const Place at(c, codes, scales, head, runs.first);
    if (p == 0) at.scale[r] = (uint8_t)b;
    if (!values) {
      copy_words<W>(reinterpret_cast<uint32_t*>(tile + key_offset<D>(r, p * E)), w);
      __syncthreads();
      uint32_t o[W];
      copy_words<W>(o, reinterpret_cast<const uint32_t*>(tile + tid * E));
      copy_words<W>(reinterpret_cast<uint32_t*>(at.codes + tid * E), o);
    } else {
      copy_words<W>(reinterpret_cast<uint32_t*>(tile + r * D + p * E), w);
      __syncthreads();
      if (tid < D) {  // 16 tokens of dimension tid
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint8_t* s = tile + 4 * i * D + tid;
          o[i] = s[0] | (uint32_t)s[D] << 8 | (uint32_t)s[2 * D] << 16 | (uint32_t)s[3 * D] << 24;
        }
        *reinterpret_cast<uint4*>(at.codes + tid * 16) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
  // Rows on their own.  (All 16 threads of a row take the branch together.)
  if (runs.single >> r & 1u) {
    uint32_t w[W];
    const uint32_t b = encode(t0 + r, w);
    const Place at(c, codes, scales, head, slots[t0 + r]);
    if (p == 0) *at.scale = (uint8_t)b;
    if (!values) {
      copy_words<W>(reinterpret_cast<uint32_t*>(at.codes + key_offset<D>(at.o, p * E)), w);
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) at.codes[(p * E + i) * 16 + at.o] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
    }
  }
}

template <int DT, int D>
__global__ __launch_bounds__(256) void kv_pages_read_kernel(KvPages c, int64_t rows, const int64_t* __restrict__ slots,
                                                            uint8_t* __restrict__ k, int64_t ldk, uint8_t* __restrict__ v,
                                                            int64_t ldv) {
  constexpr int E = D / 16, W = E / 4, kEsz = DT == NVFP4_DTYPE_BF16 ? 2 : 4;
  __shared__ __attribute__((aligned(16))) uint8_t tile[16 * (D + 4)];
  const int tid = threadIdx.x, r = tid >> 4, p = tid & 15, head = blockIdx.y;
  const bool values = blockIdx.z != 0;
  const int64_t t0 = (int64_t)blockIdx.x * kRows;
  uint8_t* const x = (values ? v + (int64_t)head * D * kEsz : k + (int64_t)head * D * kEsz) + p * E * kEsz;
  const int64_t ld = values ? ldv : ldk;
  uint8_t* const codes = values ? c.vc : c.kc;
  uint8_t* const scales = values ? c.vs : c.ks;
  const int64_t n_slots = (int64_t)c.n_pages << c.page_shift;

  // fl32(code * scale), rounded once more for bf16 (the product is exact
  // unless it is subnormal).
  auto emit = [&](int64_t row, const uint32_t w[W], uint32_t b) {
    const float s = scale_value(b);
    float f[E];
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const f32x2_t lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], true);
      f[4 * i] = lo.x * s; f[4 * i + 1] = lo.y * s; f[4 * i + 2] = hi.x * s; f[4 * i + 3] = hi.y * s;
    }
    store_elems<DT, E>(x + row * ld, f);
  };

  if (!values) {  // a key row is E-byte pieces wherever it lies
    const int64_t slot = t0 + r < rows ? slots[t0 + r] : -1;
    if (slot < 0 || slot >= n_slots) return;
    const Place at(c, codes, scales, head, slot);
    uint32_t w[W];
    copy_words<W>(w, reinterpret_cast<const uint32_t*>(at.codes + key_offset<D>(at.o, p * E)));
    emit(t0 + r, w, *at.scale);
    return;
  }
  const Runs runs(slots, rows, t0, n_slots);
  if (runs.first >= 0) {
    const Place at(c, codes, scales, head, runs.first);
    const uint32_t b = at.scale[r];
    if (tid < D) {
      const uint4 q = *reinterpret_cast<const uint4*>(at.codes + tid * 16);
      const uint32_t o[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int i = 0; i < 16; ++i) tile[i * (D + 4) + tid] = (uint8_t)(o[i >> 2] >> (8 * (i & 3)));
    }
    __syncthreads();
    uint32_t w[W];
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = *reinterpret_cast<const uint32_t*>(tile + r * (D + 4) + p * E + 4 * i);
    emit(runs.first_row + r, w, b);
  }
  if (runs.single >> r & 1u) {
    const Place at(c, codes, scales, head, slots[t0 + r]);
    uint32_t w[W] = {};
#pragma unroll
    for (int i = 0; i < E; ++i) w[i >> 2] |= (uint32_t)at.codes[(p * E + i) * 16 + at.o] << (8 * (i & 3));
    emit(t0 + r, w, *at.scale);
  }
}

// f with the dtype and head_dim as compile-time constants (checked by the ABI layer).
template <class F>
void for_types(int dtype, int dim, F f) {
  auto with = [&](auto dt) {
    if (dim == 64) f(dt, std::integral_constant<int, 64>());
    else if (dim == 128) f(dt, std::integral_constant<int, 128>());
    else f(dt, std::integral_constant<int, 256>());
  };
  if (dtype == NVFP4_DTYPE_BF16) with(std::integral_constant<int, NVFP4_DTYPE_BF16>());
  else with(std::integral_constant<int, NVFP4_DTYPE_F32>());
}

}  // namespace

hipError_t launch_kv_pages_write(const KvPages& c, const void* k, int64_t ld_k, const void* v, int64_t ld_v, int dtype,
                                 int64_t rows, const int64_t* slots, hipStream_t s) {
  const int64_t esz = dtype == NVFP4_DTYPE_BF16 ? 2 : 4;
  const dim3 grid((unsigned)((rows + kRows - 1) / kRows), c.heads, 2);
  for_types(dtype, c.dim, [&](auto dt, auto d) {
    kv_pages_write_kernel<dt(), d()><<<grid, 256, 0, s>>>(c, (const uint8_t*)k, ld_k * esz, (const uint8_t*)v, ld_v * esz, rows,
                                                          slots);
  });
  return hipGetLastError();
}

hipError_t launch_kv_pages_read(const KvPages& c, int64_t rows, const int64_t* slots, void* k, int64_t ld_k, void* v,
                                int64_t ld_v, int dtype, hipStream_t s) {
  const int64_t esz = dtype == NVFP4_DTYPE_BF16 ? 2 : 4;
  const dim3 grid((unsigned)((rows + kRows - 1) / kRows), c.heads, 2);
  for_types(dtype, c.dim, [&](auto dt, auto d) {
    kv_pages_read_kernel<dt(), d()><<<grid, 256, 0, s>>>(c, rows, slots, (uint8_t*)k, ld_k * esz, (uint8_t*)v, ld_v * esz);
  });
  return hipGetLastError();
}

}  // namespace nvfp4
