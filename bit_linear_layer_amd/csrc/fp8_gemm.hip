// Matrix product of E4M3 operands with a float32 scale per block of 128 columns
// (activations: per row, weights: per 128 rows):
//     out[m, n] = sum_b sa[m, b] sw[n / 128, b] sum_{k in b} a[m, k] w[n, k].
// One block of 128 is the depth of four 16x16x32 matrix instructions, so a tile's
// sum over a block comes out of the matrix unit by itself and enters the
// running sum with one fma per output: out += (sa sw) tmp.
//
// The weight is the instruction's first operand, the activations its second:
// a lane then holds one token (lane % 16) and four consecutive columns, needs
// one activation scale per 16-token tile and stores its columns side by side.
//
// Products are exact and sums float32: the codes become fp16 (exact) and go through
// four 16x16x32 fp16 instructions a block.  The 8-bit matrix instructions (16x16x128 and
// 16x16x32 alike) cut the products of 8 neighbouring k to multiples of 2^-13 of the
// largest's power of two before they add them (measured): a small sum of
// large products loses up to 2^-10 of their magnitudes, so they are used only where the caller allows it.
// Which k meets which inside a block is free as long as both operands agree: lane
// group g = lane / 16 takes the 16-byte pieces g and g + 4 of its row.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

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

// The s-th quarter of a fragment as an operand of the matrix instruction.
__device__ inline half8 quarter(const Frag& f, int s) { return half_of(f.p[s >> 1][2 * (s & 1)], f.p[s >> 1][2 * (s & 1) + 1]); }

// The 16 x 16 sums over one block of 128.
__device__ inline floatx4 block_product(const Frag& w, const Frag& x) {
  floatx4 c = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int s = 0; s < 4; ++s) c = __builtin_amdgcn_mfma_f32_16x16x32_f16(quarter(w, s), quarter(x, s), c, 0, 0, 0);
  return c;
}

// Where the product of two scales is beyond float32's range, sums that are not large still are not: 0 gives 0, and 2^-18
// times 2^140 gives 2^122.  Such a product leaves an infinity or NaN in the sums, so that the loops over blocks need not
// look for it; a wave that finds one in its sums over blocks [b0, b1) works out anew, from memory, the tokens with such scales.
// Both scales are at least 1 there, so that 2^-64 of each is exact.
// m: the wave's first token; w_row(i): the lane's row of weight fragment i; n: one of the wave's columns.
template <int FN, int FM, typename Rows>
__device__ inline void mend_large_scales(const Fp8GemmArgs& p, floatx4 (&acc)[FN][FM], int b0, int b1, int m, int n, Rows w_row) {
  float any = 0.0f;
#pragma unroll
  for (int i = 0; i < FN; ++i)
#pragma unroll
    for (int j = 0; j < FM; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) any = fmaf(acc[i][j][r], 0.0f, any);
  if (__ballot(any != 0.0f) == 0) return;  // NaN
  const int li = threadIdx.x & 15, lg = (threadIdx.x & 63) >> 4;
  const float* sw = p.w.scales + (int64_t)(min(n, p.N - 1) / 128) * p.w.scale_row;
  auto load = [&](const Fp8Mat& q, int row, int b) {
    Frag f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int at = (lg + 4 * h) * 16;
      f.p[h] = u32x4{0u, 0u, 0u, 0u};
      if (b * 128 + at < p.K) f.p[h] = *reinterpret_cast<const u32x4*>(q.codes + (int64_t)row * q.ld_codes + b * q.code_block + at);
    }
    return f;
  };
#pragma unroll
  for (int j = 0; j < FM; ++j) {
    const int row = min(m + j * 16 + li, p.M - 1);
    const float* sx = p.a.scales + (int64_t)row * p.a.scale_row;
    bool mine = false;
    for (int b = b0; b < b1; ++b) mine = mine || __builtin_isinf(sx[b * p.a.scale_block] * sw[b * p.w.scale_block]);
    if (__ballot(mine) == 0) continue;
    floatx4 sum[FN] = {};
    for (int b = b0; b < b1; ++b) {
      const float u = sx[b * p.a.scale_block], v = sw[b * p.w.scale_block], s = u * v;
      const bool inf = __builtin_isinf(s);
      const float sc = inf ? (u * 0x1p-64f) * (v * 0x1p-64f) : s, up = inf ? 0x1p64f : 1.0f;
      const Frag x = load(p.a, row, b);
#pragma unroll
      for (int i = 0; i < FN; ++i) {
        const floatx4 t = block_product(load(p.w, min(w_row(i), p.N - 1), b), x);
#pragma unroll
        for (int r = 0; r < 4; ++r) sum[i][r] = fmaf(t[r] * sc * up, up, sum[i][r]);
      }
    }
#pragma unroll
    for (int i = 0; i < FN; ++i) acc[i][j] = mine ? sum[i] : acc[i][j];
  }
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

// Products with few tokens, or of too few tiles to fill the chip: bound by the
// weight's bytes up to about 32 tokens, beyond by the copies into LDS and the conversions and products, in nearly equal
// parts.  Measured, us, with the join | without the copies | without the products: 3 x 34816 x 5120 38 | 28 | 37; 16 x 5120 x
// 17408 24 | 20 | 24; 32 x 34816 x 5120 44 | 36 | 43; 64 x 34816 x 5120 58 | 47 | 54; 128 x 34816 x 5120 74 | 63 | 68; 200 x 5120 x
// 17408 57 | 51 | 47, the join 7.5 of them; 256 x 5120 x 17408 64 | 56 | 50.  256 workgroups of 8 waves, one per CU, share the
// line of all (tile, block of 128) steps evenly, tile by tile; a workgroup's copies
// run D steps ahead of its products, across the ends of tiles, so that the
// stream from memory never drains.  A tile whose steps lie in one workgroup is stored; of one that a
// cut divides each workgroup leaves its float32 sums in the workspace, and
// fp8_join_kernel adds them in the order of the blocks: the result depends on the sizes only.
//
// A stage in LDS holds the weight's and the activations' rows of one block (128
// bytes each, 16-byte pieces XOR-swizzled by the row so that fragment reads are free of bank
// conflicts) and the activations' scales, all by LDS DMA.  Rows behind the last
// and pieces behind K lie behind the descriptors' ranges: such lanes write zeros.
// One barrier per step certifies the next step's stage and frees its own, whose fragments
// are in registers by then: the copies D steps ahead go there.
template <int FN, int FM, int WN, int WM, int D>
struct Ring {
  static constexpr int TN = FN * WN * 16, TM = FM * WM * 16;
  static constexpr int kW = TN * 128, kX = TM * 128;
  static constexpr int NS = (TM + 63) / 64;                  // waves that copy 64 scales
  static constexpr int CW = TN / 64, CX = TM / 64;           // copies of every wave
  static constexpr int XR = TM / 8 % 8;                      // waves that copy one more group of activation rows
  static constexpr int kBase = CW + CX;
  // Non-temporal weights.  Measured, us, without | with: 3 x 34816 x 5120 43.2 | 38.2, 16 x 5120 x 17408 26.4 | 24.9, 32 x 34816 x
  // 5120 48.7 | 43.6, 64 x 34816 x 5120 58.0 | 59.2, 128 x 34816 x 5120 74.8 | 76.0, 200 x 5120 x 17408 56.6 | 59.2.
  static constexpr int kHint = TM <= 32 ? 2 : 0;
  static constexpr int kStage = kW + kX + NS * 256;
  static_assert(WN * WM == 8 && TN % 64 == 0 && 128 % TN == 0 && XR + NS <= 8 && D * kStage <= 160 * 1024, "the copies' shares");
  static_assert((D - 1) * (kBase + 1) < 64, "vmcnt's range");
};

constexpr int kRingGroups = 256;

// The steps of workgroup g: [first, last) of the line of all.
struct Share {
  int64_t first, last;
  __host__ __device__ Share(int64_t steps, int groups, int g)
      : first(steps * g / groups), last(steps * (g + 1) / groups) {}
};

template <int FN, int FM, int WN, int WM, int D, int OUT>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2)))
void fp8_ring_kernel(const Fp8GemmArgs p, int tiles_m, int tiles_n, float* __restrict__ partial) {
  using T = Ring<FN, FM, WN, WM, D>;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wn = wave / WM, wm = wave % WM, li = lane & 15, lg = lane >> 4;
  const int blocks = (p.K + 127) / 128;
  const Share mine((int64_t)tiles_m * tiles_n * blocks, gridDim.x, blockIdx.x);

  // copies: lane l brings piece l % 8 (swizzled) of row l / 8 of a group of 8 rows
  const int q = lane >> 3, piece = ((lane & 7) ^ q) * 16;
  const int ldw = (int)p.w.ld_codes, lda = (int)p.a.ld_codes;
  constexpr int kNowhere = (int)0x80000000;
  int tile = (int)(mine.first / blocks), block = (int)(mine.first - (int64_t)tile * blocks);
  const int steps = (int)(mine.last - mine.first);
  // the copies' place in the line, D steps ahead of the products'
  int to_tile = tile, to_block = block, to_step = 0;
  i32x4 rw;
  const uint8_t* xa;
  uint32_t x_bytes;
  const float* sa;
  auto enter = [&]() __attribute__((always_inline)) {
    const int tn = to_tile / tiles_m, n0 = tn * T::TN, m0 = (to_tile - tn * tiles_m) * T::TM;
    rw = buffer_rsrc(p.w.codes + (int64_t)n0 * ldw, (uint32_t)(min(T::TN, p.N - n0) * ldw));
    xa = p.a.codes + (int64_t)m0 * lda;
    x_bytes = (uint32_t)(min(T::TM, p.M - m0) * lda);
    sa = p.a.scales + (int64_t)min(m0 + max(wave - (8 - T::NS), 0) * 64 + lane, p.M - 1) * p.a.scale_row;
  };
  auto copy = [&](uint8_t* stage) __attribute__((always_inline)) {
    const int k = to_block * 128;
    const bool there = k + piece < p.K;
    const i32x4 rx = buffer_rsrc(xa + to_block * p.a.code_block, x_bytes);
#pragma unroll
    for (int c = 0; c < T::CW; ++c)
      llvm_amdgcn_raw_buffer_load_lds(rw, (lds_u32_ptr)(stage + (wave * T::CW + c) * 1024), 16,
                                      there ? ((wave * T::CW + c) * 8 + q) * ldw + piece : kNowhere, k, 0, T::kHint);
#pragma unroll
    for (int c = 0; c < T::CX; ++c)
      llvm_amdgcn_raw_buffer_load_lds(rx, (lds_u32_ptr)(stage + T::kW + (wave * T::CX + c) * 1024), 16,
                                      there ? ((wave * T::CX + c) * 8 + q) * lda + piece : kNowhere, 0, 0, 0);
    if (wave < T::XR)
      llvm_amdgcn_raw_buffer_load_lds(rx, (lds_u32_ptr)(stage + T::kW + (8 * T::CX + wave) * 1024), 16,
                                      there ? ((8 * T::CX + wave) * 8 + q) * lda + piece : kNowhere, 0, 0, 0);
    if (wave >= 8 - T::NS)
      __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) uint32_t*)(sa + (int64_t)to_block * p.a.scale_block),
                                       (lds_u32_ptr)(stage + T::kW + T::kX + (wave - (8 - T::NS)) * 256), 4, 0, 0);
    if (to_step + 1 < steps) {  // behind the last step the last one is copied again
      ++to_step;
      if (++to_block == blocks) {
        to_block = 0;
        ++to_tile;
        enter();
      }
    }
  };

  enter();
#pragma unroll
  for (int d = 0; d < D; ++d) copy(smem + d * T::kStage);
  floatx4 acc[FN][FM];
  auto clear = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
      for (int j = 0; j < FM; ++j) acc[i][j] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
  };
  clear();
  const int key = li & 7;
  const bool vec = p.ld_out % 4 == 0 && (uintptr_t)p.out % (OUT == NVFP4_DTYPE_BF16 ? 8 : 16) == 0;
  int begun = block, stage = 0;  // begun: the tile's first block of this workgroup
  const bool extra = wave < T::XR || wave >= 8 - T::NS;
  auto landed = [&](auto sets) __attribute__((always_inline)) {  // all but the last `sets` steps' copies, in every wave
    if (extra) wait_vmem<decltype(sets)::value * (T::kBase + 1)>();
    else wait_vmem<decltype(sets)::value * T::kBase>();
    barrier_lds();
    __builtin_amdgcn_s_waitcnt(0xC07F);  // the barrier's lgkmcnt(0) again, seen by the compiler's own wait insertion
  };
  int n0, m0;
  const __attribute__((address_space(4))) float* sw;
  auto begin_tile = [&]() __attribute__((always_inline)) {
    const int tn = tile / tiles_m;
    n0 = tn * T::TN;
    m0 = (tile - tn * tiles_m) * T::TM;
    sw = (const __attribute__((address_space(4))) float*)(p.w.scales + (int64_t)(n0 / 128) * p.w.scale_row);
  };
  begin_tile();
  float next_s = sw[block * p.w.scale_block];
  auto frag = [&](const uint8_t* st, int row) __attribute__((always_inline)) {
    Frag f;
#pragma unroll
    for (int h = 0; h < 2; ++h) f.p[h] = *reinterpret_cast<const u32x4*>(st + row * 128 + (((lg + 4 * h) ^ key) << 4));
    return f;
  };
  auto scale_at = [&](const uint8_t* st, int j) __attribute__((always_inline)) {
    return *reinterpret_cast<const float*>(st + T::kW + T::kX + ((wm * FM + j) * 16 + li) * 4);
  };
  Frag w[FN], x[FM];
  float sc[FM];
  landed(std::integral_constant<int, D - 1>{});
#pragma unroll
  for (int i = 0; i < FN; ++i) w[i] = frag(smem, (wn * FN + i) * 16 + li);
#pragma unroll
  for (int j = 0; j < FM; ++j) x[j] = frag(smem, T::TN + (wm * FM + j) * 16 + li);
#pragma unroll
  for (int j = 0; j < FM; ++j) sc[j] = scale_at(smem, j);
  // A step's fragments are in registers when it begins; the next step's are read beside its products, each
  // activation fragment into the place of the one just used.
  for (int step = 0; step < steps; ++step) {
    landed(std::integral_constant<int, D - 2>{});
    const float s = next_s;
    const int next_stage = stage == D - 1 ? 0 : stage + 1;
    const uint8_t* nst = smem + next_stage * T::kStage;
    Frag next_w[FN];
    float now_sc[FM];
    floatx4 t[2][FN];
    auto add = [&](int j) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[i][j][r] = fmaf(t[j & 1][i][r], now_sc[j], acc[i][j][r]);
    };
#pragma unroll
    for (int j = 0; j < FM; ++j) now_sc[j] = sc[j] * s;
#pragma unroll
    for (int j = 0; j < FM; ++j) {
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < FN; ++i) t[j & 1][i] = block_product(w[i], x[j]);
      if (j == 0) {
#pragma unroll
        for (int i = 0; i < FN; ++i) next_w[i] = frag(nst, (wn * FN + i) * 16 + li);
      }
      x[j] = frag(nst, T::TN + (wm * FM + j) * 16 + li);
      sc[j] = scale_at(nst, j);
      if (j == 0) copy(smem + stage * T::kStage);  // every wave has this step's fragments
      if (j > 0) add(j - 1);
    }
    __builtin_amdgcn_sched_barrier(0);
    add(FM - 1);
#pragma unroll
    for (int i = 0; i < FN; ++i) w[i] = next_w[i];
    stage = next_stage;
    ++block;
    const bool ends = block == blocks || step + 1 == steps;
    if (ends) {
      mend_large_scales(p, acc, begun, block, m0 + wm * FM * 16, n0, [&](int i) { return n0 + (wn * FN + i) * 16 + li; });
      if (block == blocks && begun == 0) {
#pragma unroll
        for (int j = 0; j < FM; ++j) {
          const int m = m0 + (wm * FM + j) * 16 + li;
#pragma unroll
          for (int i = 0; i < FN; ++i) {
            const int n = n0 + (wn * FN + i) * 16 + 4 * lg;
            if (m < p.M) store4<OUT>(p.out, (int64_t)m * p.ld_out + n, acc[i][j], p.N - n, vec);
          }
        }
      } else {  // the first slot: of a tile that an earlier workgroup began; the second: of one that this one begins
        float* to = partial + ((int64_t)blockIdx.x * 2 + (begun == 0)) * (T::TN * T::TM);
#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
          for (int j = 0; j < FM; ++j)
            *reinterpret_cast<floatx4*>(to + (((wave * FN + i) * FM + j) * 64 + lane) * 4) = acc[i][j];
      }
      clear();
      begun = block = 0;
      ++tile;
      if (step + 1 < steps) begin_tile();
    }
    if (step + 1 < steps) next_s = sw[block * p.w.scale_block];
  }
  wait_vmem<0>();  // no copy may land after the workgroup's LDS is given away
}

// The sums of tiles that more than one workgroup worked on; a thread per four columns of a token.
template <int FN, int FM, int WN, int WM, int D, int OUT>
__global__ __launch_bounds__(256) void fp8_join_kernel(const Fp8GemmArgs p, int tiles_m, int groups, int64_t steps,
                                                       const float* __restrict__ partial) {
  using T = Ring<FN, FM, WN, WM, D>;
  const int tile = blockIdx.x, blocks = (p.K + 127) / 128;
  const int64_t lo = (int64_t)tile * blocks, hi = lo + blocks;
  // the workgroup of a step is the largest g with steps * g / groups <= step
  auto group_of = [&](int64_t step) {
    int g = (int)((step + 1) * groups / steps);
    g = min(g, groups - 1);
    while (g > 0 && Share(steps, groups, g).first > step) --g;
    while (g + 1 < groups && Share(steps, groups, g + 1).first <= step) ++g;
    return g;
  };
  const int g0 = group_of(lo), g1 = group_of(hi - 1);
  if (g0 == g1) return;  // stored as it was finished
  const int e = blockIdx.y * 256 + threadIdx.x;
  if (e >= T::TN * T::TM / 4) return;
  // g0 began the tile (its second slot), the others came to it from its middle (their first)
  const floatx4* at = reinterpret_cast<const floatx4*>(partial) + e;
  constexpr int kSlot = T::TN * T::TM / 4, kAhead = 4;
  floatx4 sum = at[((int64_t)g0 * 2 + 1) * kSlot];
  int g = g0 + 1;
  for (; g + kAhead <= g1 + 1; g += kAhead) {
    floatx4 v[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) v[u] = at[(int64_t)(g + u) * 2 * kSlot];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) sum += v[u];
  }
  for (; g <= g1; ++g) sum += at[(int64_t)g * 2 * kSlot];
  const int lane = e & 63, f = e >> 6, j = f % FM, i = f / FM % FN, wave = f / (FM * FN);
  const int m = tile % tiles_m * T::TM + (wave % WM * FM + j) * 16 + (lane & 15);
  const int n = tile / tiles_m * T::TN + (wave / WM * FN + i) * 16 + 4 * (lane >> 4);
  const bool vec = p.ld_out % 4 == 0 && (uintptr_t)p.out % (OUT == NVFP4_DTYPE_BF16 ? 8 : 16) == 0;
  if (m < p.M) store4<OUT>(p.out, (int64_t)m * p.ld_out + n, sum, p.N - n, vec);
}

// Large products: a workgroup has a whole tile of 256 columns x 224 tokens, 8 waves in 4 x 2, two to a SIMD; a wave owns 64
// columns x 112 tokens (112 accumulators a lane).  Per block of 128 it reads 4 + 7 fragments of 2 KB from LDS, converts
// them (176 instructions) and issues 4 * 7 * 4 matrix instructions of 16 cycles and 112 fmas (out += scale * sum).
//
// Bound: the matrix unit, the vector instructions beside it and the power limit.  Measured, 8192 x 5120 x 17408: 1175 us (1130
// to 1290 from card to card), 1.24 PFLOP/s at 1.95 GHz (a library bf16 product reaches 1.27 at 8192^3); with the copies left out 980, the fmas
// 1078, the conversions 1160, the matrix instructions 789.  The same instructions from registers alone reach 1.7.
//
// LDS holds two stages of a block: weight rows, activation rows (128 bytes each),
// the tile's activation scales; all three come by LDS DMA.  16-byte pieces are
// XOR-swizzled by the row, in the copies' addresses, so that the reads are free of
// bank conflicts.  Rows behind the last and pieces behind K lie behind the descriptors'
// ranges: such lanes write zeros.
//
// The weight's fragments stay in registers, as fp16, over a block.  A step (j, n) is two products with one quarter (32 k)
// of the activation fragment j; beside them stand fmas of the two products before, half a conversion of
// fragment j + 1 and reads of j + 2, so that no instruction waits for the one before it.  Reads are thus ahead
// by more than a fragment, and in the middle of the last but one every wave has read all that it needs of the
// stage.  The one barrier of a block stands there: it frees the stage for the block two on, and certifies the next
// block's, whose weight fragments replace the present ones beside the last products.  A block's 8 copies a
// wave are spread over 32 steps: all at once they hold up the instructions behind them (60 tiles of 40 blocks: 118 us, so 105).
struct Tile {
  static constexpr int FN = 4, FM = 7, WN = 4, WM = 2;
  static constexpr int TN = FN * WN * 16, TM = FM * WM * 16;
  static constexpr int kW = TN * 128, kX = TM * 128, kStage = kW + kX + 1024;
  // 1 KB copies of every wave; the first four waves bring one more group of activation rows, the others the scales
  static constexpr int CW = TN / 64, CX = TM / 64;
  static_assert(TM / 8 % 8 == 4 && TM <= 256, "the copies' shares");
};

template <int OUT>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2)))
void fp8_tile_kernel(const Fp8GemmArgs p, int tiles_m, int tiles_n) {
  using T = Tile;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  int tm, tn;
  tile_of(blockIdx.x, tiles_m * tiles_n, tiles_m, tiles_n, tm, tn);
  const int n0 = tn * T::TN, m0 = tm * T::TM;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wn = wave / T::WM, wm = wave % T::WM, li = lane & 15, lg = lane >> 4;
  const int blocks = (p.K + 127) / 128;

  // copies: lane l brings piece l % 8 (swizzled) of row l / 8 of a group of 8 rows
  const int ldw = (int)p.w.ld_codes, lda = (int)p.a.ld_codes;
  const i32x4 rw = buffer_rsrc(p.w.codes + (int64_t)n0 * ldw, (uint32_t)(min(T::TN, p.N - n0) * ldw));
  const uint8_t* xa = p.a.codes + (int64_t)m0 * lda;
  const uint32_t x_bytes = (uint32_t)(min(T::TM, p.M - m0) * lda);
  const float* sa = p.a.scales + (int64_t)min(m0 + max(wave - 4, 0) * 64 + lane, p.M - 1) * p.a.scale_row;
  constexpr int kNowhere = (int)0x80000000;
  constexpr int kCopies = T::CW + T::CX + 1;
  // the c-th copy of a wave's share of block b; behind the last block the last one is copied again, so that the waits need no branches
  auto copy = [&](int b, int c) __attribute__((always_inline)) {
    int l = lane;
    asm volatile("" : "+v"(l));  // the offsets are worked out anew: kept over the loop they would cost registers that it lacks
    const int q = l >> 3, g = c < T::CW ? wave * T::CW + c : c < T::CW + T::CX ? wave * T::CX + c - T::CW : 8 * T::CX + wave;
    uint8_t* to = smem + (b & 1) * T::kStage;
    const int last = min(b, blocks - 1), k = last * 128;
    if (c < T::CW) {
      const int piece = ((l & 7) ^ ((q & 3) + 4 * (c & 1))) * 16;  // by the row and the parity of the group of rows
      llvm_amdgcn_raw_buffer_load_lds(rw, (lds_u32_ptr)(to + g * 1024), 16, k + piece < p.K ? (g * 8 + q) * ldw + piece : kNowhere, k, 0, 0);
    } else if (c < kCopies - 1 || wave < 4) {
      const int piece = ((l & 7) ^ q) * 16;
      llvm_amdgcn_raw_buffer_load_lds(buffer_rsrc(xa + last * p.a.code_block, x_bytes), (lds_u32_ptr)(to + T::kW + g * 1024), 16,
                                      k + piece < p.K ? (g * 8 + q) * lda + piece : kNowhere, 0, 0, 0);
    } else {
      __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) uint32_t*)(sa + (int64_t)last * p.a.scale_block),
                                       (lds_u32_ptr)(to + T::kW + T::kX + (wave - 4) * 256), 4, 0, 0);
    }
  };
  // a wave whose columns all lie behind the last takes the last block's scales
  const auto* sw = (const __attribute__((address_space(4))) float*)(p.w.scales + (int64_t)(min(n0 + wn * 64, p.N - 1) / 128) * p.w.scale_row);

  // fragments: weight row (i, a = lane % 16) is column (i / 2) * 32 + (a / 4) * 8 + (i % 2) * 4 + a % 4 of the wave, so that a
  // lane's results of fragments 2 i and 2 i + 1 are 8 neighbouring columns
  const int wbase = (wn * 64 + (li >> 2) * 8 + (li & 3)) * 128, xbase = T::kW + (wm * T::FM * 16 + li) * 128;
  const int sbase = T::kW + T::kX + (wm * T::FM * 16 + li) * 4;
  int piece[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) piece[h] = ((lg + 4 * h) ^ (li & 7)) << 4;
  // half h of a fragment: the operands of quarters 2 h and 2 h + 1
  auto read_w = [&](const uint8_t* st, int i, int h) __attribute__((always_inline)) {
    return *reinterpret_cast<const u32x4*>(st + wbase + piece[h] + (i >> 1) * 4096 + (i & 1) * 512);
  };
  auto read_x = [&](const uint8_t* st, int j, int h) __attribute__((always_inline)) {
    return *reinterpret_cast<const u32x4*>(st + xbase + piece[h] + j * 2048);
  };
  auto read_s = [&](const uint8_t* st, int j) __attribute__((always_inline)) { return *reinterpret_cast<const float*>(st + sbase + j * 64); };
  auto quarter = [&](const u32x4& half, int s) __attribute__((always_inline)) { return half_of(half[2 * (s & 1)], half[2 * (s & 1) + 1]); };

#pragma unroll
  for (int c = 0; c < kCopies; ++c) copy(0, c);
#pragma unroll
  for (int c = 0; c < 3; ++c) copy(1, c);
  wait_vmem<3>();
  barrier_lds();
  floatx4 acc[T::FN][T::FM], t[2][2];
  half8 hw[T::FN][4], hx[4];
#pragma unroll
  for (int i = 0; i < T::FN; ++i) {
#pragma unroll
    for (int j = 0; j < T::FM; ++j) acc[i][j] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int s = 0; s < 4; ++s) hw[i][s] = quarter(read_w(smem, i, s >> 1), s);
  }
#pragma unroll
  for (int s = 0; s < 4; ++s) hx[s] = quarter(read_x(smem, 0, s >> 1), s);
  t[1][0] = t[1][1] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
  u32x4 x[2] = {read_x(smem, 1, 0), read_x(smem, 1, 1)};  // of the fragment after hx
  float sx = read_s(smem, 0), sc = 0.0f, s_now = sw[0];   // sc: the scale of the sums in t
  for (int b = 0; b < blocks; ++b) {
    const uint8_t* st = smem + (b & 1) * T::kStage;
    const uint8_t* nst = smem + ((b + 1) & 1) * T::kStage;
    const float s_next = sw[min(b + 1, blocks - 1) * p.w.scale_block];
    u32x4 w[2];
#pragma unroll
    for (int j = 0; j < T::FM; ++j) {
      half8 next[4];
      const float s_prev = sc;
#pragma unroll
      for (int n = 0; n < 8; ++n) {  // products of fragments 2 P and 2 P + 1 with quarter s
        const int P = n >> 2, s = n & 3, i = 2 * P;
        __builtin_amdgcn_sched_barrier(0);
        if (j == T::FM - 2 && n == 4) {
          wait_vmem<0>();
          barrier_lds();
          __builtin_amdgcn_s_waitcnt(0xC07F);  // the barrier's lgkmcnt(0) again, seen by the compiler's own wait insertion
          __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int u = 0; u < 2; ++u)
          t[P][u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(hw[i + u][s], hx[s], s == 0 ? floatx4{0.0f, 0.0f, 0.0f, 0.0f} : t[P][u], 0, 0, 0);
        // the two fragments before
        const int jp = P == 1 ? j : j == 0 ? T::FM - 1 : j - 1, ip = P == 1 ? 0 : 2;
        if (s > 0) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (e * 3 / 8 == s - 1) acc[ip + (e >> 2)][jp][e & 3] = fmaf(t[1 - P][e >> 2][e & 3], P == 1 ? sc : s_prev, acc[ip + (e >> 2)][jp][e & 3]);
          if (s == 3) asm volatile("" : "+v"(acc[ip][jp]), "+v"(acc[ip + 1][jp]));  // here, not where the compiler would sink them to
        }
        // half a quarter of the next fragment
        {
          const uint32_t c = x[n >> 2][n & 3];
          const half2v lo = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c, 1.0f, false), hi = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c, 1.0f, true);
          const int e = (n & 1) * 4;
          next[n >> 1][e] = lo[0];
          next[n >> 1][e + 1] = lo[1];
          next[n >> 1][e + 2] = hi[0];
          next[n >> 1][e + 3] = hi[1];
        }
        // the copies, one in four steps: the freed stage's first three, then the other stage's remaining five
        if (j == T::FM - 2 && n == 5) copy(b + 2, 0);
        if (j == T::FM - 1 && (n == 1 || n == 5)) copy(b + 2, n == 1 ? 1 : 2);
        if (j < 3 && (n == 1 || n == 5) && 2 * j + n / 5 < 5) copy(b + 1, 3 + 2 * j + n / 5);
        if (n == 0) {
          sc = sx * s_now;
          sx = j < T::FM - 1 ? read_s(st, j + 1) : read_s(nst, 0);
        }
        if (n == 4) x[0] = j < T::FM - 2 ? read_x(st, j + 2, 0) : read_x(nst, j + 2 - T::FM, 0);
        if (n == 7) x[1] = j < T::FM - 2 ? read_x(st, j + 2, 1) : read_x(nst, j + 2 - T::FM, 1);
        if (j == T::FM - 2 && n == 7) w[0] = read_w(nst, 0, 0), w[1] = read_w(nst, 1, 0);
        if (j == T::FM - 1) {
#pragma unroll
          for (int u = 0; u < 2; ++u) hw[i + u][s] = quarter(w[u], s);
          if ((s & 1) && n < 7) {
#pragma unroll
            for (int u = 0; u < 2; ++u) w[u] = read_w(nst, n == 3 ? 2 + u : i + u, n == 3 ? 0 : 1);
          }
        }
      }
#pragma unroll
      for (int s = 0; s < 4; ++s) hx[s] = next[s];
    }
    s_now = s_next;
  }
  wait_vmem<0>();  // no copy may land after the workgroup's LDS is given away
#pragma unroll
  for (int u = 0; u < 2; ++u)
#pragma unroll
    for (int r = 0; r < 4; ++r) acc[2 + u][T::FM - 1][r] = fmaf(t[1][u][r], sc, acc[2 + u][T::FM - 1][r]);
  mend_large_scales(p, acc, 0, blocks, m0 + wm * T::FM * 16, n0 + wn * 64,
                    [&](int i) { return n0 + wn * 64 + (i >> 1) * 32 + (li >> 2) * 8 + (i & 1) * 4 + (li & 3); });

  const bool vec = p.ld_out % 8 == 0 && (uintptr_t)p.out % 16 == 0;
#pragma unroll
  for (int j = 0; j < T::FM; ++j) {
    const int m = m0 + (wm * T::FM + j) * 16 + li;
    if (m >= p.M) continue;
#pragma unroll
    for (int i = 0; i < T::FN; i += 2) {
      const int n = n0 + wn * 64 + (i / 2) * 32 + lg * 8;
      const floatx4 u = acc[i][j], v = acc[i + 1][j];
      if constexpr (OUT == NVFP4_DTYPE_BF16) {
        uint16_t* o = reinterpret_cast<uint16_t*>(p.out) + (int64_t)m * p.ld_out + n;
        if (vec && n + 8 <= p.N) {
          store_stream16(o, pack_bf16x2(u[0], u[1]), pack_bf16x2(u[2], u[3]), pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
          continue;
        }
      }
      store4<OUT>(p.out, (int64_t)m * p.ld_out + n, u, p.N - n, vec);
      store4<OUT>(p.out, (int64_t)m * p.ld_out + n + 4, v, p.N - n - 4, vec);
    }
  }
}

template <int OUT>
hipError_t launch_tiles(const Fp8GemmArgs& g, hipStream_t s) {
  using T = Tile;
  const int tiles_m = (g.M + T::TM - 1) / T::TM, tiles_n = (g.N + T::TN - 1) / T::TN;
  const auto fn = fp8_tile_kernel<OUT>;
  const hipError_t e = hipFuncSetAttribute((const void*)fn, hipFuncAttributeMaxDynamicSharedMemorySize, 2 * T::kStage);
  if (e != hipSuccess) return e;
  fn<<<(unsigned)tiles_m * (unsigned)tiles_n, 512, 2 * T::kStage, s>>>(g, tiles_m, tiles_n);
  return hipGetLastError();
}

// Large products whose caller allows the 8-bit matrix instruction (the builtin with scale operands 0 is the form without
// scales: 2 % faster than unit scales).
__device__ inline floatx4 product_8bit(const Frag& w, const Frag& x) {
  const i32x8 a = {(int)w.p[0][0], (int)w.p[0][1], (int)w.p[0][2], (int)w.p[0][3],
                   (int)w.p[1][0], (int)w.p[1][1], (int)w.p[1][2], (int)w.p[1][3]};
  const i32x8 b = {(int)x.p[0][0], (int)x.p[0][1], (int)x.p[0][2], (int)x.p[0][3],
                   (int)x.p[1][0], (int)x.p[1][1], (int)x.p[1][2], (int)x.p[1][3]};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, floatx4{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0, 0, 0, 0);
}

// WN x WM = 4 waves, one per SIMD; a wave owns FN * 16
// columns x FM * 16 tokens (256 x 224 tiles: 128 x 112, 224 accumulators a
// lane).  Per block of 128 a wave reads FN + FM fragments of 2 KB from LDS for FN * FM
// matrix instructions of 32 cycles; each instruction's four fmas (out += scale *
// tmp) run three instructions later, beside the matrix unit.
//
// Bound: the matrix unit with the fmas beside it.  Measured, 8192 x 5120 x 17408: 635-715 us from card to card, 2.0-2.3 PFLOP/s
// (8192 x 34816 x 5120 1.9-2.2, 8192^3 1.9-2.2), at a clock of 1.9 GHz under this load; the same instructions and fmas from registers
// alone reach 3.1, a library product with a single scale 2.06 at this size and 2.7 at 8192^3.  Other forms at this
// size, in the version where this one took 659: 256 x 256 tiles 732 (their sums no longer fit beside the fragments in the
// vector registers and are moved to and fro), two waves per SIMD with half the accumulators each 704 (twice the
// LDS reads).
//
// LDS holds two stages of a block: weight rows, activation rows (128 bytes each),
// the tile's activation scales; all three come by LDS DMA.  16-byte pieces are
// XOR-swizzled by the row, in the copies' addresses, so that the reads are free of
// bank conflicts.  Pieces behind K and nothing else have an address behind the descriptor's
// range: such lanes write zeros.
//
// A block's regions t = 0 .. FM - 1 (one activation fragment each):
//   the weight's fragments stay in registers over a block; the next block's are
//   read in the last region, each right after its last use, and the next
//   activation fragment is read a region ahead;
//   barrier 1 (end of region 1): every wave holds its weight fragments, so the
//   stage's weight rows are free: the copies of the weight two blocks on go out in regions
//   2-5;
//   barrier 2 (end of the region before the last): every wave has read the stage's activations: the
//   copies of the activations two blocks on go out in the last region and the next
//   block's first three.  The same barrier certifies the next block, whose copies are
//   then older than the FN * WN / 2 weight copies just sent.
// Behind the last block the last one is copied again, so that the waits need no branches.
template <int FN, int FM, int WN, int WM>
struct Pipe {
  static constexpr int TN = FN * WN * 16, TM = FM * WM * 16;
  static constexpr int kW = TN * 128, kX = TM * 128, kStage = kW + kX + 1024;
  static constexpr int CW = TN / 32, CX = TM / 32;  // 1 KB copies of a wave
  static constexpr int x_share(int k) { return (CX * k + 3) / 4; }  // of the activation copies, those before the k-th of 4 regions
  static_assert(WN * WM == 4 && CW % 4 == 0 && FM >= 7 && FN % 2 == 0, "the schedule's shares");
};

template <int FN, int FM, int WN, int WM>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1, 1)))
void fp8_pipe_kernel(const Fp8GemmArgs p, int tiles_m, int tiles_n) {
  using T = Pipe<FN, FM, WN, WM>;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  int tm, tn;
  tile_of(blockIdx.x, tiles_m * tiles_n, tiles_m, tiles_n, tm, tn);
  const int n0 = tn * T::TN, m0 = tm * T::TM;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wn = wave / WM, wm = wave % WM, li = lane & 15, lg = lane >> 4;
  const int blocks = (p.K + 127) / 128;

  // copies: lane l brings piece l % 8 of row l / 8 of a group of 8 rows
  const i32x4 rw = buffer_rsrc(p.w.codes + (int64_t)n0 * p.w.ld_codes, (uint32_t)(T::TN * p.w.ld_codes));
  const i32x4 rx = buffer_rsrc(p.a.codes + (int64_t)m0 * p.a.ld_codes, (uint32_t)(T::TM * p.a.ld_codes));  // code_block is 128
  const int q = lane >> 3;
  int vw[T::CW], vx[T::CX];
  int pw[2];                              // the piece, by the parity of the group of rows
  const int px = (lane & 7) ^ q;
#pragma unroll
  for (int c = 0; c < 2; ++c) pw[c] = (lane & 7) ^ ((q & 3) + 4 * c);
#pragma unroll
  for (int c = 0; c < T::CW; ++c)
    vw[c] = min((wave * T::CW + c) * 8 + q, p.N - 1 - n0) * (int)p.w.ld_codes + pw[c & 1] * 16;
#pragma unroll
  for (int c = 0; c < T::CX; ++c)
    vx[c] = min((wave * T::CX + c) * 8 + q, p.M - 1 - m0) * (int)p.a.ld_codes + px * 16;
  constexpr int kNowhere = (int)0x80000000, kLag = 3;
  auto copy_w = [&](int b, int c) __attribute__((always_inline)) {
    const int last = min(b, blocks - 1);
    const int off = last * 128 + pw[c & 1] * 16 < p.K ? vw[c] : kNowhere;
    llvm_amdgcn_raw_buffer_load_lds(rw, (lds_u32_ptr)(smem + (b & 1) * T::kStage + (wave * T::CW + c) * 1024), 16, off, last * 128, 0, 0);
  };
  auto copy_x = [&](int b, int c) __attribute__((always_inline)) {
    const int last = min(b, blocks - 1);
    const int off = last * 128 + px * 16 < p.K ? vx[c] : kNowhere;
    llvm_amdgcn_raw_buffer_load_lds(rx, (lds_u32_ptr)(smem + (b & 1) * T::kStage + T::kW + (wave * T::CX + c) * 1024), 16, off,
                                    last * 128, 0, 0);
  };
  // the scales of rows 64 wave .. of the tile, one a lane (of following rows where a tile has fewer than 256)
  const int srow = wave * 64;
  const float* sa = p.a.scales + (int64_t)min(m0 + srow + lane, p.M - 1) * p.a.scale_row;
  auto copy_s = [&](int b) __attribute__((always_inline)) {
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) uint32_t*)(sa + (int64_t)min(b, blocks - 1) * p.a.scale_block),
                                     (lds_u32_ptr)(smem + (b & 1) * T::kStage + T::kW + T::kX + srow * 4), 4, 0, 0);
  };
  // a wave whose columns all lie behind the last takes the last block's scales
  const auto* sw = (const __attribute__((address_space(4))) float*)(p.w.scales + (int64_t)(min(n0 + wn * FN * 16, p.N - 1) / 128) * p.w.scale_row);

  // fragments: weight row (i, a = lane % 16) is column (i / 2) * 32 + (a / 4) * 8 + (i % 2) * 4 + a % 4 of the wave, so that a
  // lane's results of fragments 2 i and 2 i + 1 are 8 neighbouring columns
  const int wbase = (wn * FN * 16 + (li >> 2) * 8 + (li & 3)) * 128, xbase = T::kW + (wm * FM * 16 + li) * 128;
  int wat[2], xat[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    wat[h] = wbase + (((lg + 4 * h) ^ (li & 7)) << 4);
    xat[h] = xbase + (((lg + 4 * h) ^ (li & 7)) << 4);
  }
  auto read_w = [&](const uint8_t* st, int i) __attribute__((always_inline)) {
    Frag f;
#pragma unroll
    for (int h = 0; h < 2; ++h) f.p[h] = *reinterpret_cast<const u32x4*>(st + wat[h] + (i >> 1) * 4096 + (i & 1) * 512);
    return f;
  };
  auto read_x = [&](const uint8_t* st, int t) __attribute__((always_inline)) {
    Frag f;
#pragma unroll
    for (int h = 0; h < 2; ++h) f.p[h] = *reinterpret_cast<const u32x4*>(st + xat[h] + t * 2048);
    return f;
  };
  auto read_s = [&](const uint8_t* st, int t) __attribute__((always_inline)) {
    return *reinterpret_cast<const float*>(st + T::kW + T::kX + ((wm * FM + t) * 16 + li) * 4);
  };

  floatx4 acc[FN][FM];
#pragma unroll
  for (int i = 0; i < FN; ++i)
#pragma unroll
    for (int j = 0; j < FM; ++j) acc[i][j] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};

#pragma unroll
  for (int c = 0; c < T::CW; ++c) copy_w(0, c);
#pragma unroll
  for (int c = 0; c < T::CX; ++c) copy_x(0, c);
  copy_s(0);
#pragma unroll
  for (int c = 0; c < T::CW; ++c) copy_w(1, c);
#pragma unroll
  for (int c = 0; c < T::x_share(1); ++c) copy_x(1, c);
  copy_s(1);
  wait_vmem<T::CW + T::x_share(1) + 1>();
  barrier_lds();
  Frag w[FN], x[2];
  float sc[FM];
#pragma unroll
  for (int i = 0; i < FN; ++i) w[i] = read_w(smem, i);
  x[0] = read_x(smem, 0);
  {
    const float s = sw[0];
#pragma unroll
    for (int t = 0; t < FM; ++t) sc[t] = read_s(smem, t) * s;
  }
  for (int b = 0; b < blocks; ++b) {
    const uint8_t* st = smem + (b & 1) * T::kStage;
    const uint8_t* nst = smem + ((b + 1) & 1) * T::kStage;
    float next_sw = 0.0f, next_sc[FM];
    floatx4 tmp[kLag + 1];
    auto add = [&](int o) __attribute__((always_inline)) {
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[o % FN][o / FN][r] = fmaf(tmp[o % (kLag + 1)][r], sc[o / FN], acc[o % FN][o / FN][r]);
    };
#pragma unroll
    for (int t = 0; t < FM; ++t) {
      // copies of this region, one beside each of its first matrix instructions
      const int x_lo = t == FM - 1 ? 0 : t < 3 ? T::x_share(t + 1) : 0, x_hi = t == FM - 1 ? T::x_share(1) : t < 3 ? T::x_share(t + 2) : 0;
      const int w_lo = t >= 2 && t < 6 ? (t - 2) * (T::CW / 4) : 0, w_hi = t >= 2 && t < 6 ? (t - 1) * (T::CW / 4) : 0;
#pragma unroll
      for (int i = 0; i < FN; ++i) {
        __builtin_amdgcn_sched_barrier(0);
        const int n = t * FN + i;
        if (i == 1) x[(t + 1) & 1] = t < FM - 1 ? read_x(st, t + 1) : read_x(nst, 0);
        tmp[n % (kLag + 1)] = product_8bit(w[i], x[t & 1]);
        if (n >= kLag) add(n - kLag);
        // the next block's scales: early enough that nothing waits for them
        if (t == 1 && i == 2) next_sw = sw[min(b + 1, blocks - 1) * p.w.scale_block];
        if (t == FM - 1 && i == 0) {
#pragma unroll
          for (int j = 0; j < FM; ++j) next_sc[j] = read_s(nst, j);
        }
        if (t == FM - 1) w[i] = read_w(nst, i);
        const int c = i - 1;
        if (c >= 0 && c < x_hi - x_lo) copy_x(t < 3 ? b + 1 : b + 2, x_lo + c);
        else if (c >= 0 && c - (x_hi - x_lo) < w_hi - w_lo) copy_w(b + 2, w_lo + c - (x_hi - x_lo));
        else if (t == FM - 1 && c == x_hi) copy_s(b + 2);
      }
      __builtin_amdgcn_sched_barrier(0);
      if (t == FM - 1) {
#pragma unroll
        for (int o = FM * FN - kLag; o < FM * FN; ++o) add(o);
#pragma unroll
        for (int j = 0; j < FM; ++j) next_sc[j] *= next_sw;
      }
      if (t == 1) {
        barrier_lds();
        __builtin_amdgcn_s_waitcnt(0xC07F);  // the barrier's lgkmcnt(0) again, seen by the compiler's own wait insertion
      }
      if (t == FM - 2) {
        wait_vmem<T::CW>();
        barrier_lds();
        __builtin_amdgcn_s_waitcnt(0xC07F);
      }
    }
#pragma unroll
    for (int t = 0; t < FM; ++t) sc[t] = next_sc[t];
    if constexpr (FM % 2 == 1) x[0] = x[1];
  }
  wait_vmem<0>();  // no copy may land after the workgroup's LDS is given away
  mend_large_scales(p, acc, 0, blocks, m0 + wm * FM * 16, n0 + wn * FN * 16,
                    [&](int i) { return n0 + wn * FN * 16 + (i >> 1) * 32 + (li >> 2) * 8 + (i & 1) * 4 + (li & 3); });

  const bool vec = p.ld_out % 8 == 0 && (uintptr_t)p.out % 16 == 0;
  uint16_t* out = reinterpret_cast<uint16_t*>(p.out);
#pragma unroll
  for (int j = 0; j < FM; ++j) {
    const int m = m0 + (wm * FM + j) * 16 + li;
    if (m >= p.M) continue;
#pragma unroll
    for (int i = 0; i < FN; i += 2) {
      const int n = n0 + wn * FN * 16 + (i / 2) * 32 + lg * 8;
      uint16_t* o = out + (int64_t)m * p.ld_out + n;
      const floatx4 u = acc[i][j], v = acc[i + 1][j];
      if (vec && n + 8 <= p.N) {
        store_stream16(o, pack_bf16x2(u[0], u[1]), pack_bf16x2(u[2], u[3]), pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
      } else {
#pragma unroll
        for (int r = 0; r < 8; ++r)
          if (n + r < p.N) o[r] = (uint16_t)f32_to_bf16_bits(r < 4 ? u[r] : v[r - 4]);
      }
    }
  }
}

template <int FN, int FM, int WN, int WM>
hipError_t launch_pipe(const Fp8GemmArgs& g, hipStream_t s) {
  using T = Pipe<FN, FM, WN, WM>;
  const int tiles_m = (g.M + T::TM - 1) / T::TM, tiles_n = (g.N + T::TN - 1) / T::TN;
  const auto fn = fp8_pipe_kernel<FN, FM, WN, WM>;
  const hipError_t e = hipFuncSetAttribute((const void*)fn, hipFuncAttributeMaxDynamicSharedMemorySize, 2 * T::kStage);
  if (e != hipSuccess) return e;
  fn<<<(unsigned)tiles_m * (unsigned)tiles_n, 256, 2 * T::kStage, s>>>(g, tiles_m, tiles_n);
  return hipGetLastError();
}

template <int FN, int FM, int WN, int WM, int D, int OUT>
hipError_t launch_ring_as(const Fp8GemmArgs& g, float* ws, hipStream_t s) {
  using T = Ring<FN, FM, WN, WM, D>;
  static_assert(T::TN * T::TM <= 128 * 224, "a partial tile's room in the workspace");
  const int tiles_m = (g.M + T::TM - 1) / T::TM, tiles_n = (g.N + T::TN - 1) / T::TN, blocks = (g.K + 127) / 128;
  const int64_t tiles = (int64_t)tiles_m * tiles_n, steps = tiles * blocks;
  // At least 4 steps a workgroup, where a tile has them: fewer sums to join.  Measured, us with at least 1, 2, 4, 8:
  // 1 x 1024 x 5120 13.3, 11.8, 11.1, 11.4; 40 x 2048 x 2048 13.3, 11.3, 11.7, 13.9; 128 x 1024 x 5120 18.9, 16.2, 14.7, 16.8;
  // 200 x 1024 x 5120 24.4, 21.3, 19.7, 23.1; 77 x 1000 x 2064 float32 13.3, 11.9, 12.5, 16.5.
  const int64_t want = tiles > steps / 4 ? tiles : steps / 4;
  const int groups = (int)(want < kRingGroups ? want : kRingGroups);
  const auto fn = fp8_ring_kernel<FN, FM, WN, WM, D, OUT>;
  hipError_t e = hipFuncSetAttribute((const void*)fn, hipFuncAttributeMaxDynamicSharedMemorySize, D * T::kStage);
  if (e != hipSuccess) return e;
  fn<<<groups, 512, D * T::kStage, s>>>(g, tiles_m, tiles_n, ws);
  if ((e = hipGetLastError()) != hipSuccess || blocks == 1 || tiles % groups == 0) return e;  // whole tiles each: nothing to join
  fp8_join_kernel<FN, FM, WN, WM, D, OUT><<<dim3((unsigned)tiles, (T::TN * T::TM / 4 + 255) / 256), 256, 0, s>>>(g, tiles_m, groups, steps, ws);
  return hipGetLastError();
}

template <int FN, int FM, int WN, int WM, int D>
hipError_t launch_ring(const Fp8GemmArgs& g, float* ws, hipStream_t s) {
  return g.out_dtype == NVFP4_DTYPE_BF16 ? launch_ring_as<FN, FM, WN, WM, D, NVFP4_DTYPE_BF16>(g, ws, s)
                                         : launch_ring_as<FN, FM, WN, WM, D, NVFP4_DTYPE_F32>(g, ws, s);
}

// Tokens of the ring kernel's tiles.  Above 128 by the tiles' number and the time of a step, 1.3 us for 128 tokens and 2.1 for 224.
// Measured, us, 128 | 224: 200 x 5120 x 17408 62 | 57; 256 x 5120 x 17408 64 | 90; 384 x 5120 x 17408 91 | 96; 448 x 5120 x
// 17408 112 | 97; 512 x 5120 x 17408 114 | 133; 224 x 5120 x 5120 28 | 30; 512 x 5120 x 5120 46 | 53; 640 x 5120 x 5120 53 | 55.
int ring_tokens(int64_t m) {
  if (m <= 16) return 16;
  if (m <= 32) return 32;
  if (m <= 64) return 64;
  if (m <= 128) return 128;
  return (m + 127) / 128 * 5 < (m + 223) / 224 * 8 ? 128 : 224;
}

}  // namespace

// Two partial tiles of each workgroup.  More tokens never need less, so that one workspace serves smaller calls too.
size_t fp8_gemm_workspace(int64_t m) {
  const int tm = m <= 128 ? ring_tokens(m) : 224;
  return (size_t)kRingGroups * 2 * 128 * tm * sizeof(float);
}

// By the steps (a block of a tile) of the busiest workgroup: 1.3 or 2.1 us each for an even share of 128 x 128 or 128 x 224 tiles,
// whose partial sums and join cost 10 more, against whole 256 x 224 tiles with 2.6 to 2.9 us a step, or 1.55 with the 8-bit instruction.
// Measured, us, shared | whole | whole with the 8-bit instruction: 224 x 34816 x 5120 108 | 126 | 76; 512 x 5120 x 5120 51 | 105
// | -; 448 x 5120 x 17408 95 | 370 | 188; 1024 x 5120 x 5120 78 | 108 | 61; 1024 x 34816 x 5120 432 | 344 | 214; 2048 x 5120 x
// 17408 400 | 349 | 205; 8192 x 5120 x 17408 1467 | 1175 | 635-715.
namespace {
enum class Form { kRing, kTile, kPipe };
Form form_of(const Fp8GemmArgs& g) {
  if (g.M <= 128) return Form::kRing;
  const int64_t blocks = (g.K + 127) / 128, tm = ring_tokens(g.M);
  const int64_t whole = ((g.M + 223) / 224 * (((int64_t)g.N + 255) / 256) + 255) / 256 * blocks;
  const int64_t shared = (g.M + tm - 1) / tm * (((int64_t)g.N + 127) / 128) * blocks / kRingGroups * (tm == 128 ? 5 : 8) + 40;
  if (g.cut_sums && whole * 6 <= shared) return Form::kPipe;
  return whole * 12 <= shared ? Form::kTile : Form::kRing;
}
}  // namespace

bool fp8_gemm_shares(const Fp8GemmArgs& g) { return form_of(g) != Form::kPipe; }

hipError_t launch_fp8_gemm(const Fp8GemmArgs& g, float* ws, hipStream_t s) {
  const Form form = form_of(g);
  if (form == Form::kPipe) return launch_pipe<8, 7, 2, 2>(g, s);
  if (form == Form::kTile) return g.out_dtype == NVFP4_DTYPE_BF16 ? launch_tiles<NVFP4_DTYPE_BF16>(g, s) : launch_tiles<NVFP4_DTYPE_F32>(g, s);
  switch (ring_tokens(g.M)) {
    case 16: return launch_ring<1, 1, 8, 1, 8>(g, ws, s);
    case 32: return launch_ring<1, 2, 8, 1, 7>(g, ws, s);
    case 64: return launch_ring<1, 4, 8, 1, 6>(g, ws, s);
    case 128: return launch_ring<2, 4, 4, 2, 4>(g, ws, s);
    default: return launch_ring<2, 7, 4, 2, 3>(g, ws, s);
  }
}

}  // namespace nvfp4
