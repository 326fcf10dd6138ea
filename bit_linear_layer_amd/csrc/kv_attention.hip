// Attention over the paged FP8 KV cache for a batch of sequences that share
// a prefix.
//
// For a query row r and the tokens t that it sees,
//   o_r = sum_t softmax_t(c q_r . k_t) v_t,
// computed in one pass: with the running maximum M (in log2 units), the sum
// l = sum 2^(x_t - M) and o = sum 2^(x_t - M) v_t over the tokens so far,
// another set of tokens with maximum M' multiplies l and o by 2^(M - max) and
// adds its own.  Parts of a row's tokens handled by different waves and
// workgroups join by the same rule, in a fixed order.
//
// Tiles.  A tile is up to 16 query rows that share a kv head and a token
// range: the q_len * group rows of one sequence, or of all sequences where
// the tokens are the shared prefix.  A wave takes steps of 64 tokens:
//   S^T = K Q^T   (16 x 16 x 32 MFMA; A = 16 tokens x 32 dimensions)
//   O^T += V^T P^T (A = 16 dimensions x 32 tokens)
// Both products are formed transposed, so a lane owns one query row (column
// lane % 16): the maximum and the sum are per-lane scalars, and the lane's 16
// softmax weights of a step are, in register order, the 16 tokens of block
// lane / 16 -- exactly its slice of the second product's B operand, with no
// data moved between lanes.  To that end row i of key tile tau is token
// 4 tau + i % 4 of block i / 4 of the step.  Key and value bytes go from
// global memory to registers in 16-byte pieces (the cache layout is made for
// that) and become bf16 in the conversion instruction, the key's power-of-two
// scale included; the value's scale multiplies the softmax weight, exactly.
//
// Work is divided evenly whatever the lengths: the tiles' token ranges, in
// units of 256 tokens (one step for each of the workgroup's 4 waves), form one
// line that is cut into equal shares, one per workgroup.  A tile that a cut
// divides leaves partial (M, l, o) in the workspace, in slot tile + workgroup
// (distinct for every piece, since one of the two grows from piece to piece),
// and a second kernel joins them.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "device_util.h"
#include "kv_pages.h"

namespace nvfp4 {

namespace {

using namespace dev;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256, kWaves = 4;
constexpr int kStep = 64;       // tokens of one wave's step
constexpr int kTileRows = 16;
constexpr float kLowest = -3.0e38f;  // stands for "no token yet"; finite, so differences are never NaN

// One pass over tiles of rows: what the stream kernel and the join share.
struct Pass {
  int batch;      // sequences (1 where the rows of all share their tokens)
  int rows;       // query rows of a sequence and kv head: q_len * group
  int q_len, group;
  int row_tiles;  // ceil(rows / kTileRows)
  int prefix_len; // shared tokens this pass reads for every tile
  const int* lens;  // null: no tokens of the sequences' own
  int max_len;
  int workgroups;
  int direct;     // every tile is whole in one workgroup and nothing joins it: write the output
  float* ml;      // partials: [slot][16][2], then [slot][16][D]
  float* o;
};

__device__ __host__ inline int ceil_div(int a, int b) { return (a + b - 1) / b; }

__device__ inline int own_len(const Pass& p, int b) {
  return p.lens == nullptr ? 0 : max(min(p.lens[b], p.max_len), -1);
}
__device__ inline int tile_units(const Pass& p, int len) {
  const int steps = ceil_div(p.prefix_len, kStep) + ceil_div(max(len, 0), kStep);
  return max(1, ceil_div(steps, kWaves));  // a tile without tokens is one empty unit
}

// Units of the sequences before `b` (sum over one tile each), and where a
// position on that line lies.  All threads call it; the answer is uniform.
struct Line {
  int64_t total;       // units of all sequences, one tile each
  int64_t share;       // units of a workgroup, all tiles counted
  int64_t* scratch;    // LDS, kWaves + 2
  int per;
  int64_t before;      // units before this thread's sequences
  __device__ Line(const Pass& p, int tiles_per_seq, int64_t* scratch_) : scratch(scratch_) {
    per = ceil_div(p.batch, kThreads);
    const int b0 = threadIdx.x * per;
    int64_t sum = 0;
    for (int b = b0; b < min(b0 + per, p.batch); ++b) sum += tile_units(p, own_len(p, b));
    int64_t incl = sum;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int64_t up = __shfl_up(incl, off);
      if (lane >= off) incl += up;
    }
    if (lane == 63) scratch[wave] = incl;
    __syncthreads();
    before = incl - sum;
    total = 0;
    for (int w = 0; w < kWaves; ++w) {
      if (w < wave) before += scratch[w];
      total += scratch[w];
    }
    const int64_t all = total * tiles_per_seq;
    share = (all + p.workgroups - 1) / p.workgroups;
  }
  // The sequence that holds position v of the line, and the units before it.
  __device__ void find(const Pass& p, int64_t v, int* seq, int64_t* seq_before) {
    int64_t at = before;
    const int b0 = threadIdx.x * per;
    for (int b = b0; b < min(b0 + per, p.batch); ++b) {
      const int u = tile_units(p, own_len(p, b));
      if (v >= at && v < at + u) {
        scratch[kWaves] = b;
        scratch[kWaves + 1] = at;
      }
      at += u;
    }
    __syncthreads();
    *seq = (int)scratch[kWaves];
    *seq_before = scratch[kWaves + 1];
    __syncthreads();
  }
  // The units before sequence b.
  __device__ int64_t before_seq(const Pass& p, int b) {
    const int b0 = threadIdx.x * per;
    if (b >= b0 && b < b0 + per) {
      int64_t at = before;
      for (int i = b0; i < b; ++i) at += tile_units(p, own_len(p, i));
      scratch[kWaves] = at;
    }
    __syncthreads();
    const int64_t at = scratch[kWaves];
    __syncthreads();
    return at;
  }
};

// 8 E4M3 bytes -> 8 bf16 values times the power of two `s` (exact).
__device__ inline bf16x8 decode8(uint32_t a, uint32_t b, float s) {
  const bf16x2_t p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)a, s, false);
  const bf16x2_t p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)a, s, true);
  const bf16x2_t p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)b, s, false);
  const bf16x2_t p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)b, s, true);
  return bf16x8{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
}

__device__ inline float byte_scale(uint32_t word, int byte) {
  return __uint_as_float(((word >> (8 * byte)) & 0xFFu) << 23);
}

// The leading bf16 term of each of 8 floats, which keep what is left.
__device__ inline bf16x8 take_term(float f[8]) {
  bf16x8 r;
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const uint32_t w = pack_bf16x2(f[i], f[i + 1]);
    const bf16x2_t t = __builtin_bit_cast(bf16x2_t, w);
    r[i] = t[0];
    r[i + 1] = t[1];
    f[i] -= __uint_as_float(w << 16);
    f[i + 1] -= __uint_as_float(w & 0xFFFF0000u);
  }
  return r;
}

// 1 / l, 0 for a row without tokens.
__device__ inline float inverse_sum(float l) { return l > 0.0f ? 1.0f / l : 0.0f; }

template <int DT>
__device__ inline void store_out4(const KvAttnArgs& a, int token, int head, int d, const float* v) {
  if constexpr (DT == NVFP4_DTYPE_BF16) {
    uint16_t* const p = (uint16_t*)a.out + token * a.ld_out + (int64_t)head * a.c.dim + d;
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
  } else {
    float* const p = (float*)a.out + token * a.ld_out + (int64_t)head * a.c.dim + d;
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  }
}

// T = bf16 terms of a query element and of a softmax weight: 1 for bf16
// queries (exact; the weights are rounded to 8 bits, relative 2^-9 each), 3
// for float32 (24 bits).
template <int DT, int D>
__global__ __launch_bounds__(kThreads) void kv_attention_kernel(KvAttnArgs a, Pass p) {
  constexpr int T = DT == NVFP4_DTYPE_BF16 ? 1 : 3;
  constexpr int KJ = D / 64;   // 16-byte pieces of a token that a lane holds
  constexpr int DT16 = D / 16; // output tiles of 16 dimensions
  constexpr int kPad = D + 4;
  __shared__ __attribute__((aligned(16))) float lds_o[kWaves][kTileRows][kPad];
  __shared__ float lds_ml[kWaves][kTileRows][2];
  __shared__ int64_t lds_line[kWaves + 2];

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i = lane & 15, g = lane >> 4;
  const int tiles_per_seq = a.c.heads * p.row_tiles;
  const int prefix_steps = ceil_div(p.prefix_len, kStep);
  const int page_blocks_shift = a.c.page_shift - 4, page_blocks_mask = (1 << page_blocks_shift) - 1;

  Line line(p, tiles_per_seq, lds_line);
  int64_t unit = (int64_t)blockIdx.x * line.share;
  const int64_t last_unit = min(unit + line.share, line.total * tiles_per_seq);
  if (unit >= last_unit) return;
  int seq;
  int64_t seq_before;
  line.find(p, unit / tiles_per_seq, &seq, &seq_before);

  int len = own_len(p, seq), units = tile_units(p, len);
  int x = (int)((unit - seq_before * tiles_per_seq) / units);  // tile of the sequence
  int u0 = (int)(unit - seq_before * tiles_per_seq - (int64_t)x * units);

  while (true) {
    const int u1 = (int)min((int64_t)units, u0 + (last_unit - unit));
    const int kvh = x / p.row_tiles, row0 = (x - kvh * p.row_tiles) * kTileRows;
    const int steps = prefix_steps + ceil_div(max(len, 0), kStep);
    const int tile = seq * tiles_per_seq + x;

    // This lane's query row and the first own token that it does not see.
    const int row = min(row0 + i, p.rows - 1);
    const int row_token = row / p.group;
    const int64_t token = (int64_t)seq * p.q_len + row_token;
    const int limit = len - p.q_len + 1 + row_token;
    const int tile_last = min(row0 + kTileRows, p.rows) - 1;
    const int limit_first = len - p.q_len + 1 + row0 / p.group, limit_last = len - p.q_len + 1 + tile_last / p.group;

    bf16x8 qf[T][2 * KJ];
    {
      const int head = kvh * p.group + row - row_token * p.group;
#pragma unroll
      for (int j = 0; j < 2 * KJ; ++j) {
        const int64_t at = token * a.ld_q + (int64_t)head * D + (4 * (j >> 1) + g) * 16 + 8 * (j & 1);
        if constexpr (T == 1) {
          qf[0][j] = *reinterpret_cast<const bf16x8*>((const uint16_t*)a.q + at);
        } else {
          const float* s = (const float*)a.q + at;
          const float4 lo = *reinterpret_cast<const float4*>(s), hi = *reinterpret_cast<const float4*>(s + 4);
          float f[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
          for (int t = 0; t < T; ++t) qf[t][j] = take_term(f);
        }
      }
    }

    float m = kLowest, l = 0.0f;
    f32x4 o[DT16];
#pragma unroll
    for (int d = 0; d < DT16; ++d) o[d] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    // Where a step's tokens are: `list` of pages, first token `base`, tokens
    // of the list `n` (those that any row of the tile sees).
    auto step_list = [&](int s, const int*& list, int& base, int& n) {
      if (s < prefix_steps) {
        list = a.prefix_pages;
        base = s * kStep;
        n = p.prefix_len;
      } else {
        list = a.table + seq * a.ld_table;
        base = (s - prefix_steps) * kStep;
        n = limit_last;
      }
    };
    // A wave's next step from s on that holds a visible token, or -1.
    auto next_step = [&](int s) {
      const int end = min(u1 * kWaves, steps);
      if (s >= end) return -1;
      if (s >= prefix_steps && (s - prefix_steps) * kStep >= limit_last) return -1;  // later ones neither
      return s;
    };
    // Page ids of the lane's key block (i / 4) and value block (g); blocks
    // past the last token take the last one's page and are masked below.
    auto page_ids = [&](int s, int& pk, int& pv) {
      const int* list;
      int base, n;
      step_list(s, list, base, n);
      const int last = (n - 1) >> 4;
      pk = list[min((base >> 4) + (i >> 2), last) >> page_blocks_shift];
      pv = list[min((base >> 4) + g, last) >> page_blocks_shift];
    };
    // Byte offset of token block `blk` (of its page) in codes; scales are at / D.
    auto block_at = [&](int blk) { return (kvh << a.c.page_shift) + (blk & page_blocks_mask) * 16; };

    uint4 kq[4][KJ], ksc;
    auto load_keys = [&](int s, int pk) {
      const int* list;
      int base, n;
      step_list(s, list, base, n);
      const int page = (unsigned)pk < (unsigned)a.c.n_pages ? pk : 0;
      const int at = block_at(min((base >> 4) + (i >> 2), (n - 1) >> 4));
      const uint8_t* src = a.c.kc + page * a.c.ld_codes + (int64_t)at * D + g * 64 + (i & 3) * 16;
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int j = 0; j < KJ; ++j) kq[t][j] = *reinterpret_cast<const uint4*>(src + t * (4 * D) + j * 256);
      ksc = *reinterpret_cast<const uint4*>(a.c.ks + page * a.c.ld_scales + at);
    };

    int s = next_step(u0 * kWaves + wave);
    int pk = 0, pv = 0;
    if (s >= 0) {
      page_ids(s, pk, pv);
      load_keys(s, pk);
    }
    while (s >= 0) {
      const int* list;
      int base, n;
      step_list(s, list, base, n);
      const bool prefix = s < prefix_steps;
      const bool bad = (unsigned)pv >= (unsigned)a.c.n_pages;
      const int sn = next_step(s + kWaves);
      int pkn = 0, pvn = 0;
      if (sn >= 0) page_ids(sn, pkn, pvn);

      // values of this step
      uint4 vq[DT16], vsc;
      {
        const int page = bad ? 0 : pv;
        const int at = block_at(min((base >> 4) + g, (n - 1) >> 4));
        const uint8_t* src = a.c.vc + page * a.c.ld_codes + (int64_t)at * D + i * 16;
#pragma unroll
        for (int d = 0; d < DT16; ++d) vq[d] = *reinterpret_cast<const uint4*>(src + d * 256);
        vsc = *reinterpret_cast<const uint4*>(a.c.vs + page * a.c.ld_scales + at);
      }

      // scores: sc[t][r] is token 4 t + r of block g
      f32x4 sc[4];
      const uint32_t kw[4] = {ksc.x, ksc.y, ksc.z, ksc.w};
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const float ks = byte_scale(kw[t], i & 3);
        f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < KJ; ++j) {
          const bf16x8 k0 = decode8(kq[t][j].x, kq[t][j].y, ks), k1 = decode8(kq[t][j].z, kq[t][j].w, ks);
#pragma unroll
          for (int e = T - 1; e >= 0; --e) {
            acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k0, qf[e][2 * j], acc, 0, 0, 0);
            acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k1, qf[e][2 * j + 1], acc, 0, 0, 0);
          }
        }
        sc[t] = acc;
      }
      if (sn >= 0) load_keys(sn, pkn);

      const uint32_t vw[4] = {vsc.x, vsc.y, vsc.z, vsc.w};
      float vs[4][4];
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) vs[t][r] = byte_scale(vw[t], r);

      // Tokens that this row does not see, and bytes of the cache that hold
      // no token that any row sees (they may be NaN codes: 0 * NaN).
      const bool masked = prefix ? base + kStep > n : base + kStep > limit_first;
      if (masked || __any(bad)) {
        const int first = base + 16 * g;
        const int sees = bad ? 0 : (prefix ? n : limit) - first;  // of this row in block g
        const int holds = bad ? 0 : n - first;                   // of any row
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            sc[t][r] = 4 * t + r < sees ? sc[t][r] : -__builtin_inff();
            vs[t][r] = 4 * t + r < sees ? vs[t][r] : 0.0f;
          }
        uint32_t keep[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const int c = min(max(holds - 4 * t, 0), 4);
          keep[t] = c == 4 ? 0xFFFFFFFFu : (1u << (8 * c)) - 1u;
        }
#pragma unroll
        for (int d = 0; d < DT16; ++d) {
          vq[d].x &= keep[0];
          vq[d].y &= keep[1];
          vq[d].z &= keep[2];
          vq[d].w &= keep[3];
        }
      }

      float top = fmaxf(fmaxf(sc[0][0], sc[0][1]), fmaxf(sc[0][2], sc[0][3]));
#pragma unroll
      for (int t = 1; t < 4; ++t) top = fmaxf(top, fmaxf(fmaxf(sc[t][0], sc[t][1]), fmaxf(sc[t][2], sc[t][3])));
      top = fmaxf(top, __shfl_xor(top, 16));
      top = fmaxf(top, __shfl_xor(top, 32));
      const float mn = fmaxf(m, top * a.scale_log2);
      if (__any(mn > m)) {
        const float f = __builtin_amdgcn_exp2f(m - mn);
        l *= f;
#pragma unroll
        for (int d = 0; d < DT16; ++d) o[d] *= f;
        m = mn;
      }
      float w[16];
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float e = __builtin_amdgcn_exp2f(fmaf(sc[t][r], a.scale_log2, -m));
          l += e;
          w[4 * t + r] = e * vs[t][r];
        }
      bf16x8 pf[T][2];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int t = 0; t < T; ++t) pf[t][h] = take_term(w + 8 * h);

#pragma unroll
      for (int d = 0; d < DT16; ++d) {
        const bf16x8 v0 = decode8(vq[d].x, vq[d].y, 1.0f), v1 = decode8(vq[d].z, vq[d].w, 1.0f);
#pragma unroll
        for (int e = T - 1; e >= 0; --e) {
          o[d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v0, pf[e][0], o[d], 0, 0, 0);
          o[d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v1, pf[e][1], o[d], 0, 0, 0);
        }
      }
      s = sn;
      pv = pvn;
    }

    // Join the four waves.
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    if (g == 0) {
      lds_ml[wave][i][0] = m;
      lds_ml[wave][i][1] = l;
    }
#pragma unroll
    for (int d = 0; d < DT16; ++d) *reinterpret_cast<f32x4*>(&lds_o[wave][i][16 * d + 4 * g]) = o[d];
    __syncthreads();
    const bool whole = p.direct && u0 == 0 && u1 == units;
    const int64_t slot = (int64_t)tile + blockIdx.x;
    for (int e = threadIdx.x; e < kTileRows * (D / 4); e += kThreads) {
      const int r = e / (D / 4), d = (e - r * (D / 4)) * 4;
      if (row0 + r >= p.rows) break;
      float top = lds_ml[0][r][0];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) top = fmaxf(top, lds_ml[w][r][0]);
      float sum = 0.0f;
      f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const float f = __builtin_amdgcn_exp2f(lds_ml[w][r][0] - top);
        sum += lds_ml[w][r][1] * f;
        acc += *reinterpret_cast<const f32x4*>(&lds_o[w][r][d]) * f;
      }
      if (whole) {
        if (len >= 0) {
          const float inv = inverse_sum(sum);
          const float v[4] = {acc[0] * inv, acc[1] * inv, acc[2] * inv, acc[3] * inv};
          const int rt = (row0 + r) / p.group;
          store_out4<DT>(a, seq * p.q_len + rt, kvh * p.group + row0 + r - rt * p.group, d, v);
        }
      } else {
        *reinterpret_cast<f32x4*>(p.o + (slot * kTileRows + r) * D + d) = acc;
        if (d == 0) *reinterpret_cast<float2*>(p.ml + (slot * kTileRows + r) * 2) = make_float2(top, sum);
      }
    }
    __syncthreads();

    unit += u1 - u0;
    if (unit >= last_unit) break;
    u0 = 0;
    if (++x == tiles_per_seq) {
      x = 0;
      ++seq;
      len = own_len(p, seq);
      units = tile_units(p, len);
    }
  }
}

// Joins the pieces of the rows: of the sequence's own pass and, where the
// prefix was computed for all rows together, of that pass.  A workgroup
// takes one tile of the own pass, a wave one row at a time.
template <int DT, int D>
__global__ __launch_bounds__(kThreads) void kv_attention_join_kernel(KvAttnArgs a, Pass own, Pass shared) {
  constexpr int V = D / 64;  // dimensions of a lane
  __shared__ int64_t lds_line[kWaves + 2];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int tiles_per_seq = a.c.heads * own.row_tiles;
  const int tile = blockIdx.x, seq = tile / tiles_per_seq, x = tile - seq * tiles_per_seq;
  const int kvh = x / own.row_tiles, row0 = (x - kvh * own.row_tiles) * kTileRows;
  const int len = own_len(own, seq);
  Line line(own, tiles_per_seq, lds_line);
  const int units = tile_units(own, len);
  const int64_t first = line.before_seq(own, seq) * tiles_per_seq + (int64_t)x * units;
  const int w0 = (int)(first / line.share), w1 = (int)((first + units - 1) / line.share);
  if (len < 0) return;
  if (own.direct && w0 == w1) return;

  int64_t shared_share = 1;
  const int shared_units = shared.batch ? tile_units(shared, 0) : 0;
  if (shared.batch) shared_share = ((int64_t)shared_units * a.c.heads * shared.row_tiles + shared.workgroups - 1) / shared.workgroups;

  for (int r = wave; r < kTileRows && row0 + r < own.rows; r += kWaves) {
    const int row = row0 + r, row_token = row / own.group, h = row - row_token * own.group;
    const int token = seq * own.q_len + row_token;
    float m = kLowest, l = 0.0f, acc[V] = {};
    auto add = [&](const Pass& p, int64_t at) {
      const float2 ml = *reinterpret_cast<const float2*>(p.ml + at * 2);
      if (ml.y == 0.0f) return;  // no token in this piece
      const float mn = fmaxf(m, ml.x), f = __builtin_amdgcn_exp2f(m - mn), fp = __builtin_amdgcn_exp2f(ml.x - mn);
      l = l * f + ml.y * fp;
      const float* src = p.o + at * D + lane * V;
#pragma unroll
      for (int e = 0; e < V; ++e) acc[e] = acc[e] * f + src[e] * fp;
      m = mn;
    };
    if (shared.batch) {
      const int64_t pr = (int64_t)token * shared.group + h;
      const int t = kvh * shared.row_tiles + (int)(pr / kTileRows);
      const int64_t u = (int64_t)t * shared_units;
      for (int64_t w = u / shared_share; w <= (u + shared_units - 1) / shared_share; ++w)
        add(shared, (t + w) * kTileRows + pr % kTileRows);
    }
    for (int w = w0; w <= w1; ++w) add(own, ((int64_t)tile + w) * kTileRows + r);
    const float inv = inverse_sum(l);
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] *= inv;
    const int64_t at = token * a.ld_out + (int64_t)(kvh * own.group + h) * D + lane * V;
    if constexpr (DT == NVFP4_DTYPE_F32) {
#pragma unroll
      for (int e = 0; e < V; ++e) ((float*)a.out)[at + e] = acc[e];
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) ((uint16_t*)a.out)[at + e] = (uint16_t)f32_to_bf16_bits(acc[e]);
    }
  }
}

// ------------------------------------------------------------ host side

struct Plan {
  Pass own{}, shared{};  // shared.batch == 0: no such pass
  bool join;
  size_t floats;
};

Plan make_plan(const KvAttnArgs& a) {
  Plan pl{};
  Pass& own = pl.own;
  own.batch = a.batch;
  own.q_len = a.q_len;
  own.group = a.group;
  own.rows = a.q_len * a.group;
  own.row_tiles = ceil_div(own.rows, kTileRows);
  own.lens = a.lens;
  own.max_len = a.max_len;
  const bool share = a.batch > 1 && a.prefix_len >= 256;
  own.prefix_len = share ? 0 : a.prefix_len;
  own.direct = !share;
  const int max_units = ceil_div(ceil_div(own.prefix_len, kStep) + ceil_div(own.max_len, kStep), kWaves);
  const int64_t own_tiles = (int64_t)own.batch * a.c.heads * own.row_tiles;
  own.workgroups = (int)min(own_tiles * max(max_units, 1), (int64_t)(a.c.dim == 256 ? 256 : 512));
  pl.join = share || max_units > 1;
  size_t slots = (size_t)own_tiles + own.workgroups;
  size_t at = pl.join ? slots * kTileRows * (2 + a.c.dim) : 0;
  if (share) {
    Pass& sh = pl.shared;
    sh.batch = 1;
    sh.q_len = a.batch * a.q_len;
    sh.group = a.group;
    sh.rows = sh.q_len * a.group;
    sh.row_tiles = ceil_div(sh.rows, kTileRows);
    sh.prefix_len = a.prefix_len;
    const int64_t tiles = (int64_t)a.c.heads * sh.row_tiles;
    sh.workgroups = (int)min(tiles * ceil_div(ceil_div(a.prefix_len, kStep), kWaves), (int64_t)(a.c.dim == 256 ? 256 : 512));
    at += (size_t)(tiles + sh.workgroups) * kTileRows * (2 + a.c.dim);
  }
  pl.floats = at;
  return pl;
}

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

size_t kv_attention_workspace(const KvAttnArgs& a) {
  return a.batch == 0 ? 16 : 16 + sizeof(float) * make_plan(a).floats;
}

hipError_t launch_kv_attention(const KvAttnArgs& a, void* ws, hipStream_t s) {
  Plan pl = make_plan(a);
  const int64_t own_tiles = (int64_t)pl.own.batch * a.c.heads * pl.own.row_tiles;
  float* at = (float*)ws;
  auto place = [&](Pass& p, int64_t tiles) {
    const int64_t slots = tiles + p.workgroups;
    p.o = at;
    p.ml = at + slots * kTileRows * a.c.dim;
    at = p.ml + slots * kTileRows * 2;
  };
  place(pl.own, own_tiles);
  if (pl.shared.batch) place(pl.shared, (int64_t)a.c.heads * pl.shared.row_tiles);
  hipError_t err = hipSuccess;
  for_types(a.dtype, a.c.dim, [&](auto dt, auto d) {
    if (pl.shared.batch) {
      kv_attention_kernel<dt(), d()><<<pl.shared.workgroups, kThreads, 0, s>>>(a, pl.shared);
      if ((err = hipGetLastError()) != hipSuccess) return;
    }
    kv_attention_kernel<dt(), d()><<<pl.own.workgroups, kThreads, 0, s>>>(a, pl.own);
    if ((err = hipGetLastError()) != hipSuccess || !pl.join) return;
    kv_attention_join_kernel<dt(), d()><<<(int)own_tiles, kThreads, 0, s>>>(a, pl.own, pl.shared);
    err = hipGetLastError();
  });
  return err;
}

}  // namespace nvfp4
