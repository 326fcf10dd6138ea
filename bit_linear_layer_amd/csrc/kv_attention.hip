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
// units of one step for each wave that takes other tokens (256 tokens here),
// form one line that is cut into equal shares, one per workgroup or, for many
// short tiles, per wave.  A tile that a cut divides leaves partial (M, l, o)
// in the workspace, in slot tile + share (distinct for every piece, since one
// of the two grows from piece to piece), and a second kernel joins them.
// Larger tiles, for more rows, are described at rows_body and wide_body.
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
constexpr int kStep = 64;       // tokens of one wave's step (16-row tiles)
constexpr int kTileRows = 16;
// Larger tiles rescale their accumulators only when a row's maximum has grown by
// more than 2^kSlack: at every growth of any of 32 rows it would be more than
// half of the steps of a few thousand tokens (512-token chunks of four prompts
// 213 -> 203 us).  Weights then reach 2^6 and round to bf16 as any others, also the
// largest one, which would otherwise be 1: the error against 64 bits is 0.0021
// of the output's root mean square instead of 0.0018, the output's own rounding
// 0.0017.  16-row tiles wait for memory and keep the maximum exact.
constexpr float kSlack = 6.0f;
constexpr float kLowest = -3.0e38f;  // stands for "no token yet"; finite, so differences are never NaN

// The running maximum M of a row and its weights' exponents c x - M, x a score.
// M = c max(x) is rounded, so even the largest score's exponent is off by up to
// 2^-25 |M|, which the sum l and the output o share.  From |M| = 2^28 on that would
// soon be more than a float's exponent holds (scores around 2^32: sums of 0 or
// infinity), while a score's own rounding is 2^4 and more in the exponent.
// There c and M are kept scaled by the power of two that brings M below 2^28: a
// score n roundings below the largest then has a weight of 2^(-8 n) at most, as
// good as nothing, though not as little as it should.  Only a new maximum
// changes the scale, so a step without one costs nothing.
struct Maximum {
  float c, m;  // scaled
  __device__ explicit Maximum(float scale) : c(scale), m(kLowest) {}
  __device__ float exponent(float x) const { return fmaf(x, c, -m); }
  __device__ bool passed(float top, float slack) const { return top * c > m + slack; }
  // M, not scaled
  __device__ float value(float scale) const { return ldexpf(m, __builtin_amdgcn_frexp_expf(scale) - __builtin_amdgcn_frexp_expf(c)); }
  // M becomes at least that of a score `top`: what that multiplies l and o by.
  __device__ float raise(float scale, float top) {
    const float old = value(scale), now = fmaxf(old, top * scale);
    // |M| < 2^128 scale bounds the exponent, also where M is still kLowest
    const int k = min(max(__builtin_amdgcn_frexp_expf(now) - 28, 0), max(__builtin_amdgcn_frexp_expf(scale) + 100, 0));
    c = ldexpf(scale, -k);
    m = ldexpf(now, -k);
    return __builtin_amdgcn_exp2f(old - now);
  }
};

// One pass over tiles of rows: what the stream kernel and the join share.
struct Pass {
  int batch;      // sequences (1 where the rows of all share their tokens)
  int rows;       // query rows of a sequence and kv head: q_len * group
  int q_len, group;
  int tile_rows;  // query rows of a tile
  int step;       // tokens of a wave's step
  int step_waves; // waves of a workgroup that take different steps
  int row_tiles;  // ceil(rows / tile_rows)
  int prefix_len; // shared tokens this pass reads for every tile
  const int* lens;  // null: no tokens of the sequences' own
  int max_len;
  int workgroups;
  int start;      // what a tile's beginning and end take, in units
  int solo;       // a share is a wave's, not a workgroup's (16-row tiles, step_waves 1)
  int direct;     // every tile is whole in one workgroup and nothing joins it: write the output
  float* ml;      // partials: [slot][tile_rows][2] and [slot][tile_rows][D]
  float* o;
  int2* head;     // [tile]: the workgroup with its first unit, and the number of its pieces
};

__device__ __host__ inline int ceil_div(int a, int b) { return (a + b - 1) / b; }

__device__ inline int own_len(const Pass& p, int b) {
  return p.lens == nullptr ? 0 : max(min(p.lens[b], p.max_len), -1);
}
__device__ __host__ inline int pass_shares(const Pass& p) { return p.solo ? p.workgroups * kWaves : p.workgroups; }
__device__ inline int ceil_pow2(int a, int b) { return (a + b - 1) >> __builtin_ctz(b); }
// Units of row tile `rt` of a sequence with `len` own tokens: those that its
// last row sees.  A tile without tokens is one empty unit.
__device__ inline int tile_units(const Pass& p, int len, int rt) {
  if (len < 0) return 1;  // no sequence, no result
  const int last = min((rt + 1) * p.tile_rows, p.rows) - 1;
  const int seen = max(len - p.q_len + 1 + (p.q_len == 1 ? 0 : last / p.group), 0);
  return max(1, ceil_pow2(ceil_pow2(p.prefix_len, p.step) + ceil_pow2(seen, p.step), p.step_waves));
}

// The tiles lie on a line of units: sequence by sequence, row tile by row
// tile, and of each the kv heads, which all have the same units.  All threads
// call this; the answers are uniform.
struct Line {
  int64_t units;       // of all row tiles, one head each
  int start;           // what counts as units before each tile's own
  int64_t share, all;  // of a share and in total, starts included, all heads counted
  int64_t* scratch;    // LDS, 2 * kWaves
  int per;
  int64_t before;      // units before this thread's row tiles, starts included
  __device__ Line(const Pass& p, int heads, int64_t* scratch_) : scratch(scratch_) {
    const int n = pass_shares(p), tiles = p.batch * p.row_tiles;
    per = ceil_div(tiles, kThreads);
    if (tiles == 1) {  // no scan (one sequence's first tokens: 8.6 -> 7.4 us)
      units = tile_units(p, own_len(p, 0), 0);
      before = 0;
    } else {
      int64_t sum = 0;
      each(p, [&](int, int, int u) { sum += u; });
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
      units = 0;
      for (int w = 0; w < kWaves; ++w) {
        if (w < wave) before += scratch[w];
        units += scratch[w];
      }
    }
    // where shares are a few units, they would only become more uneven
    start = units * heads >= 4 * (int64_t)n ? p.start : 0;
    before += (int64_t)start * min((int64_t)threadIdx.x * per, (int64_t)tiles);
    all = (units + (int64_t)start * tiles) * heads;
    share = (all + n - 1) / n;
  }
  // The row tile in which share `wg` begins, and what lies before it on the
  // line (one head each); in a solo pass wave w asks for share wg + w.
  __device__ void find(const Pass& p, int heads, int wg, int* seq, int* rt, int64_t* units_before) {
    *seq = *rt = 0;
    *units_before = 0;
    if (p.batch * p.row_tiles == 1) return;
    const int n = p.solo ? kWaves : 1;
    int64_t want[kWaves];
    for (int w = 0; w < n; ++w) want[w] = (wg + w) * share / heads;
    __syncthreads();  // the scan's sums are read
    int64_t pos = before;
    each(p, [&](int b, int r, int u) {
      u += start;
      for (int w = 0; w < n; ++w)
        if (want[w] >= pos && want[w] < pos + u) {
          scratch[2 * w] = (int64_t)b << 32 | r;
          scratch[2 * w + 1] = pos;
        }
      pos += u;
    });
    __syncthreads();
    const int mine = p.solo ? threadIdx.x >> 6 : 0;
    *seq = (int)(scratch[2 * mine] >> 32);
    *rt = (int)scratch[2 * mine];
    *units_before = scratch[2 * mine + 1];
  }

 private:
  template <class F>
  __device__ void each(const Pass& p, F f) const {  // this thread's row tiles
    const int e0 = threadIdx.x * per, n = min(per, p.batch * p.row_tiles - e0);
    if (n <= 0) return;
    int b = p.row_tiles == 1 ? e0 : e0 / p.row_tiles, r = e0 - b * p.row_tiles, len = own_len(p, b);
    for (int k = 0; k < n; ++k) {
      f(b, r, tile_units(p, len, r));
      if (++r == p.row_tiles) {
        r = 0;
        len = own_len(p, min(++b, p.batch - 1));
      }
    }
  }
};

// A walk over a share, tile by tile, and of each the units [u0, u1).
// SOLO: each wave walks a share of its own.
template <bool SOLO>
struct Walk {
  int wg;  // the share's number
  int64_t at, end, last;  // on the line: this piece, the share's end
  int heads;
  int seq, rt, kvh, tile;  // sequence, its row tile and kv head; the tile's place on the line
  int len, units;          // of the sequence, of the tile
  int u0, u1;
  bool any;
  // Workgroups are dealt to the 8 XCDs in turn; each XCD gets neighbouring
  // shares, which read the same pages (row tiles of a head, parts of one
  // sequence) and find them in its L2.
  __device__ Walk(const KvAttnArgs& a, const Pass& p, int dealt, int64_t* scratch) {
    const int q = p.workgroups / 8, r = p.workgroups % 8, xcd = dealt % 8;
    wg = xcd * q + min(xcd, r) + dealt / 8;
    const int first = SOLO ? wg * kWaves : wg;  // share of the workgroup's first wave
    wg = SOLO ? first + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) : first;
    heads = a.c.heads;
    Line line(p, heads, scratch);
    share = uniform(line.share);
    start = __builtin_amdgcn_readfirstlane(line.start);
    at = wg * share;
    last = uniform(min(at + share, line.all));
    any = at < last;
    if (!SOLO && !any) return;
    int64_t before;
    line.find(p, heads, first, &seq, &rt, &before);  // (past the end nothing is found)
    if (!any) return;
    seq = __builtin_amdgcn_readfirstlane(seq);
    rt = __builtin_amdgcn_readfirstlane(rt);
    before = uniform(before) * heads;
    len = __builtin_amdgcn_readfirstlane(own_len(p, seq));
    units = __builtin_amdgcn_readfirstlane(tile_units(p, len, rt));
    kvh = __builtin_amdgcn_readfirstlane((int)((at - before) / (start + units)));
    place(p, __builtin_amdgcn_readfirstlane((int)(at - before - (int64_t)kvh * (start + units))));
    if (u0 == u1) any = next(p);
  }
  __device__ bool next(const Pass& p) {
    do {
      at = end;
      if (at >= last) return false;
      if (++kvh == heads) {
        kvh = 0;
        if (++rt == p.row_tiles) {
          rt = 0;
          ++seq;
          len = __builtin_amdgcn_readfirstlane(own_len(p, seq));
        }
        units = __builtin_amdgcn_readfirstlane(tile_units(p, len, rt));
      }
      place(p, 0);
    } while (u0 == u1);  // a start only
    return true;
  }
  // every unit of the tile is this workgroup's
  __device__ bool whole() const { return u0 == 0 && u1 == units; }

 private:
  int64_t share;
  int start;
  // A value that all lanes hold, in scalar registers.
  static __device__ int64_t uniform(int64_t v) {
    return (int64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)v) | (int64_t)__builtin_amdgcn_readfirstlane((int)(v >> 32)) << 32;
  }
  // The share's part of the tile, `from` units (starts included) after its first.
  __device__ void place(const Pass& p, int from) {
    const int64_t tile_end = at - from + start + units;
    end = min(tile_end, last);
    u0 = max(from - start, 0);
    u1 = max(from - start + (int)(end - at), 0);
    tile = (seq * p.row_tiles + rt) * heads + kvh;
    // the join wants to know: the share of unit 0 and the number of pieces
    if (p.head != nullptr && u0 == 0 && u1 > 0 && (threadIdx.x & (SOLO ? 63 : kThreads - 1)) == 0)
      p.head[tile] = make_int2(wg, (int)((tile_end - 1) / share - wg) + 1);
  }
};

// v of the lane with number at / 4 (__shfl computes that number anew at each use).
__device__ inline float from_lane(int at, float v) {
  return __int_as_float(__builtin_amdgcn_ds_bpermute(at, __float_as_int(v)));
}

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

// The bytes of a dword that hold one of the first n tokens.
__device__ inline uint32_t keep_bytes(int n) {
  const int c = min(max(n, 0), 4);
  return c == 4 ? 0xFFFFFFFFu : (1u << (8 * c)) - 1u;
}

// A token's value may hold NaN codes.  Where only some rows of a tile see the
// token, its weight is 0 for the others, and 0 * NaN would reach them: so in
// the steps that hold such tokens the NaN codes are taken out of the bytes
// before the product (drop_nan), and the rows that see one get the NaN when
// their results are in memory (put_nan, from the cache once more; without NaN
// codes in these few tokens it is not called).

// Bit 7 of every byte that is a NaN code (0x7F, 0xFF).
__device__ inline uint32_t nan_bytes(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }
__device__ inline uint32_t nan_bytes(const uint4& v) { return nan_bytes(v.x) | nan_bytes(v.y) | nan_bytes(v.z) | nan_bytes(v.w); }

// Takes the NaN codes out of 16 codes; not zero if there were any.
__device__ inline uint32_t drop_nan(uint4& v) {
  uint32_t any = 0;
  auto word = [&](uint32_t& w) {
    asm("" : "+v"(w));  // what a test before computed is not kept: it would take as many registers again
    const uint32_t n = nan_bytes(w);
    w &= ~(n | (n - (n >> 7)));
    any |= n;
  };
  word(v.x);
  word(v.y);
  word(v.z);
  word(v.w);
  return any;
}

// Writes NaN into the results of row r of the tile, in each dimension that has a
// NaN code among the tokens that the row sees, from the first step (of STEP
// tokens) on that some row of the tile does not see.  This lane has the
// dimensions d .. d + 3 of d = first, first + stride ..
template <int DT, int D, int ROWS, int STEP, class W>
__device__ __attribute__((always_inline)) inline void put_nan(const KvAttnArgs& a, const Pass& p, const W& t, int r, int first, int stride) {
  // All is worked out anew from these: what the tile began with would have to
  // be kept in scalar registers, of which there are too few.
  int seq = t.seq, kvh = t.kvh, rt = t.rt, len = t.len;
  asm("" : "+v"(seq), "+v"(kvh), "+v"(rt), "+v"(len));
  const int row = rt * ROWS + r;
  if (row >= p.rows) return;
  const int row_token = row / p.group, limit = len - p.q_len + 1 + row_token;
  const int64_t token = (int64_t)seq * p.q_len + row_token;
  const int64_t at_out = token * a.ld_out + (int64_t)(kvh * p.group + row - row_token * p.group) * D;
  float* const partial = p.direct && t.whole() ? nullptr : p.o + (((int64_t)t.tile + t.wg) * ROWS + r) * D;
  const int page_blocks_shift = a.c.page_shift - 4, page_blocks_mask = (1 << page_blocks_shift) - 1;
  const int* const list = a.table + seq * a.ld_table;
  // (the tile's rows are ROWS tokens apart at most)
#pragma unroll 1
  for (int block = max(limit - ROWS, 0) / STEP * (STEP / 16); 16 * block < limit; ++block) {
    const int id = list[block >> page_blocks_shift];
    if ((unsigned)id >= (unsigned)a.c.n_pages) continue;
    const int64_t at = (int64_t)((kvh << a.c.page_shift) + (block & page_blocks_mask) * 16) * D;
    const uint8_t* const src = a.c.vc + (uint64_t)(unsigned)id * (uint64_t)a.c.ld_codes + at;
    const int sees = limit - 16 * block;
#pragma unroll 1
    for (int e = 0; e < 4 * (D / stride); ++e) {
      const int d = first + (e >> 2) * stride + (e & 3);
      const uint4 v = *reinterpret_cast<const uint4*>(src + d * 16);
      if (nan_bytes(make_uint4(v.x & keep_bytes(sees), v.y & keep_bytes(sees - 4), v.z & keep_bytes(sees - 8), v.w & keep_bytes(sees - 12))) == 0)
        continue;
      if (partial != nullptr) partial[d] = __builtin_nanf("");
      else if constexpr (DT == NVFP4_DTYPE_BF16) ((uint16_t*)a.out)[at_out + d] = 0x7FC0;
      else ((float*)a.out)[at_out + d] = __builtin_nanf("");
    }
  }
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
// queries (exact; the weights are rounded to 8 bits, at most 2^-8 of each),
// 3 for float32 (24 bits).
template <int DT>
constexpr int kTerms = DT == NVFP4_DTYPE_BF16 ? 1 : 3;

// LDS of a stream workgroup.  The queries' fragments lie there because all
// four waves use the same ones and their registers are wanted for bytes in
// flight (D = 256: 32 of 256).
template <int DT, int D>
struct StreamLds {
  float *part_a, *part_b;  // a wave's accumulators each: 16 * D
  uint4* q;                // [kTerms][D / 32][64], SOLO: for each wave
  float (*ml)[32][2];
  int64_t* line;
  int* nan_tile;           // the tile whose values had NaN codes taken out (any other number: perhaps none)
};

// PAIR: two workgroups share a CU, i.e. 256 registers a wave.
// SOLO: each wave has tiles of its own, from its queries to its result: for
// many short tiles, where four waves to a tile would mostly wait for each
// other and for the hand-over of their sums.
// OWN: the sequences' own tokens are among the pass's, not the shared prefix alone.
template <int DT, int D, bool PAIR, bool SOLO, bool OWN>
__device__ __attribute__((always_inline)) inline void stream_body(const KvAttnArgs& a, const Pass& p, const int wg,
                                                                  const StreamLds<DT, D>& lds) {
  constexpr int T = kTerms<DT>;
  constexpr int SW = SOLO ? 1 : kWaves;  // waves that share a tile
  constexpr int KJ = D / 64;   // 16-byte pieces of a token that a lane holds
  constexpr int DT16 = D / 16; // output tiles of 16 dimensions

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i = lane & 15, g = lane >> 4;
  const int lane16 = 4 * (lane ^ 16), lane32 = 4 * (lane ^ 32);  // see from_lane
  const int prefix_steps = ceil_div(p.prefix_len, kStep);
  const int page_blocks_shift = a.c.page_shift - 4, page_blocks_mask = (1 << page_blocks_shift) - 1;

  Walk<SOLO> t(a, p, wg, lds.line);
  if (!t.any) return;
  do {
    const int u0 = t.u0, u1 = t.u1, seq = t.seq, len = t.len, tile = t.tile;
    const int kvh = t.kvh, row0 = t.rt * kTileRows;

    // This lane's query row and the first own token that it does not see.
    const int row = min(row0 + i, p.rows - 1);
    const int row_token = row / p.group;
    const int64_t token = (int64_t)seq * p.q_len + row_token;
    const int limit = len - p.q_len + 1 + row_token;
    const int tile_last = min(row0 + kTileRows, p.rows) - 1;
    const int limit_first = len - p.q_len + 1 + row0 / p.group, limit_last = len - p.q_len + 1 + tile_last / p.group;
    const int steps = prefix_steps + ceil_div(max(limit_last, 0), kStep);  // with a visible token

    const int head = kvh * p.group + row - row_token * p.group;
    uint4* const queries = SOLO ? lds.q + wave * (T * 2 * KJ * 64) : lds.q;
    for (int j = SOLO ? 0 : wave; j < 2 * KJ; j += SOLO ? 1 : kWaves) {
      const int64_t at = token * a.ld_q + (int64_t)head * D + (4 * (j >> 1) + g) * 16 + 8 * (j & 1);
      if constexpr (T == 1) {
        queries[j * 64 + lane] = *reinterpret_cast<const uint4*>((const uint16_t*)a.q + at);
      } else {
        const float* s = (const float*)a.q + at;
        const float4 lo = *reinterpret_cast<const float4*>(s), hi = *reinterpret_cast<const float4*>(s + 4);
        float f[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
        for (int t = 0; t < T; ++t) queries[(t * 2 * KJ + j) * 64 + lane] = __builtin_bit_cast(uint4, take_term(f));
      }
    }

    Maximum most(a.scale_log2);
    float l = 0.0f;
    f32x4 o[DT16];
#pragma unroll
    for (int d = 0; d < DT16; ++d) o[d] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    // Where a step's tokens are: a list of pages, the first token `base`, and
    // the tokens of the list that any row of the tile sees.
    struct Where {
      const int* list;
      int base, n;
    };
    auto where = [&](int s) __attribute__((always_inline)) {
      if (s < prefix_steps) return Where{a.prefix_pages, s * kStep, p.prefix_len};
      return Where{a.table + seq * a.ld_table, (s - prefix_steps) * kStep, limit_last};
    };
    // A wave's next step from s on that holds a visible token, or -1.
    auto next_step = [&](int s) {
      return s < min(u1 * SW, steps) ? s : -1;
    };
    // Blocks past the last token take the last one's page and are masked below.
    auto block_of = [&](const Where& w, int b) { return min((w.base >> 4) + b, (w.n - 1) >> 4); };
    auto slot_of = [&](int blk) { return (kvh << a.c.page_shift) + (blk & page_blocks_mask) * 16; };
    auto row_of = [&](int id, int64_t ld) {
      return (uint64_t)((unsigned)id < (unsigned)a.c.n_pages ? (unsigned)id : 0u) * (uint64_t)(uint32_t)ld;
    };
    // Page ids of the lane's key block (i / 4) and value block (g).
    auto page_ids = [&](int s, int& pk, int& pv) __attribute__((always_inline)) {
      const Where w = where(s);
      pk = w.list[block_of(w, i >> 2) >> page_blocks_shift];
      pv = w.list[block_of(w, g) >> page_blocks_shift];
    };

    // With D = 256 a step's keys and values together do not fit the registers
    // of two waves per SIMD beside the accumulators: half of the values are
    // asked for when the keys are used up, and the next keys when the first
    // half of the values is.
    constexpr bool kLate = D == 256 && PAIR;
    constexpr int kFirst = kLate ? DT16 / 2 : DT16;
    uint4 kq[4][KJ], ksc;
    auto load_keys = [&](int s, int pk) __attribute__((always_inline)) {
      const int at = slot_of(block_of(where(s), i >> 2));
      const uint8_t* src = a.c.kc + row_of(pk, a.c.ld_codes) + (uint32_t)(at * D + g * 64 + (i & 3) * 16);
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int j = 0; j < KJ; ++j) kq[t][j] = *reinterpret_cast<const uint4*>(src + t * (4 * D) + j * 256);
      ksc = *reinterpret_cast<const uint4*>(a.c.ks + row_of(pk, a.c.ld_scales) + (uint32_t)at);
    };

    int s = next_step(SOLO ? u0 : u0 * SW + wave);
    int pk = 0, pv = 0;
    if (s >= 0) {
      page_ids(s, pk, pv);
      load_keys(s, pk);
    }
    bool nan = false;  // NaN codes were taken out
    if constexpr (!SOLO) __syncthreads();  // the queries are in LDS
    while (s >= 0) {
      const Where w = where(s);
      const bool prefix = s < prefix_steps;
      const bool bad = (unsigned)pv >= (unsigned)a.c.n_pages;
      const int sn = next_step(s + SW);
      int pkn = 0, pvn = 0;
      if (sn >= 0) page_ids(sn, pkn, pvn);

      // values of this step
      uint4 vq[DT16], vsc;
      const uint8_t* vsrc;
      {
        const int at = slot_of(block_of(w, g));
        vsrc = a.c.vc + row_of(pv, a.c.ld_codes) + (uint32_t)(at * D + i * 16);
#pragma unroll
        for (int d = 0; d < kFirst; ++d) vq[d] = *reinterpret_cast<const uint4*>(vsrc + d * 256);
        vsc = *reinterpret_cast<const uint4*>(a.c.vs + row_of(pv, a.c.ld_scales) + (uint32_t)at);
      }

      // scores: sc[t][r] is token 4 t + r of block g
      f32x4 sc[4];
      float ks[4];
      {
        const uint32_t kw[4] = {ksc.x, ksc.y, ksc.z, ksc.w};
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          ks[t] = byte_scale(kw[t], i & 3);
          sc[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
      }
#pragma unroll
      for (int j = 0; j < KJ; ++j)
#pragma unroll
        for (int e = T - 1; e >= 0; --e) {
          const bf16x8 q0 = __builtin_bit_cast(bf16x8, queries[(e * 2 * KJ + 2 * j) * 64 + lane]);
          const bf16x8 q1 = __builtin_bit_cast(bf16x8, queries[(e * 2 * KJ + 2 * j + 1) * 64 + lane]);
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            sc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(decode8(kq[t][j].x, kq[t][j].y, ks[t]), q0, sc[t], 0, 0, 0);
            sc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(decode8(kq[t][j].z, kq[t][j].w, ks[t]), q1, sc[t], 0, 0, 0);
          }
        }
      if constexpr (kLate) {
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int d = kFirst; d < DT16; ++d) vq[d] = *reinterpret_cast<const uint4*>(vsrc + d * 256);
      } else if (sn >= 0) {
        load_keys(sn, pkn);
      }

      // Tokens that this row does not see, and bytes of the cache that hold
      // no token that any row sees (they may be NaN codes and infinite
      // scales: 0 * NaN).
      const bool masked = prefix ? w.base + kStep > w.n : w.base + kStep > limit_first;
      if (masked || __any(bad)) {
        const int first = w.base + 16 * g;
        const int sees = bad ? 0 : (prefix ? w.n : limit) - first;  // of this row in block g
        const int holds = bad ? 0 : w.n - first;                    // of any row
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int r = 0; r < 4; ++r) sc[t][r] = 4 * t + r < sees ? sc[t][r] : -__builtin_inff();
        uint32_t keep[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) keep[t] = keep_bytes(holds - 4 * t);
        vsc.x &= keep[0];
        vsc.y &= keep[1];
        vsc.z &= keep[2];
        vsc.w &= keep[3];
#pragma unroll
        for (int d = 0; d < DT16; ++d) {
          vq[d].x &= keep[0];
          vq[d].y &= keep[1];
          vq[d].z &= keep[2];
          vq[d].w &= keep[3];
        }
        if (OWN && !prefix && limit_first < limit_last && w.base + kStep > limit_first) {
          uint32_t any = 0;
          if constexpr (kLate) {  // (tested first, as below, it would spill 100 registers more)
#pragma unroll
            for (int d = 0; d < DT16; ++d) {
              any |= drop_nan(vq[d]);
              __builtin_amdgcn_sched_barrier(0);
            }
            nan |= __any(any != 0);
          } else {
#pragma unroll
            for (int d = 0; d < DT16; ++d) any |= nan_bytes(vq[d]);
            if (__builtin_expect(__any(any != 0), 0)) {
              nan = true;
#pragma unroll
              for (int d = 0; d < DT16; ++d) drop_nan(vq[d]);
            }
          }
        }
      }

      float top = fmaxf(fmaxf(sc[0][0], sc[0][1]), fmaxf(sc[0][2], sc[0][3]));
#pragma unroll
      for (int t = 1; t < 4; ++t) top = fmaxf(top, fmaxf(fmaxf(sc[t][0], sc[t][1]), fmaxf(sc[t][2], sc[t][3])));
      top = fmaxf(top, from_lane(lane16, top));
      top = fmaxf(top, from_lane(lane32, top));
      if (__any(most.passed(top, 0.0f))) {
        const float f = most.raise(a.scale_log2, top);
        l *= f;
#pragma unroll
        for (int d = 0; d < DT16; ++d) o[d] *= f;
      }
      float wt[16];
      const uint32_t vw[4] = {vsc.x, vsc.y, vsc.z, vsc.w};
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float e = __builtin_amdgcn_exp2f(most.exponent(sc[t][r]));
          l += e;
          wt[4 * t + r] = e * byte_scale(vw[t], r);
        }
      bf16x8 pf[T][2];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int t = 0; t < T; ++t) pf[t][h] = take_term(wt + 8 * h);

#pragma unroll
      for (int d = 0; d < DT16; ++d) {
        if (kLate && d == kFirst) {
          __builtin_amdgcn_sched_barrier(0);
          if (sn >= 0) load_keys(sn, pkn);
        }
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

    float m = most.value(a.scale_log2);
    if (!SOLO && nan) *lds.nan_tile = tile;

    // Join the four waves, register by register: 2 and 3 hand theirs to 0 and
    // 1, then 1 to 0.
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    auto give = [&](float* to) __attribute__((always_inline)) {
      if (g == 0) {
        lds.ml[wave][i][0] = m;
        lds.ml[wave][i][1] = l;
      }
#pragma unroll
      for (int d = 0; d < DT16; ++d) *reinterpret_cast<f32x4*>(to + (d * 64 + lane) * 4) = o[d];
    };
    auto take = [&](const float* from, int other) __attribute__((always_inline)) {
      const float mo = lds.ml[other][i][0], mn = fmaxf(m, mo);
      const float f = __builtin_amdgcn_exp2f(m - mn), fo = __builtin_amdgcn_exp2f(mo - mn);
      l = l * f + lds.ml[other][i][1] * fo;
#pragma unroll
      for (int d = 0; d < DT16; ++d) o[d] = o[d] * f + *reinterpret_cast<const f32x4*>(from + (d * 64 + lane) * 4) * fo;
      m = mn;
    };
    if constexpr (!SOLO) {
      if (wave >= 2) give(wave == 2 ? lds.part_a : lds.part_b);
      __syncthreads();
      if (wave < 2) take(wave == 0 ? lds.part_a : lds.part_b, wave + 2);
      if (wave == 1) give(lds.part_b);
      __syncthreads();
      if (wave == 0) take(lds.part_b, 1);
    }
    if (SOLO || wave == 0) {
      const bool whole = p.direct && t.whole();
      const int64_t at = ((int64_t)tile + t.wg) * kTileRows + i;
      if (row0 + i < p.rows) {
        if (!whole) {
          if (g == 0) *reinterpret_cast<float2*>(p.ml + at * 2) = make_float2(m, l);
#pragma unroll
          for (int d = 0; d < DT16; ++d) *reinterpret_cast<f32x4*>(p.o + at * D + 16 * d + 4 * g) = o[d];
        } else if (len >= 0) {
          const float inv = inverse_sum(l);
#pragma unroll
          for (int d = 0; d < DT16; ++d) {
            const float v[4] = {o[d][0] * inv, o[d][1] * inv, o[d][2] * inv, o[d][3] * inv};
            store_out4<DT>(a, (int)token, head, 16 * d + 4 * g, v);
          }
        }
      }
      if constexpr (OWN)
        if (__builtin_expect(SOLO ? nan : __builtin_amdgcn_readfirstlane(*lds.nan_tile) == tile, 0))
          put_nan<DT, D, kTileRows, kStep>(a, p, t, i, 4 * g, 16);
    }
    if constexpr (!SOLO) __syncthreads();  // the queries and the hand-over are read
  } while (t.next(p));
}

// Two workgroups of a pass on a CU, except where one keeps more bytes in
// flight than two would.
template <int DT, int D>
constexpr bool kPaired = DT == NVFP4_DTYPE_BF16 && D < 256;

template <int DT, int D, bool SOLO>
__global__ __launch_bounds__(kThreads, (kPaired<DT, D>) ? 2 : 1) void kv_attention_kernel(KvAttnArgs a, Pass p) {
  __shared__ __attribute__((aligned(16))) float part_a[16 * D], part_b[16 * D];
  __shared__ uint4 q[kTerms<DT> * (D / 32) * 64 * (SOLO ? kWaves : 1)];
  __shared__ float ml[kWaves][32][2];
  __shared__ int64_t line[2 * kWaves];
  __shared__ int nan_tile;
  stream_body<DT, D, kPaired<DT, D>, SOLO, true>(a, p, blockIdx.x, StreamLds<DT, D>{part_a, part_b, q, ml, line, &nan_tile});
}

// The same for more rows (bf16): tiles of 32 * WM rows (WM = 1, 2; with D =
// 256 also 4) on 32 x 32 x 16 MFMA.  A wave owns 32 rows; WM waves work on the same tokens (a region of the
// step's LDS stage), 4 / WM regions hold different tokens.  Reading the bytes
// of 64 tokens (D = 128) from L2 for each wave on its own would ask for the
// whole 64 bytes a cycle of a CU's path to L2, so they come once per region
// by LDS DMA, two stages deep, laid out as the lanes read them: piece
// (tile of 32 tokens, 32 dimensions) is 1 KB, lane l's 16 bytes at 16 l.
//   key piece: row i = l % 32 is token 16 h + 4 (i / 8) + i % 4 with
//   h = i / 4 % 2, dimensions 16 (2 j + l / 32) ..; so register r of the
//   scores is token r of block l / 32, again the second product's B operand.
//   value piece: dimension l % 32, the 16 tokens of block l / 32.
template <int D, int WM>
struct RowsShape {
  static constexpr int kWM = WM, kWT = kWaves / WM;
  static constexpr int kTT = D == 256 ? 1 : 2;                 // 32-token tiles of a step
  static constexpr int kStepTokens = 32 * kTT;
  static constexpr int kD32 = D / 32;
  static constexpr int kHalf = kStepTokens * D;                // key (or value) bytes of a region
  static constexpr int kPieces = kHalf / 1024 / WM;            // key (or value) pieces that a wave copies,
  static constexpr int kTiles = kPieces > kD32 ? kPieces / kD32 : 1;  // ... of so many 32-token tiles
  static constexpr int kStageBytes = kWT * 2 * kHalf;
  static constexpr int kRows = 32 * WM;
  // Query fragments that a wave keeps in LDS and not in registers (D = 256:
  // accumulators 128 and queries 64 of 256 leave too few).
  static constexpr int kQueriesLds = D == 256 ? (WM == 4 ? 6 : WM == 2 ? 2 : 0) : 0;
};

// LDS DMA of 16 bytes a lane: lane l's go to `to` + 16 l (`to` uniform).  As
// the builtin, it would make every LDS read of the compiler's wait for every
// copy in flight; written out, the kernel's own wait_vmem and barrier order
// it (and no other instruction here uses m0).
__device__ __attribute__((always_inline)) inline void copy_to_lds16(const uint8_t* from, const uint8_t* to) {
  const uint32_t at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const uint8_t*)to;
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
               :: "s"(__builtin_amdgcn_readfirstlane(at)), "v"(from) : "memory");
}

struct RowsLds {
  uint8_t* stages;  // 2 * kStageBytes
  float (*scales)[2][kStep];  // of a wave's tokens: keys', values'
  float (*ml)[32][2];
  int64_t* line;
  uint4* q;  // [kWaves][kQueriesLds][64]
  int* nan_tile;  // see StreamLds
};

template <int D, int WM, bool OWN>  // OWN: see stream_body
__device__ __attribute__((always_inline)) inline void rows_body(const KvAttnArgs& a, const Pass& p, const int wg, const RowsLds& lds) {
  typedef RowsShape<D, WM> C;
  constexpr int TT = C::kTT, D32 = C::kD32, PW = C::kPieces, NT = C::kTiles;
  uint8_t* const stages = lds.stages;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave % WM, wt = wave / WM;
  const int i = lane & 31, h = lane >> 5;
  const int prefix_steps = ceil_div(p.prefix_len, C::kStepTokens);
  const int page_blocks_shift = a.c.page_shift - 4, page_blocks_mask = (1 << page_blocks_shift) - 1;

  // What this lane copies of a key piece, a value piece and the scales.
  const int kh = (lane >> 2) & 1;
  const int key_src = ((lane & 31) >> 3) * (4 * D) + h * 64 + (lane & 3) * 16;
  const int value_src = i * 16;
  const int scale_token = lane & (C::kStepTokens - 1);
  const int key_token = 16 * kh + 4 * (i >> 3) + (i & 3);

  Walk<false> t(a, p, wg, lds.line);
  if (!t.any) return;
  do {
    const int u0 = t.u0, u1 = t.u1, seq = t.seq, len = t.len, tile = t.tile;
    const int kvh = t.kvh, row0 = t.rt * C::kRows;
    const int row = min(row0 + 32 * wm + i, p.rows - 1);
    const int row_token = row / p.group;
    const int64_t token = (int64_t)seq * p.q_len + row_token;
    const int limit = len - p.q_len + 1 + row_token;  // first own token that this row does not see
    const int limit_first = len - p.q_len + 1 + min(row0 + 32 * wm, p.rows - 1) / p.group;
    const int limit_tile = len - p.q_len + 1 + row0 / p.group;  // ... that the tile's first row does not see
    const int limit_last = len - p.q_len + 1 + (min(row0 + C::kRows, p.rows) - 1) / p.group;
    const int steps = prefix_steps + ceil_div(max(limit_last, 0), C::kStepTokens);  // with a visible token
    const int u_end = min(u1, ceil_div(steps, C::kWT));

    constexpr int QL = C::kQueriesLds, QR = 2 * D32 - QL;
    uint4* const queries = lds.q + wave * QL * 64 + lane;
    bf16x8 qf[QR];
    {
      const int64_t at = token * a.ld_q + (int64_t)(kvh * p.group + row - row_token * p.group) * D + h * 16;
#pragma unroll
      for (int j = 0; j < 2 * D32; ++j) {
        const uint4 q = *reinterpret_cast<const uint4*>((const uint16_t*)a.q + at + (j >> 1) * 32 + 8 * (j & 1));
        if (j < QR) qf[j] = __builtin_bit_cast(bf16x8, q);
        else queries[(j - QR) * 64] = q;
      }
    }
    auto query = [&](int j) __attribute__((always_inline)) {
      return j < QR ? qf[j < QR ? j : 0] : __builtin_bit_cast(bf16x8, queries[(j < QR ? 0 : j - QR) * 64]);
    };

    Maximum most(a.scale_log2);
    float l = 0.0f;
    floatx16 o[D32];
#pragma unroll
    for (int d = 0; d < D32; ++d) o[d] = floatx16{};

    struct Where {
      const int* list;
      int base, n, all;  // the step's first token; tokens of the list that any row sees, that all rows of the tile see
    };
    auto where = [&](int s) __attribute__((always_inline)) {
      if (!OWN || s < prefix_steps) return Where{a.prefix_pages, s * C::kStepTokens, p.prefix_len, p.prefix_len};
      return Where{a.table + seq * a.ld_table, (s - prefix_steps) * C::kStepTokens, limit_last, limit_tile};
    };
    // Step of this region in unit u; past the last one, that one again (so
    // every wave copies as much, and nothing reads it).
    auto step_of = [&](int u) { return min(u * C::kWT + wt, steps - 1); };
    // The blocks a lane copies from: of its key pieces, of its value pieces,
    // and that of its token for the scales.
    auto col_of_piece = [&](int k) { return NT == 1 ? wm * PW % D32 + k : k % D32; };
    auto block_of = [&](const Where& w, int b) { return min((w.base >> 4) + b, (w.n - 1) >> 4); };
    auto slot_of = [&](int blk) { return (kvh << a.c.page_shift) + (blk & page_blocks_mask) * 16; };
    auto row_of = [&](int id, int64_t ld) {
      return (uint64_t)((unsigned)id < (unsigned)a.c.n_pages ? (unsigned)id : 0u) * (uint64_t)(uint32_t)ld;
    };
    int pages[2 * NT + 1];
    auto load_pages = [&](int u) __attribute__((always_inline)) {
      const Where w = where(step_of(u));
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int tile = NT == 1 ? wm * PW / D32 : t;
        pages[t] = w.list[block_of(w, 2 * tile + kh) >> page_blocks_shift];
        pages[NT + t] = w.list[block_of(w, 2 * tile + h) >> page_blocks_shift];
      }
      pages[2 * NT] = w.list[block_of(w, scale_token >> 4) >> page_blocks_shift];
    };
    // Starts the copy of unit u; its scales go through registers to the
    // wave's own table (put_scales), as floats.
    uint32_t key_scale = 0, value_scale = 0;
    uint64_t bad = 0, bad_next = 0;  // bit t for token t of the stage if its page does not exist
    auto copy = [&](int u, uint8_t* stage) __attribute__((always_inline)) {
      const Where w = where(step_of(u));
      uint8_t* const region = stage + wt * (2 * C::kHalf) + wm * PW * 1024;
      const uint8_t *kp[NT], *vp[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int tile = NT == 1 ? wm * PW / D32 : t;
        kp[t] = a.c.kc + row_of(pages[t], a.c.ld_codes) + (uint32_t)(slot_of(block_of(w, 2 * tile + kh)) * D + key_src);
        vp[t] = a.c.vc + row_of(pages[NT + t], a.c.ld_codes) + (uint32_t)(slot_of(block_of(w, 2 * tile + h)) * D + value_src);
      }
#pragma unroll
      for (int k = 0; k < PW; ++k)
        copy_to_lds16(kp[NT == 1 ? 0 : k / D32] + col_of_piece(k) * 128, region + k * 1024);
#pragma unroll
      for (int k = 0; k < PW; ++k)
        copy_to_lds16(vp[NT == 1 ? 0 : k / D32] + col_of_piece(k) * 512, region + C::kHalf + k * 1024);
      const uint64_t at = row_of(pages[2 * NT], a.c.ld_scales) + (uint32_t)(slot_of(block_of(w, scale_token >> 4)) + (lane & 15));
      key_scale = a.c.ks[at];
      value_scale = a.c.vs[at];
      bad_next = __ballot((unsigned)pages[2 * NT] >= (unsigned)a.c.n_pages);
    };
    float* const key_scales = lds.scales[wave][0];
    float* const value_scales = lds.scales[wave][1];
    auto put_scales = [&]() __attribute__((always_inline)) {
      key_scales[lane] = __uint_as_float(key_scale << 23);
      value_scales[lane] = __uint_as_float(value_scale << 23);
      bad = bad_next;
    };
    // Bytes that hold no token that any row sees may be NaN codes, and their
    // scales infinite (0 * NaN): each wave clears those of the pieces that it
    // copied, and takes out the NaN codes that only some rows see.
    auto clear = [&](int u, uint8_t* stage) __attribute__((always_inline)) {
      const int s = u * C::kWT + wt;
      const Where w = where(min(s, steps - 1));
      if (bad == 0 && s < steps && w.base + C::kStepTokens <= w.all) return;
      asm volatile("");  // a real branch: the steps that take it are few
      uint8_t* const values = stage + wt * (2 * C::kHalf) + C::kHalf + wm * PW * 1024 + lane * 16;
      uint32_t any = 0;
      if (OWN && w.all < w.n && w.base + C::kStepTokens > w.all) {
#pragma unroll
        for (int k = 0; k < PW; ++k) any |= nan_bytes(*reinterpret_cast<const uint4*>(values + k * 1024));
        any = __any(any != 0);
        if (any == 0 && bad == 0 && s < steps && w.base + C::kStepTokens <= w.n) return;
      }
      for (int k = 0; k < PW; ++k) {
        const int block = 32 * (NT == 1 ? wm * PW / D32 : k / D32) + 16 * h;
        const int holds = s >= steps || (bad >> block & 1u) ? 0 : w.n - (w.base + block);
        uint4 v = *reinterpret_cast<const uint4*>(values + k * 1024);
        v = make_uint4(v.x & keep_bytes(holds), v.y & keep_bytes(holds - 4), v.z & keep_bytes(holds - 8), v.w & keep_bytes(holds - 12));
        if (any != 0) drop_nan(v);
        *reinterpret_cast<uint4*>(values + k * 1024) = v;
      }
      if (any != 0) *lds.nan_tile = tile;
    };

    // One step.  The fragments (keys, then values) are read kAhead before
    // their use and converted one ahead, and the order is pinned
    // (sched_barrier): left alone, the compiler reads each right before its
    // conversion and converts it right before its product, and the wave waits
    // for both.
    constexpr int kAhead = D == 256 ? 2 : 3, F = TT * D32;
    auto step = [&](int u, uint8_t* stage) __attribute__((always_inline)) {
      const int s = u * C::kWT + wt;
      const Where w = where(min(s, steps - 1));
      const int held = s >= steps ? 0 : w.n;  // tokens of the list that any row sees
      const int row_sees = s >= steps ? 0 : s < prefix_steps ? w.n : limit;
      const int all_see = s >= steps ? 0 : s < prefix_steps ? w.n : limit_first;
      const int base = w.base;
      const bool masked = bad != 0 || base + C::kStepTokens > all_see;
      uint8_t* const keys = stage + wt * (2 * C::kHalf) + lane * 16;
      uint8_t* const values = keys + C::kHalf;

      if (masked) {
        asm volatile("");
        if (lane < 32 * TT && (base + lane >= held || (bad >> lane & 1u))) value_scales[lane] = 0.0f;
      }

      floatx16 sc[TT];
      float ks[TT];
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        ks[t] = key_scales[32 * t + key_token];
        sc[t] = floatx16{};
      }
      // The conversions of fragment f + 1 go between the two products of f.
      auto key_at = [&](int f) { return *reinterpret_cast<const uint4*>(keys + ((f % TT) * D32 + f / TT) * 1024); };
      auto value_at = [&](int f) { return *reinterpret_cast<const uint4*>(values + ((f % TT) * D32 + f / TT) * 1024); };
      uint4 fr[kAhead];
#pragma unroll
      for (int f = 0; f < kAhead; ++f) fr[f] = key_at(f);
      bf16x8 c0 = decode8(fr[0].x, fr[0].y, ks[0]), c1 = decode8(fr[0].z, fr[0].w, ks[0]);
#pragma unroll
      for (int f = 0; f < F; ++f) {  // tile f % TT, dimensions 32 (f / TT) ..
        const int t = f % TT, j = f / TT;
        fr[f % kAhead] = f + kAhead < F ? key_at(f + kAhead) : value_at(f + kAhead - F);
        const uint4 q = fr[(f + 1) % kAhead];
        const float kn = f + 1 < F ? ks[(f + 1) % TT] : 1.0f;
        sc[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(c0, query(2 * j), sc[t], 0, 0, 0);
        const bf16x8 n0 = decode8(q.x, q.y, kn);
        __builtin_amdgcn_sched_barrier(0);
        sc[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(c1, query(2 * j + 1), sc[t], 0, 0, 0);
        const bf16x8 n1 = decode8(q.z, q.w, kn);
        __builtin_amdgcn_sched_barrier(0);
        c0 = n0;
        c1 = n1;
      }
      f32x4 vs[TT][4];
#pragma unroll
      for (int t = 0; t < TT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) vs[t][r] = *reinterpret_cast<const f32x4*>(value_scales + 32 * t + 16 * h + 4 * r);
      __builtin_amdgcn_sched_barrier(0);

      if (masked) {
        asm volatile("");
#pragma unroll
        for (int t = 0; t < TT; ++t) {
          const int sees = (bad >> (32 * t + 16 * h) & 1u) ? 0 : row_sees - (base + 32 * t + 16 * h);
#pragma unroll
          for (int r = 0; r < 16; ++r) sc[t][r] = r < sees ? sc[t][r] : -__builtin_inff();
        }
      }

      float top = kLowest;
#pragma unroll
      for (int t = 0; t < TT; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r) top = fmaxf(top, sc[t][r]);
      top = fmaxf(top, __shfl_xor(top, 32));
      if (__any(most.passed(top, kSlack))) {
        const float f = most.raise(a.scale_log2, top);
        l *= f;
#pragma unroll
        for (int d = 0; d < D32; ++d) o[d] *= f;
      }
      bf16x8 pf[TT][2];
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        float e[16];
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          e[r] = __builtin_amdgcn_exp2f(most.exponent(sc[t][r]));
          l += e[r];
        }
#pragma unroll
        for (int r = 0; r < 16; ++r) e[r] *= vs[t][r >> 2][r & 3];
        pf[t][0] = take_term(e);
        pf[t][1] = take_term(e + 8);
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int f = 0; f < F; ++f) {
        const int t = f % TT, d = f / TT;
        if (f + kAhead < F) fr[(f + F) % kAhead] = value_at(f + kAhead);
        const uint4 v = fr[(f + 1 + F) % kAhead];
        o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(c0, pf[t][0], o[d], 0, 0, 0);
        const bf16x8 n0 = f + 1 < F ? decode8(v.x, v.y, 1.0f) : c0;
        __builtin_amdgcn_sched_barrier(0);
        o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(c1, pf[t][1], o[d], 0, 0, 0);
        const bf16x8 n1 = f + 1 < F ? decode8(v.z, v.w, 1.0f) : c1;
        __builtin_amdgcn_sched_barrier(0);
        c0 = n0;
        c1 = n1;
      }
    };

    // Unit u is in one stage while u + 1 is copied into the other: a wave's
    // own copies have landed (wait_vmem) and every wave is done reading the
    // stage that is overwritten (the barrier).
    if (u0 < u_end) {
      load_pages(u0);
      copy(u0, stages + (u0 & 1) * C::kStageBytes);
      load_pages(u0 + 1);
      for (int u = u0; u < u_end; ++u) {
        wait_vmem<0>();
        asm volatile("" ::: "memory");  // only the wait says that the bytes read below are there
        put_scales();
        clear(u, stages + (u & 1) * C::kStageBytes);
        barrier_lds();
        copy(u + 1, stages + (~u & 1) * C::kStageBytes);
        load_pages(u + 2);
        step(u, stages + (u & 1) * C::kStageBytes);
      }
      wait_vmem<0>();  // copies past the last unit
    }

    float m = most.value(a.scale_log2);

    // Join the regions: waves of wt > 0 hand theirs to the wave of wt = 0
    // with the same rows (register by register).
    l += __shfl_xor(l, 32);
    barrier_lds();
    constexpr int kOut = D32 * 16;  // accumulator registers
    if constexpr (C::kWT > 1) {
      float* const given = reinterpret_cast<float*>(stages);
      if (wt > 0) {
        const int at = ((wt - 1) * WM + wm) * kOut * 64 + lane;
#pragma unroll
        for (int r = 0; r < kOut; ++r) given[at + r * 64] = o[r >> 4][r & 15];
        if (h == 0) {
          lds.ml[wave][i][0] = m;
          lds.ml[wave][i][1] = l;
        }
      }
      barrier_lds();
      if (wt == 0) {
        float top = m;
#pragma unroll
        for (int w = 1; w < C::kWT; ++w) top = fmaxf(top, lds.ml[w * WM + wm][i][0]);
        const float f0 = __builtin_amdgcn_exp2f(m - top);
        l *= f0;
#pragma unroll
        for (int d = 0; d < D32; ++d) o[d] *= f0;
#pragma unroll
        for (int w = 1; w < C::kWT; ++w) {
          const float f = __builtin_amdgcn_exp2f(lds.ml[w * WM + wm][i][0] - top);
          l += lds.ml[w * WM + wm][i][1] * f;
          const int at = ((w - 1) * WM + wm) * kOut * 64 + lane;
#pragma unroll
          for (int r = 0; r < kOut; ++r) o[r >> 4][r & 15] += given[at + r * 64] * f;
        }
        m = top;
      }
    }
    const int r = 32 * wm + i;  // row of the tile
    const bool whole = p.direct && t.whole();
    const int64_t at = ((int64_t)tile + t.wg) * C::kRows + r;
    if (wt == 0 && row0 + r < p.rows) {
      if (!whole) {
        if (h == 0) *reinterpret_cast<float2*>(p.ml + at * 2) = make_float2(m, l);
#pragma unroll
        for (int d = 0; d < D32; ++d)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            *reinterpret_cast<f32x4*>(p.o + at * D + 32 * d + 8 * e + 4 * h) =
                f32x4{o[d][4 * e], o[d][4 * e + 1], o[d][4 * e + 2], o[d][4 * e + 3]};
      } else if (len >= 0) {
        const float inv = inverse_sum(l);
#pragma unroll
        for (int d = 0; d < D32; ++d)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float v[4] = {o[d][4 * e] * inv, o[d][4 * e + 1] * inv, o[d][4 * e + 2] * inv, o[d][4 * e + 3] * inv};
            store_out4<NVFP4_DTYPE_BF16>(a, (int)token, kvh * p.group + row - row_token * p.group, 32 * d + 8 * e + 4 * h, v);
          }
      }
    }
    if constexpr (OWN)
      if (__builtin_expect(wt == 0 && __builtin_amdgcn_readfirstlane(*lds.nan_tile) == tile, 0))
        put_nan<NVFP4_DTYPE_BF16, D, C::kRows, C::kStepTokens>(a, p, t, r, 4 * h, 8);
    barrier_lds();
  } while (t.next(p));
}

template <int D, int WM>
__global__ __launch_bounds__(kThreads, WM == 1 ? 1 : 2) void kv_attention_rows_kernel(KvAttnArgs a, Pass p) {
  typedef RowsShape<D, WM> C;
  __shared__ __attribute__((aligned(16))) uint8_t stages[2 * C::kStageBytes];
  __shared__ __attribute__((aligned(16))) float scales[kWaves][2][kStep];
  __shared__ float ml[kWaves][32][2];
  __shared__ int64_t line[2 * kWaves];
  __shared__ uint4 q[C::kQueriesLds * kWaves * 64 + 1];
  __shared__ int nan_tile;
  rows_body<D, WM, true>(a, p, blockIdx.x, RowsLds{stages, scales, ml, line, q, &nan_tile});
}

// Tiles of 128 rows, D <= 128: the four waves own 32 each and all work on the same
// tokens.  Here the conversion to bf16 would be made four times over, and the
// instructions a wave issues are what bounds it, so each wave converts a
// quarter of the step and the stage holds bf16: fragment (tile of 32 tokens,
// 16 dimensions) of the keys, or (tile, 32 dimensions, half of a block's
// tokens) of the values, 1 KB each, lane l's 8 values at 16 l.  The bytes go
// through registers: asked for a step ahead, converted after the step's
// products, one barrier a step.  (With D = 256 the accumulators and queries
// take 192 of 256 registers, and this form spills 120; it stays with rows_body.
// That spills too there: 14 registers with 128 rows, none of them used within a
// step, 35 with 64 rows, of which a step reloads 7, behind the copies of the
// next one; in the joint launch 34 to 64.)
template <int D>
struct WideShape {
  static constexpr int kTT = 2;                           // 32-token tiles of a step
  static constexpr int kStepTokens = 32 * kTT;
  static constexpr int kD32 = D / 32;
  static constexpr int kPieces = kTT * kD32 / 4;          // raw KB of keys, and of values, of a wave
  static constexpr int kHalf = kStepTokens * D * 2;       // bytes of a stage's keys, or values
  static constexpr int kStageBytes = 2 * kHalf;
  static constexpr int kRows = 128;
  };

struct WideLds {
  uint8_t* stages;          // 2 * kStageBytes
  float (*scales)[kStep];   // values' scales of each stage
  uint64_t* bad;            // of each stage: bit t for token t if its page does not exist
  int64_t* line;
  int* nan_tile;            // see StreamLds; [2], tiles in turn
};

template <int D, bool OWN>  // OWN: see stream_body
__device__ __attribute__((always_inline)) inline void wide_body(const KvAttnArgs& a, const Pass& p, const int wg, const WideLds& lds) {
  typedef WideShape<D> C;
  static_assert(D <= 128, "no registers for wider heads");
  constexpr int TT = C::kTT, D32 = C::kD32, PW = C::kPieces, ST = C::kStepTokens;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i = lane & 31, h = lane >> 5;
  const int prefix_steps = ceil_div(p.prefix_len, ST);
  const int page_blocks_shift = a.c.page_shift - 4, page_blocks_mask = (1 << page_blocks_shift) - 1;

  // What this lane converts (see rows_body): PW pieces of one 32-token tile.
  const int my_tile = wave * PW / D32, my_col = wave * PW % D32;
  const int kh = (lane >> 2) & 1, key_row = 4 * (i >> 3) + (i & 3);  // block of the tile, token of the block
  const int key_src = (i >> 3) * (4 * D) + h * 64 + (lane & 3) * 16 + my_col * 128;
  const int value_src = i * 16 + my_col * 512;
  const int scale_token = lane & (ST - 1);
  int turn = 0;

  Walk<false> t(a, p, wg, lds.line);
  if (!t.any) return;
  do {
    const int u0 = t.u0, u1 = t.u1, seq = t.seq, len = t.len, tile = t.tile;
    const int kvh = t.kvh, row0 = t.rt * C::kRows;
    const int row = min(row0 + 32 * wave + i, p.rows - 1);
    const int row_token = row / p.group;
    const int64_t token = (int64_t)seq * p.q_len + row_token;
    const int limit = len - p.q_len + 1 + row_token;  // first own token that this row does not see
    const int limit_first = len - p.q_len + 1 + min(row0 + 32 * wave, p.rows - 1) / p.group;
    const int limit_tile = len - p.q_len + 1 + row0 / p.group;  // ... that the tile's first row does not see
    const int limit_last = len - p.q_len + 1 + (min(row0 + C::kRows, p.rows) - 1) / p.group;
    const int steps = prefix_steps + ceil_div(max(limit_last, 0), ST);  // with a visible token
    const int u_end = min(u1, steps);

    bf16x8 qf[2 * D32];
    {
      const int64_t at = token * a.ld_q + (int64_t)(kvh * p.group + row - row_token * p.group) * D + h * 16;
#pragma unroll
      for (int j = 0; j < 2 * D32; ++j)
        qf[j] = *reinterpret_cast<const bf16x8*>((const uint16_t*)a.q + at + (j >> 1) * 32 + 8 * (j & 1));
    }

    Maximum most(a.scale_log2);
    float l = 0.0f;
    floatx16 o[D32];
#pragma unroll
    for (int d = 0; d < D32; ++d) o[d] = floatx16{};

    struct Where {
      const int* list;
      int base, n, all;  // see rows_body
    };
    auto where = [&](int u) __attribute__((always_inline)) {
      const int s = min(u, steps - 1);
      if (!OWN || s < prefix_steps) return Where{a.prefix_pages, s * ST, p.prefix_len, p.prefix_len};
      return Where{a.table + seq * a.ld_table, (s - prefix_steps) * ST, limit_last, limit_tile};
    };
    auto block_of = [&](const Where& w, int b) { return min((w.base >> 4) + b, (w.n - 1) >> 4); };
    auto slot_of = [&](int blk) { return (kvh << a.c.page_shift) + (blk & page_blocks_mask) * 16; };
    auto row_of = [&](int id, int64_t ld) {
      return (uint64_t)((unsigned)id < (unsigned)a.c.n_pages ? (unsigned)id : 0u) * (uint64_t)(uint32_t)ld;
    };

    int key_page = 0, value_page = 0;
    auto load_pages = [&](const Where& w) __attribute__((always_inline)) {
      key_page = w.list[block_of(w, 2 * my_tile + kh) >> page_blocks_shift];
      value_page = w.list[block_of(w, 2 * my_tile + h) >> page_blocks_shift];
    };
    uint4 kraw[PW], vraw[PW];
    uint32_t kscale = 0;
    bool value_gone = false;
    // A step's loads in four parts (see step()).
    constexpr int kLoadParts = 4;
    const uint8_t* src = nullptr;
    auto load_part = [&](const Where& w, int part) __attribute__((always_inline)) {
      const int kat = slot_of(block_of(w, 2 * my_tile + kh));
      if (part == 0) {
        src = a.c.kc + row_of(key_page, a.c.ld_codes) + (uint32_t)(kat * D + key_src);
#pragma unroll
        for (int k = 0; k < PW; ++k) kraw[k] = *reinterpret_cast<const uint4*>(src + k * 128);
      } else if (part == 1) {
        src = a.c.vc + row_of(value_page, a.c.ld_codes) + (uint32_t)(slot_of(block_of(w, 2 * my_tile + h)) * D + value_src);
#pragma unroll
        for (int k = 0; k < PW; ++k) vraw[k] = *reinterpret_cast<const uint4*>(src + k * 512);
      } else if (part == 2) {
        kscale = a.c.ks[row_of(key_page, a.c.ld_scales) + (uint32_t)(kat + key_row)];
      } else {
        value_gone = (unsigned)value_page >= (unsigned)a.c.n_pages;
      }
    };
    auto load = [&](const Where& w) __attribute__((always_inline)) {
#pragma unroll
      for (int part = 0; part < kLoadParts; ++part) load_part(w, part);
    };
    const int to_frag = (my_tile * D32 + my_col) * 2048 + lane * 16;
    constexpr int kPutParts = 4 * PW;
    auto put_part = [&](int stage, int part) __attribute__((always_inline)) {
      uint8_t* const to = lds.stages + stage * C::kStageBytes + to_frag + part / 2 % PW * 2048 + (part & 1) * 1024;
      const uint4 q = part < 2 * PW ? kraw[part / 2 % PW] : vraw[part / 2 % PW];
      const uint32_t lo = part & 1 ? q.z : q.x, hi = part & 1 ? q.w : q.y;
      if (part < 2 * PW) *reinterpret_cast<bf16x8*>(to) = decode8(lo, hi, __uint_as_float(kscale << 23));
      else *reinterpret_cast<bf16x8*>(to + C::kHalf) = decode8(lo, hi, 1.0f);
    };
    auto put = [&](int stage) __attribute__((always_inline)) {
#pragma unroll
      for (int part = 0; part < kPutParts; ++part) put_part(stage, part);
    };
    // Bytes that hold no token that any row sees may be NaN codes, and their
    // scales infinite (0 * NaN): zeros instead; and NaN codes that only some
    // rows see are taken out.
    auto clear = [&](const Where& w, int stage) __attribute__((always_inline)) {
      const bool gone = __any(value_gone);
      if (!gone && w.base + ST <= w.all) return;
      uint32_t any = 0;
      if (OWN && w.all < w.n && w.base + ST > w.all) {
#pragma unroll
        for (int k = 0; k < PW; ++k) any |= nan_bytes(vraw[k]);
        any = __any(any != 0);
        if (any == 0 && !gone && w.base + ST <= w.n) return;
      }
      uint8_t* const to = lds.stages + stage * C::kStageBytes + C::kHalf + to_frag;
      const int holds = value_gone ? 0 : w.n - (w.base + 32 * my_tile + 16 * h);
#pragma unroll
      for (int k = 0; k < PW; ++k) {
        uint4 v = make_uint4(vraw[k].x & keep_bytes(holds), vraw[k].y & keep_bytes(holds - 4),
                             vraw[k].z & keep_bytes(holds - 8), vraw[k].w & keep_bytes(holds - 12));
        if (any != 0) drop_nan(v);
        *reinterpret_cast<bf16x8*>(to + k * 2048) = decode8(v.x, v.y, 1.0f);
        *reinterpret_cast<bf16x8*>(to + k * 2048 + 1024) = decode8(v.z, v.w, 1.0f);
      }
      if (any != 0) lds.nan_tile[turn] = tile;
    };
    // The values' scales, by wave 0, another step ahead: lane t's token t.
    int scale_page = 0;
    uint32_t vscale = 0;
    uint64_t gone = 0;
    auto load_scale_page = [&](const Where& w) __attribute__((always_inline)) {
      scale_page = w.list[block_of(w, scale_token >> 4) >> page_blocks_shift];
    };
    auto load_scales = [&](const Where& w) __attribute__((always_inline)) {
      vscale = a.c.vs[row_of(scale_page, a.c.ld_scales) + (uint32_t)(slot_of(block_of(w, scale_token >> 4)) + (lane & 15))];
      gone = __ballot((unsigned)scale_page >= (unsigned)a.c.n_pages);
    };
    auto put_scales = [&](const Where& w, int stage) __attribute__((always_inline)) {
      const bool none = w.base + scale_token >= w.n || (gone >> scale_token & 1u);
      lds.scales[stage][lane] = none ? 0.0f : __uint_as_float(vscale << 23);
      if (lane == 0) lds.bad[stage] = gone;
    };

    // One step, with the next one's bytes asked for and converted inside.  A
    // wave issues one instruction in about 5 cycles and a product occupies
    // the matrix unit for 32, so after each product come a few other
    // instructions: the next step's addresses and loads in the first half,
    // the softmax of the second tile and the conversions in the second.
    // sched_barrier pins that order (and the fragments' reads, kAhead
    // before their product); the compiler's own bunches products and reads.
    // The parts with products run at raised priority: without it the older of
    // two waves on a SIMD always wins, finishes its share early and leaves the
    // other alone (at equal shares of 75 units 155 and 205 us, now 160 and
    // 184).
    constexpr int kAhead = 4, F = 2 * TT * D32, FT = 2 * D32;
    auto step = [&](const Where& w, bool prefix, int stage, const Where& next, const Where& after) __attribute__((always_inline)) {
      const uint8_t* const keys = lds.stages + stage * C::kStageBytes + lane * 16;
      const uint8_t* const values = keys + C::kHalf;
      const float* const scales = lds.scales[stage];
      // key product f: tile f / 2 % TT, 16 dimensions; value product f: tile
      // f / FT, 32 dimensions and half the tokens
      auto key_at = [&](int f) {
        return *reinterpret_cast<const bf16x8*>(keys + ((f / 2 % TT) * D32 + f / (2 * TT)) * 2048 + (f & 1) * 1024);
      };
      auto value_at = [&](int f) { return *reinterpret_cast<const bf16x8*>(values + f * 1024); };
      floatx16 sc[TT];
#pragma unroll
      for (int k = 0; k < TT; ++k) sc[k] = floatx16{};
      bf16x8 fr[kAhead];
#pragma unroll
      for (int f = 0; f < kAhead; ++f) fr[f] = key_at(f);
      const uint64_t bad64 = lds.bad[stage];
#pragma unroll
      for (int f = 0; f < F; ++f) {
        const bf16x8 k = fr[f % kAhead];
        sc[f / 2 % TT] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k, qf[2 * (f / (2 * TT)) + (f & 1)], sc[f / 2 % TT], 0, 0, 0);
        fr[f % kAhead] = f + kAhead < F ? key_at(f + kAhead) : value_at(f + kAhead - F);
        if (f < kLoadParts) load_part(next, f);
        if (f == kLoadParts) load_pages(after);
        __builtin_amdgcn_sched_barrier(0);
      }
      f32x4 vs[TT][4];
#pragma unroll
      for (int k = 0; k < TT; ++k)
#pragma unroll
        for (int r = 0; r < 4; ++r) vs[k][r] = *reinterpret_cast<const f32x4*>(scales + 32 * k + 16 * h + 4 * r);
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_setprio(0);

      const uint32_t bad_lo = __builtin_amdgcn_readfirstlane((uint32_t)bad64), bad_hi = __builtin_amdgcn_readfirstlane((uint32_t)(bad64 >> 32));
      if ((bad_lo | bad_hi) != 0 || w.base + ST > (prefix ? w.n : limit_first)) {
        asm volatile("");
#pragma unroll
        for (int k = 0; k < TT; ++k) {
          const int sees = ((k ? bad_hi : bad_lo) >> (16 * h) & 1u) ? 0 : (prefix ? w.n : limit) - (w.base + 32 * k + 16 * h);
#pragma unroll
          for (int r = 0; r < 16; ++r) sc[k][r] = r < sees ? sc[k][r] : -__builtin_inff();
        }
      }

      float top = kLowest;
#pragma unroll
      for (int k = 0; k < TT; ++k)
#pragma unroll
        for (int r = 0; r < 16; ++r) top = fmaxf(top, sc[k][r]);
      top = fmaxf(top, __shfl_xor(top, 32));
      if (__any(most.passed(top, kSlack))) {
        const float f = most.raise(a.scale_log2, top);
        l *= f;
#pragma unroll
        for (int d = 0; d < D32; ++d) o[d] *= f;
      }
      uint32_t pf[TT][8];  // pairs of weights as bf16
      auto weight_pair = [&](int k, int r) __attribute__((always_inline)) {
        const float e0 = __builtin_amdgcn_exp2f(most.exponent(sc[k][r]));
        const float e1 = __builtin_amdgcn_exp2f(most.exponent(sc[k][r + 1]));
        l += e0;
        l += e1;
        pf[k][r >> 1] = pack_bf16x2(e0 * vs[k][r >> 2][r & 3], e1 * vs[k][r >> 2][(r & 3) + 1]);
      };
      auto weights = [&](int k, int half) __attribute__((always_inline)) {
        return __builtin_bit_cast(bf16x8, u32x4{pf[k][4 * half], pf[k][4 * half + 1], pf[k][4 * half + 2], pf[k][4 * half + 3]});
      };
      auto product = [&](int f) __attribute__((always_inline)) {
        const bf16x8 v = fr[(f + F) % kAhead];
        o[f % FT / 2] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v, weights(f / FT, f & 1), o[f % FT / 2], 0, 0, 0);
        if (f + kAhead < F) fr[(f + F) % kAhead] = value_at(f + kAhead);
      };
#pragma unroll
      for (int r = 0; r < 16; r += 2) weight_pair(0, r);
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int f = 0; f < FT; ++f) {
        product(f);
#pragma unroll
        for (int r = 0; r < 16 / FT; r += 2) weight_pair(1, f * (16 / FT) + r);
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int f = 0; f < FT; ++f) {
        product((TT - 1) * FT + f);
        if (f >= FT - kPutParts) put_part(stage ^ 1, f - (FT - kPutParts));
        __builtin_amdgcn_sched_barrier(0);
      }
      clear(next, stage ^ 1);
      if (wave == 0) put_scales(next, stage ^ 1);
    };

    bool nan = false;  // NaN codes were taken out
    if (u0 < u_end) {
      Where w = where(u0), next = where(u0 + 1);
      load_pages(w);
      load(w);
      load_pages(next);
      if (wave == 0) {
        load_scale_page(w);
        load_scales(w);
        put_scales(w, u0 & 1);
        load_scale_page(next);
        load_scales(next);
        load_scale_page(where(u0 + 2));
      }
      put(u0 & 1);
      clear(w, u0 & 1);
      barrier_lds();
      for (int u = u0; u < u_end; ++u) {
        const Where after = where(u + 2);
        step(w, u < prefix_steps, u & 1, next, after);
        if (wave == 0) {
          load_scales(after);
          load_scale_page(where(u + 3));
        }
        w = next;
        next = after;
        barrier_lds();  // the other stage is full, and no wave reads this one any more
      }
      nan = __builtin_amdgcn_readfirstlane(lds.nan_tile[turn]) == tile;
      turn ^= 1;  // (a wave is at most one tile with a step ahead of the others)
    }
    const float m = most.value(a.scale_log2);

    l += __shfl_xor(l, 32);
    const int r = 32 * wave + i;  // row of the tile
    const bool whole = p.direct && t.whole();
    const int64_t at = ((int64_t)tile + t.wg) * C::kRows + r;
    if (row0 + r < p.rows) {
      if (!whole) {
        if (h == 0) *reinterpret_cast<float2*>(p.ml + at * 2) = make_float2(m, l);
#pragma unroll
        for (int d = 0; d < D32; ++d)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            *reinterpret_cast<f32x4*>(p.o + at * D + 32 * d + 8 * e + 4 * h) =
                f32x4{o[d][4 * e], o[d][4 * e + 1], o[d][4 * e + 2], o[d][4 * e + 3]};
      } else if (len >= 0) {
        const float inv = inverse_sum(l);
#pragma unroll
        for (int d = 0; d < D32; ++d)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float v[4] = {o[d][4 * e] * inv, o[d][4 * e + 1] * inv, o[d][4 * e + 2] * inv, o[d][4 * e + 3] * inv};
            store_out4<NVFP4_DTYPE_BF16>(a, (int)token, kvh * p.group + row - row_token * p.group, 32 * d + 8 * e + 4 * h, v);
          }
      }
    }
    if constexpr (OWN)
      if (__builtin_expect(nan, 0)) put_nan<NVFP4_DTYPE_BF16, D, C::kRows, ST>(a, p, t, r, 4 * h, 8);
  } while (t.next(p));
}

template <int D>
__global__ __launch_bounds__(kThreads, 2) void kv_attention_wide_kernel(KvAttnArgs a, Pass p) {
  typedef WideShape<D> C;
  __shared__ __attribute__((aligned(16))) uint8_t stages[2 * C::kStageBytes];
  __shared__ __attribute__((aligned(16))) float scales[2][kStep];
  __shared__ uint64_t bad[2];
  __shared__ int64_t line[2 * kWaves];
  __shared__ int nan_tile[2];
  wide_body<D, true>(a, p, blockIdx.x, WideLds{stages, scales, bad, line, nan_tile});
}

// The shared prefix and the sequences' own tokens in one launch: the first is
// bound by the matrix and vector units, the second by memory, so that each
// uses what the other leaves.  Where there is more work than places on the
// chip (`slots`), the grid fills those once and is divided by the time that
// both passes take, which depends on the lengths: so the workgroups divide it
// themselves, each finding the same number.  The two kinds are spread among
// each other by eights, since workgroups are dealt to the 8 XCDs in turn.
// (64 sequences of 64 to 1024 tokens after 16384, 256 dimensions: 66 us and join;
// divided on the host for half of the longest length, with further own
// workgroups that follow as places became free, 71 to 84 from run to run.)
// WM = 0: 16-row tiles for the prefix as well.
struct Split {
  int slots;           // 0: every unit has a workgroup, shared.workgroups of them for the prefix
  float shared_time;   // of one workgroup for the whole prefix pass, us
  float own_unit_time; // ... for a unit of an own tile
};

// The prefix has this many at least (a multiple of 8), also where the sequences
// have nearly all of the work.  24, 64 and 112 took the same time in 52 shapes (64 to 256
// sequences of up to 64 and 512 tokens after 1024 to 4096).
constexpr int kSharedLeast = 64;

__device__ inline int shared_slots(const KvAttnArgs& a, const Split& split, const Pass& shared, const Pass& own, int64_t* scratch) {
  const float own_time = (float)(Line(own, a.c.heads, scratch).units * a.c.heads) * split.own_unit_time;
  __syncthreads();  // the scratch is free again
  const int n = (int)((float)split.slots * split.shared_time / (split.shared_time + own_time)) & ~7;
  return __builtin_amdgcn_readfirstlane(max(min(n, shared.workgroups), min(kSharedLeast, shared.workgroups)));
}

template <int DT, int D, int WM, bool SOLO>
__global__ __launch_bounds__(kThreads, DT == NVFP4_DTYPE_BF16 ? 2 : 1) void kv_attention_both_kernel(KvAttnArgs a, Pass shared, Pass own, Split split) {
  constexpr bool kWide = WM == 4 && D <= 128;
  constexpr int kStage = WM == 0 ? 0 : kWide ? WideShape<D>::kStageBytes : RowsShape<D, WM == 0 ? 2 : WM>::kStageBytes;
  constexpr int kPart = SOLO && WM != 0 ? 0 : 16 * D * (int)sizeof(float);  // a solo wave hands nothing over
  constexpr int kStreamBytes = 2 * kPart + kTerms<DT> * (D / 32) * 1024 * (SOLO ? kWaves : 1);
  constexpr int kRowsQ = WM == 0 || kWide ? 0 : RowsShape<D, WM == 0 ? 2 : WM>::kQueriesLds * kWaves * 64;
  __shared__ __attribute__((aligned(16))) uint8_t stages[2 * kStage > kStreamBytes ? 2 * kStage : kStreamBytes];
  __shared__ __attribute__((aligned(16))) float scales[kWaves][2][kStep];
  __shared__ uint64_t bad[2];
  __shared__ uint4 q[kRowsQ + 1];
  __shared__ float ml[kWaves][32][2];
  __shared__ int64_t line[2 * kWaves];
  __shared__ int nan_tile[2];
  const int b = blockIdx.x;
  bool first = b < shared.workgroups;
  int wg = first ? b : b - shared.workgroups;
  if (split.slots) {
    const int n = shared_slots(a, split, shared, own, line), eights = split.slots / 8;
    const int e = b >> 3, k = e * (n >> 3) / eights;
    first = (e + 1) * (n >> 3) / eights > k;
    wg = (first ? k : e - k) * 8 + (b & 7);
    shared.workgroups = n;
    own.workgroups = split.slots - n;
  }
  const StreamLds<DT, D> stream{(float*)stages, (float*)(stages + kPart), (uint4*)(stages + 2 * kPart), ml, line, nan_tile};
  if (!first) {
    stream_body<DT, D, DT == NVFP4_DTYPE_BF16, SOLO, true>(a, own, wg, stream);
  } else if constexpr (WM == 0) {
    stream_body<DT, D, DT == NVFP4_DTYPE_BF16, false, false>(a, shared, wg, stream);
  } else if constexpr (kWide) {
    wide_body<D, false>(a, shared, wg, WideLds{stages, scales[0], bad, line, nan_tile});
  } else {
    rows_body<D, WM, false>(a, shared, wg, RowsLds{stages, scales, ml, line, q, nan_tile});
  }
}

// Joins the pieces of the rows: of the sequence's own pass and, where the
// prefix was computed for all rows together, of that pass.  D / 4 lanes take
// a row.  S = 1: as many rows as that gives, for many rows of few pieces;
// S = 4: the four waves share the pieces of a row, for few rows cut into many.
// The lanes of a row first read (M, l) of a piece each and find the weights,
// then the pieces' o, kBatch loads at a time.
template <int DT, int D, int S>
__global__ __launch_bounds__(kThreads) void kv_attention_join_kernel(KvAttnArgs a, Pass own, Pass shared) {
  constexpr int LR = D / 4, RW = 64 / LR;  // lanes of a row, rows of a wave
  constexpr int R = RW * kWaves / S;       // rows of a workgroup at a time
  constexpr int kBatch = 4;
  __shared__ float lds_ml[kWaves][RW][2];
  __shared__ __attribute__((aligned(16))) float lds_o[kWaves][RW][D];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int k = lane & (LR - 1), group = lane / LR, part = S == 1 ? 0 : wave;
  const int seq = blockIdx.x / a.c.heads, kvh = blockIdx.x - seq * a.c.heads;
  if (own_len(own, seq) < 0) return;

  for (int row0 = blockIdx.y * R; row0 < own.rows; row0 += gridDim.y * R) {
    const int row = row0 + (S == 1 ? wave * RW : 0) + group;
    const int rc = min(row, own.rows - 1);
    const int row_token = rc / own.group, hd = rc - row_token * own.group;
    const int token = seq * own.q_len + row_token;
    // the row's pieces: the row in the first one's slot, and their number
    const int tx = rc / own.tile_rows, tile = (seq * own.row_tiles + tx) * a.c.heads + kvh;
    const int2 head = own.head[tile];
    const bool done = row >= own.rows || (own.direct && head.y == 1);  // nothing there, or written by its workgroup
    const int n_own = done ? 0 : head.y;
    const int64_t own_at = ((int64_t)tile + head.x) * own.tile_rows + (rc - tx * own.tile_rows);
    int n_shared = 0;
    int64_t shared_at = 0;
    if (shared.batch) {
      const int pr = token * shared.group + hd, pt = pr / shared.tile_rows, t = pt * a.c.heads + kvh;
      const int2 sh = shared.head[t];
      n_shared = done ? 0 : sh.y;
      shared_at = ((int64_t)t + sh.x) * shared.tile_rows + (pr - pt * shared.tile_rows);
    }
    const int n = n_own + n_shared;
    // row of piece j (of the first one where the row has none: any valid place)
    auto place = [&](int j, bool& is_own) {
      is_own = j >= n_shared;
      return is_own ? own_at + (int64_t)max(min(j - n_shared, n_own - 1), 0) * own.tile_rows
                    : shared_at + (int64_t)j * shared.tile_rows;
    };
    const int most = (int)wave_max((float)n);  // (exact: n is at most a few thousand)

    float m = kLowest, l = 0.0f;
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int c = 0; c < most; c += LR * S) {
      const int j = c + k * S + part;
      float2 ml = make_float2(kLowest, 0.0f);
      if (j < n) {
        bool is_own;
        const int64_t at = place(j, is_own);
        ml = *reinterpret_cast<const float2*>((is_own ? own.ml : shared.ml) + at * 2);
      }
      float mn = fmaxf(m, ml.x);
#pragma unroll
      for (int off = LR / 2; off > 0; off >>= 1) mn = fmaxf(mn, __shfl_xor(mn, off));
      // A piece without tokens (weight 0) holds nothing.  One whose tokens have no
      // weight left (-0) adds nothing but its NaN: 0 * NaN.
      const float e = __builtin_amdgcn_exp2f(ml.x - mn);
      const float f = ml.y == 0.0f ? 0.0f : e == 0.0f ? -0.0f : e;
      float sum = ml.y * f;
#pragma unroll
      for (int off = LR / 2; off > 0; off >>= 1) sum += __shfl_xor(sum, off);
      const float old = __builtin_amdgcn_exp2f(m - mn);
      l = l * old + sum;
      acc *= old;
      m = mn;
      const int count = min(LR, ceil_div(most - c, S));
      for (int q0 = 0; q0 < count; q0 += kBatch) {
        f32x4 v[kBatch];
        float wq[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
          const int q = min(q0 + b, LR - 1);
          const float wf = __shfl(f, group * LR + q);
          wq[b] = q0 + b < LR ? wf : 0.0f;
          bool is_own;
          const int64_t at = place(min(c + q * S + part, max(n - 1, 0)), is_own);
          v[b] = __float_as_uint(wq[b]) != 0 ? *reinterpret_cast<const f32x4*>((is_own ? own.o : shared.o) + at * D + 4 * k) : f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
          if (__builtin_expect(__any(__float_as_uint(wq[b]) == 0x80000000u), 0)) {
#pragma unroll
            for (int x = 0; x < 4; ++x) v[b][x] = wq[b] == 0.0f && v[b][x] == v[b][x] ? 0.0f : v[b][x];
          }
          acc += v[b] * wq[b];
        }
      }
    }
    if constexpr (S > 1) {
      if (k == 0) {
        lds_ml[wave][group][0] = m;
        lds_ml[wave][group][1] = l;
      }
      *reinterpret_cast<f32x4*>(&lds_o[wave][group][4 * k]) = acc;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < S; ++w) m = fmaxf(m, lds_ml[w][group][0]);
      l = 0.0f;
      acc = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int w = 0; w < S; ++w) {
        const float f = __builtin_amdgcn_exp2f(lds_ml[w][group][0] - m);
        l += lds_ml[w][group][1] * f;
        acc += *reinterpret_cast<const f32x4*>(&lds_o[w][group][4 * k]) * f;
      }
      __syncthreads();
    }
    if (!done && part == 0) {
      const float inv = inverse_sum(l);
      const float v[4] = {acc[0] * inv, acc[1] * inv, acc[2] * inv, acc[3] * inv};
      store_out4<DT>(a, token, kvh * own.group + hd, 4 * k, v);
    }
  }
}

// ------------------------------------------------------------ host side

struct Plan {
  Pass own{}, shared{};  // shared.batch == 0: no such pass
  bool join;
  int join_waves;  // waves of a row in the join
  Split split;     // of launch_both
  size_t floats;
};

int64_t pass_tiles(const KvAttnArgs& a, const Pass& p) { return (int64_t)p.batch * a.c.heads * p.row_tiles; }
// Units if every sequence has max_len tokens.
int64_t pass_units(const KvAttnArgs& a, const Pass& p) {
  const int steps = ceil_div(p.prefix_len, p.step) + ceil_div(p.max_len, p.step);
  return pass_tiles(a, p) * max(1, ceil_div(steps, p.step_waves));
}
// Floats of a pass's part of the workspace: partials, and the tiles' heads.
size_t pass_floats(const KvAttnArgs& a, const Pass& p) {
  return (size_t)(pass_tiles(a, p) + pass_shares(p)) * p.tile_rows * (2 + a.c.dim) + (2 * (size_t)pass_tiles(a, p) + 3) / 4 * 4;
}

// Tiles from which on each is one wave's: half of the waves that the chip holds
// (2 workgroups of 4 on 256 CUs).  Measured, a workgroup to a tile -> a wave,
// 4 query rows, 128 dimensions: 1024 tiles of 1 to 512 tokens 24.1 -> 25.4 us,
// of up to 1024 tokens after a prefix of 512 46.7 -> 43.8; 2048 tiles of 1 to
// 512 tokens 38.9 -> 37.7, of 64 after a prefix of 256 41.5 -> 27.2; 1024 tiles
// of 64 dimensions and up to 300 tokens 18.5 -> 14.9; 2048 in float32 62 -> 46.
constexpr int64_t kSoloTiles = 1024;

// Tile shape and number of workgroups of a pass with its rows, prefix_len
// and max_len set: 16-row tiles for up to stream_rows rows.
void shape_pass(const KvAttnArgs& a, Pass& p, int stream_rows) {
  int per_cu;
  if (a.dtype == NVFP4_DTYPE_F32 || p.rows <= stream_rows) {
    p.tile_rows = kTileRows;
    p.step = kStep;
    p.step_waves = kWaves;
    per_cu = a.dtype == NVFP4_DTYPE_F32 || (a.c.dim == 256 && stream_rows == kTileRows) ? 1 : 2;
  } else {
    const int wm = p.rows <= 32 ? 1 : p.rows <= 64 ? 2 : 4;
    p.tile_rows = 32 * wm;
    p.step = a.c.dim == 256 ? 32 : 64;
    p.step_waves = kWaves / wm;
    per_cu = wm == 1 ? 1 : 2;
  }
  p.row_tiles = ceil_div(p.rows, p.tile_rows);
  if (p.tile_rows == kTileRows && pass_tiles(a, p) >= kSoloTiles && p.batch > 1) {
    p.solo = 1;
    p.step_waves = 1;
  }
  // Queries, page ids and first bytes come one after another before a tile's
  // first product, and its result leaves after the last.  Counted as 1, 2, 3
  // units: 256 sequences of 1 to 512 tokens 35.5, 35.9, 35.6 us (0: 37.9), in
  // float32 36.7, 38.2, 40.1 (46.9); a whole prompt of 4096, whose first tiles
  // see few tokens, 234, 207, 195 (317), with 4 and 6 196 and 198.
  p.start = p.tile_rows == kTileRows ? 1 : 3;
  const int64_t units = pass_units(a, p);
  p.workgroups = (int)min(p.solo ? (units + kWaves - 1) / kWaves : units, (int64_t)(256 * per_cu));
}

Plan make_plan(const KvAttnArgs& a) {
  Plan pl{};
  Pass& own = pl.own;
  own.batch = a.batch;
  own.q_len = a.q_len;
  own.group = a.group;
  own.rows = a.q_len * a.group;
  own.lens = a.lens;
  own.max_len = a.max_len;
  // Computing the prefix for all sequences at once saves reading and
  // converting it for each and costs partial results and their join.  Measured,
  // us for each -> at once, 4 query rows a kv head, own lengths up to 64 (400):
  //   128 dimensions, 8 kv heads      prefix 512               1024                      2048
  //   2 sequences               12.1 -> 12.8              12.8 -> 13.1              13.6 -> 13.5 (13.8 -> 13.9)
  //   8                         12.5 -> 13.0              14.4 -> 13.6 (14.9, 14.8) 19.7 -> 15.2 (21.5 -> 15.6)
  //   16                        13.9 -> 17.1              18.6 -> 17.9 (19.7, 17.9) 20.4 -> 18.9 (22.7 -> 18.2)
  //   64                        17.3 -> 24.1 (25.0, 24.1) 21.5 -> 28.0 (29.7, 28.7) 30.8 -> 27.2 (39.5 -> 28.1)
  //   256                       34.5 -> 30.4              52.8 -> 35.7              84.5 -> 40.8
  // So: from 1024 tokens on (512 with 2048 own tiles, one per sequence and kv
  // head; with 1024 27.6 against 25.1), and where sequences, kv heads and prefix tokens
  // multiply to 2^16 (fewer are 0.3 to 1 us slower).  With 512 to 1023 own tiles
  // each place of the chip has a whole one, which nothing has to join: there from
  // 1536 tokens on (26.5 -> 26.1; 64 dimensions 20.9 -> 21.7, 2048 24.0 -> 24.0).
  // 256 dimensions (1024 tokens: 44.6 -> 41.7) and float32 (36.4 -> 31.0) gain before
  // that.  It remains slower with 2 kv heads and own lengths of 64: 128 dimensions,
  // 64 sequences after 2048 19.2 -> 21.2; 256 dimensions, 32 to 128 sequences after 1024
  // to 2048 up to 1.28 times.  More rows of their own fill larger tiles and cost
  // another launch: 20 and 48 rows of 8 kv heads, 32 sequences after 4096 53 -> 53 and
  // 66 -> 69, after 8192 84 -> 64 and 106 -> 97; 16 after 8192 (2^20) 56 -> 53 and
  // 64 -> 66; 64 rows 129 -> 137.
  const int64_t tiles = (int64_t)a.batch * a.c.heads, shared_tokens = tiles * a.prefix_len;
  const bool whole_tiles = a.dtype == NVFP4_DTYPE_BF16 && a.c.dim <= 128 && tiles >= 512 && tiles < kSoloTiles;
  const int least = whole_tiles ? 1536 : tiles >= 2048 ? 512 : 1024;
  const bool share = a.batch > 1 && (own.rows <= kTileRows ? a.prefix_len >= least && shared_tokens >= 1 << 16
                                                           : own.rows <= 48 && shared_tokens >= 3 << 19);
  own.prefix_len = share ? 0 : a.prefix_len;
  own.direct = !share;
  shape_pass(a, own, kTileRows);
  const int own_steps = ceil_div(own.prefix_len, own.step) + ceil_div(own.max_len, own.step);
  pl.join = share || own_steps > own.step_waves;
  if (share) {
    Pass& sh = pl.shared;
    sh.batch = 1;
    sh.q_len = a.batch * a.q_len;
    sh.group = a.group;
    sh.rows = sh.q_len * a.group;
    sh.prefix_len = a.prefix_len;
    // together with an own pass of 16-row tiles (launch_both), two such tiles
    // rather than one of 32: that one's LDS would leave one workgroup to a CU
    shape_pass(a, sh, own.tile_rows == kTileRows ? 2 * kTileRows : kTileRows);

    // The units' times with both kinds on the chip, for a workgroup: 2.6 us for
    // one of 64 or 128 rows (3.4 with 256 dimensions), 5 per 128 dimensions for
    // 256 tokens of 16 rows.  float32 gains nothing: its tiles are all alike.
    constexpr int slots = 512;  // two workgroups on each of 256 CUs
    const int64_t sh_units = pass_units(a, sh), own_units = pass_units(a, own);
    if (a.dtype == NVFP4_DTYPE_BF16 && own.tile_rows == kTileRows &&
        sh_units + (own.solo ? (own_units + kWaves - 1) / kWaves : own_units) > slots) {
      const float narrow = 5.0f * a.c.dim / 128;
      const float wide = sh.tile_rows == kTileRows ? narrow : a.c.dim == 256 ? 3.4f : 2.6f;
      sh.workgroups = (int)min((sh_units + 7) / 8 * 8, (int64_t)slots - 16);
      own.workgroups = slots - min(kSharedLeast, sh.workgroups);
      pl.split = {slots, (float)sh_units * wide, own.solo ? narrow / 4 : narrow};
    }
  }
  pl.floats = pl.join ? pass_floats(a, own) : 0;
  int64_t pieces = own.workgroups / pass_tiles(a, own);
  if (share) {
    pl.floats += pass_floats(a, pl.shared);
    pieces += pl.shared.workgroups / pass_tiles(a, pl.shared);
  }
  pl.join_waves = pieces > 16 ? kWaves : 1;
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

template <int DT, int D>
hipError_t launch_pass(const KvAttnArgs& a, const Pass& p, hipStream_t s) {
  if (p.solo) {
    kv_attention_kernel<DT, D, true><<<p.workgroups, kThreads, 0, s>>>(a, p);
  } else if (p.tile_rows == kTileRows) {
    kv_attention_kernel<DT, D, false><<<p.workgroups, kThreads, 0, s>>>(a, p);
  } else if constexpr (DT == NVFP4_DTYPE_BF16) {
    if (p.tile_rows == 32) kv_attention_rows_kernel<D, 1><<<p.workgroups, kThreads, 0, s>>>(a, p);
    else if (p.tile_rows == 64) kv_attention_rows_kernel<D, 2><<<p.workgroups, kThreads, 0, s>>>(a, p);
    else if constexpr (D <= 128) kv_attention_wide_kernel<D><<<p.workgroups, kThreads, 0, s>>>(a, p);
    else kv_attention_rows_kernel<D, 4><<<p.workgroups, kThreads, 0, s>>>(a, p);
  }
  return hipGetLastError();
}

// The prefix of all and the sequences' own tokens.
template <int DT, int D, bool SOLO>
hipError_t launch_both(const KvAttnArgs& a, const Plan& pl, hipStream_t s) {
  const Pass &shared = pl.shared, &own = pl.own;
  const int grid = pl.split.slots ? pl.split.slots : shared.workgroups + own.workgroups;
  if (shared.tile_rows == kTileRows) {
    kv_attention_both_kernel<DT, D, 0, SOLO><<<grid, kThreads, 0, s>>>(a, shared, own, pl.split);
  } else if constexpr (DT == NVFP4_DTYPE_BF16) {
    if (shared.tile_rows == 64) kv_attention_both_kernel<DT, D, 2, SOLO><<<grid, kThreads, 0, s>>>(a, shared, own, pl.split);
    else kv_attention_both_kernel<DT, D, 4, SOLO><<<grid, kThreads, 0, s>>>(a, shared, own, pl.split);
  }
  return hipGetLastError();
}

template <int DT, int D, int S>
hipError_t launch_join(const KvAttnArgs& a, const Plan& pl, hipStream_t s) {
  const dim3 grid(a.batch * a.c.heads, min(ceil_div(pl.own.rows, 256 / D * kWaves / S), 65535));
  kv_attention_join_kernel<DT, D, S><<<grid, kThreads, 0, s>>>(a, pl.own, pl.shared);
  return hipGetLastError();
}

}  // namespace

size_t kv_attention_workspace(const KvAttnArgs& a) {
  return a.batch == 0 ? 16 : 16 + sizeof(float) * make_plan(a).floats;
}

hipError_t launch_kv_attention(const KvAttnArgs& a, void* ws, hipStream_t s) {
  Plan pl = make_plan(a);
  float* at = (float*)ws;
  auto place = [&](Pass& p) {
    const int64_t rows = (pass_tiles(a, p) + pass_shares(p)) * p.tile_rows;
    p.o = at;
    p.ml = at + rows * a.c.dim;
    p.head = (int2*)(p.ml + rows * 2);
    at += pass_floats(a, p);
  };
  if (pl.join) place(pl.own);
  if (pl.shared.batch) place(pl.shared);
  hipError_t err = hipSuccess;
  for_types(a.dtype, a.c.dim, [&](auto dt, auto d) {
    if (pl.shared.batch && pl.own.tile_rows == kTileRows) {
      err = pl.own.solo ? launch_both<dt(), d(), true>(a, pl, s) : launch_both<dt(), d(), false>(a, pl, s);
      if (err != hipSuccess) return;
    } else {
      if (pl.shared.batch && (err = launch_pass<dt(), d()>(a, pl.shared, s)) != hipSuccess) return;
      if ((err = launch_pass<dt(), d()>(a, pl.own, s)) != hipSuccess || !pl.join) return;
    }
    err = pl.join_waves == 1 ? launch_join<dt(), d(), 1>(a, pl, s) : launch_join<dt(), d(), kWaves>(a, pl, s);
  });
  return err;
}

}  // namespace nvfp4
