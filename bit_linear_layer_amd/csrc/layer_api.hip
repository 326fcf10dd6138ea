// C ABI of the 8-bit linear layers, the query/key norm with rotation, the short
// convolution and the gated delta rule's next tokens: argument validation
// (before any HIP call) and dispatch.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "internal.h"
#include "layer_ops.h"
#include "nvfp4.h"

using namespace nvfp4;

namespace {

constexpr int64_t kIndexLimit = (int64_t)1 << 31;
constexpr int64_t kCodeStrideLimit = (int64_t)1 << 22;  // a tile's offsets fit 32 bits
constexpr int64_t kSizeLimit = (int64_t)1 << 40;        // products of two sizes stay far inside 64 bits
constexpr int64_t kGridLimit = (int64_t)1 << 24;        // workgroups of 256 threads, in a grid of less than 2^32

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }

int elem_size(int dtype) { return dtype == NVFP4_DTYPE_BF16 ? 2 : dtype == NVFP4_DTYPE_F32 ? 4 : 0; }

// A dense operand whose rows hold `width` elements of `esz` bytes and start on 16 bytes.
int check_rows(const void* p, int64_t rows, int64_t ld, int64_t width, int esz) {
  if (ld < width || ld % (16 / esz) != 0) return NVFP4_ERR_STRIDE;
  if (ld >= kSizeLimit || rows * (ld / 256 + 1) >= kSizeLimit / 256) return NVFP4_ERR_RANGE;
  return aligned(p, 16) ? NVFP4_OK : NVFP4_ERR_ALIGN;
}

int check_fp8_shape(int64_t rows, int64_t cols) {
  if (rows < 0 || cols <= 0 || cols % 16 != 0) return NVFP4_ERR_SHAPE;
  if (rows >= kIndexLimit || cols >= kCodeStrideLimit) return NVFP4_ERR_RANGE;
  return NVFP4_OK;
}

int64_t pieces_of(int64_t cols) { return (cols + 127) / 128; }

// An E4M3 matrix (rows may be 0, then its pointers are not looked at).
int check_fp8(const nvfp4_fp8_tensor* t, Fp8Mat& out) {
  if (t == nullptr) return NVFP4_ERR_NULL;
  if (t->block_rows != 1 && t->block_rows != 128) return NVFP4_ERR_SHAPE;
  const int st = check_fp8_shape(t->rows, t->cols);
  if (st != NVFP4_OK) return st;
  if (t->ld_codes < t->cols || t->ld_codes % 16 != 0 || t->ld_scales < pieces_of(t->cols)) return NVFP4_ERR_STRIDE;
  if (t->ld_codes >= kCodeStrideLimit || t->ld_scales >= kCodeStrideLimit) return NVFP4_ERR_RANGE;
  if (t->rows >= kSizeLimit / t->ld_codes) return NVFP4_ERR_RANGE;
  if (t->block_rows == 1 && t->rows >= kSizeLimit / t->ld_scales) return NVFP4_ERR_RANGE;
  if (t->rows > 0) {
    if (t->codes == nullptr || t->scales == nullptr) return NVFP4_ERR_NULL;
    if (!aligned(t->codes, 16) || !aligned(t->scales, 4)) return NVFP4_ERR_ALIGN;
  }
  out = Fp8Mat{t->codes, t->scales, t->ld_codes, 128, t->ld_scales, 1};
  return NVFP4_OK;
}

// The sizes and the output of a product (a's and w's matrices already checked).
int check_product(int64_t m, int64_t n, int64_t k, void* out, int out_dtype, int64_t ld_out, Fp8GemmArgs& g) {
  g.cut_sums = (out_dtype & NVFP4_FP8_CUT_SUMS) != 0;
  out_dtype &= ~NVFP4_FP8_CUT_SUMS;
  const int esz = elem_size(out_dtype);
  if (esz == 0) return NVFP4_ERR_DTYPE;
  if (g.cut_sums && out_dtype != NVFP4_DTYPE_BF16) return NVFP4_ERR_FLAGS;
  if (n <= 0) return NVFP4_ERR_SHAPE;
  if (ld_out < n) return NVFP4_ERR_STRIDE;
  if (ld_out >= kIndexLimit || m >= kSizeLimit / ld_out) return NVFP4_ERR_RANGE;
  // every tile is larger (16 to 224 tokens x 128 columns, 224 x 256): grids stay below 2^32 threads, and a tile's last row and
  // column inside 32 bits
  if ((m <= 64 ? (n + 31) / 32 : (n + 63) / 64 * ((m + 63) / 64)) >= kGridLimit) return NVFP4_ERR_RANGE;
  if (m == 0) return NVFP4_OK;
  if (out == nullptr) return NVFP4_ERR_NULL;
  if (!aligned(out, (uintptr_t)esz)) return NVFP4_ERR_ALIGN;
  g.out = out;
  g.ld_out = ld_out;
  g.out_dtype = out_dtype;
  g.M = (int)m;
  g.N = (int)n;
  g.K = (int)k;
  return NVFP4_OK;
}

// The workspace of nvfp4_fp8_linear: the product's, then codes, then scales [pieces, rows].  Codes as [pieces, rows, 128],
// so that what a step reads lies together (with the 8-bit instruction 64 x 34816 x 5120 took 47 us instead of 42.5 the other
// way), or as [rows, 128 pieces] where the product needs that.
int64_t up16(int64_t bytes) { return (bytes + 15) / 16 * 16; }

int check_heads(const nvfp4_head_rows* r, int64_t tokens, int head_dim, int esz) {
  if (r->heads < 1 || r->heads > 4096) return NVFP4_ERR_SHAPE;
  const int64_t unit = 16 / esz, most = kIndexLimit;
  // a stride that is not used counts as 0
  const bool rows = tokens > 1, several = r->heads > 1;
  const int64_t lds[2] = {rows ? r->ld_x : 0, rows ? r->ld_out : 0}, hds[2] = {several ? r->head_x : 0, several ? r->head_out : 0};
  for (int i = 0; i < 2; ++i) {
    if (lds[i] < 0 || hds[i] < 0 || lds[i] % unit != 0 || hds[i] % unit != 0) return NVFP4_ERR_STRIDE;
    if (lds[i] >= most || hds[i] >= most) return NVFP4_ERR_RANGE;
    // no two (token, head) places may overlap: the heads of a token lie together, or the tokens of a head do
    const bool by_token = (!several || hds[i] >= head_dim) && (!rows || lds[i] >= (r->heads - 1) * hds[i] + head_dim);
    const bool by_head = (!rows || lds[i] >= head_dim) && (!several || hds[i] >= (tokens - 1) * lds[i] + head_dim);
    if (!by_token && !by_head) return NVFP4_ERR_STRIDE;
  }
  if (tokens == 0) return NVFP4_OK;
  if (r->x == nullptr || r->out == nullptr) return NVFP4_ERR_NULL;
  // in place every element is read by the thread that writes it
  if (r->x == r->out && (lds[0] != lds[1] || hds[0] != hds[1])) return NVFP4_ERR_STRIDE;
  if (!aligned(r->x, 16) || !aligned(r->out, 16) || !aligned(r->weight, 4)) return NVFP4_ERR_ALIGN;
  return NVFP4_OK;
}

int check_rope(const nvfp4_rope* r, int64_t tokens, int head_dim) {
  if (r->rotary_dim < 16 || r->rotary_dim > head_dim || r->rotary_dim % 16 != 0 || r->axes < 1 || r->axes > 255)
    return NVFP4_ERR_SHAPE;
  if (r->ld_positions < tokens && r->ld_positions != 0) return NVFP4_ERR_STRIDE;
  if (r->ld_positions >= kSizeLimit) return NVFP4_ERR_RANGE;
  if (tokens == 0) return NVFP4_OK;
  if (r->positions == nullptr || r->inv_freq == nullptr) return NVFP4_ERR_NULL;
  if (!aligned(r->positions, 8) || !aligned(r->inv_freq, 4)) return NVFP4_ERR_ALIGN;
  return NVFP4_OK;
}

}  // namespace

extern "C" {

int nvfp4_fp8_quantize(const void* x, int x_dtype, int64_t ld_x, const nvfp4_fp8_tensor* q, int flags, void* stream) {
  Fp8Mat m{};
  int st = check_fp8(q, m);
  if (st != NVFP4_OK) return st;
  const int esz = elem_size(x_dtype);
  if (esz == 0) return NVFP4_ERR_DTYPE;
  if (flags != NVFP4_FP8_SCALE_F32 && flags != NVFP4_FP8_SCALE_POW2) return NVFP4_ERR_FLAGS;
  if (q->rows == 0) return NVFP4_OK;
  if (x == nullptr) return NVFP4_ERR_NULL;
  if ((st = check_rows(x, q->rows, ld_x, q->cols, esz)) != NVFP4_OK) return st;
  const bool pow2 = flags == NVFP4_FP8_SCALE_POW2;
  if (q->block_rows == 1)
    return status_from_hip(launch_fp8_quantize_rows(x, x_dtype, q->rows, q->cols, ld_x, m, pow2, (hipStream_t)stream));
  if ((q->rows + 127) / 128 * pieces_of(q->cols) >= kGridLimit / 4) return NVFP4_ERR_RANGE;  // workgroups of 1024 threads
  return status_from_hip(launch_fp8_quantize_blocks(x, x_dtype, q->rows, q->cols, ld_x, m, pow2, (hipStream_t)stream));
}

size_t nvfp4_fp8_gemm_workspace_bytes(int64_t rows) {
  return rows < 0 || rows >= kIndexLimit ? 0 : fp8_gemm_workspace(rows);
}

int nvfp4_fp8_gemm(const nvfp4_fp8_tensor* a, const nvfp4_fp8_tensor* w, void* out, int out_dtype, int64_t ld_out,
                   void* workspace, size_t workspace_bytes, void* stream) {
  Fp8GemmArgs g{};
  int st = check_fp8(a, g.a);
  if (st != NVFP4_OK || (st = check_fp8(w, g.w)) != NVFP4_OK) return st;
  if (a->block_rows != 1 || w->block_rows != 128 || a->cols != w->cols) return NVFP4_ERR_SHAPE;
  if ((st = check_product(a->rows, w->rows, a->cols, out, out_dtype, ld_out, g)) != NVFP4_OK) return st;
  if (a->rows == 0) return NVFP4_OK;
  if (workspace == nullptr || workspace_bytes < nvfp4_fp8_gemm_workspace_bytes(a->rows)) return NVFP4_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return NVFP4_ERR_ALIGN;
  return status_from_hip(launch_fp8_gemm(g, (float*)workspace, (hipStream_t)stream));
}

size_t nvfp4_fp8_linear_workspace_bytes(int64_t rows, int64_t cols) {
  if (check_fp8_shape(rows, cols) != NVFP4_OK || rows >= kSizeLimit / cols) return 0;
  return fp8_gemm_workspace(rows) + (size_t)(rows * pieces_of(cols) * (128 + 4));
}

int nvfp4_fp8_linear(const void* x, int x_dtype, int64_t rows, int64_t ld_x, const nvfp4_fp8_tensor* w, void* out,
                     int out_dtype, int64_t ld_out, void* workspace, size_t workspace_bytes, void* stream) {
  Fp8GemmArgs g{};
  int st = check_fp8(w, g.w);
  if (st != NVFP4_OK) return st;
  if (w->block_rows != 128) return NVFP4_ERR_SHAPE;
  const int esz = elem_size(x_dtype);
  if (esz == 0) return NVFP4_ERR_DTYPE;
  const size_t need = nvfp4_fp8_linear_workspace_bytes(rows, w->cols);
  if (need == 0) return rows < 0 ? NVFP4_ERR_SHAPE : NVFP4_ERR_RANGE;
  if ((st = check_product(rows, w->rows, w->cols, out, out_dtype, ld_out, g)) != NVFP4_OK) return st;
  if (rows == 0) return NVFP4_OK;
  if (x == nullptr) return NVFP4_ERR_NULL;
  if ((st = check_rows(x, rows, ld_x, w->cols, esz)) != NVFP4_OK) return st;
  if (workspace == nullptr || workspace_bytes < need) return NVFP4_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return NVFP4_ERR_ALIGN;
  uint8_t* codes = (uint8_t*)workspace + up16((int64_t)fp8_gemm_workspace(rows));
  const int64_t wide = pieces_of(w->cols) * 128;
  const bool together = fp8_gemm_shares(g);
  g.a = Fp8Mat{codes, (float*)(codes + rows * wide), together ? 128 : wide, together ? rows * 128 : 128, 1, rows};
  const hipError_t e = launch_fp8_quantize_rows(x, x_dtype, rows, w->cols, ld_x, g.a, false, (hipStream_t)stream);
  if (e != hipSuccess) return status_from_hip(e);
  return status_from_hip(launch_fp8_gemm(g, (float*)workspace, (hipStream_t)stream));
}

int nvfp4_qk_norm_rope(const nvfp4_head_rows* q, const nvfp4_head_rows* k, int dtype, int64_t tokens, int head_dim, float eps,
                       float weight_offset, const nvfp4_rope* rope, void* stream) {
  if (q == nullptr && k == nullptr) return NVFP4_ERR_NULL;
  const int esz = elem_size(dtype);
  if (esz == 0) return NVFP4_ERR_DTYPE;
  if (tokens < 0 || (head_dim != 64 && head_dim != 128 && head_dim != 256)) return NVFP4_ERR_SHAPE;
  if (tokens >= kGridLimit) return NVFP4_ERR_RANGE;
  int st;
  RopeArgs a{};
  const nvfp4_head_rows* both[2] = {q, k};
  bool norm = false;
  for (int i = 0; i < 2; ++i) {
    if (both[i] == nullptr) continue;
    if ((st = check_heads(both[i], tokens, head_dim, esz)) != NVFP4_OK) return st;
    a.rows[i] = *both[i];
    norm = norm || both[i]->weight != nullptr;
  }
  if (rope != nullptr) {
    if ((st = check_rope(rope, tokens, head_dim)) != NVFP4_OK) return st;
    a.rope = *rope;
  }
  if (norm && (!(eps >= 0x1p-126f) || !isfinite(eps) || !isfinite(weight_offset))) return NVFP4_ERR_VALUE;
  if (tokens == 0) return NVFP4_OK;
  a.dtype = dtype;
  a.head_dim = head_dim;
  a.tokens = tokens;
  a.eps = eps;
  a.weight_offset = weight_offset;
  return status_from_hip(launch_qk_norm_rope(a, (hipStream_t)stream));
}

int nvfp4_causal_conv(const nvfp4_conv* c, int dtype, void* stream) {
  if (c == nullptr) return NVFP4_ERR_NULL;
  const int esz = elem_size(dtype);
  if (esz == 0) return NVFP4_ERR_DTYPE;
  if (c->width < 2 || c->width > 4 || c->channels < 8 || c->channels % 8 != 0 || c->tokens < 0 || c->batch < 0)
    return NVFP4_ERR_SHAPE;
  if (c->channels >= (int64_t)1 << 20 || c->tokens >= kIndexLimit || c->batch >= kIndexLimit ||
      c->tokens * c->channels >= (int64_t)1 << 36)
    return NVFP4_ERR_RANGE;
  if (c->state != nullptr) {
    if (c->n_states < 1) return NVFP4_ERR_SHAPE;
    if (c->ld_state < (c->width - 1) * c->channels || c->ld_state % (16 / esz) != 0) return NVFP4_ERR_STRIDE;
    if (c->n_states >= kIndexLimit || c->ld_state >= kIndexLimit) return NVFP4_ERR_RANGE;
    if (c->slots == nullptr && c->batch > c->n_states) return NVFP4_ERR_SHAPE;
  }
  if (c->tokens == 0 || c->batch == 0) return NVFP4_OK;
  if (c->starts == nullptr && c->tokens % c->batch != 0) return NVFP4_ERR_SHAPE;
  if (c->x == nullptr || c->y == nullptr || c->weight == nullptr) return NVFP4_ERR_NULL;
  if (c->x == c->y) return NVFP4_ERR_VALUE;  // the inputs before a run of tokens would be gone
  int st;
  if ((st = check_rows(c->x, c->tokens, c->ld_x, c->channels, esz)) != NVFP4_OK) return st;
  if ((st = check_rows(c->y, c->tokens, c->ld_y, c->channels, esz)) != NVFP4_OK) return st;
  if (c->ld_x >= kIndexLimit || c->ld_y >= kIndexLimit) return NVFP4_ERR_RANGE;
  if (!aligned(c->weight, 16) || !aligned(c->bias, 4) || !aligned(c->starts, 4) || !aligned(c->state, 16) ||
      !aligned(c->slots, 4))
    return NVFP4_ERR_ALIGN;
  return status_from_hip(launch_causal_conv(*c, dtype, (hipStream_t)stream));
}

int nvfp4_gdn_step(const nvfp4_gdn_inputs* in, int in_dtype, int64_t batch, int64_t q_len, int k_heads, int v_heads,
                   int normalize_qk, float* states, int64_t n_states, int64_t ld_states, const int32_t* slots,
                   const uint8_t* fresh, void* o, int o_dtype, int64_t ld_o, void* stream) {
  if (in == nullptr) return NVFP4_ERR_NULL;
  const int esz = elem_size(in_dtype), osz = elem_size(o_dtype);
  if (esz == 0 || osz == 0) return NVFP4_ERR_DTYPE;
  if (batch < 0 || q_len < 1 || k_heads < 1 || v_heads < 1 || v_heads % k_heads != 0 || v_heads > 4096 || n_states < 1)
    return NVFP4_ERR_SHAPE;
  if (batch >= kIndexLimit || q_len >= kIndexLimit || batch * q_len >= kIndexLimit || n_states >= kIndexLimit)
    return NVFP4_ERR_RANGE;
  const int64_t kw = (int64_t)k_heads * 128, vw = (int64_t)v_heads * 128;
  if (ld_states < vw * 128 || ld_states % 4 != 0) return NVFP4_ERR_STRIDE;
  if (ld_states >= kIndexLimit) return NVFP4_ERR_RANGE;
  if (slots == nullptr && batch > n_states) return NVFP4_ERR_SHAPE;
  if (batch == 0) return NVFP4_OK;
  if (in->q == nullptr || in->k == nullptr || in->v == nullptr || in->beta == nullptr || in->g == nullptr || o == nullptr ||
      states == nullptr)
    return NVFP4_ERR_NULL;
  int st;
  const int64_t rows = batch * q_len;
  if ((st = check_rows(in->q, rows, in->ld_q, kw, esz)) != NVFP4_OK) return st;
  if ((st = check_rows(in->k, rows, in->ld_k, kw, esz)) != NVFP4_OK) return st;
  if ((st = check_rows(in->v, rows, in->ld_v, vw, esz)) != NVFP4_OK) return st;
  if (in->ld_beta < v_heads || in->ld_g < v_heads || ld_o < vw) return NVFP4_ERR_STRIDE;
  if (in->ld_beta >= kIndexLimit || in->ld_g >= kIndexLimit || ld_o >= kIndexLimit) return NVFP4_ERR_RANGE;
  if (!aligned(in->beta, (uintptr_t)esz) || !aligned(in->g, (uintptr_t)esz) || !aligned(o, (uintptr_t)osz) ||
      !aligned(states, 16) || !aligned(slots, 4))
    return NVFP4_ERR_ALIGN;
  const GdnStepArgs a{*in, in_dtype, o_dtype, (int)batch, (int)q_len, k_heads, v_heads, normalize_qk != 0,
                      states, n_states, ld_states, slots, fresh, o, ld_o};
  return status_from_hip(launch_gdn_step(a, (hipStream_t)stream));
}

}  // extern "C"
