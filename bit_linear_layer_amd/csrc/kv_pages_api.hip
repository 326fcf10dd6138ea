// C ABI of the paged FP8 KV cache and its attention: argument validation
// (before any HIP call) and dispatch.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "internal.h"
#include "kv_pages.h"
#include "nvfp4.h"

using namespace nvfp4;

namespace {

constexpr int64_t kIndexLimit = (int64_t)1 << 31;
constexpr int64_t kLengthLimit = (int64_t)1 << 30;  // tokens and rows round up to whole steps and tiles in 32 bits
constexpr int64_t kRowLimit = ((int64_t)1 << 28) - 15;  // workgroups of 256 threads for 16 rows each, in a grid of less than 2^32

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }

int elem_size(int dtype) { return dtype == NVFP4_DTYPE_BF16 ? 2 : dtype == NVFP4_DTYPE_F32 ? 4 : 0; }

// The sizes of a cache (not its pointers).
int check_pages_shape(const nvfp4_kv_pages* c, KvPages& out) {
  if (c == nullptr) return NVFP4_ERR_NULL;
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return NVFP4_ERR_SHAPE;
  if (c->page_size < 16 || c->page_size > 4096 || (c->page_size & (c->page_size - 1)) != 0) return NVFP4_ERR_SHAPE;
  if (c->kv_heads < 1 || c->kv_heads > 4096 || c->n_pages < 1) return NVFP4_ERR_SHAPE;
  if (c->n_pages >= kIndexLimit || c->n_pages * c->page_size >= kIndexLimit) return NVFP4_ERR_RANGE;
  out.n_pages = (int)c->n_pages;
  out.heads = c->kv_heads;
  out.dim = c->head_dim;
  out.page_shift = __builtin_ctz((unsigned)c->page_size);
  return NVFP4_OK;
}

int check_pages(const nvfp4_kv_pages* c, KvPages& out) {
  const int st = check_pages_shape(c, out);
  if (st != NVFP4_OK) return st;
  if (c->k_codes == nullptr || c->v_codes == nullptr || c->k_scales == nullptr || c->v_scales == nullptr)
    return NVFP4_ERR_NULL;
  const int64_t per = (int64_t)c->kv_heads * c->page_size;
  if (c->ld_codes < per * c->head_dim || c->ld_codes % 16 != 0) return NVFP4_ERR_STRIDE;
  if (c->ld_scales < per || c->ld_scales % 16 != 0) return NVFP4_ERR_STRIDE;
  if (c->ld_codes >= kIndexLimit || c->ld_scales >= kIndexLimit) return NVFP4_ERR_RANGE;
  if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16) || !aligned(c->k_scales, 16) || !aligned(c->v_scales, 16))
    return NVFP4_ERR_ALIGN;
  out.kc = c->k_codes;
  out.vc = c->v_codes;
  out.ks = c->k_scales;
  out.vs = c->v_scales;
  out.ld_codes = c->ld_codes;
  out.ld_scales = c->ld_scales;
  return NVFP4_OK;
}

// A dense operand whose rows hold `width` elements of `esz` bytes.
int check_rows(const void* p, int64_t ld, int64_t width, int esz) {
  if (ld < width || ld % (16 / esz) != 0) return NVFP4_ERR_STRIDE;
  return aligned(p, 16) ? NVFP4_OK : NVFP4_ERR_ALIGN;
}

// The sizes of a batch over cache `c` (already in a.c), not its pointers.
int check_batch(const nvfp4_kv_batch* b, int q_heads, int dtype, KvAttnArgs& a) {
  if (b == nullptr) return NVFP4_ERR_NULL;
  if (elem_size(dtype) == 0) return NVFP4_ERR_DTYPE;
  if (q_heads < 1 || q_heads % a.c.heads != 0) return NVFP4_ERR_SHAPE;
  if (b->batch < 0 || b->q_len < 1 || b->max_len < 0 || b->prefix_len < 0) return NVFP4_ERR_SHAPE;
  if (b->batch >= kIndexLimit || b->q_len >= kIndexLimit || b->max_len >= kLengthLimit || b->prefix_len >= kLengthLimit)
    return NVFP4_ERR_RANGE;
  if (b->batch * b->q_len >= kLengthLimit / q_heads) return NVFP4_ERR_RANGE;
  // a column of workgroups of 256 threads for each sequence and kv head, in a grid of less than 2^32
  if (b->batch * a.c.heads >= (int64_t)1 << 24) return NVFP4_ERR_RANGE;
  a.dtype = dtype;
  a.q_heads = q_heads;
  a.group = q_heads / a.c.heads;
  a.batch = (int)b->batch;
  a.q_len = (int)b->q_len;
  a.max_len = (int)b->max_len;
  a.prefix_len = (int)b->prefix_len;
  return NVFP4_OK;
}

}  // namespace

extern "C" {

int nvfp4_kv_pages_write(const nvfp4_kv_pages* cache, const void* k, int64_t ld_k, const void* v, int64_t ld_v,
                         int x_dtype, int64_t rows, const int64_t* slots, void* stream) {
  KvPages c{};
  int st = check_pages(cache, c);
  if (st != NVFP4_OK) return st;
  const int esz = elem_size(x_dtype);
  if (esz == 0) return NVFP4_ERR_DTYPE;
  if (rows < 0) return NVFP4_ERR_SHAPE;
  if (rows >= kRowLimit) return NVFP4_ERR_RANGE;
  if (rows == 0) return NVFP4_OK;
  if (k == nullptr || v == nullptr || slots == nullptr) return NVFP4_ERR_NULL;
  const int64_t width = (int64_t)c.heads * c.dim;
  if ((st = check_rows(k, ld_k, width, esz)) != NVFP4_OK) return st;
  if ((st = check_rows(v, ld_v, width, esz)) != NVFP4_OK) return st;
  if (!aligned(slots, 8)) return NVFP4_ERR_ALIGN;
  return status_from_hip(launch_kv_pages_write(c, k, ld_k, v, ld_v, x_dtype, rows, slots, (hipStream_t)stream));
}

int nvfp4_kv_pages_read(const nvfp4_kv_pages* cache, int64_t rows, const int64_t* slots, void* k_out, int64_t ld_k,
                        void* v_out, int64_t ld_v, int out_dtype, void* stream) {
  KvPages c{};
  int st = check_pages(cache, c);
  if (st != NVFP4_OK) return st;
  const int esz = elem_size(out_dtype);
  if (esz == 0) return NVFP4_ERR_DTYPE;
  if (rows < 0) return NVFP4_ERR_SHAPE;
  if (rows >= kRowLimit) return NVFP4_ERR_RANGE;
  if (rows == 0) return NVFP4_OK;
  if (k_out == nullptr || v_out == nullptr || slots == nullptr) return NVFP4_ERR_NULL;
  const int64_t width = (int64_t)c.heads * c.dim;
  if ((st = check_rows(k_out, ld_k, width, esz)) != NVFP4_OK) return st;
  if ((st = check_rows(v_out, ld_v, width, esz)) != NVFP4_OK) return st;
  if (!aligned(slots, 8)) return NVFP4_ERR_ALIGN;
  return status_from_hip(launch_kv_pages_read(c, rows, slots, k_out, ld_k, v_out, ld_v, out_dtype, (hipStream_t)stream));
}

size_t nvfp4_kv_pages_attention_workspace_bytes(const nvfp4_kv_pages* cache, const nvfp4_kv_batch* batch, int q_heads,
                                                int dtype) {
  KvAttnArgs a{};
  if (check_pages_shape(cache, a.c) != NVFP4_OK) return 0;
  if (check_batch(batch, q_heads, dtype, a) != NVFP4_OK) return 0;
  return kv_attention_workspace(a);
}

int nvfp4_kv_pages_attention(const nvfp4_kv_pages* cache, const nvfp4_kv_batch* batch, const void* q, int64_t ld_q,
                             int dtype, int q_heads, float scale, void* out, int64_t ld_out, void* workspace,
                             size_t workspace_bytes, void* stream) {
  KvAttnArgs a{};
  int st = check_pages(cache, a.c);
  if (st != NVFP4_OK) return st;
  if ((st = check_batch(batch, q_heads, dtype, a)) != NVFP4_OK) return st;
  a.scale_log2 = scale * 1.44269504088896341f;
  if (!(scale > 0.0f) || !isfinite(a.scale_log2)) return NVFP4_ERR_VALUE;
  if (a.batch == 0) return NVFP4_OK;
  if (q == nullptr || out == nullptr) return NVFP4_ERR_NULL;
  const int esz = elem_size(dtype);
  const int64_t width = (int64_t)q_heads * a.c.dim;
  if ((st = check_rows(q, ld_q, width, esz)) != NVFP4_OK) return st;
  if ((st = check_rows(out, ld_out, width, esz)) != NVFP4_OK) return st;
  if (a.max_len > 0) {
    if (batch->table == nullptr || batch->lens == nullptr) return NVFP4_ERR_NULL;
    if (batch->table_cols < (a.max_len + (int64_t)cache->page_size - 1) / cache->page_size) return NVFP4_ERR_SHAPE;
    if (batch->ld_table < batch->table_cols) return NVFP4_ERR_STRIDE;
  }
  if (a.prefix_len > 0 && batch->prefix_pages == nullptr) return NVFP4_ERR_NULL;
  if (!aligned(batch->table, 4) || !aligned(batch->lens, 4) || !aligned(batch->prefix_pages, 4)) return NVFP4_ERR_ALIGN;
  const size_t need = kv_attention_workspace(a);
  if (workspace == nullptr || workspace_bytes < need) return NVFP4_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return NVFP4_ERR_ALIGN;
  a.q = q; a.ld_q = ld_q;
  a.out = out; a.ld_out = ld_out;
  a.lens = batch->lens;
  a.table = batch->table; a.ld_table = batch->ld_table;
  a.prefix_pages = batch->prefix_pages;
  return status_from_hip(launch_kv_attention(a, workspace, (hipStream_t)stream));
}

}  // extern "C"
