// Paged FP8 KV cache: the parts shared by the write, the read and the
// attention kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "internal.h"

namespace nvfp4 {

// nvfp4_kv_pages with the sizes the kernels index with.
struct KvPages {
  uint8_t *kc, *vc, *ks, *vs;
  int64_t ld_codes, ld_scales;
  int n_pages, heads, dim;
  int page_shift;  // log2(page_size)
};

struct KvAttnArgs {
  KvPages c;
  const void* q; int64_t ld_q;
  void* out; int64_t ld_out;
  int dtype;
  int q_heads, group;
  int batch, q_len;  // batch * q_len * q_heads < 2^30
  const int* lens;   // null: all zero
  int max_len;
  const int* table; int64_t ld_table;
  const int* prefix_pages;
  int prefix_len;
  float scale_log2;  // scale * log2(e)
};

hipError_t launch_kv_pages_write(const KvPages& c, const void* k, int64_t ld_k, const void* v, int64_t ld_v, int dtype,
                                 int64_t rows, const int64_t* slots, hipStream_t s);
hipError_t launch_kv_pages_read(const KvPages& c, int64_t rows, const int64_t* slots, void* k, int64_t ld_k, void* v,
                                int64_t ld_v, int dtype, hipStream_t s);
size_t kv_attention_workspace(const KvAttnArgs& a);
hipError_t launch_kv_attention(const KvAttnArgs& a, void* ws, hipStream_t s);

}  // namespace nvfp4
