// Stand-ins for the launchers of the paged KV cache, for kv_pages_api.hip
// built as plain host C++ under AddressSanitizer / UBSan: each records its
// call and keeps away from the (device) pointers.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../bit_linear_layer_amd/csrc/kv_pages.h"

namespace {
int g_calls = 0;
nvfp4::KvPages g_pages;
nvfp4::KvAttnArgs g_args;
}  // namespace

extern "C" int nvfp4_kv_stub_calls(void) { return g_calls; }
extern "C" int nvfp4_kv_stub_page_shift(void) { return g_pages.page_shift; }
extern "C" int nvfp4_kv_stub_group(void) { return g_args.group; }

namespace nvfp4 {

hipError_t launch_kv_pages_write(const KvPages& c, const void*, int64_t, const void*, int64_t, int, int64_t,
                                 const int64_t*, hipStream_t) {
  g_pages = c;
  ++g_calls;
  return hipSuccess;
}
hipError_t launch_kv_pages_read(const KvPages& c, int64_t, const int64_t*, void*, int64_t, void*, int64_t, int,
                                hipStream_t) {
  g_pages = c;
  ++g_calls;
  return hipSuccess;
}
size_t kv_attention_workspace(const KvAttnArgs& a) { return 16 + (size_t)a.batch * a.q_len * a.q_heads * a.c.dim * 4; }
hipError_t launch_kv_attention(const KvAttnArgs& a, void*, hipStream_t) {
  g_pages = a.c;
  g_args = a;
  ++g_calls;
  return hipSuccess;
}

}  // namespace nvfp4
