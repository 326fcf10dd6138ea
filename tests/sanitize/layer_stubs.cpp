// Stand-ins for the launchers behind layer_api.hip, for a host build of it under
// AddressSanitizer / UBSan: each records its call and keeps away from the
// (device) pointers.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../bit_linear_layer_amd/csrc/layer_ops.h"

namespace {
int g_calls = 0;
int64_t g_seen[4];
hipError_t record(int64_t a = 0, int64_t b = 0, int64_t c = 0, int64_t d = 0) {
  ++g_calls;
  g_seen[0] = a; g_seen[1] = b; g_seen[2] = c; g_seen[3] = d;
  return hipSuccess;
}
}  // namespace

extern "C" int nvfp4_layer_stub_calls(void) { return g_calls; }
extern "C" int64_t nvfp4_layer_stub_seen(int i) { return g_seen[i]; }

namespace nvfp4 {

hipError_t launch_fp8_quantize_rows(const void*, int, int64_t rows, int64_t cols, int64_t, const Fp8Mat& q, bool, hipStream_t) {
  return record(rows, cols, q.ld_codes, q.scale_block);
}
hipError_t launch_fp8_quantize_blocks(const void*, int, int64_t rows, int64_t cols, int64_t, const Fp8Mat& q, bool, hipStream_t) {
  return record(rows, cols, q.ld_codes, q.scale_block);
}
size_t fp8_gemm_workspace(int64_t m) { return (m <= 16 ? 1 : 8) << 22; }
bool fp8_gemm_shares(const Fp8GemmArgs& g) { return g.M <= 128; }
hipError_t launch_fp8_gemm(const Fp8GemmArgs& g, float*, hipStream_t) { return record(g.M, g.N, g.K, g.ld_out); }
hipError_t launch_qk_norm_rope(const RopeArgs& a, hipStream_t) { return record(a.tokens, a.rows[0].heads, a.rows[1].heads, a.rope.rotary_dim); }
hipError_t launch_causal_conv(const nvfp4_conv& c, int, hipStream_t) { return record(c.tokens, c.channels, c.batch, c.width); }
hipError_t launch_gdn_step(const GdnStepArgs& a, hipStream_t) { return record(a.batch, a.q_len, a.hk, a.hv); }

}  // namespace nvfp4
