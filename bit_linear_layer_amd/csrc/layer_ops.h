// Launchers of the 8-bit linear layers, the query/key norm with rotation, the
// short convolution and the gated delta rule's next tokens.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "nvfp4.h"

namespace nvfp4 {

// E4M3 codes with a float32 scale per block: the 128 codes of (row, block b)
// begin at codes[row * ld_codes + b * code_block], its scale is at
// scales[row * scale_row + b * scale_block] (rows counted in block_rows).
struct Fp8Mat {
  uint8_t* codes;
  float* scales;
  int64_t ld_codes, code_block, scale_row, scale_block;
};

hipError_t launch_fp8_quantize_rows(const void* x, int dtype, int64_t rows, int64_t cols, int64_t ld_x, const Fp8Mat& q,
                                    bool pow2, hipStream_t s);
hipError_t launch_fp8_quantize_blocks(const void* x, int dtype, int64_t rows, int64_t cols, int64_t ld_x, const Fp8Mat& q,
                                      bool pow2, hipStream_t s);

struct Fp8GemmArgs {
  Fp8Mat a, w;  // a: block_rows 1, w: block_rows 128
  void* out;
  int64_t ld_out;
  int out_dtype;
  int M, N, K;
  bool cut_sums;  // the 8-bit matrix instructions are allowed
};
size_t fp8_gemm_workspace(int64_t m);  // bytes for products of up to 2^31 columns with m tokens
// Whether the product reads a's blocks wherever they lie; else a.code_block has to be 128.
bool fp8_gemm_shares(const Fp8GemmArgs& g);
hipError_t launch_fp8_gemm(const Fp8GemmArgs& g, float* ws, hipStream_t s);

struct RopeArgs {
  nvfp4_head_rows rows[2];  // queries, keys; heads 0 where absent
  nvfp4_rope rope;          // rotary_dim 0 where absent
  int dtype, head_dim;
  int64_t tokens;
  float eps, weight_offset;
};
hipError_t launch_qk_norm_rope(const RopeArgs& a, hipStream_t s);

hipError_t launch_causal_conv(const nvfp4_conv& c, int dtype, hipStream_t s);

struct GdnStepArgs {
  nvfp4_gdn_inputs in;
  int in_dtype, o_dtype;
  int batch, q_len, hk, hv, normalize;
  float* states;
  int64_t n_states, ld_states;
  const int32_t* slots;
  const uint8_t* fresh;
  void* o;
  int64_t ld_o;
};
hipError_t launch_gdn_step(const GdnStepArgs& a, hipStream_t s);

}  // namespace nvfp4
