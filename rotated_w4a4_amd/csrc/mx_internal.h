// Host-side interface between the C ABI layer and the MXFP4 kernel launchers.
#pragma once

#include "rw4_internal.h"

namespace rw4 {

// block: Hadamard block (128, 256, 512) or 1 for no transform; sign_mask [K] or null.
struct MxRows {
  const void* x;
  bool bf16;
  int64_t rows, K;
  int64_t stride_row, stride_k;  // elements
  int block;
  const uint32_t* sign_mask;
  uint8_t* q;
  uint8_t* s;
};

// Rows with stride_k = 1 and 16-byte rows.
hipError_t launch_mx_quantize(const MxRows& a, hipStream_t st);
// Rows of any strides, mx_pack_blocks(rows, K, block) <= kMxPackMostBlocks.
hipError_t launch_mx_pack(const MxRows& a, hipStream_t st);
hipError_t launch_mx_dequantize(const uint8_t* q, const uint8_t* s, int64_t M, int64_t K, void* out, bool out_bf16,
                                int64_t ldo, hipStream_t st);
// mx_gemm_fits(M, N, K).
hipError_t launch_mx_gemm(const uint8_t* qa, const uint8_t* sa, const uint8_t* qw, const uint8_t* sw, int64_t M,
                          int64_t N, int64_t K, void* y, bool y_bf16, int64_t ldy, hipStream_t st);

}  // namespace rw4
