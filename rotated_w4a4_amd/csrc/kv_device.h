// Device-side pieces shared by the KV cache kernels: head rows spread over
// lanes (8 consecutive channels a lane, D / 8 lanes a row).
#pragma once

#include "rw4_device.h"

namespace rw4 {

template <int M>
__device__ __forceinline__ void lane_stage(float (&v)[8], int lane) {
  const float sign = (lane & M) ? -1.0f : 1.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = sign * v[e] + lane_xor<M>(v[e]);
}

// y H_D (Sylvester order, entries +-1) of a row.
template <int L>
__device__ __forceinline__ void row_hadamard(float (&v)[8], int lane) {
  fwht8(v);
  lane_stage<1>(v, lane);
  lane_stage<2>(v, lane);
  lane_stage<4>(v, lane);
  if constexpr (L > 8) lane_stage<8>(v, lane);
  if constexpr (L > 16) lane_stage<16>(v, lane);
}

__device__ __forceinline__ void store_row8(void* base, bool bf16, int64_t off, const float (&v)[8]) {
  if (bf16) {
    __bf16 h[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = static_cast<__bf16>(v[i]);  // round to nearest even
    *reinterpret_cast<uint4*>(reinterpret_cast<__bf16*>(base) + off) = *reinterpret_cast<const uint4*>(h);
  } else {
    float4* dst = reinterpret_cast<float4*>(reinterpret_cast<float*>(base) + off);
    dst[0] = make_float4(v[0], v[1], v[2], v[3]);
    dst[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

// 1 / sqrt(D) of the head's Hadamard.
template <int D>
constexpr float kHeadPost = D == 64 ? 0.125f : D == 256 ? 0.0625f : 0.08838834764831845f;

}  // namespace rw4
