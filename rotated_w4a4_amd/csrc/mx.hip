// MXFP4: rotation and quantization of rows, and reading them back.
//
//   y = x R           R the block Hadamard / sqrt(block), block 128, 256 or 512,
//                     with an optional +-1 diagonal in front, or the identity
//   E = clamp(floor(log2 max |y|) - 2, -127, 127) over 32 channels (-127 for zeros)
//   code = y 2^-E rounded to {0, 0.5, 1, 1.5, 2, 3, 4, 6} with its sign, ties to
//          the even code, what lies above 6 to 6
//
// A block whose maximum is not finite gets the scale 255 (NaN) and codes 0.
//
// Exactness.  Codes and exponents are those of the exact y.  The butterflies run
// in fp32 and keep a bound of their error: each of the n stages rounds every
// intermediate once, all intermediates of an output are at most S = sum |x| over
// the Hadamard block, so |u - exact| <= n 2^-24 S (1 + tiny); forming y = u c 2^-E
// and the two values below costs 3 roundings of at most S more, and the sum S
// itself is short of the exact one by less than 2^-19 of it, so
//   d = (n + 5) 2^-24 S c 2^-E
// covers everything.  A lane converts y - d and y + d: where the codes of both
// are the same they are the code of the exact value.  Otherwise, or where the
// maximum could lie on either side of a power of two, the wave evaluates its rows
// again in fp64 (about one wave of 512 values in 50 for Gaussian values in blocks
// of 128).  fp64 for every row would take several times as long, fp32 alone would
// decide ties by the order of its additions: with blocks of 256 and bf16 values,
// exact ties are common.
#include <type_traits>

#include "mx_internal.h"
#include "rw4_device.h"

namespace rw4 {

namespace {

constexpr int kSpan = 512;    // channels of a wave: 8 for each lane

template <int BLOCK>
constexpr int kStages = BLOCK == 1 ? 0 : BLOCK == 128 ? 7 : BLOCK == 256 ? 8 : 9;
template <int BLOCK>
constexpr double kPost64 = BLOCK == 1     ? 1.0
                           : BLOCK == 128 ? 0.08838834764831843
                           : BLOCK == 256 ? 0.0625
                                          : 0.04419417382415922;
template <int BLOCK>
constexpr float kPost32 = float(kPost64<BLOCK>);

__device__ __forceinline__ float two_to(int e) { return __uint_as_float(uint32_t(e + 127) << 23); }  // -126..127

// Eight values as FP4 codes, value e in bits 4 e .. 4 e + 3; round to nearest
// even, saturating.
__device__ __forceinline__ uint32_t fp4_word(const float (&v)[8]) {
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], 1.0f, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], 1.0f, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], 1.0f, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], 1.0f, 3);
  return w;
}

// The lanes of a 16-lane row hold the words word_of(l) of their 128 channels:
// after the DPP lane stages of rw4_device.h (blocks of 128 and more) a signed
// permutation, without a transform in order.
template <int BLOCK>
__device__ __forceinline__ int word_of(int l) {
  return BLOCK == 1 ? l : h128_lane_word(l);
}

// Maximum over the 4 lanes whose words make one block of 32 channels: lanes that
// agree in l & 8 and, behind the permutation, in the parity of l & 7 (f(l) >> 2 =
// 2 (l / 8) + parity), so the lane masks 3 and 6; else the lane's quad.
template <int BLOCK>
__device__ __forceinline__ uint32_t block_max(uint32_t m) {
  if constexpr (BLOCK == 1) {
    m = max(m, uint32_t(__builtin_amdgcn_mov_dpp(int(m), 0xB1, 0xF, 0xF, true)));
    return max(m, uint32_t(__builtin_amdgcn_mov_dpp(int(m), 0x4E, 0xF, 0xF, true)));
  } else {
    m = max(m, uint32_t(__builtin_amdgcn_mov_dpp(int(m), 0x1B, 0xF, 0xF, true)));            // lane ^ 3
    const int t = __builtin_amdgcn_mov_dpp(int(m), 0x141, 0xF, 0xF, true);                   // lane ^ 7
    return max(m, uint32_t(__builtin_amdgcn_mov_dpp(t, 0xB1, 0xF, 0xF, true)));              // ^ 1: lane ^ 6
  }
}

// Sum over the lanes of a Hadamard block.
template <int BLOCK>
__device__ __forceinline__ float block_sum(float s) {
  s += lane_xor<1>(s);
  s += lane_xor<2>(s);
  s += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(s), 0x141, 0xF, 0xF, true));  // lane ^ 7
  s += lane_xor<8>(s);
  if constexpr (BLOCK >= 256) s += lane_xor<16>(s);
  if constexpr (BLOCK >= 512) s += lane_xor<32>(s);
  return s;
}

// The four scale bytes of 128 channels from the lanes that hold them: byte b in
// its place, or-ed over lanes with different b.
template <int BLOCK>
__device__ __forceinline__ uint32_t gather_scales(uint32_t byte, int l) {
  uint32_t w = byte << (8 * (word_of<BLOCK>(l) >> 2));
  if constexpr (BLOCK == 1) {
    w |= uint32_t(__builtin_amdgcn_mov_dpp(int(w), 0x141, 0xF, 0xF, true));  // lane ^ 7: the other quad of 8 lanes
  } else {
    w |= uint32_t(__builtin_amdgcn_mov_dpp(int(w), 0xB1, 0xF, 0xF, true));  // lane ^ 1: the other parity
  }
  return w | uint32_t(__builtin_amdgcn_mov_dpp(int(w), 0x128, 0xF, 0xF, true));  // lane ^ 8
}

// What a lane stores: 8 codes of word `word` of its 128 channels, and in lane 0
// of each 16 the four scale bytes.
struct MxWord {
  uint32_t codes, scales;
  int word;
};

__device__ __forceinline__ double shfl_xor64(double v, int mask) { return __shfl_xor(v, mask); }

// The rows of the wave in fp64, in channel order (rarely called).
template <int BLOCK, class Load>
__device__ __forceinline__ MxWord encode64(Load load, int lane) {
  float v[8];
  load(v);
  double u[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) u[e] = v[e];
  if constexpr (BLOCK > 1) {
#pragma unroll
    for (int h = 1; h < 8; h <<= 1)
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if ((e & h) == 0) {
          const double a = u[e], b = u[e | h];
          u[e] = a + b;
          u[e | h] = a - b;
        }
#pragma unroll 1
    for (int m = 1; m < BLOCK / 8; m <<= 1)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const double o = shfl_xor64(u[e], m);
        u[e] = (lane & m) ? o - u[e] : u[e] + o;
      }
#pragma unroll
    for (int e = 0; e < 8; ++e) u[e] *= kPost64<BLOCK>;
  }
  unsigned long long top = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) top = max(top, (unsigned long long)(__double_as_longlong(u[e])) & 0x7FFFFFFFFFFFFFFFull);
  top = max(top, (unsigned long long)(__shfl_xor((long long)(top), 1)));
  top = max(top, (unsigned long long)(__shfl_xor((long long)(top), 2)));
  const bool finite = top < 0x7FF0000000000000ull;
  int E = int(top >> 52) - 1023 - 2;  // a zero or a subnormal lies below -127
  E = E < -127 ? -127 : E > 127 ? 127 : E;
  MxWord r;
  r.codes = 0;
  r.word = lane & 15;
  const double inv = ldexp(1.0, -E);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const double a = fabs(u[e]) * inv;
    // ties between codes i and i + 1 go to the even one
    const uint32_t n = uint32_t(a > 0.25) + uint32_t(a >= 0.75) + uint32_t(a > 1.25) + uint32_t(a >= 1.75) +
                       uint32_t(a > 2.5) + uint32_t(a >= 3.5) + uint32_t(a > 5.0);
    r.codes |= (n | (u[e] < 0.0 ? 8u : 0u)) << (4 * e);
  }
  if (!finite) r.codes = 0;
  r.scales = gather_scales<1>(finite ? uint32_t(E + 127) : 255u, lane & 15);
  return r;
}

// The lane's 8 channels of a row (16 lanes hold 128, the wave 512), encoded.
// load gives the values again; every lane of the wave takes part.
template <int BLOCK, class Load>
__device__ __forceinline__ MxWord encode(float (&v)[8], Load load, int lane) {
  const int l = lane & 15;
  if constexpr (BLOCK == 1) {
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(v[e]) & 0x7FFFFFFFu);
    top = block_max<1>(top);
    const bool finite = top < 0x7F800000u;
    const int E = max(int(top >> 23) - 127 - 2, -127);
    const float inv = two_to(-E);  // 2^-126 .. 2^127 (E <= 125): exact, also from subnormals
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = finite ? fmaf(v[e], inv, 0.0f) : 0.0f;  // -0 becomes 0
    return MxWord{fp4_word(v), gather_scales<1>(finite ? uint32_t(E + 127) : 255u, l), l};
  } else {
    constexpr int n = kStages<BLOCK>;
    float S = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) S += fabsf(v[e]);
    S = block_sum<BLOCK>(S);
    fwht8(v);
    lane_stages_dpp(v, (__builtin_popcount(l & 5) & 1) ? -1.0f : 1.0f, (__builtin_popcount(l & 6) & 1) ? -1.0f : 1.0f,
                    (l & 4) ? -1.0f : 1.0f, (l & 8) ? -1.0f : 1.0f);
    if constexpr (BLOCK >= 256) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = butterfly_x<16>(v[e], lane);
    }
    if constexpr (BLOCK >= 512) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = butterfly_x<32>(v[e], lane);
    }
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(v[e]) & 0x7FFFFFFFu);
    top = block_max<BLOCK>(top);
    const float err = S * (kPost32<BLOCK> * float(n + 5) * 0x1p-24f);
    const float most = __uint_as_float(top) * kPost32<BLOCK>;
    const uint32_t at = __float_as_uint(most + err) >> 23;
    const int E = max(int(at) - 127 - 2, -127);
    const float inv = two_to(-E), d = err * inv;
    const float c = kPost32<BLOCK> * parity_sign(l) * inv;
    float lo[8], hi[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      lo[e] = fmaf(v[e], c, -d);
      hi[e] = fmaf(v[e], c, d);
    }
    const uint32_t w = fp4_word(hi);  // v c + 0 is not -0
    // Sums beyond 2^100 (and what is not finite) could leave fp32; below 2^-90 the
    // products above could lose bits; without any value all is zero.
    const bool sure = w == fp4_word(lo) && at == __float_as_uint(most - err) >> 23 && S < 0x1p100f && S > 0x1p-90f;
    if (__builtin_amdgcn_ballot_w64(!sure && S != 0.0f) != 0) return encode64<BLOCK>(load, lane);
    return MxWord{w, gather_scales<BLOCK>(uint32_t(E + 127), l), h128_lane_word(l)};
  }
}

__device__ __forceinline__ void store_word(const MxRows& a, int64_t row, int64_t k0, int lane, const MxWord& r) {
  // k0: first channel of the wave's span
  const int64_t g = (k0 >> 7) + (lane >> 4);
  *reinterpret_cast<uint32_t*>(a.q + row * (a.K >> 1) + 64 * g + 4 * r.word) = r.codes;
  if ((lane & 15) == 0) *reinterpret_cast<uint32_t*>(a.s + (g * a.rows + row) * 4) = r.scales;
}

// ---------------------------------------------------------------------------
// Rows with unit stride: a wave takes 512 channels of a row, the grid walks the
// spans of all rows in order; the next span is loaded before the current one is
// computed.
// ---------------------------------------------------------------------------
template <bool BF16, int BLOCK, bool SIGNED>
__global__ __launch_bounds__(256) void mx_quantize_kernel(MxRows a) {
  const int lane = threadIdx.x & 63;
  const int64_t spans = (a.K + kSpan - 1) / kSpan;
  const int64_t waves = int64_t(gridDim.x) * 4, first = int64_t(blockIdx.x) * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t step_row = waves / spans, step_span = waves % spans;
  int64_t row = first / spans, span = first % spans;
  auto load = [&](int64_t r, int64_t sp, float (&v)[8]) {
    const int64_t k = sp * kSpan + 8 * lane;
    if (k < a.K) {
      RowSrc<BF16> src{a.x, a.stride_row};
      if constexpr (SIGNED) SignedSrc<RowSrc<BF16>>{src, a.sign_mask}.load8(r, k, v);
      else src.load8(r, k, v);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = 0.0f;
    }
  };
  float next[8];
  if (row < a.rows) load(row, span, next);
  while (row < a.rows) {
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = next[e];
    int64_t row2 = row + step_row, span2 = span + step_span;
    if (span2 >= spans) {
      span2 -= spans;
      ++row2;
    }
    if (row2 < a.rows) load(row2, span2, next);
    const MxWord r = encode<BLOCK>(v, [&](float(&w)[8]) { load(row, span, w); }, lane);
    if (span * kSpan + 8 * lane < a.K) store_word(a, row, span * kSpan, lane, r);
    row = row2;
    span = span2;
  }
}

// ---------------------------------------------------------------------------
// Rows of any strides (weights [K, N]): a block brings 32 rows x 512 channels
// into LDS, its lanes along whichever stride is 1, then encodes them from there.
// Channel k of a row lies at k + k / 8, so that 64 lanes reading every ninth
// word hit all banks; rows are an odd number of words apart for the writes.
// ---------------------------------------------------------------------------
constexpr int kPackRows = 32;
constexpr int kPackRow = kSpan + kSpan / 8 + 1;

template <bool BF16, int BLOCK, bool SIGNED>
__global__ __launch_bounds__(256) void mx_pack_kernel(MxRows a, int64_t spans) {
  __shared__ float tile[kPackRows * kPackRow];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t row0 = (blockIdx.x / spans) * kPackRows, k0 = (blockIdx.x % spans) * kSpan;
  const int64_t rows = a.rows - row0 < kPackRows ? a.rows - row0 : kPackRows;
  const int64_t channels = a.K - k0 < kSpan ? a.K - k0 : kSpan;
  const bool along_rows = a.stride_row <= a.stride_k;
  const StridedSrc<BF16> src{a.x, a.stride_k, a.stride_row};
#pragma unroll 8
  for (int i = 0; i < kPackRows * kSpan / 256; ++i) {
    const int at = i * 256 + tid;
    const int r = along_rows ? at % kPackRows : at / kSpan, k = along_rows ? at / kPackRows : at % kSpan;
    float v = 0.0f;
    if (r < rows && k < channels) {
      v = src.at(row0 + r, k0 + k);
      if constexpr (SIGNED) v = __uint_as_float(__float_as_uint(v) ^ a.sign_mask[k0 + k]);
    }
    tile[r * kPackRow + k + (k >> 3)] = v;
  }
  __syncthreads();
  for (int r = wave; r < rows; r += 4) {
    auto load = [&](float(&v)[8]) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = tile[r * kPackRow + 9 * lane + e];
    };
    float v[8];
    load(v);
    const MxWord w = encode<BLOCK>(v, load, lane);
    if (8 * lane < channels) store_word(a, row0 + r, k0, lane, w);
  }
}

// ---------------------------------------------------------------------------
// Reading back: 8 codes a lane.  Values are exact in bf16 and fp32.
// ---------------------------------------------------------------------------
template <bool BF16>
__global__ __launch_bounds__(256) void mx_dequantize_kernel(const uint8_t* q, const uint8_t* s, int64_t M, int64_t K,
                                                            void* out, int64_t ldo) {
  typedef float v2f __attribute__((ext_vector_type(2)));
  const int64_t words = K >> 3, step = int64_t(gridDim.x) * 256, all = M * words;
  int64_t at = int64_t(blockIdx.x) * 256 + threadIdx.x;
  int64_t row = at / words, word = at % words;
  const int64_t step_row = step / words, step_word = step % words;
  for (; at < all; at += step) {
    const uint32_t w = reinterpret_cast<const uint32_t*>(q)[at];
    const uint32_t e = s[((word >> 4) * M + row) * 4 + ((word >> 2) & 3)];
    v2f p[4];
    p[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0);
    p[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
    p[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2);
    p[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = ldexpf(p[i >> 1][i & 1], int(e) - 127);
      v[i] = e == 255 ? __builtin_nanf("") : x;
    }
    const int64_t o = row * ldo + 8 * word;
    if constexpr (BF16) {
      uint32_t b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)  // exact: the lower halves are zero (NaN: its upper half is NaN)
        b[i] = (__float_as_uint(v[2 * i]) >> 16) | (__float_as_uint(v[2 * i + 1]) & 0xFFFF0000u);
      *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(out) + o) = make_uint4(b[0], b[1], b[2], b[3]);
    } else {
      float4* dst = reinterpret_cast<float4*>(reinterpret_cast<float*>(out) + o);
      dst[0] = make_float4(v[0], v[1], v[2], v[3]);
      dst[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
    row += step_row;
    word += step_word;
    if (word >= words) {
      word -= words;
      ++row;
    }
  }
}

// f(type of x, block, signed) for the run-time values.
template <class F>
hipError_t by_kind(const MxRows& a, F f) {
  using T = std::true_type;
  using N = std::false_type;
  auto by_sign = [&](auto bf16, auto block) { return a.sign_mask ? f(bf16, block, T{}) : f(bf16, block, N{}); };
  auto by_block = [&](auto bf16) {
    switch (a.block) {
      case 1: return f(bf16, std::integral_constant<int, 1>{}, N{});
      case 128: return by_sign(bf16, std::integral_constant<int, 128>{});
      case 256: return by_sign(bf16, std::integral_constant<int, 256>{});
      default: return by_sign(bf16, std::integral_constant<int, 512>{});
    }
  };
  return a.bf16 ? by_block(T{}) : by_block(N{});
}

}  // namespace

hipError_t launch_mx_quantize(const MxRows& a, hipStream_t st) {
  const int64_t spans = (a.K + kSpan - 1) / kSpan, items = a.rows * spans;
  const int64_t full = 256 * 8;  // 8 blocks of 4 waves a CU
  const int64_t need = (items + 3) / 4, blocks = need < full ? need : full;
  return by_kind(a, [&](auto bf16, auto block, auto sign) {
    hipLaunchKernelGGL((mx_quantize_kernel<decltype(bf16)::value, decltype(block)::value, decltype(sign)::value>),
                       dim3(unsigned(blocks)), dim3(256), 0, st, a);
    return hipGetLastError();
  });
}

hipError_t launch_mx_pack(const MxRows& a, hipStream_t st) {
  const int64_t spans = (a.K + kSpan - 1) / kSpan, blocks = (a.rows + kPackRows - 1) / kPackRows * spans;
  if (blocks > (int64_t(1) << 23)) return hipErrorInvalidValue;  // a grid has fewer than 2^32 threads
  return by_kind(a, [&](auto bf16, auto block, auto sign) {
    hipLaunchKernelGGL((mx_pack_kernel<decltype(bf16)::value, decltype(block)::value, decltype(sign)::value>),
                       dim3(unsigned(blocks)), dim3(256), 0, st, a, spans);
    return hipGetLastError();
  });
}

hipError_t launch_mx_dequantize(const uint8_t* q, const uint8_t* s, int64_t M, int64_t K, void* out, bool out_bf16,
                                int64_t ldo, hipStream_t st) {
  const int64_t need = (M * (K >> 3) + 255) / 256, full = 256 * 16, blocks = need < full ? need : full;
  if (out_bf16)
    hipLaunchKernelGGL((mx_dequantize_kernel<true>), dim3(unsigned(blocks)), dim3(256), 0, st, q, s, M, K, out, ldo);
  else
    hipLaunchKernelGGL((mx_dequantize_kernel<false>), dim3(unsigned(blocks)), dim3(256), 0, st, q, s, M, K, out, ldo);
  return hipGetLastError();
}

}  // namespace rw4
