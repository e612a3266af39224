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
// Exactness.  Codes and exponents are decided in fp32 where that is certain.  The
// butterflies run in fp32 and keep a bound of their error: each of the n stages rounds
// every intermediate once, and the intermediates of a stage that an output depends on add
// up to at most S = sum |x| over the Hadamard block, so |u - exact| <= n 2^-24 S (1 +
// tiny).  Forming y = u c 2^-E costs the roundings of c 2^-E and of the result, 2^-24 of
// |y| < 8 each.  With
//   d = (n + 1/8) 2^-24 S c 2^-E + 2^-20
// (the eighth for S's own roundings, below 2^-19 of it) a lane converts y - d and y + d:
// where the codes of both are the same they are the code of the exact value.  Where they
// differ (about one wave of 512 Gaussian values in 60 in blocks of 128) the wave
// evaluates those values again in fp64 (settle), or all of its rows where they are many
// or the maximum could lie on either side of a power of two (encode64).  fp64 for every
// row would take several times as long, fp32 alone would decide ties by the order of
// its additions: with blocks of 256 and bf16 values, exact ties are common.
//   In fp64 a sum of at most 13 additions, times the rounded 1 / sqrt(block), is off by
// less than 15 2^-53 S / sqrt(block).  Sums of multiples of a unit below 2^53 units are
// exact, and so is the factor 1/16.  For 128 and 512 borders are m 2^k sqrt(2) units, m =
// 1, 3, 5, 7: no whole number below 2^46 comes closer to one of those than 2^-46.9 of it,
// and the two roundings are 2^-52 together, so such sums are decided as the exact y is.
// Larger ones can fall on a border's wrong side (124395540479019 is 5 2^44 sqrt(2) but for
// 2^-54.6), and fp64 loses what is 2^53 times smaller than the sum.
#include <type_traits>

#include "mx_index.h"
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

// A lane's value and that of lane ^ M (16 or 32): of the lane whose bit M is clear, and
// of the other.  Exchanging the upper halves (odd rows of 16) of a register with the
// lower ones (even rows) of its copy leaves just that.
struct Both {
  uint32_t clear, set;
};
template <int M>
__device__ __forceinline__ Both both(uint32_t v) {
  static_assert(M == 16 || M == 32, "lane masks of the swaps");
  if constexpr (M == 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    return Both{r[0], r[1]};
  } else {
    const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return Both{r[0], r[1]};
  }
}
// The butterfly over lane bit M.
template <int M>
__device__ __forceinline__ float lane_stage_swap(float v, int lane) {
  const Both b = both<M>(__float_as_uint(v));
  return fmaf((lane & M) ? -1.0f : 1.0f, __uint_as_float(b.set), __uint_as_float(b.clear));
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

// v of lane ^ 1, 2, 7 or 8 (CTRL a DPP control), in 64 bits.
template <int CTRL>
__device__ __forceinline__ double dpp64(double v) {
  const long long b = __double_as_longlong(v);
  const uint32_t lo = uint32_t(__builtin_amdgcn_mov_dpp(int(b), CTRL, 0xF, 0xF, true));
  const uint32_t hi = uint32_t(__builtin_amdgcn_mov_dpp(int(b >> 32), CTRL, 0xF, 0xF, true));
  return __longlong_as_double((long long)((uint64_t(hi) << 32) | lo));
}
template <int CTRL>
__device__ __forceinline__ void lane_stage64(double (&u)[8], bool negative) {
  const double c = negative ? -1.0 : 1.0;
#pragma unroll
  for (int e = 0; e < 8; ++e) u[e] = fma(dpp64<CTRL>(u[e]), c, u[e]);
}

template <int M>
__device__ __forceinline__ void lane_stage64_swap(double (&u)[8], int lane) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint64_t b = uint64_t(__double_as_longlong(u[e]));
    const Both lo = both<M>(uint32_t(b)), hi = both<M>(uint32_t(b >> 32));
    const double clear = __longlong_as_double((long long)((uint64_t(hi.clear) << 32) | lo.clear));
    const double set = __longlong_as_double((long long)((uint64_t(hi.set) << 32) | lo.set));
    u[e] = fma((lane & M) ? -1.0 : 1.0, set, clear);
  }
}

// The sum over lane bit M.
template <int M>
__device__ __forceinline__ double sum64_swap(double v) {
  const uint64_t b = uint64_t(__double_as_longlong(v));
  const Both lo = both<M>(uint32_t(b)), hi = both<M>(uint32_t(b >> 32));
  return __longlong_as_double((long long)((uint64_t(hi.clear) << 32) | lo.clear)) +
         __longlong_as_double((long long)((uint64_t(hi.set) << 32) | lo.set));
}

// |x| as an fp32 number on the same side of every number of few bits: where x lies
// between two fp32 numbers, the one whose last bit is 1.
__device__ __forceinline__ float to_odd(double x) {
  const float f = float(x);
  const double rest = x - double(f);
  const uint32_t bits = __float_as_uint(f);
  const uint32_t odd = bits + (rest > 0.0 ? 1u : rest < 0.0 ? ~0u : 0u);
  return __uint_as_float((bits & 1u) ? bits : odd);
}

// The wave's rows in fp64, in the lanes' order of the stages of encode (rarely called).
template <int BLOCK>
__device__ __forceinline__ MxWord encode64(const float (&v)[8], int lane) {
  const int l = lane & 15;
  double u[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) u[e] = v[e];
#pragma unroll
  for (int h = 1; h < 8; h <<= 1)
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if ((e & h) == 0) {
        const double a = u[e], b = u[e | h];
        u[e] = a + b;
        u[e | h] = a - b;
      }
  lane_stage64<0xB1>(u, __builtin_popcount(l & 5) & 1);   // lane ^ 1
  lane_stage64<0x4E>(u, __builtin_popcount(l & 6) & 1);   // lane ^ 2
  lane_stage64<0x141>(u, (l & 4) != 0);                   // lane ^ 7
  lane_stage64<0x128>(u, (l & 8) != 0);                   // lane ^ 8
  if constexpr (BLOCK >= 256) lane_stage64_swap<16>(u, lane);
  if constexpr (BLOCK >= 512) lane_stage64_swap<32>(u, lane);
  const double c = kPost64<BLOCK> * double(parity_sign(l));
  double most = 0.0;
  bool finite = true;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    u[e] *= c;
    finite = finite && fabs(u[e]) < __builtin_huge_val();
    most = fmax(most, fabs(u[e]));
  }
  // over the lanes of the block (as block_max): the upper half of a number that is not finite above all others
  uint32_t top = finite ? uint32_t(uint64_t(__double_as_longlong(most)) >> 32) : 0x7FF00000u;
  top = block_max<BLOCK>(top);
  finite = top < 0x7FF00000u;
  int E = int(top >> 20) - 1023 - 2;  // a zero or a subnormal lies below -127
  E = E < -127 ? -127 : E > 127 ? 127 : E;
  const double inv = __longlong_as_double((long long)(1023 - E) << 52);
  float f[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float a = finite ? to_odd(fabs(u[e]) * inv) : 0.0f;
    f[e] = finite && u[e] < 0.0 ? -a : a;
  }
  return MxWord{fp4_word(f), gather_scales<BLOCK>(finite ? uint32_t(E + 127) : 255u, l), h128_lane_word(l)};
}

// The codes of y + d (w) and y - d (other) differ here and there: those values again,
// one of each Hadamard block at a time.  Every lane adds its part of the output in fp64:
// output (o, e) of a lane and an element takes x of (m, j) with the sign
// (-1)^(|o & m| + |e & j|).  A few of a wave's values cost less this way than its rows
// (a quarter of the instructions, which the wave also has to fetch): 2048 x 4096 bf16
// 7.0 us, 7.8 with encode64 for all of them, 6.1 without either.
template <int BLOCK>
__device__ __forceinline__ uint32_t settle(const float (&x)[8], uint32_t w, uint32_t other, float inv, int lane) {
  constexpr int kLanes = BLOCK / 8;
  constexpr uint64_t kBits = ~uint64_t(0) >> (64 - kLanes);
  const int base = lane & (64 - kLanes), m = lane & (kLanes - 1);
  uint32_t open = w ^ other;
  for (uint64_t lanes = __builtin_amdgcn_ballot_w64(open != 0); lanes != 0;
       lanes = __builtin_amdgcn_ballot_w64(open != 0)) {
    const uint64_t mine = (lanes >> base) & kBits;  // none in the lane's block: its first value, not stored
    const int from = base + (mine != 0 ? __builtin_ctzll(mine) : 0);
    const uint32_t its = uint32_t(__builtin_amdgcn_ds_bpermute(4 * from, int(open)));
    const int e = its != 0 ? __builtin_ctz(its) >> 2 : 0;
    const int o = h128_lane_word(from & 15) | (from & (kLanes - 1) & ~15);
    const uint32_t signs = ((e & 1) ? 0xAAu : 0u) ^ ((e & 2) ? 0xCCu : 0u) ^ ((e & 4) ? 0xF0u : 0u) ^
                           ((__builtin_popcount(o & m) & 1) ? 0xFFu : 0u);
    double u = 0.0;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      u += double(__uint_as_float(__float_as_uint(x[j]) ^ ((signs << (31 - j)) & 0x80000000u)));
    u += dpp64<0xB1>(u);
    u += dpp64<0x4E>(u);
    u += dpp64<0x141>(u);
    u += dpp64<0x128>(u);
    if constexpr (BLOCK >= 256) u = sum64_swap<16>(u);
    if constexpr (BLOCK >= 512) u = sum64_swap<32>(u);
    u *= kPost64<BLOCK>;
    const float a = to_odd(fabs(u) * double(inv)), f = u < 0.0 ? -a : a;
    const uint32_t code = uint32_t(__builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0, f, f, 1.0f, 0)) & 15u;
    if (its != 0 && lane == from) {
      w = (w & ~(15u << (4 * e))) | code << (4 * e);
      open &= ~(15u << (4 * e));
    }
  }
  return w;
}

// The lane's 8 channels of a row (16 lanes hold 128, the wave 512), encoded.
// Every lane of the wave takes part.
template <int BLOCK>
__device__ __forceinline__ MxWord encode(const float (&x)[8], int lane) {
  float v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = x[e];
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
      for (int e = 0; e < 8; ++e) v[e] = lane_stage_swap<16>(v[e], lane);
    }
    if constexpr (BLOCK >= 512) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = lane_stage_swap<32>(v[e], lane);
    }
    float most8 = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) most8 = fmaxf(most8, fabsf(v[e]));  // NaN is seen in S
    const uint32_t top = block_max<BLOCK>(__float_as_uint(most8));
    const float err = S * (kPost32<BLOCK> * (n + 0.125f) * 0x1p-24f), most_err = S * (kPost32<BLOCK> * (n + 3) * 0x1p-24f);
    const float most = __uint_as_float(top) * kPost32<BLOCK>;
    const uint32_t at = __float_as_uint(most + most_err) >> 23;
    const int E = max(int(at) - 127 - 2, -127);
    const float inv = two_to(-E), d = fmaf(err, inv, 0x1p-20f);
    const float c = kPost32<BLOCK> * parity_sign(l) * inv;
    float lo[8], hi[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      lo[e] = fmaf(v[e], c, -d);
      hi[e] = fmaf(v[e], c, d);
    }
    uint32_t w = fp4_word(hi);  // zeros: of d, 0
    const uint32_t other = S != 0.0f ? fp4_word(lo) : w;
    // Sums beyond 2^100 (and what is not finite) could leave fp32; below 2^-90 the
    // products above could lose bits; without any value all is zero.
    const bool known = (at == __float_as_uint(most - most_err) >> 23 && S < 0x1p100f && S > 0x1p-90f) || S == 0.0f;
    const uint64_t open = __builtin_amdgcn_ballot_w64(w != other || !known);
    if (open != 0) {
      if (__builtin_popcountll(open) > 4 || __builtin_amdgcn_ballot_w64(!known) != 0) return encode64<BLOCK>(x, lane);
      w = settle<BLOCK>(x, w, other, inv, lane);
    }
    return MxWord{w, gather_scales<BLOCK>(uint32_t(E + 127), l), h128_lane_word(l)};
  }
}

// ---------------------------------------------------------------------------
// Rows with unit stride: a wave keeps one span of 512 channels and walks rows, the
// waves of a block side by side along a row.  The next row's values are on their way
// while the current ones are computed.  QUAD: 4 consecutive rows at a time, whose
// scales go out together, 16 bytes a group (where there are rows enough for every
// wave: at 4096 x 14336 single words took 5 us more); the last ones singly.
//   Lanes behind the last channel load zeros and store out of range, where the hardware
// drops it: a branch around a store would make the compiler wait for everything in
// flight, the next row's values among it.  Rows are at most 2^28, so the offsets of
// four groups' scales stay in 32 bits.
//   Bound by the vector units, some 18 instructions a channel, and memory: 4096 x 14336
// bf16, block 128, 32 us (149 MB at 4.7 TB/s, where a copy reaches 4.9; with the 4 rows as a
// loop, whose waits count less exactly, 34).  1333 x 8192 fp32, block 256, signs, 12 us
// (49 MB at 4.2 TB/s: two to three rows a wave, whose first loads nothing covers).  4096 x
// 8192 bf16 from memory 18.5 us without a transform, 20.9, 23.4 and 26.6 with blocks of
// 128, 256 and 512 (30.4 with signs), fp32 31 to 33 with any.
// ---------------------------------------------------------------------------
template <bool BF16, int BLOCK, bool SIGNED, bool QUAD>
__global__ __launch_bounds__(256) void mx_quantize_kernel(MxRows a, uint32_t spans, uint32_t walkers) {
  typedef unsigned int v4u __attribute__((ext_vector_type(4)));
  constexpr int kSize = BF16 ? 2 : 4, kLoads = BF16 ? 1 : 2, kRows = QUAD ? 4 : 1;
  const int lane = threadIdx.x & 63, g = lane >> 4;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + (threadIdx.x >> 6));
  const int64_t k0 = int64_t(wave % spans) * kSpan;
  const int rows = int(a.rows), stride = int(walkers) * kRows;
  int row = int(wave / spans) * kRows;
  if (wave / spans >= walkers || row >= rows) return;
  const int channels = int(a.K - k0 < kSpan ? a.K - k0 : kSpan);
  const char* const x = reinterpret_cast<const char*>(a.x) + k0 * kSize;
  struct Raw {
    v4u v[kLoads];
  };
  auto load = [&](int r) {
    const __amdgpu_buffer_rsrc_t from = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<char*>(x + r * a.stride_row * kSize), 0, channels * kSize, 0x00020000);
    Raw raw;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) raw.v[i] = __builtin_amdgcn_raw_buffer_load_b128(from, lane * (8 * kSize) + 16 * i, 0, 0);
    return raw;
  };
  uint32_t sign[8] = {};
  if constexpr (SIGNED) {
    const __amdgpu_buffer_rsrc_t from =
        __builtin_amdgcn_make_buffer_rsrc(const_cast<uint32_t*>(a.sign_mask + k0), 0, channels * 4, 0x00020000);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const v4u m = __builtin_amdgcn_raw_buffer_load_b128(from, lane * 32 + 16 * i, 0, 0);
#pragma unroll
      for (int e = 0; e < 4; ++e) sign[4 * i + e] = m[e];
    }
  }
  const uint32_t group = uint32_t(a.rows) * 4;  // bytes from one group's scales to the next
  const uint32_t scale_range = group * ((channels >> 7) - 1);  // in front of the last group's
  // -16: beyond every range, and the 16 bytes from there do not pass the end of 32 bits
  const int scale_at = (lane & 15) == 0 && 128 * g < channels ? int(g * group) : -16;
  auto encode_row = [&](const Raw& raw, int r) {  // stores its codes; its scales
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if constexpr (BF16) v[e] = (e & 1) ? bf16_hi(raw.v[0][e >> 1]) : bf16_lo(raw.v[0][e >> 1]);
      else v[e] = __uint_as_float(raw.v[(e >> 2) % kLoads][e & 3]);
      if constexpr (SIGNED) v[e] = __uint_as_float(__float_as_uint(v[e]) ^ sign[e]);
    }
    const MxWord w = encode<BLOCK>(v, lane);
    __builtin_amdgcn_raw_buffer_store_b32(
        w.codes, __builtin_amdgcn_make_buffer_rsrc(a.q + r * (a.K >> 1) + (k0 >> 1), 0, channels >> 1, 0x00020000),
        64 * g + 4 * w.word, 0, 0);
    return w.scales;
  };
  auto scales_of = [&](int r) { return a.s + ((k0 >> 7) * a.rows + r) * 4; };
  Raw next = load(row);
  if constexpr (QUAD) {
    for (; row + 4 <= rows; row += stride) {
      v4u scales;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const Raw raw = next;
        const int r2 = i < 3 ? row + i + 1 : row + stride;
        next = load(r2 < rows ? r2 : row);
        scales[i] = encode_row(raw, row + i);
      }
      __builtin_amdgcn_raw_buffer_store_b128(
          scales, __builtin_amdgcn_make_buffer_rsrc(scales_of(row), 0, int(scale_range + 16), 0x00020000), scale_at, 0, 0);
    }
  }
  for (; row < rows; row += QUAD ? 1 : stride) {  // QUAD: the last rows, fewer than 4
    const Raw raw = next;
    const int r2 = row + (QUAD ? 1 : stride);
    next = load(r2 < rows ? r2 : row);
    const uint32_t scales = encode_row(raw, row);
    __builtin_amdgcn_raw_buffer_store_b32(
        scales, __builtin_amdgcn_make_buffer_rsrc(scales_of(row), 0, int(scale_range + 4), 0x00020000), scale_at, 0, 0);
  }
}

// ---------------------------------------------------------------------------
// Rows of any strides (weights [K, N]): a block brings some rows of one Hadamard block
// (128 channels at least) into LDS, then encodes them from there, 16 lanes or more a
// row.  VECTOR: rows lie side by side (stride_row 1) and 16-byte loads fit; otherwise
// single values, the lanes along whichever stride is the smaller.  Channel k of a row
// lies at k + k / 8, so that lanes reading every ninth word hit all banks; rows are an
// odd number of words apart for the writes.
//   Bound by memory: 4096 x 4096 fp32 as [K, N], block 128, 18 us (76 MB at 4.2 TB/s,
// vector units 73 % busy); 4 blocks a CU, of which some load while others encode.  Single
// values wait for their loads: from memory 4096 x 4097 bf16 19.8 us where 16-byte loads of
// 4096 x 4096 take 13.7, [N, K] of an odd pitch 20.1, every second channel 26.9 (fp32 45).
// ---------------------------------------------------------------------------
template <int BLOCK>
struct Pack {
  static constexpr int span = mx_pack_span(BLOCK), rows = mx_pack_rows(BLOCK);
  static constexpr int row = span + span / 8 + 1, lanes = span / 8;
};

template <bool BF16, int BLOCK, bool SIGNED, bool VECTOR>
__global__ __launch_bounds__(256) void mx_pack_kernel(MxRows a, int64_t spans) {
  using P = Pack<BLOCK>;
  __shared__ float tile[P::rows * P::row];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t row0 = (blockIdx.x / spans) * P::rows, k0 = (blockIdx.x % spans) * P::span;  // spans are whole
  const int rows = int(a.rows - row0 < P::rows ? a.rows - row0 : P::rows);
  auto put = [&](int r, int k, float v) {
    if constexpr (SIGNED) v = __uint_as_float(__float_as_uint(v) ^ a.sign_mask[k0 + k]);
    tile[r * P::row + k + (k >> 3)] = v;
  };
  if constexpr (VECTOR) {
    constexpr int E = BF16 ? 8 : 4, kAcross = P::rows / E, kPasses = P::span * kAcross / 256;
    const int r = (tid % kAcross) * E;
    const char* from = reinterpret_cast<const char*>(a.x) + (row0 + (r < rows ? r : 0)) * (BF16 ? 2 : 4);
#pragma unroll
    for (int i0 = 0; i0 < kPasses; i0 += 8) {
      uint4 w[8];
#pragma unroll
      for (int i = 0; i < 8 && i0 + i < kPasses; ++i) {
        const int k = (i0 + i) * (256 / kAcross) + tid / kAcross;
        w[i] = *reinterpret_cast<const uint4*>(from + (k0 + k) * a.stride_k * (BF16 ? 2 : 4));  // rows is a multiple of E
      }
#pragma unroll
      for (int i = 0; i < 8 && i0 + i < kPasses; ++i) {
        const int k = (i0 + i) * (256 / kAcross) + tid / kAcross;
        const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
        for (int e = 0; e < E; ++e)
          put(r + e, k, BF16 ? ((e & 1) ? bf16_hi(u[e >> 1]) : bf16_lo(u[e >> 1])) : __uint_as_float(u[e & 3]));
      }
    }
  } else {
    const bool along_rows = a.stride_row <= a.stride_k;
    const StridedSrc<BF16> src{a.x, a.stride_k, a.stride_row};
#pragma unroll 8
    for (int i = 0; i < P::rows * P::span / 256; ++i) {
      const int at = i * 256 + tid;
      const int r = along_rows ? at % P::rows : at / P::span, k = along_rows ? at / P::rows : at % P::span;
      put(r, k, src.at(row0 + (r < rows ? r : 0), k0 + k));
    }
  }
  __syncthreads();
  constexpr int kTogether = 64 / P::lanes;  // rows of a wave
  const int l = lane % P::lanes;
  for (int r0 = wave * kTogether; r0 < rows; r0 += 4 * kTogether) {
    const int r = r0 + lane / P::lanes;
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = tile[r * P::row + 9 * l + e];
    const MxWord w = encode<BLOCK>(v, lane);
    if (r < rows) {
      const int64_t g = (k0 >> 7) + (l >> 4);
      *reinterpret_cast<uint32_t*>(a.q + (row0 + r) * (a.K >> 1) + 64 * g + 4 * w.word) = w.codes;
      if ((lane & 15) == 0) *reinterpret_cast<uint32_t*>(a.s + (g * a.rows + row0 + r) * 4) = w.scales;
    }
  }
}

// ---------------------------------------------------------------------------
// Reading back: a wave keeps one span of 512 channels, 8 a lane, and walks rows, four at
// a time, the next four on their way.  Values below 2^128 are exact in bf16 and fp32, others infinite.  Lanes
// behind the last channel load zeros and store out of range, where it is dropped.
//   Bound by memory: 4096 x 14336 to bf16 24.5 us (149 MB at 6.1 TB/s).
// ---------------------------------------------------------------------------
constexpr int kBackRows = 4;
constexpr int kStream = 2;  // stores as non-temporal: 4096 x 14336 takes 24.7 us, 34.9 through the caches

template <bool BF16>
__global__ __launch_bounds__(256) void mx_dequantize_kernel(const uint8_t* __restrict__ q, const uint8_t* __restrict__ s,
                                                            int64_t M, int64_t K, void* __restrict__ out, int64_t ldo,
                                                            uint32_t spans, uint32_t walkers) {
  typedef float v2f __attribute__((ext_vector_type(2)));
  typedef unsigned int v4u __attribute__((ext_vector_type(4)));
  constexpr int kSize = BF16 ? 2 : 4;
  const int lane = threadIdx.x & 63;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + (threadIdx.x >> 6));
  const int64_t k0 = int64_t(wave % spans) * kSpan;
  int64_t row = int64_t(wave / spans) * kBackRows;
  if (wave / spans >= walkers) return;
  const int channels = int(K - k0 < kSpan ? K - k0 : kSpan);
  // the lane's scale byte in its group's words of the rows, rows at most 2^28
  const uint32_t group = uint32_t(M) * 4, at = uint32_t(lane >> 4) * group;
  const int shift = 8 * ((lane >> 2) & 3);
  struct Raw {
    uint32_t codes[kBackRows], scales[kBackRows];
  };
  auto load = [&](int64_t r, Raw& raw) {
#pragma unroll
    for (int i = 0; i < kBackRows; ++i) {
      const int64_t n = r + i < M ? r + i : M - 1;
      raw.codes[i] = __builtin_amdgcn_raw_buffer_load_b32(
          __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(q + n * (K >> 1) + (k0 >> 1)), 0, channels >> 1, 0x00020000),
          lane * 4, 0, 0);
      raw.scales[i] = __builtin_amdgcn_raw_buffer_load_b32(
          __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(s + ((k0 >> 7) * M + n) * 4), 0,
                                            int(group * ((channels >> 7) - 1) + 4), 0x00020000),
          int(at), 0, 0);
    }
  };
  Raw next;
  load(row, next);
  while (row < M) {
    const Raw raw = next;
    const int64_t row2 = row + int64_t(walkers) * kBackRows;
    load(row2 < M ? row2 : row, next);
#pragma unroll
    for (int i = 0; i < kBackRows; ++i) {
      const uint32_t w = raw.codes[i], e = (raw.scales[i] >> shift) & 255u;
      const v2f p[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0), __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1),
                        __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2), __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3)};
      uint32_t v[8];
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const float x = ldexpf(p[c >> 1][c & 1], int(e) - 127);
        v[c] = __float_as_uint(e == 255u ? __builtin_nanf("") : x);
      }
      // rows behind the last one: an empty range
      const int64_t n = row + i;
      const __amdgpu_buffer_rsrc_t to = __builtin_amdgcn_make_buffer_rsrc(
          reinterpret_cast<char*>(out) + (n < M ? n * ldo + k0 : 0) * kSize, 0, n < M ? channels * kSize : 0, 0x00020000);
      if constexpr (BF16) {
        v4u b;
#pragma unroll
        for (int c = 0; c < 4; ++c)  // exact: the lower halves are zero (NaN: its upper half is NaN)
          b[c] = (v[2 * c] >> 16) | (v[2 * c + 1] & 0xFFFF0000u);
        __builtin_amdgcn_raw_buffer_store_b128(b, to, lane * 16, 0, kStream);
      } else {
        __builtin_amdgcn_raw_buffer_store_b128(v4u{v[0], v[1], v[2], v[3]}, to, lane * 32, 0, kStream);
        __builtin_amdgcn_raw_buffer_store_b128(v4u{v[4], v[5], v[6], v[7]}, to, lane * 32 + 16, 0, kStream);
      }
    }
    row = row2;
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
  const int64_t spans = (a.K + kSpan - 1) / kSpan;  // at most 2^14
  const int64_t full = 256 * 32;                    // waves the card holds
  const bool quad = a.rows * spans >= 4 * full;
  const int64_t most = quad ? (a.rows + 3) / 4 : a.rows;
  int64_t walkers = full / spans > 1 ? full / spans : 1;
  walkers = walkers < most ? walkers : most;
  const dim3 grid{unsigned((spans * walkers + 3) / 4)};
  return by_kind(a, [&](auto bf16, auto block, auto sign) {
    constexpr bool B = decltype(bf16)::value, S = decltype(sign)::value;
    constexpr int L = decltype(block)::value;
    if (quad)
      hipLaunchKernelGGL((mx_quantize_kernel<B, L, S, true>), grid, dim3(256), 0, st, a, uint32_t(spans), uint32_t(walkers));
    else
      hipLaunchKernelGGL((mx_quantize_kernel<B, L, S, false>), grid, dim3(256), 0, st, a, uint32_t(spans), uint32_t(walkers));
    return hipGetLastError();
  });
}

hipError_t launch_mx_pack(const MxRows& a, hipStream_t st) {
  const int64_t size = a.bf16 ? 2 : 4;
  const bool vector = a.stride_row == 1 && (a.stride_k * size) % 16 == 0 && (a.rows * size) % 16 == 0 &&
                      (reinterpret_cast<uintptr_t>(a.x) & 15) == 0;
  return by_kind(a, [&](auto bf16, auto block, auto sign) {
    using P = Pack<decltype(block)::value>;
    const int64_t spans = a.K / P::span, blocks = mx_pack_blocks(a.rows, a.K, a.block);
    if (vector)
      hipLaunchKernelGGL((mx_pack_kernel<decltype(bf16)::value, decltype(block)::value, decltype(sign)::value, true>),
                         dim3(unsigned(blocks)), dim3(256), 0, st, a, spans);
    else
      hipLaunchKernelGGL((mx_pack_kernel<decltype(bf16)::value, decltype(block)::value, decltype(sign)::value, false>),
                         dim3(unsigned(blocks)), dim3(256), 0, st, a, spans);
    return hipGetLastError();
  });
}

hipError_t launch_mx_dequantize(const uint8_t* q, const uint8_t* s, int64_t M, int64_t K, void* out, bool out_bf16,
                                int64_t ldo, hipStream_t st) {
  const int64_t spans = (K + kSpan - 1) / kSpan, most = (M + kBackRows - 1) / kBackRows;
  int64_t walkers = 256 * 32 / spans > 1 ? 256 * 32 / spans : 1;  // as many waves as the card holds
  walkers = walkers < most ? walkers : most;
  const dim3 grid{unsigned((spans * walkers + 3) / 4)};
  if (out_bf16)
    hipLaunchKernelGGL((mx_dequantize_kernel<true>), grid, dim3(256), 0, st, q, s, M, K, out, ldo, uint32_t(spans),
                       uint32_t(walkers));
  else
    hipLaunchKernelGGL((mx_dequantize_kernel<false>), grid, dim3(256), 0, st, q, s, M, K, out, ldo, uint32_t(spans),
                       uint32_t(walkers));
  return hipGetLastError();
}

}  // namespace rw4
