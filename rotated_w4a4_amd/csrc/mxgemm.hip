// MXFP4 GEMM on the gfx950 matrix cores.
//
//   Y[m, n] = sum over blocks b of 32 channels of
//             2^(ea[m, b] + ew[n, b]) sum over k in b of a[m, k] w[n, k]
//
// with FP4 E2M1 codes and E8M0 scales on both sides, which the scaled MFMA takes as
// they are stored: a lane supplies 32 codes (16 bytes) of one row, which are one
// block, and that block's scale byte.  Sums are fp32.  A scale of 255 makes its
// products NaN.
//
// Operand layout: for 32 x 32 x 64, lane l supplies row l % 32, channels 32 (l / 32)
// .. + 32; for 16 x 16 x 128, row l % 16, channels 32 (l / 16) .. + 32.  The weights
// are the row operand and the tokens the column operand, so that a lane ends with
// one token and 4 consecutive channels at a time: D[8 (r / 4) + 4 (l / 32) + r % 4]
// [l % 32], r = 0..15, and D[4 (l / 16) + r][l % 16], r = 0..3.
#include <type_traits>

#include "mx_internal.h"
#include "rw4_device.h"

namespace rw4 {

namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef unsigned int v4u __attribute__((ext_vector_type(4)));
typedef unsigned int v2u __attribute__((ext_vector_type(2)));
typedef __bf16 v4bf __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void lds_void_t;

constexpr int kFp4 = 4;  // MFMA operand format FP4 E2M1

__device__ __forceinline__ v8i fp4_operand(const v4u& c) {
  return v8i{int(c[0]), int(c[1]), int(c[2]), int(c[3]), 0, 0, 0, 0};  // FP4 reads four registers
}

// A block's place among the tiles: blocks go round-robin over the 8 XCDs, so each XCD
// gets one contiguous range of tiles, walked in bands of 8 tile rows, column by
// column: the tiles resident on one XCD share their rows and columns in its L2.
__device__ __forceinline__ void mx_tile(int64_t b, int64_t blocks, int64_t tiles_m, int64_t& mt, int64_t& nt) {
  const int64_t x = b & 7, i = b >> 3, q = blocks >> 3, r = blocks & 7;
  const int64_t l = x * q + (x < r ? x : r) + i;
  const int64_t tiles_n = blocks / tiles_m;
  constexpr int64_t kBand = 8;
  const int64_t band = l / (kBand * tiles_n), first = band * kBand;
  const int64_t in_band = tiles_m - first < kBand ? tiles_m - first : kBand;
  const int64_t li = l - first * tiles_n;
  mt = first + li % in_band;
  nt = li / in_band;
}

template <bool BF16>
__device__ __forceinline__ void store_one(void* y, int64_t at, float v) {
  if constexpr (BF16) reinterpret_cast<__bf16*>(y)[at] = static_cast<__bf16>(v);  // round to nearest even
  else reinterpret_cast<float*>(y)[at] = v;
}

// ---------------------------------------------------------------------------
// Many rows: BM tokens x BN channels a block, WM x WN waves.  K goes in stages of
// 256 channels, which the DMA brings from memory into one of two LDS buffers while
// the other is computed on (one barrier a stage).  A row of a stage is 128 bytes,
// eight 16-byte chunks, chunk c at place c ^ (row & 7), so that 8 lanes reading one
// chunk of 8 rows hit all banks; the DMA writes LDS in lane order, so the exchange is
// in the addresses it reads from.  The scales of a stage go straight into registers
// (4 bytes for 128 channels of a row, rows side by side), a stage ahead.
// ---------------------------------------------------------------------------
constexpr int kStageK = 256, kStageRow = kStageK / 2;

template <int BM, int BN, int WM, int WN>
struct Tile {
  static constexpr int waves = WM * WN, threads = 64 * waves;
  static constexpr int TM = BM / WM / 32, TN = BN / WN / 32;  // 32 x 32 tiles of a wave
  static constexpr int bytes = (BM + BN) * kStageRow;
  static constexpr int loads = (BM + BN) / 8 / waves;  // DMA instructions of a wave, 8 rows each
  static_assert((BM + BN) % (8 * waves) == 0 && BM % (8 * waves) == 0, "whole DMA instructions of one operand");
};

template <int BM, int BN, int WM, int WN, bool BF16>
__global__ __launch_bounds__(64 * WM * WN) void mx_gemm_kernel(
    const uint8_t* __restrict__ qa, const uint32_t* __restrict__ sa, const uint8_t* __restrict__ qw,
    const uint32_t* __restrict__ sw, int64_t M, int64_t N, int64_t K, void* __restrict__ y, int64_t ldy,
    int64_t tiles_m) {
  using T = Tile<BM, BN, WM, WN>;
  constexpr int TM = T::TM, TN = T::TN;
  // two objects: the compiler sees that the DMA into one never writes what is read from the other
  __shared__ __align__(16) uint8_t buf0[T::bytes];
  __shared__ __align__(16) uint8_t buf1[T::bytes];

  const int tid = threadIdx.x, lane = tid & 63, n = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  int64_t mt, nt;
  mx_tile(blockIdx.x, gridDim.x, tiles_m, mt, nt);
  const int64_t m0 = mt * BM, n0 = nt * BN, row_bytes = K / 2, G = K / kGroup;
  const int rows_a = int(M - m0 < BM ? M - m0 : BM), rows_w = int(N - n0 < BN ? N - n0 : BN);

  // rows beyond the last one read that again; what they give is not stored
  const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(qa + m0 * row_bytes), 0,
                                                                      int(rows_a * row_bytes), 0x00020000);
  const __amdgpu_buffer_rsrc_t rw = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(qw + n0 * row_bytes), 0,
                                                                      int(rows_w * row_bytes), 0x00020000);
  constexpr int LA = BM / 8 / T::waves, LW = T::loads - LA;
  uint32_t from_a[LA], from_w[LW];
  const int sub = lane >> 3, chunk = ((lane & 7) ^ sub) * 16;
#pragma unroll
  for (int i = 0; i < LA; ++i) {
    const int r = (wave * LA + i) * 8 + sub;
    from_a[i] = uint32_t((r < rows_a ? r : rows_a - 1) * row_bytes + chunk);
  }
#pragma unroll
  for (int i = 0; i < LW; ++i) {
    const int r = (wave * LW + i) * 8 + sub;
    from_w[i] = uint32_t((r < rows_w ? r : rows_w - 1) * row_bytes + chunk);
  }
  auto bring = [&](uint8_t* to, int64_t stage) {  // behind the last channel: other rows' codes or zeros, not used
    const int at = int(stage * kStageRow);
#pragma unroll
    for (int i = 0; i < LA; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void_t*)(to + (wave * LA + i) * 1024), 16, int(from_a[i]), at, 0, 0);
#pragma unroll
    for (int i = 0; i < LW; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_void_t*)(to + BM * kStageRow + (wave * LW + i) * 1024), 16,
                                               int(from_w[i]), at, 0, 0);
  };

  // scales: word g of a row holds the bytes of its channels 128 g ..; shifted so that
  // byte 0 and byte 2 are the lane half's blocks of the two products of 64 channels
  int row_a[TM], row_w[TN];
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int r = (wm * TM + i) * 32 + n;
    row_a[i] = r < rows_a ? r : rows_a - 1;
  }
#pragma unroll
  for (int i = 0; i < TN; ++i) {
    const int r = (wn * TN + i) * 32 + n;
    row_w[i] = r < rows_w ? r : rows_w - 1;
  }
  struct Scales {
    uint32_t a[2][TM], w[2][TN];
  };
  auto load_scales = [&](int64_t stage, Scales& to) {
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const int64_t g = 2 * stage + p < G ? 2 * stage + p : G - 1;
      const uint32_t* pa = sa + g * M + m0;
      const uint32_t* pw = sw + g * N + n0;
#pragma unroll
      for (int i = 0; i < TM; ++i) to.a[p][i] = pa[row_a[i]];
#pragma unroll
      for (int i = 0; i < TN; ++i) to.w[p][i] = pw[row_w[i]];
    }
  };

  v16f acc[TN][TM];
#pragma unroll
  for (int i = 0; i < TN; ++i)
#pragma unroll
    for (int j = 0; j < TM; ++j) acc[i][j] = v16f{};

  int off[4];  // of the lane's chunk of each product in a tile of 32 rows
#pragma unroll
  for (int k = 0; k < 4; ++k) off[k] = n * kStageRow + (((2 * k + h) ^ (n & 7)) * 16);
  const int base_a = wm * TM * 32 * kStageRow, base_w = (BM + wn * TN * 32) * kStageRow;

  struct Operands {
    v4u a[TM], w[TN];
  };
  auto read = [&](const uint8_t* from, int k, Operands& to) {
#pragma unroll
    for (int i = 0; i < TN; ++i) to.w[i] = *reinterpret_cast<const v4u*>(from + base_w + off[k] + i * 32 * kStageRow);
#pragma unroll
    for (int i = 0; i < TM; ++i) to.a[i] = *reinterpret_cast<const v4u*>(from + base_a + off[k] + i * 32 * kStageRow);
  };
  auto multiply = [&](const Operands& o, const uint32_t (&xa)[TM], const uint32_t (&xw)[TN], auto second) {
    constexpr int kByte = decltype(second)::value ? 2 : 0;
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
      for (int j = 0; j < TM; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fp4_operand(o.w[i]), fp4_operand(o.a[j]), acc[i][j],
                                                                    kFp4, kFp4, kByte, int(xw[i]), kByte, int(xa[j]));
  };

  Scales next;
  const int64_t stages = (G + 1) / 2;
  bring(buf0, 0);
  load_scales(0, next);
  auto stage = [&](const uint8_t* from, uint8_t* to, int64_t s) {
    __syncthreads();  // this stage has arrived, the other buffer is read
    Scales x;
#pragma unroll
    for (int p = 0; p < 2; ++p) {
#pragma unroll
      for (int i = 0; i < TM; ++i) x.a[p][i] = next.a[p][i] >> (8 * h);
#pragma unroll
      for (int i = 0; i < TN; ++i) x.w[p][i] = next.w[p][i] >> (8 * h);
    }
    if (s + 1 < stages) {
      bring(to, s + 1);
      load_scales(s + 1, next);
    }
    Operands o[2];
    read(from, 0, o[0]);
    read(from, 1, o[1]);
    multiply(o[0], x.a[0], x.w[0], std::false_type{});
    const bool two = 2 * s + 1 < G;
    if (two) read(from, 2, o[0]);
    multiply(o[1], x.a[0], x.w[0], std::true_type{});
    if (two) {
      read(from, 3, o[1]);
      multiply(o[0], x.a[1], x.w[1], std::false_type{});
      multiply(o[1], x.a[1], x.w[1], std::true_type{});
    }
  };
  for (int64_t s = 0; s < stages; s += 2) {
    stage(buf0, buf1, s);
    if (s + 1 < stages) stage(buf1, buf0, s + 1);
  }
  __syncthreads();

  // Output: 32 tokens at a time through the wave's own part of LDS into rows of 16-byte chunks.
  constexpr int E = BF16 ? 2 : 4, kCols = TN * 32, kOut = kCols * E + 16, kChunks = kCols * E / 16;
  constexpr int kWaveBytes = 32 * kOut;
  static_assert((T::waves / 2) * kWaveBytes <= T::bytes, "output rows of half of the waves in each buffer");
  uint8_t* out = (wave < T::waves / 2 ? buf0 : buf1) + (wave % (T::waves / 2)) * kWaveBytes;
  const bool aligned = (ldy * E) % 16 == 0 && (reinterpret_cast<uintptr_t>(y) & 15) == 0;
  const int64_t c0 = n0 + wn * kCols;
#pragma unroll
  for (int j = 0; j < TM; ++j) {
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const v4f v{acc[i][j][4 * b], acc[i][j][4 * b + 1], acc[i][j][4 * b + 2], acc[i][j][4 * b + 3]};
        uint8_t* dst = out + n * kOut + (i * 32 + 8 * b + 4 * h) * E;
        if constexpr (BF16) {
          v4bf p;
#pragma unroll
          for (int e = 0; e < 4; ++e) p[e] = static_cast<__bf16>(v[e]);  // round to nearest even
          *reinterpret_cast<v4bf*>(dst) = p;
        } else {
          *reinterpret_cast<v4f*>(dst) = v;
        }
      }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int it = 0; it < 32 * kChunks / 64; ++it) {
      const int idx = it * 64 + lane, r = idx / kChunks, c = idx % kChunks;
      const int64_t m = m0 + (wm * TM + j) * 32 + r, col = c0 + c * (16 / E);
      const v4u v = *reinterpret_cast<const v4u*>(out + r * kOut + c * 16);
      if (m < M && col < N) {
        if (aligned && col + 16 / E <= N) {
          *reinterpret_cast<v4u*>(reinterpret_cast<uint8_t*>(y) + (m * ldy + col) * E) = v;
        } else {
#pragma unroll
          for (int e = 0; e < 16 / E; ++e)
            if (col + e < N) {
              if constexpr (BF16) reinterpret_cast<uint16_t*>(y)[m * ldy + col + e] = uint16_t(v[e / 2] >> (16 * (e & 1)));
              else reinterpret_cast<uint32_t*>(y)[m * ldy + col + e] = v[e];
            }
        }
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

// ---------------------------------------------------------------------------
// Few rows: a block takes 16 channels and up to 16 MT tokens (grid y: chunks of
// them), its 8 waves split K in slices of 128 channels, two consecutive ones at a
// time, so that a wave reads whole 128-byte lines of the weights.  Weights go
// straight to registers, the next slices are loaded before the current ones are
// multiplied, the waves' sums meet in LDS.
// ---------------------------------------------------------------------------
constexpr int kFewWaves = 8, kFewPair = 2;

template <int MT, bool BF16>
__global__ __launch_bounds__(64 * kFewWaves) void mx_gemm_few_kernel(
    const uint8_t* __restrict__ qa, const uint32_t* __restrict__ sa, const uint8_t* __restrict__ qw,
    const uint32_t* __restrict__ sw, int64_t M, int64_t N, int64_t K, void* __restrict__ y, int64_t ldy) {
  __shared__ __align__(16) float sums[kFewWaves][MT * 16][20];  // 16 channels of a token, +4: fewer bank conflicts
  const int tid = threadIdx.x, lane = tid & 63, n = lane & 15, g4 = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t n0 = int64_t(blockIdx.x) * 16, m0 = int64_t(blockIdx.y) * (16 * MT), row_bytes = K / 2;
  const int G = int(K / kGroup);
  const int64_t row_w = n0 + n < N ? n0 + n : N - 1;  // rows beyond the last one read that again
  const uint8_t* pw = qw + row_w * row_bytes + 16 * g4;
  int64_t row_a[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) row_a[i] = m0 + 16 * i + n < M ? m0 + 16 * i + n : M - 1;

  struct Slice {
    v4u w, a[MT];
    uint32_t xw, xa[MT];
  };
  auto load = [&](int g, Slice& s) {
    g = g < G ? g : G - 1;
    s.w = *reinterpret_cast<const v4u*>(pw + int64_t(g) * 64);
    s.xw = sw[g * N + row_w];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      s.a[i] = *reinterpret_cast<const v4u*>(qa + row_a[i] * row_bytes + int64_t(g) * 64 + 16 * g4);
      s.xa[i] = sa[g * M + row_a[i]];
    }
  };
  v4f acc[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) acc[i] = v4f{};
  constexpr int kStep = kFewWaves * kFewPair;
  Slice cur[kFewPair], next[kFewPair];
  int g = wave * kFewPair;
  if (g < G) {
#pragma unroll
    for (int p = 0; p < kFewPair; ++p) load(g + p, cur[p]);
  }
  for (; g < G; g += kStep) {
    if (g + kStep < G) {
#pragma unroll
      for (int p = 0; p < kFewPair; ++p) load(g + kStep + p, next[p]);
    }
#pragma unroll
    for (int p = 0; p < kFewPair; ++p) {
      if (g + p < G) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
          acc[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fp4_operand(cur[p].w), fp4_operand(cur[p].a[i]), acc[i],
                                                                    kFp4, kFp4, 0, int(cur[p].xw >> (8 * g4)), 0,
                                                                    int(cur[p].xa[i] >> (8 * g4)));
      }
    }
#pragma unroll
    for (int p = 0; p < kFewPair; ++p) cur[p] = next[p];
  }
#pragma unroll
  for (int i = 0; i < MT; ++i) *reinterpret_cast<v4f*>(&sums[wave][16 * i + n][4 * g4]) = acc[i];
  __syncthreads();
  for (int at = tid; at < MT * 256; at += 64 * kFewWaves) {
    const int t = at >> 4, c = at & 15;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kFewWaves; ++w) v += sums[w][t][c];
    if (m0 + t < M && n0 + c < N) store_one<BF16>(y, (m0 + t) * ldy + n0 + c, v);
  }
}

}  // namespace

hipError_t launch_mx_gemm(const uint8_t* qa, const uint8_t* sa, const uint8_t* qw, const uint8_t* sw, int64_t M,
                          int64_t N, int64_t K, void* y, bool y_bf16, int64_t ldy, hipStream_t st) {
  const uint32_t* xa = reinterpret_cast<const uint32_t*>(sa);
  const uint32_t* xw = reinterpret_cast<const uint32_t*>(sw);
  auto few = [&](auto mt) {
    constexpr int MT = decltype(mt)::value;
    const int64_t blocks = (N + 15) / 16, chunks = (M + 16 * MT - 1) / (16 * MT);
    if (blocks > (int64_t(1) << 22)) return hipErrorInvalidValue;
    const dim3 grid{unsigned(blocks), unsigned(chunks), 1u};
    if (y_bf16)
      hipLaunchKernelGGL((mx_gemm_few_kernel<MT, true>), grid, dim3(64 * kFewWaves), 0, st, qa, xa, qw, xw, M, N, K, y, ldy);
    else
      hipLaunchKernelGGL((mx_gemm_few_kernel<MT, false>), grid, dim3(64 * kFewWaves), 0, st, qa, xa, qw, xw, M, N, K, y, ldy);
    return hipGetLastError();
  };
  auto many = [&](auto bm, auto bn, auto wm, auto wn) {
    constexpr int BM = decltype(bm)::value, BN = decltype(bn)::value, WM = decltype(wm)::value, WN = decltype(wn)::value;
    const int64_t tiles_m = (M + BM - 1) / BM, blocks = tiles_m * ((N + BN - 1) / BN);
    if (blocks > (int64_t(1) << 22)) return hipErrorInvalidValue;
    const dim3 grid{unsigned(blocks)}, threads{64 * WM * WN};
    if (y_bf16)
      hipLaunchKernelGGL((mx_gemm_kernel<BM, BN, WM, WN, true>), grid, threads, 0, st, qa, xa, qw, xw, M, N, K, y, ldy,
                         tiles_m);
    else
      hipLaunchKernelGGL((mx_gemm_kernel<BM, BN, WM, WN, false>), grid, threads, 0, st, qa, xa, qw, xw, M, N, K, y, ldy,
                         tiles_m);
    return hipGetLastError();
  };
  using std::integral_constant;
  if (M <= 16) return few(integral_constant<int, 1>{});
  if (M <= 64) return few(integral_constant<int, 4>{});
  const integral_constant<int, 128> k128{};
  const integral_constant<int, 2> k2{};
  return many(k128, k128, k2, k2);
}

}  // namespace rw4
