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
// Every kernel uses v_mfma_scale_f32_16x16x128_f8f6f4: lane l supplies row l % 16,
// channels 32 (l / 16) .. + 32.  (With random codes, where the card's power limits the
// matrix units, it reaches 6.85 PFLOP/s in a loop of nothing else; 32 x 32 x 64, which
// reads and writes twice the accumulators for each product, 5.4-6.15; on zeros both
// 9.4.)  The weights are the row operand and the tokens the column operand, so that a
// lane ends with one token and 4 consecutive channels: D[4 (l / 16) + r][l % 16].
#include <type_traits>

#include "mx_index.h"
#include "mx_internal.h"
#include "rw4_device.h"

namespace rw4 {

namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef unsigned int v4u __attribute__((ext_vector_type(4)));
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
// Many rows: BM tokens x BN channels a block, WM x WN waves of TM x TN tiles of 16 x 16.
// K goes in stages of 256 channels (whole 128-byte lines of the rows) through a ring of
// LDS buffers that the DMA fills (RING more than 2 where the tiles are small and a
// stage's products take less than the memory's latency).  A stage is two steps of 128
// channels; the operands of a step are read from LDS during the products of the step
// before, also across stages.  So the reads of a buffer are over when its stage's second
// step begins: there the wait for the next stage's arrival, the barrier, and the start
// of the DMA into the buffer just read, which has RING - 1 stages' time to arrive.
//   Operands: a second set of registers takes the next step's where there is room
// (TWICE); the 256 x 256 tile reads each one into the registers of the same one as soon
// as its last product of the step is issued.
//   A row of a stage is eight 16-byte chunks, chunk c at place c ^ (row & 7), so that 8
// lanes reading one chunk of 8 rows hit all banks; the DMA writes LDS in lane order,
// so the exchange is in the addresses it reads from.
//   Bound, operands in the cache.  256 x 256: matrix units 60 % of a CU's busy cycles at
// 4096 x 4096, K = 14336, 104 us (4.6 PFLOP/s; the products alone 89 us, where power limits
// them, the loads alone 66).  128 x 128: the loads through L2 (55 to 65 GB/s a CU, some
// 64 KB of them in flight: a microsecond's latency under load) and LDS beside the
// products, 2048 x 4096, K = 4096, 21.4 us (3.2 PFLOP/s, 4.9 of it launch, first loads and
// output).  64 x 64: the loads' latency, 61 x 11008, K = 4096, 7.2 us (25 MB at 3.5 TB/s).
// ---------------------------------------------------------------------------
constexpr int kStageRow = kGroup;  // bytes of 256 channels

template <int BM, int BN, int WM, int WN>
struct Tile {
  static constexpr int waves = WM * WN, threads = 64 * waves;
  static constexpr int TM = BM / WM / 16, TN = BN / WN / 16;  // 16 x 16 tiles of a wave
  static constexpr bool twice = TM * TN <= 16;               // two sets of operands
  // a stage in LDS: codes, then the scale words of its two groups of 128 channels
  static constexpr int codes = (BM + BN) * kStageRow, words = (BM + BN) * 4, bytes = codes + 2 * words;
  // DMA instructions of a wave for a stage: 8 rows' codes, and 64 rows' words of a group each
  static constexpr int LA = BM / 8 / waves, LW = BN / 8 / waves, pieces = 2 * (BM + BN) / 64;
  static constexpr int LX = (pieces + waves - 1) / waves, loads = LA + LW + LX;
  static_assert(BM % (8 * waves) == 0 && BN % (8 * waves) == 0 && BM % 64 == 0 && BN % 64 == 0, "whole DMA instructions");
};

// Until at most N vector-memory instructions of the wave are in flight; LDS reads go on.
template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 0xF) | (0x7 << 4) | (0xF << 8) | ((N >> 4) << 14));
}
// The same, and all LDS reads of the wave are done.
template <int N>
__device__ __forceinline__ void wait_vm_lds() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 0xF) | (0x7 << 4) | (0x0 << 8) | ((N >> 4) << 14));
}
__device__ __forceinline__ void block_barrier() { asm volatile("s_barrier" ::: "memory"); }

template <int BM, int BN, int WM, int WN, int RING, bool BF16>
__global__ __launch_bounds__(64 * WM * WN, 1) void mx_gemm_kernel(
    const uint8_t* __restrict__ qa, const uint32_t* __restrict__ sa, const uint8_t* __restrict__ qw,
    const uint32_t* __restrict__ sw, int64_t M, int64_t N, int64_t K, void* __restrict__ y, int64_t ldy,
    int64_t tiles_m) {
  using T = Tile<BM, BN, WM, WN>;
  constexpr int TM = T::TM, TN = T::TN;
  // objects of their own: the compiler sees that the DMA into one never writes what is read from another
  static_assert(RING == 2 || RING == 3, "buffers of the ring");
  __shared__ __align__(16) uint8_t buf0[T::bytes];
  __shared__ __align__(16) uint8_t buf1[T::bytes];
  __shared__ __align__(16) uint8_t buf2[RING > 2 ? T::bytes : 16];

  const int tid = threadIdx.x, lane = tid & 63, n = lane & 15, h = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  int64_t mt, nt;
  mx_tile(blockIdx.x, gridDim.x, tiles_m, mt, nt);
  const int64_t m0 = mt * BM, n0 = nt * BN, row_bytes = K / 2;
  const int G = int(K / kGroup);
  const int rows_a = int(M - m0 < BM ? M - m0 : BM), rows_w = int(N - n0 < BN ? N - n0 : BN);

  // rows beyond the last one read that again; what they give is not stored
  const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(qa + m0 * row_bytes), 0,
                                                                      int(rows_a * row_bytes), 0x00020000);
  const __amdgpu_buffer_rsrc_t rw = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(qw + n0 * row_bytes), 0,
                                                                      int(rows_w * row_bytes), 0x00020000);
  uint32_t from_a[T::LA], from_w[T::LW];
  const int sub = lane >> 3, chunk = ((lane & 7) ^ sub) * 16;
#pragma unroll
  for (int i = 0; i < T::LA; ++i) {
    const int r = (wave * T::LA + i) * 8 + sub;
    from_a[i] = uint32_t((r < rows_a ? r : rows_a - 1) * row_bytes + chunk);
  }
#pragma unroll
  for (int i = 0; i < T::LW; ++i) {
    const int r = (wave * T::LW + i) * 8 + sub;
    from_w[i] = uint32_t((r < rows_w ? r : rows_w - 1) * row_bytes + chunk);
  }
  const int stages = (G + 1) / 2;
  // One of the wave's T::loads DMA instructions of a stage (behind the last stage: that
  // again, not used; behind the last channel: the next row's codes or zeros).
  auto bring = [&](uint8_t* to, int stage, int i) {
    const int s = stage < stages ? stage : stages - 1;
    if (i < T::LA) {
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void_t*)(to + (wave * T::LA + i) * 1024), 16, int(from_a[i]),
                                               s * kStageRow, 0, 0);
    } else if (i < T::LA + T::LW) {
      i -= T::LA;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_void_t*)(to + BM * kStageRow + (wave * T::LW + i) * 1024), 16,
                                               int(from_w[i]), s * kStageRow, 0, 0);
    } else {
      // 64 rows' words of a group; zeros behind the tile's last row, and for a last stage's
      // second half that has no channels: whatever the codes there are, products of two
      // operands of scale 2^-127 are below the smallest fp32 number, so they add nothing.
      // Where there are fewer pieces than waves, the last one again.
      int p = wave * T::LX + i - T::LA - T::LW;
      p = p < T::pieces ? p : T::pieces - 1;
      constexpr int kHalf = T::pieces / 2;
      const int half = p >= kHalf ? 1 : 0, row = 64 * (p - half * kHalf);  // of the tokens, then the channels
      const int g = 2 * s + half;
      const bool a = row < BM;
      const uint32_t* from = a ? sa + g * M + m0 : sw + g * N + n0;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          __builtin_amdgcn_make_buffer_rsrc(const_cast<uint32_t*>(from), 0, g < G ? (a ? rows_a : rows_w) * 4 : 0,
                                            0x00020000),
          (lds_void_t*)(to + T::codes + p * 256), 4, ((a ? row : row - BM) + lane) * 4, 0, 0, 0);
    }
  };

  v4f acc[TN][TM];
#pragma unroll
  for (int i = 0; i < TN; ++i)
#pragma unroll
    for (int j = 0; j < TM; ++j) acc[i][j] = v4f{};

  int off[2];  // of the lane's chunk of a step in a tile of 16 rows
#pragma unroll
  for (int k = 0; k < 2; ++k) off[k] = n * kStageRow + (((4 * k + h) ^ (n & 7)) * 16);
  const int base_a = wm * TM * 16 * kStageRow, base_w = (BM + wn * TN * 16) * kStageRow;
  const int base_xa = T::codes + (wm * TM * 16 + n) * 4 + h, base_xw = T::codes + (BM + wn * TN * 16 + n) * 4 + h;

  constexpr int kSets = T::twice ? 2 : 1, P = TN * TM;
  v4u w[kSets][TN], t[kSets][TM];
  uint32_t xw[kSets][TN], xt[kSets][TM];  // scale bytes
  auto read_w = [&](const uint8_t* from, int k, int set, int i) {
    w[set][i] = *reinterpret_cast<const v4u*>(from + off[k] + base_w + i * 16 * kStageRow);
    xw[set][i] = from[base_xw + k * T::words + i * 64];
  };
  auto read_t = [&](const uint8_t* from, int k, int set, int j) {
    t[set][j] = *reinterpret_cast<const v4u*>(from + off[k] + base_a + j * 16 * kStageRow);
    xt[set][j] = from[base_xa + k * T::words + j * 64];
  };
  // f(i) for i < COUNT, spread over the P products of a step from the first one on
  auto spread = [&](int at, auto count, auto f) {
    constexpr int kCount = decltype(count)::value, kEach = (kCount + P - 1) / P;
#pragma unroll
    for (int e = 0; e < kEach; ++e)
      if (at * kEach + e < kCount) f(at * kEach + e);
  };
  using Reads = std::integral_constant<int, TN + TM>;
  using Loads = std::integral_constant<int, T::loads>;
  // The products of a step; operands of step k2 of `from` are read meanwhile.
  auto step = [&](int set, const uint8_t* from, int k2, auto meanwhile) {
#pragma unroll
    for (int j = 0; j < TM; ++j)
#pragma unroll
      for (int i = 0; i < TN; ++i) {
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fp4_operand(w[set][i]), fp4_operand(t[set][j]), acc[i][j],
                                                                     kFp4, kFp4, 0, int(xw[set][i]), 0, int(xt[set][j]));
        if constexpr (T::twice) {
          spread(j * TN + i, Reads{}, [&](int e) {
            if (e < TN) read_w(from, k2, 1 - set, e);
            else read_t(from, k2, 1 - set, e - TN);
          });
        } else {
          if (j == TM - 1) read_w(from, k2, 0, i);
          if (i == TN - 1) read_t(from, k2, 0, j);
        }
        meanwhile(j * TN + i);
        __builtin_amdgcn_sched_barrier(0);
      }
  };

#pragma unroll
  for (int i = 0; i < T::loads; ++i) bring(buf0, 0, i);
#pragma unroll
  for (int i = 0; i < T::loads; ++i) bring(buf1, 1, i);
  if constexpr (RING > 2) {
#pragma unroll
    for (int i = 0; i < T::loads; ++i) bring(buf2, 2, i);
  }
  wait_vm<(RING - 1) * T::loads>();
  block_barrier();
#pragma unroll
  for (int i = 0; i < TN; ++i) read_w(buf0, 0, 0, i);
#pragma unroll
  for (int j = 0; j < TM; ++j) read_t(buf0, 0, 0, j);
  // Stage s in `cur`, whose first operands are read; reads those of the next one.
  auto stage = [&](uint8_t* cur, const uint8_t* next, int s) {
    step(0, cur, 1, [](int) {});
    wait_vm_lds<(RING - 2) * T::loads>();  // the next stage has arrived, this wave has read the last of this one
    block_barrier();                       // for all waves
    step(kSets - 1, next, 0, [&](int at) { spread(at, Loads{}, [&](int i) { bring(cur, s + RING, i); }); });
  };
  int s = 0;
  for (; s + RING <= stages; s += RING) {
    stage(buf0, buf1, s);
    if constexpr (RING == 2) {
      stage(buf1, buf0, s + 1);
    } else {
      stage(buf1, buf2, s + 1);
      stage(buf2, buf0, s + 2);
    }
  }
  if (s < stages) stage(buf0, buf1, s);
  if constexpr (RING > 2) {
    if (s + 1 < stages) stage(buf1, buf2, s + 1);
  }
  __syncthreads();  // the DMA behind the last stage included

  // Output: 32 tokens at a time through the wave's own part of LDS into rows of 16-byte chunks.
  constexpr int E = BF16 ? 2 : 4, kCols = TN * 16, kOut = kCols * E + 16, kChunks = kCols * E / 16;
  constexpr int kWaveBytes = 32 * kOut, kEach = T::waves / 2;
  static_assert(kEach * kWaveBytes <= T::bytes, "output rows of half of the waves in each buffer");
  uint8_t* out = (wave < kEach ? buf0 : buf1) + (wave % kEach) * kWaveBytes;
  const bool aligned = (ldy * E) % 16 == 0 && (reinterpret_cast<uintptr_t>(y) & 15) == 0;
  const int64_t c0 = n0 + wn * kCols;
#pragma unroll
  for (int j = 0; j < TM / 2; ++j) {
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const v4f v = acc[i][2 * j + b];
        uint8_t* dst = out + (16 * b + n) * kOut + (16 * i + 4 * h) * E;
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
    const int64_t first = m0 + wm * TM * 16 + j * 32;
    if (aligned && c0 + kCols <= N) {
#pragma unroll
      for (int it = 0; it < 32 * kChunks / 64; ++it) {
        const int idx = it * 64 + lane, r = idx / kChunks, c = idx % kChunks;
        const v4u v = *reinterpret_cast<const v4u*>(out + r * kOut + c * 16);
        if (first + r < M)  // nothing in the kernel reads y back
          __builtin_nontemporal_store(v, reinterpret_cast<v4u*>(reinterpret_cast<uint8_t*>(y) + ((first + r) * ldy + c0) * E + c * 16));
      }
    } else {  // rows that are not 16-byte aligned, or end in the tile: neighbouring lanes store neighbouring values
      typedef typename std::conditional<BF16, uint16_t, uint32_t>::type Word;
      constexpr int kRows = kCols < 64 ? 64 / kCols : 1, kPasses = kCols < 64 ? 1 : kCols / 64;  // of an instruction
      const int r0 = kCols < 64 ? lane / kCols : 0, c1 = kCols < 64 ? lane % kCols : lane;
#pragma unroll
      for (int i = 0; i < 32; i += 8 * kRows) {
        Word v[8][kPasses];  // read together: the stores below wait for them once
#pragma unroll
        for (int e = 0; e < 8; ++e)
#pragma unroll
          for (int p = 0; p < kPasses; ++p)
            v[e][p] = *reinterpret_cast<const Word*>(out + (i + e * kRows + r0) * kOut + (c1 + 64 * p) * E);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int64_t m = first + i + e * kRows + r0;
#pragma unroll
          for (int p = 0; p < kPasses; ++p)
            if (m < M && c0 + c1 + 64 * p < N) reinterpret_cast<Word*>(y)[m * ldy + c0 + c1 + 64 * p] = v[e][p];
        }
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

// ---------------------------------------------------------------------------
// Few tiles (a few dozen rows, or few channels): 32 tokens x 32 channels a block, whose
// 4 waves take 128 channels each of a stage of 512 (256 bytes of a row) for the whole
// tile and add up in LDS at the end.  The ring, the DMA and the exchange of chunks (place
// c ^ (row & 15)) as above; a wave's operands of a stage are read during its products of
// the stage before.
//   A CU takes in 55 to 65 GB/s by way of L2 in these kernels, as much as it has in flight
// over the latency, so where 64 x 64 tiles are fewer than the CUs smaller ones are faster,
// though they read more: 61 tokens x 4096 channels, K = 14336, in the cache 8.8 us against
// 15.6, from memory 13.1 against 23.3 (64 x 64 tiles whose waves split K like here took
// 17, 32 x 32 straight from memory to registers 16, both in the cache).
// ---------------------------------------------------------------------------
constexpr int kSplitTile = kMxSplitTile, kSplitWaves = 4, kSplitRow = 256, kSplitRing = 4;
constexpr int kSplitCodes = 2 * kSplitTile * kSplitRow, kSplitBytes = kSplitCodes + kSplitWaves * 2 * kSplitTile * 4;
constexpr int kSplitLoads = kSplitCodes / 1024 / kSplitWaves + 1;  // DMA instructions of a wave for a stage

template <bool BF16>
__global__ __launch_bounds__(64 * kSplitWaves) void mx_gemm_split_kernel(
    const uint8_t* __restrict__ qa, const uint32_t* __restrict__ sa, const uint8_t* __restrict__ qw,
    const uint32_t* __restrict__ sw, int64_t M, int64_t N, int64_t K, void* __restrict__ y, int64_t ldy, int64_t tiles_m) {
  __shared__ __align__(16) uint8_t buf0[kSplitBytes];
  __shared__ __align__(16) uint8_t buf1[kSplitBytes];
  __shared__ __align__(16) uint8_t buf2[kSplitBytes];
  __shared__ __align__(16) uint8_t buf3[kSplitBytes];
  const int tid = threadIdx.x, lane = tid & 63, n = lane & 15, h = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  int64_t mt, nt;
  mx_tile(blockIdx.x, gridDim.x, tiles_m, mt, nt);
  const int64_t m0 = mt * kSplitTile, n0 = nt * kSplitTile, row_bytes = K / 2;
  const int G = int(K / kGroup), stages = (G + kSplitWaves - 1) / kSplitWaves;
  const int rows_a = int(M - m0 < kSplitTile ? M - m0 : kSplitTile), rows_w = int(N - n0 < kSplitTile ? N - n0 : kSplitTile);

  // codes: wave 0, 1 bring the tokens' rows, 2, 3 the channels', 4 rows an instruction
  const bool of_a = wave < 2;
  const int rows = of_a ? rows_a : rows_w;
  const __amdgpu_buffer_rsrc_t from = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(of_a ? qa + m0 * row_bytes : qw + n0 * row_bytes), 0, int(rows * row_bytes), 0x00020000);
  uint32_t src[kSplitLoads - 1];
#pragma unroll
  for (int i = 0; i < kSplitLoads - 1; ++i) {
    const int r = (wave & 1) * 16 + 4 * i + h;  // rows beyond the last one read that again
    src[i] = uint32_t((r < rows ? r : rows - 1) * row_bytes + (n ^ (r & 15)) * 16);
  }
  // scales: a wave brings its own group's words, the tokens' in lanes 0 .. 31, then the channels'
  const int sr = lane & 31;
  const uint32_t* const scale0 = lane < 32 ? sa + m0 + (sr < rows_a ? sr : rows_a - 1) : sw + n0 + (sr < rows_w ? sr : rows_w - 1);
  const int64_t scale_step = lane < 32 ? M : N;
  auto bring = [&](uint8_t* to, int stage) {  // behind the last stage that again, behind the last channel other codes, not used
    const int s = stage < stages ? stage : stages - 1;
#pragma unroll
    for (int i = 0; i < kSplitLoads - 1; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (lds_void_t*)(to + (wave * (kSplitLoads - 1) + i) * 1024), 16, int(src[i]),
                                               s * kSplitRow, 0, 0);
    const int g = s * kSplitWaves + wave < G ? s * kSplitWaves + wave : G - 1;
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(scale0 + g * scale_step),
                                     (lds_void_t*)(to + kSplitCodes + wave * 256), 4, 0, 0);
  };

  v4f acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = v4f{};
  v4u w[2][2], t[2][2];
  uint32_t xw[2][2], xt[2][2];
  const int off = n * kSplitRow + (((4 * wave + h) ^ n) * 16), off_x = kSplitCodes + wave * 256 + n * 4 + h;
  auto read = [&](const uint8_t* b, int set) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      t[set][i] = *reinterpret_cast<const v4u*>(b + off + i * 16 * kSplitRow);
      w[set][i] = *reinterpret_cast<const v4u*>(b + off + (2 + i) * 16 * kSplitRow);
      xt[set][i] = b[off_x + i * 64];
      xw[set][i] = b[off_x + (2 + i) * 64];
    }
  };
  bring(buf0, 0);
  bring(buf1, 1);
  bring(buf2, 2);
  bring(buf3, 3);
  wait_vm<(kSplitRing - 1) * kSplitLoads>();
  block_barrier();
  read(buf0, 0);
  // Stage s in `cur`, whose operands are read; reads those of the next one.
  auto stage = [&](uint8_t* cur, const uint8_t* next, int set, int s) {
    wait_vm_lds<(kSplitRing - 2) * kSplitLoads>();  // the next stage has arrived, this wave has read this one
    block_barrier();                                // for all waves
    bring(cur, s + kSplitRing);
    read(next, 1 - set);
    if (s * kSplitWaves + wave < G) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fp4_operand(w[set][i]), fp4_operand(t[set][j]),
                                                                       acc[i][j], kFp4, kFp4, 0, int(xw[set][i]), 0,
                                                                       int(xt[set][j]));
    }
  };
  int s = 0;
  for (; s + kSplitRing <= stages; s += kSplitRing) {
    stage(buf0, buf1, 0, s);
    stage(buf1, buf2, 1, s + 1);
    stage(buf2, buf3, 0, s + 2);
    stage(buf3, buf0, 1, s + 3);
  }
  if (s < stages) stage(buf0, buf1, 0, s);
  if (s + 1 < stages) stage(buf1, buf2, 1, s + 1);
  if (s + 2 < stages) stage(buf2, buf3, 0, s + 2);
  __syncthreads();  // the DMA behind the last stage included

  // the waves' sums, one buffer each: [32 tokens][32 channels], 4 floats of padding a token
  constexpr int kRow = kSplitTile + 4;
  static_assert(kSplitTile * kRow * 4 <= kSplitBytes, "sums of a wave in a buffer");
  float* mine = reinterpret_cast<float*>(wave == 0 ? buf0 : wave == 1 ? buf1 : wave == 2 ? buf2 : buf3);
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) *reinterpret_cast<v4f*>(mine + (16 * j + n) * kRow + 16 * i + 4 * h) = acc[i][j];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kSplitTile * kSplitTile / (64 * kSplitWaves); ++i) {
    const int at = i * 64 * kSplitWaves + tid, token = at / kSplitTile, c = at % kSplitTile, from_at = token * kRow + c;
    const float v = (reinterpret_cast<const float*>(buf0)[from_at] + reinterpret_cast<const float*>(buf1)[from_at]) +
                    (reinterpret_cast<const float*>(buf2)[from_at] + reinterpret_cast<const float*>(buf3)[from_at]);
    if (token < rows_a && c < rows_w) store_one<BF16>(y, (m0 + token) * ldy + n0 + c, v);
  }
}

// ---------------------------------------------------------------------------
// Single tokens and a few more: a block takes 16 channels and up to 16 tokens, its 8
// waves split K in slices of 128 channels, PAIR consecutive ones at a time, so that a
// wave reads whole lines of the rows: 2 (128 bytes), 4 for longer rows.  Operands go
// straight to registers, the next slices are loaded before the current ones are
// multiplied, the waves' sums meet in LDS.
//   Bound by the launch, then by the weights' bytes: 1 x 4096 x 4096 3.9 us, 1 x 65536 x
// 4096 26.6 (5.4 TB/s), 1 x 14336 x 14336 21.1 (5.2 TB/s).  PAIR 2 / 4, us: 1 x 65536 x 4096
// 26.6 / 29.5, 1 x 11008 x 4096 6.4 / 7.2, 1 x 4096 x 14336 7.0 / 7.3, 1 x 14336 x 14336
// 22.7 / 21.1, 1 x 28672 x 8192 29.5 / 23.8, 1 x 4096 x 8192 6.6 / 5.3 (rows of 4 KB share
// their memory channels).
// ---------------------------------------------------------------------------
constexpr int kFewWaves = 8, kFewTokens = 16, kFewChannels = kMxFewChannels;

template <int PAIR, bool BF16>
__global__ __launch_bounds__(64 * kFewWaves) void mx_gemm_few_kernel(
    const uint8_t* __restrict__ qa, const uint32_t* __restrict__ sa, const uint8_t* __restrict__ qw,
    const uint32_t* __restrict__ sw, int M, int64_t N, int64_t K, void* __restrict__ y, int64_t ldy) {
  __shared__ __align__(16) float sums[kFewWaves][kFewTokens][kFewChannels + 4];  // +4: fewer bank conflicts
  const int tid = threadIdx.x, lane = tid & 63, n = lane & 15, h = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t n0 = int64_t(blockIdx.x) * kFewChannels, row_bytes = K / 2;
  const int G = int(K / kGroup);
  // rows beyond the last one read that again; what they give is not stored
  const int64_t row_a = n < M ? n : M - 1, row_w = n0 + n < N ? n0 + n : N - 1;

  struct Slice {
    v4u w, t;
    uint32_t xw, xt;
  };
  auto load = [&](int g, Slice& s) {
    g = g < G ? g : G - 1;
    const int64_t at = int64_t(g) * 64 + 16 * h;
    s.w = *reinterpret_cast<const v4u*>(qw + row_w * row_bytes + at);
    s.xw = sw[g * N + row_w];
    s.t = *reinterpret_cast<const v4u*>(qa + row_a * row_bytes + at);
    s.xt = sa[g * int64_t(M) + row_a];
  };
  v4f acc{};
  constexpr int kStep = kFewWaves * PAIR;
  Slice cur[PAIR], next[PAIR];
  int g = wave * PAIR;
  if (g < G) {
#pragma unroll
    for (int p = 0; p < PAIR; ++p) load(g + p, cur[p]);
  }
  for (; g < G; g += kStep) {
    if (g + kStep < G) {
#pragma unroll
      for (int p = 0; p < PAIR; ++p) load(g + kStep + p, next[p]);
    }
#pragma unroll
    for (int p = 0; p < PAIR; ++p)
      if (g + p < G)
        acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fp4_operand(cur[p].w), fp4_operand(cur[p].t), acc, kFp4, kFp4,
                                                               0, int(cur[p].xw >> (8 * h)), 0, int(cur[p].xt >> (8 * h)));
#pragma unroll
    for (int p = 0; p < PAIR; ++p) cur[p] = next[p];
  }
  *reinterpret_cast<v4f*>(&sums[wave][n][4 * h]) = acc;
  __syncthreads();
  if (tid < kFewTokens * kFewChannels) {
    const int token = tid / kFewChannels, c = tid % kFewChannels;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kFewWaves; ++w) v += sums[w][token][c];
    if (token < M && n0 + c < N) store_one<BF16>(y, token * ldy + n0 + c, v);
  }
}

}  // namespace

hipError_t launch_mx_gemm(const uint8_t* qa, const uint8_t* sa, const uint8_t* qw, const uint8_t* sw, int64_t M,
                          int64_t N, int64_t K, void* y, bool y_bf16, int64_t ldy, hipStream_t st) {
  const uint32_t* xa = reinterpret_cast<const uint32_t*>(sa);
  const uint32_t* xw = reinterpret_cast<const uint32_t*>(sw);
  auto few = [&](auto pair) {
    constexpr int P = decltype(pair)::value;
    const dim3 grid{unsigned((N + kFewChannels - 1) / kFewChannels)}, threads{64 * kFewWaves};
    if (y_bf16)
      hipLaunchKernelGGL((mx_gemm_few_kernel<P, true>), grid, threads, 0, st, qa, xa, qw, xw, int(M), N, K, y, ldy);
    else
      hipLaunchKernelGGL((mx_gemm_few_kernel<P, false>), grid, threads, 0, st, qa, xa, qw, xw, int(M), N, K, y, ldy);
    return hipGetLastError();
  };
  auto split = [&]() {
    const int64_t tiles_m = (M + kSplitTile - 1) / kSplitTile, blocks = tiles_m * ((N + kSplitTile - 1) / kSplitTile);
    const dim3 grid{unsigned(blocks)}, threads{64 * kSplitWaves};
    if (y_bf16)
      hipLaunchKernelGGL((mx_gemm_split_kernel<true>), grid, threads, 0, st, qa, xa, qw, xw, M, N, K, y, ldy, tiles_m);
    else
      hipLaunchKernelGGL((mx_gemm_split_kernel<false>), grid, threads, 0, st, qa, xa, qw, xw, M, N, K, y, ldy, tiles_m);
    return hipGetLastError();
  };
  auto many = [&](auto bm, auto bn, auto wm, auto wn, auto ring) {
    constexpr int BM = decltype(bm)::value, BN = decltype(bn)::value, WM = decltype(wm)::value, WN = decltype(wn)::value,
                  R = decltype(ring)::value;
    const int64_t tiles_m = (M + BM - 1) / BM, blocks = tiles_m * ((N + BN - 1) / BN);
    const dim3 grid{unsigned(blocks)}, threads{64 * WM * WN};
    if (y_bf16)
      hipLaunchKernelGGL((mx_gemm_kernel<BM, BN, WM, WN, R, true>), grid, threads, 0, st, qa, xa, qw, xw, M, N, K, y, ldy,
                         tiles_m);
    else
      hipLaunchKernelGGL((mx_gemm_kernel<BM, BN, WM, WN, R, false>), grid, threads, 0, st, qa, xa, qw, xw, M, N, K, y, ldy,
                         tiles_m);
    return hipGetLastError();
  };
  using std::integral_constant;
  const integral_constant<int, 2> k2{};
  const integral_constant<int, 3> k3{};
  const integral_constant<int, 4> k4{};
  const integral_constant<int, 64> k64{};
  const integral_constant<int, 128> k128{};
  const integral_constant<int, 256> k256{};
  switch (mx_kernel_for(M, N, K)) {
    case MxKernel::Few2: return few(k2);
    case MxKernel::Few4: return few(k4);
    case MxKernel::Split: return split();
    case MxKernel::Tile64: return many(k64, k64, k2, k2, k3);
    case MxKernel::Tile128: return many(k128, k128, k2, k2, k2);
    default: return many(k256, k256, k4, k2, k2);
  }
}

}  // namespace rw4
