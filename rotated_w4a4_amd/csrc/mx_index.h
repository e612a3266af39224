// Grids of the MXFP4 kernels and the choice of the product's: constants and arithmetic
// without any device code, so that host compilers can check them too.
#pragma once

#include <stdint.h>

namespace rw4 {

// Blocks of a grid, at most (512 threads each: a grid has fewer than 2^32).
constexpr int64_t kMxMostBlocks = int64_t(1) << 22;
// Channels of a block of the kernel for single tokens, and the tile's side of the one
// whose waves split K.
constexpr int kMxFewChannels = 16, kMxSplitTile = 32;

// Few2, Few4: single tokens, so many slices of 128 channels at a time; Split: 32 x 32
// tiles; the others: tiles of so many tokens and channels.
enum class MxKernel { Few2, Few4, Split, Tile64, Tile128, Tile256 };

constexpr int64_t mx_tiles(int64_t M, int64_t N, int64_t side) {
  return ((M + side - 1) / side) * ((N + side - 1) / side);
}

// Measured at M x N, us, the launch included, operands from memory (several sets in turn,
// larger than the cache together): K = 4096, in brackets 14336, or the K that is named.
constexpr MxKernel mx_kernel_for(int64_t M, int64_t N, int64_t K) {
  const bool longer = K > 4096;
  // Single tokens / 32 x 32:  1 x 4096 4.1 (8.2) / 4.4 (10.4), 4 x 4096 4.1 (8.5) / 4.5 (10.4), 1 x 65536
  //   26.7 (83.1) / 31.3 (82.6).  By tokens alone, which costs 4 tokens of many channels some time: 4 x
  //   14336 9.4 (24.2) / 8.8 (21.5), 4 x 65536 31.5 (92.4) / 31.8 (83.1), 4 x 28672 16.3 (42.3), 64 x 64 13.4 (39.1).
  //   8 tokens in the cache: x 4096 4.0 / 4.4, x 14336 8.7 / 7.8.
  // 2 slices / 4:  K = 2048 1 x 65536 14.5 / 19.3, 4096 1 x 8192 5.7 / 5.3 and 1 x 65536 26.7 / 29.6, 8192
  //   1 x 4096 7.2 / 6.0 and 1 x 65536 62.9 / 50.3
  if (M <= 4 && N <= kMxMostBlocks * kMxFewChannels) return longer ? MxKernel::Few4 : MxKernel::Few2;
  // 32 x 32 / 64 x 64, by small tiles:  61 x 4096 (256) 5.0 (13.1) / 6.5 (23.3), 64 x 4608 (288) 7.9 (20.3) /
  //   8.5 (23.5), 32 x 11008 (344) 10.0 (24.0) / 9.2 (24.9), 61 x 6144 (384) 8.9 (21.0) / 8.8 (23.7), 128 x
  //   4096 (512) 7.0 (19.6) / 6.6 (23.2), 61 x 11008 (688) 12.6 (30.5) / 9.5 (25.6)
  //   between: 128 x 4096 K = 4224 8.7 / 9.0, 5120 10.0 / 10.0, 8192 12.8 / 14.5; 32 x 11008, which reads most for
  //   its tiles, 4224 11.9 / 9.7, 5120 12.6 / 10.9, 8192 16.4 / 16.2
  //   below: 61 x 4096 1024 4.0 / 4.1, 2048 4.2 / 4.7; 64 x 4608 1024 4.9 / 4.1, 2048 5.6 / 4.8
  if (mx_tiles(M, N, kMxSplitTile) <= (longer ? 512 : 288)) return MxKernel::Split;
  // 64 x 64, 128 x 128: up to 3 of the small tiles for each CU
  //   512 x 4096 (512 small tiles) 10.9 / 14.9, 384 x 8192 (768) 17.6 / 17.7, 1024 x 4096 (1024) 18.9 / 15.9
  //   the same at K = 2048 6.6 / 8.4, 9.7 / 9.5, 10.4 / 9.2, at 512 4.4 / 5.0, 5.5 / 5.1, 6.6 / 5.5
  if (mx_tiles(M, N, 64) <= 768) return MxKernel::Tile64;
  // 128 x 128, 256 x 256: the large tiles where they fill 7/8 of the rounds of a block for
  // each CU that they take
  //   2048 x 4096 (128 large tiles) 23.4 / 30.0, 2048 x 8192 (256) 47.8 / 37.9, 4096 x 8192 (512) 89.9 / 73.9; in the
  //   cache 3000 x 6144 (288) 47.0 / 58.6, 2048 x 14336 (448) 66.3 / 64.6.  2048 x 6144 (192) is even in the
  //   cache, 30.5 / 30.7, and 38.3 / 32.0 from memory
  //   K = 2048: 2048 x 4096 12.8 / 17.6, 4096 x 4096 23.6 / 23.1, 4096 x 8192 56.3 / 48.0; K = 512, mostly output:
  //   7.1 / 9.9, 12.2 / 12.5, 21.7 / 26.0
  //   (128 x 256 tiles, 4 or 8 waves, in the cache: 21.8 to 23.6 at 2048 x 4096, 118 at 4096 x 4096, K = 14336)
  const int64_t large = mx_tiles(M, N, 256), rounds = (large + 255) / 256;
  return 8 * large >= 7 * 256 * rounds ? MxKernel::Tile256 : MxKernel::Tile128;
}

// Whether the kernel's grid holds the tiles: the other kernels have 2^13 at most.
constexpr bool mx_gemm_fits(int64_t M, int64_t N, int64_t K) {
  return mx_kernel_for(M, N, K) != MxKernel::Tile256 || mx_tiles(M, N, 256) <= kMxMostBlocks;
}

// The kernel for rows of any strides takes so many rows and channels a block (Hadamard
// blocks of 256 and 512: a whole one).
constexpr int mx_pack_rows(int block) { return block < 512 ? 64 : 32; }
constexpr int mx_pack_span(int block) { return block < 128 ? 128 : block; }
constexpr int64_t kMxPackMostBlocks = (int64_t(1) << 24) - 1;  // of 256 threads: a grid has fewer than 2^32
// K is a multiple of the block, and of 128.
constexpr int64_t mx_pack_blocks(int64_t rows, int64_t K, int block) {
  return (rows + mx_pack_rows(block) - 1) / mx_pack_rows(block) * (K / mx_pack_span(block));
}

}  // namespace rw4
