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

// Measured at M x N, K = 4096 (in brackets 14336), us, the launch included.
constexpr MxKernel mx_gemm_kernel(int64_t M, int64_t N, int64_t K) {
  const bool longer = K > 4096;
  //   Single tokens / 32 x 32:  1 x 4096 3.9 (7.3) / 4.4 (7.9), 4 x 4096 3.8 (7.6) / 4.4 (8.0), 4 x 14336
  //   8.2 (23.2) / 7.8 (20.0), 8 x 4096 4.0 / 4.4, 8 x 14336 8.7 / 7.8; 1 x 65536 26.6 / 30.9, 8 x 65536 35.6 / 31.5
  if (M <= 4 && N <= kMxMostBlocks * kMxFewChannels) return longer ? MxKernel::Few4 : MxKernel::Few2;
  //   32 x 32 / 64 x 64, by small tiles:  61 x 4096 (256) 4.9 (8.8) / 6.3 (15.6), 32 x 11008 (344)
  //   7.9 / 6.8, 61 x 6144 (384) 7.0 (14.3) / 6.6 (16.0), 128 x 4096 (512) 6.9 (14.5) / 6.4 (15.8),
  //   61 x 11008 (688) 9.5 / 6.9, 256 x 4096 (1024) 11.5 (25.2) / 7.0 (16.7)
  if (mx_tiles(M, N, kMxSplitTile) <= (longer ? 512 : 288)) return MxKernel::Split;
  // 64 x 64, 128 x 128: up to 3 of the small tiles for each CU
  //   512 x 4096 (512 small tiles) 10.1 (25.4) / 13.3 (38.3), 256 x 11008 (688) 13.0 / 13.4,
  //   384 x 8192 (768) 13.2 / 13.4, 1024 x 4096 (1024) 17.0 (50.2) / 14.2 (42.1)
  if (mx_tiles(M, N, 64) <= 768) return MxKernel::Tile64;
  // 128 x 128, 256 x 256: the large tiles where they fill 7/8 of the rounds of a block for
  // each CU that they take
  //   2048 x 4096 (128 large tiles) 21.4 (62.8) / 29.2 (84.8), 2048 x 6144 (192) 30.5 / 30.7, 2048 x 8192 (256)
  //   39.8 / 36.6, 3000 x 6144 (288) 47.0 / 58.6, 2048 x 14336 (448) 66.3 / 64.6, 4096 x 4096 (256) (123.7) / (104.2)
  //   (128 x 256 tiles, 4 or 8 waves: 21.8 to 23.6 at 2048 x 4096, 118 at 4096 x 4096, K = 14336)
  const int64_t large = mx_tiles(M, N, 256), rounds = (large + 255) / 256;
  return 8 * large >= 7 * 256 * rounds ? MxKernel::Tile256 : MxKernel::Tile128;
}

// Whether the kernel's grid holds the tiles: the other kernels have 2^13 at most.
constexpr bool mx_gemm_fits(int64_t M, int64_t N, int64_t K) {
  return mx_gemm_kernel(M, N, K) != MxKernel::Tile256 || mx_tiles(M, N, 256) <= kMxMostBlocks;
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
