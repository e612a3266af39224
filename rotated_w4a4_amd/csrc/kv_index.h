// Index bounds of the KV cache kernels: constants and arithmetic without any
// device code, so that host compilers can check them too.
#pragma once

#include <stdint.h>

namespace rw4 {

// Tokens of one request, at most: kv_slots refuses more, kv_attention clamps longer
// lengths.  The kernels hold key indexes in 32 bits and look up to two steps, or
// 32 tiles of page ids, ahead of the last key.
constexpr int kMostKeys = 0x7FFFFFFF - 8191;

constexpr int clamp_keys(int64_t len, int64_t room) {
  const int64_t most = room < kMostKeys ? room : int64_t(kMostKeys);
  return int(len < 0 ? 0 : len > most ? most : len);
}

// The kernel for few rows fetches the page ids of 32 tiles at a time, one a
// lane: lane n has the half n & 1 (16 keys) of tile n / 2, the tiles of a wave
// 128 keys apart.  The lane's first key lies this far behind the first tile's.
constexpr int ids_ahead(int lane) { return 128 * (lane >> 1) + 16 * (lane & 1); }
static_assert(kMostKeys <= 0x7FFFFFFF - ids_ahead(63) - 128, "key indexes stay in 32 bits");

// Whether the kernel for many rows gives every block a whole unit instead of
// cutting the line of all units' steps into equal shares.  That needs `whole` units
// or more (0: never), so that the grid is full for a while, a grid with a block for
// each, and no unit that is longer than a share: the last block to start would else
// run on alone.
constexpr bool whole_units(int64_t units, int64_t whole, int64_t grid, int64_t longest, int64_t steps, int blocks) {
  return whole > 0 && units >= whole && units <= grid && longest * blocks <= steps;
}

// The kernel for few rows where a unit's keys are bounded (a window with sinks): units
// take whole shares, so that no block works on two of them.  A share cut anywhere
// starts and merges two units or more, which costs as much as 8 steps, so even shares
// may be up to twice as long and 8 steps longer than equal ones.  Steps a share and us,
// equal / even, 8 KV heads of 128, single tokens:
//   64 requests, window 2048            12, 54.9 / 17, 43.5
//   64 of 1 to 3000 keys, window 2048   9, 55.1 / 17, 38.5
//   64 requests, window 512             4, 27.7 / 5, 21.0
//   64 requests, window 8192            43, 135 / 65, 134
constexpr int64_t even_most(int64_t equal) { return 2 * equal + 8; }
// With more than 64 requests the even share is a whole unit, where there are `whole` of
// them or more and the grid has blocks for all.
constexpr bool whole_few(int64_t units, int64_t whole, int64_t grid, int64_t longest, int64_t steps, int blocks) {
  return whole > 0 && units >= whole && units <= grid && longest <= even_most((steps + blocks - 1) / blocks);
}

// Blocks of the kernel for many rows, for so many units at most: a block for each,
// or those that share the line where a grid (fewer than 2^32 threads) has no room.
constexpr int64_t wide_grid(int64_t units, int64_t blocks) {
  return units > blocks && units < (int64_t(1) << 24) ? units : blocks;
}

}  // namespace rw4
