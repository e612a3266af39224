// Attention over the paged INT4 KV cache.
//
//   s_j = scale sk_j (q . ck_j),  out = sum_j softmax(s)_j sv_j cv_j
//
// with the stored codes ck, cv and one fp32 scale per cached row.  One pass
// over the keys with the running maximum m and sum l of the softmax (base 2:
// scale log2(e) is folded into sk), so a key's codes are read once:
//   m' = max(m, s_j),  l' = l 2^(m - m') + sum 2^(s_j - m'),
//   o' = o 2^(m - m') + sum 2^(s_j - m') sv_j cv_j.
// The codes are exact in bf16 and the scales stay outside the products (sk
// multiplies the score, sv the probability), so scores of bf16 queries are
// exact up to the fp32 accumulation.  Probabilities enter the second product as
// three bf16 parts where anything is fp32 (PRECISE; fp32 queries are split the same
// way), else as two (2^-16) in the kernel for few rows, which is bound by memory,
// and as one fp16 number (2^-11) in the kernel for many rows, where a second product
// would cost time: little against the output's own rounding, 2^-8.
//
// Work.  A unit is a tile of query rows (row = query token x query head of one
// KV head) of one request and KV head.  The keys of all units, in steps of 64
// or 128, form one line that is cut into equal shares, one for each block of
// the grid, so ragged batches are balanced whatever their lengths: a share
// holds the end of one unit, whole units and the start of another.  Whole
// units write their output; the pieces of cut ones leave unnormalized partial
// results (o, m, l) in the workspace, at most two for each block, for the
// combine kernel.  Every block works the line out by itself from kv_len and
// cu_q: no plan, no copy to the host, and a captured graph follows its lengths.
#include "kv_device.h"
#include "kv_index.h"
#include "kv_internal.h"

#include <type_traits>

namespace rw4 {

namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v4f_u __attribute__((ext_vector_type(4), aligned(4)));
typedef int v6i __attribute__((ext_vector_type(6)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef __bf16 v32bf __attribute__((ext_vector_type(32)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef _Float16 v32h __attribute__((ext_vector_type(32)));
typedef unsigned int v4u __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// Probabilities may reach 2^kSlack before the maximum is raised (2^kHalfSlack where
// they enter products as fp16).
constexpr float kSlack = 8.0f, kHalfSlack = 7.0f;
constexpr int kCUs = 256;
constexpr int kNarrowRows = 16;
constexpr int kNarrowStep = 128;  // keys of a step: 32 for each of a block's 4 waves
constexpr int kWideRows = 128, kWideStep = 64;
// Blocks of a grid for each CU, at most: the workspace has room for the borders of these.
constexpr int kNarrowBlocksMost = 3, kWideBlocksMost = 3;
constexpr int kMaxBlocks = kCUs * (kNarrowBlocksMost > kWideBlocksMost ? kNarrowBlocksMost : kWideBlocksMost);
// Up to this many rows of a request the kernel for few rows is used.  Measured on
// requests of 4000 keys and 8 KV heads, few / many rows, us:
//               batch of 32                          batch of 4
//   D = 128     32 rows 71 / 80, 48 82 / 90,         31 / 29, 31 / 32,
//               64 118 / 89                          36 / 33
//   D = 64      32 rows 55 / 56, 48 63 / 61          23 / 25, 25 / 27
//   D = 256     48 rows 173 / 182, 64 191 / 175      52 / 43, 51 / 44
//   fp32, 128   64 rows 144 / 176, 96 210 / 179      37 / 45, 50 / 47
//   fp32, 64    64 rows 118 / 125, 96 174 / 126      29 / 32, 40 / 33
//   fp32, 256   48 rows 258 / 297, 64 335 / 297      57 / 69, 59 / 69
template <int D, bool PRECISE>
constexpr int kNarrowMost = PRECISE ? 64 : D == 64 ? 32 : 48;

// ---------------------------------------------------------------------------
// The line of work.
// ---------------------------------------------------------------------------
struct Req {
  int q0, qn, kv;   // first query token, query tokens, keys
  int tiles;        // row tiles
  int lo, span;     // first key any row sees (a multiple of 64) and keys from there on; with sinks 0, and a tile's positions
};

__device__ __forceinline__ int round16(int n) { return (n + 15) & ~15; }

__device__ __forceinline__ int clamp_int(int64_t v, int64_t hi) { return int(v < 0 ? 0 : v > hi ? hi : v); }

__device__ __forceinline__ Req request(const AttnArgs& a, int b, int rows) {
  Req r;
  const int q1 = clamp_int(a.cu_q[b + 1], a.T);
  r.q0 = clamp_int(a.cu_q[b], a.T);
  r.qn = q1 > r.q0 ? q1 - r.q0 : 0;
  r.kv = clamp_keys(a.kv_len[b], a.table_width << a.cache.log2_page);
  r.tiles = (r.qn * a.group + rows - 1) / rows;  // T * heads < 2^31
  r.lo = 0;
  if (a.window > 0) {
    const int64_t first = int64_t(r.kv) - r.qn + 1 - a.window;
    r.lo = first > 0 ? int(first) & ~63 : 0;
  }
  r.span = r.kv - r.lo;
  if (a.sinks > 0) {  // positions of a tile (Places), at most: its rows' windows start at most qn - 1 or a tile's tokens apart
    const int tokens = (rows + a.group - 2) / a.group + 1;
    const int64_t most = int64_t(round16(a.sinks)) + a.window + (r.qn < tokens ? r.qn : tokens) + 15;
    r.lo = 0;
    r.span = most < r.kv ? int(most) : r.kv;
  }
  return r;
}

// With sinks a unit works on positions instead of keys: the sinks, then the keys from
// the first one of its rows' windows on, without those between.  Position w is key w in
// front of `head` and key w + gap from there on (gap 0 where nothing lies between);
// GRAIN: keys that stay side by side, from a multiple of GRAIN on.
template <bool SINKS, int GRAIN>
struct Places {
  int head, gap;
  // lo: first key of the windows of the unit's rows
  __device__ __forceinline__ Places(const AttnArgs& a, int lo) : head(0), gap(0) {
    if constexpr (SINKS) {
      head = (a.sinks + GRAIN - 1) & ~(GRAIN - 1);
      lo &= ~(GRAIN - 1);
      gap = lo > head ? lo - head : 0;
    }
  }
  __device__ __forceinline__ int key(int w) const { return SINKS && w >= head ? w + gap : w; }
  // of a key of the windows
  __device__ __forceinline__ int place(int j) const { return SINKS ? j - gap : j; }
};

template <typename T>
__device__ __forceinline__ T wave_prefix(T v, int lane) {
  for (int d = 1; d < kWave; d <<= 1) {
    const T o = __shfl_up(v, d);
    if (lane >= d) v += o;
  }
  return v;
}
// The same for 32 bits in six DPP additions: shifts by 1, 2, 4, 8 within rows of
// 16 lanes, then the rows' last lanes broadcast to the rows behind.
__device__ __forceinline__ int wave_prefix_dpp(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);  // lane 15 to row 1, lane 47 to row 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);  // lane 31 to rows 2 and 3
  return v;
}
// The largest of the lanes up to each one, of values from 0 on, the same way.
__device__ __forceinline__ int wave_upmost_dpp(int v) {
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, true));
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, true));
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, true));
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, true));
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false));
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false));
  return v;
}
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t uniform(int64_t v) {
  return int64_t(uint32_t(uniform(int(v)))) | (int64_t(uniform(int(v >> 32))) << 32);
}

__device__ __forceinline__ int req_steps(const Req& r, int step) {
  return r.span > 0 ? (r.span + step - 1) / step : 1;
}

// The piece of a unit at a position of the line.
struct Piece {
  Req r;
  int b, head, tile;   // request, KV head, row tile
  int steps, at;       // steps of the unit, the position's step in it
};

// Orders a wave's own LDS writes and reads for the compiler (the hardware
// executes a wave's LDS operations in order).
__device__ __forceinline__ void wave_lds_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// How a kernel cuts the work: query rows of a unit, keys of a step, blocks that
// share the line, what whole_units goes by, and whether even_share and whole_few do instead.
struct Cut {
  int rows, step, blocks, whole;
  bool few = false;
  __device__ __forceinline__ bool take_whole(int64_t units, int64_t longest, int64_t steps) const {
    return few ? whole_few(units, whole, gridDim.x, longest, steps, blocks)
               : whole_units(units, whole, gridDim.x, longest, steps, blocks);
  }
};

// Steps before each thread's requests (256 threads take consecutive ones), and
// the requests themselves where a thread has one.
struct Line {
  long long before[257];
  Req reqs[256];
  long long wave_sum[4], wave_units[4];
  int wave_longest[4];
  bool by_units;  // a step for each unit
  int even;       // > 0: units take whole shares of so many steps (even_share), their last one may be cut short
};

// Steps with the room that a unit takes on the line.
__device__ __forceinline__ int even_steps(int steps, int even) { return even > 0 ? (steps + even - 1) / even * even : steps; }

// A share of which every unit can have whole ones of its own within the grid's blocks:
// the longest unit in as many equal parts as fit (tried in steps of a sixteenth: a
// few tries at most); 0: none up to even_most.  A lane's
// request has `units` of `steps`, all together `total` steps.  Every lane of the wave
// takes part.
__device__ __forceinline__ int even_share(int units, int steps, int total, int blocks) {
  const int longest = __builtin_amdgcn_readlane(wave_upmost_dpp(units > 0 ? steps : 0), kWave - 1);
  const int equal = total > blocks ? (total + blocks - 1) / blocks : 1, most = int(even_most(equal));  // total < 2^31
  for (int parts = (longest + equal - 1) / equal; parts > 0; parts -= 1 + (parts >> 4)) {
    const int share = (longest + parts - 1) / parts;
    if (share > most) break;
    const int need = wave_prefix_dpp(units * ((steps + share - 1) / share));
    if (__builtin_amdgcn_readlane(need, kWave - 1) <= blocks) return share;
  }
  return 0;
}

// Up to 64 requests, and 32 bits for their steps: a lane each, every wave by
// itself and with the same results, so no barrier (they write the same values).

__device__ __forceinline__ bool line_build_wave(const AttnArgs& a, const Cut& cut, Line& line) {
  const int lane = threadIdx.x & (kWave - 1);
  Req r{};
  if (lane < int(a.B)) r = request(a, lane, cut.rows);
  const int units = r.tiles * a.cache.heads, steps = req_steps(r, cut.step);
  if (__ballot(float(units) * float(steps) > 0x1p24f)) return false;  // sums below 2^30
  int own = units * steps, upto = wave_prefix_dpp(own);
  bool by_units = false;
  int even = 0;
  if (cut.few) {
    even = even_share(units, steps, __builtin_amdgcn_readlane(upto, kWave - 1), cut.blocks);
    own = units * even_steps(steps, even);
    upto = wave_prefix_dpp(own);
  } else if (cut.whole > 0) {
    const int upto_units = wave_prefix_dpp(units);
    // of every lane's request in the place of the longest
    by_units = !__ballot(!cut.take_whole(__builtin_amdgcn_readlane(upto_units, kWave - 1), units > 0 ? steps : 0,
                                         __builtin_amdgcn_readlane(upto, kWave - 1)));
    if (by_units) {
      own = units;
      upto = upto_units;
    }
  }
  line.before[lane] = upto - own;
  line.reqs[lane] = r;
  if (lane == kWave - 1) line.before[256] = upto;
  if (lane == 0) {
    line.by_units = by_units;
    line.even = even;
  }
  wave_lds_order();
  return true;
}

__device__ __forceinline__ void line_build(const AttnArgs& a, const Cut& cut, Line& line) {
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  const int B = int(a.B), per = (B + 255) / 256;
  if (B <= kWave && line_build_wave(a, cut, line)) return;
  const int b0 = tid * per < B ? tid * per : B, b1 = b0 + per < B ? b0 + per : B;
  long long sum = 0, units = 0;
  int longest = 0;
  for (int b = b0; b < b1; ++b) {
    const Req r = request(a, b, cut.rows);
    const int steps = req_steps(r, cut.step);
    sum += (long long)(r.tiles) * a.cache.heads * steps;
    units += (long long)(r.tiles) * a.cache.heads;
    if (r.tiles > 0) longest = max(longest, steps);
    if (per == 1) line.reqs[tid] = r;
  }
  long long upto = wave_prefix(sum, lane), upto_units = 0;
  if (lane == kWave - 1) line.wave_sum[wave] = upto;
  if (cut.whole > 0) {
    upto_units = wave_prefix(units, lane);
    for (int d = 1; d < kWave; d <<= 1) longest = max(longest, __shfl_xor(longest, d));
    if (lane == kWave - 1) {
      line.wave_units[wave] = upto_units;
      line.wave_longest[wave] = longest;
    }
  }
  __syncthreads();
  bool by_units = false;
  if (cut.whole > 0) {
    const long long all = line.wave_sum[0] + line.wave_sum[1] + line.wave_sum[2] + line.wave_sum[3];
    const long long all_units = line.wave_units[0] + line.wave_units[1] + line.wave_units[2] + line.wave_units[3];
    longest = max(max(line.wave_longest[0], line.wave_longest[1]), max(line.wave_longest[2], line.wave_longest[3]));
    by_units = cut.take_whole(all_units, longest, all);
    if (by_units) {
      sum = units;
      upto = upto_units;
    }
  }
  if (tid == 0) {
    line.by_units = by_units;
    line.even = 0;
  }
  long long before = upto - sum;
  for (int w = 0; w < wave; ++w) before += by_units ? line.wave_units[w] : line.wave_sum[w];
  line.before[tid] = before;
  if (tid == 255) line.before[256] = before + sum;
  __syncthreads();
}

__device__ __forceinline__ int64_t line_total(const Line& line) { return uniform(int64_t(line.before[256])); }

// A block's share: at least one step.
__device__ __forceinline__ int64_t line_share(int64_t total, int blocks) {
  const int64_t share = (total + blocks - 1) / blocks;
  return share > 0 ? share : 1;
}

// The piece at position pos < total; every wave finds it by itself.
__device__ __forceinline__ Piece line_find(const AttnArgs& a, const Cut& cut, const Line& line, int64_t pos) {
  const int lane = threadIdx.x & (kWave - 1);
  const int per = (int(a.B) + 255) / 256;
  int seg = -1;  // the last thread whose requests start at or before pos
  const int blocks64 = int(a.B) <= kWave ? 1 : 4;
  for (int i = 0; i < blocks64; ++i) seg += __popcll(__ballot(line.before[kWave * i + lane] <= pos));
  Piece p;
  const bool by_units = uniform(int(line.by_units));
  const int even = uniform(line.even);
  int room;
  p.b = seg * per;
  int64_t local = pos - uniform(int64_t(line.before[seg]));
  for (;; ++p.b) {  // ends at the last request at the latest: pos lies on the line
    const Req r = per == 1 ? line.reqs[p.b] : request(a, p.b, cut.rows);
    p.r = Req{uniform(r.q0), uniform(r.qn), uniform(r.kv), uniform(r.tiles), uniform(r.lo), uniform(r.span)};
    p.steps = by_units ? 1 : req_steps(p.r, cut.step);
    room = even_steps(p.steps, even);
    const int64_t all = int64_t(p.r.tiles) * a.cache.heads * room;
    if (local < all || p.b + 1 >= int(a.B)) break;
    local -= all;
  }
  int unit;
  if (local >> 31) {
    unit = int(local / room);
    p.at = int(local % room);
  } else {
    unit = int(local) / room;
    p.at = int(local) % room;
  }
  p.head = unit % a.cache.heads;
  p.tile = p.r.tiles - 1 - unit / a.cache.heads;  // the rows that see most first
  return p;
}

// The workspace: a descriptor for each border between blocks, then the
// partial results, two for each block: its first piece, and the one that the
// next block goes on with.
struct Border {
  int pieces;       // of the unit cut here for the first time; 0: none is
  int first;        // slot of its first piece (the others are 2 w, 2 (w + 1), ...)
  int q0, qn, head, tile;
  int unused[2];
};
__device__ __forceinline__ Border* borders(const AttnArgs& a) { return reinterpret_cast<Border*>(a.workspace); }
__device__ __forceinline__ float* partials(const AttnArgs& a) {
  return reinterpret_cast<float*>(reinterpret_cast<char*>(a.workspace) + kMaxBlocks * sizeof(Border));
}
__device__ __forceinline__ int piece_slot(int w, bool first) { return 2 * w + (first ? 0 : 1); }

// Block w writes what the combine kernel has to do at the border in front of
// it; `it` is its first piece (steps left unused without one).
__device__ __forceinline__ void write_border(const AttnArgs& a, int w, bool any, const Piece& it, int64_t share) {
  if (threadIdx.x != 0) return;
  Border d{};
  if (any && it.at > 0 && it.at <= share) {  // cut here, and not before
    d.pieces = 2 + int((it.steps - it.at - 1) / share);
    d.first = piece_slot(w - 1, it.at == share);
    d.q0 = it.r.q0;
    d.qn = it.r.qn;
    d.head = it.head;
    d.tile = it.tile;
  }
  borders(a)[w] = d;
}

// Keys [begin, end) that query token i of a request sees (besides the sinks in front of begin).
__device__ __forceinline__ void row_range(const AttnArgs& a, const Req& r, int i, int& begin, int& end) {
  const int place = r.kv - r.qn + i;
  end = a.causal ? place + 1 : r.kv;
  begin = 0;
  if (a.window > 0) {
    const int64_t first = int64_t(place) + 1 - a.window;
    begin = first > 0 ? int(first) : 0;
  }
}

// ---------------------------------------------------------------------------
// Operands.
// ---------------------------------------------------------------------------
// A 16-byte chunk's 32 codes as bf16 or fp16, in the order of the stored pairs:
// elements 8 i .. 8 i + 7 are channels 8 pair_order(i) .. of the chunk.
__device__ __forceinline__ v6i chunk_pairs(const v4u& w) {
  // a pair (a, b) opens into X[0:32] = a & A, X[32:64] = (a & ~A) | (b & ~C), X[64:96] = b & C
  return v6i{int(w[0] & kSgnA), int((w[0] & ~kSgnA) | (w[3] & ~kSgnC)), int(w[3] & kSgnC),
             int(w[1] & kSgnA), int((w[1] & ~kSgnA) | (w[2] & ~kSgnC)), int(w[2] & kSgnC)};
}
__device__ __forceinline__ v32bf open_chunk(const v4u& w) {
  return __builtin_amdgcn_cvt_scalef32_pk32_bf16_fp6(chunk_pairs(w), 8.0f);  // E2M3 c / 8 times 8
}
__device__ __forceinline__ v32h open_chunk_half(const v4u& w) {
  return __builtin_amdgcn_cvt_scalef32_pk32_f16_fp6(chunk_pairs(w), 8.0f);
}
__device__ __forceinline__ int pair_order(int i) { return i == 0 ? 0 : i == 1 ? 3 : i == 2 ? 1 : 2; }

__device__ __forceinline__ v8bf part8(const v32bf& x, int i) {
  v8bf r;
#pragma unroll
  for (int e = 0; e < 8; ++e) r[e] = x[8 * i + e];
  return r;
}

// The same 8 of an fp16 chunk, as the 16 bytes that are stored.
__device__ __forceinline__ v8bf part8(const v32h& x, int i) {
  v8h r;
#pragma unroll
  for (int e = 0; e < 8; ++e) r[e] = x[8 * i + e];
  return __builtin_bit_cast(v8bf, r);
}

// x = sum of N bf16 parts (N = 3: exact up to the smallest exponents).
template <int N>
__device__ __forceinline__ void split_bf16(float x, __bf16 (&part)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    part[i] = static_cast<__bf16>(x);  // round to nearest even
    x -= static_cast<float>(part[i]);
  }
}

// 8 query channels as N operands.
template <int N>
__device__ __forceinline__ void query_operand(const AttnArgs& a, int64_t off, bool live, v8bf (&out)[N]) {
  if (!live) {
#pragma unroll
    for (int i = 0; i < N; ++i) out[i] = v8bf{};
    return;
  }
  if (a.q_bf16) {
    out[0] = *reinterpret_cast<const v8bf*>(reinterpret_cast<const __bf16*>(a.q) + off);
#pragma unroll
    for (int i = 1; i < N; ++i) out[i] = v8bf{};
  } else {
    float v[8];
    RowSrc<false>{a.q, 0}.load8(0, off, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      __bf16 p[N];
      split_bf16<N>(v[e], p);
#pragma unroll
      for (int i = 0; i < N; ++i) out[i][e] = p[i];
    }
  }
}

__device__ __forceinline__ v8bf lds_transposed(const char* p0, const char* p1) {
  typedef __attribute__((address_space(3))) v4s* lds_v4s;
  const v4s a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s)(p0));
  const v4s b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s)(p1));
  typedef short v8s __attribute__((ext_vector_type(8)));
  const v8s r = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
  return __builtin_bit_cast(v8bf, r);
}

// Keeps a rarely taken, uniform branch a branch: as selects its work would be
// done for every step.
__device__ __forceinline__ void keep_branch() { asm volatile(""); }

// Bits 0 .. n - 1 (n of any size).
__device__ __forceinline__ uint32_t bits_below(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }

// Offset of a slot of a page (-1: page 0, read but not used); the strides of
// pages are below 2^32 and those of slots below 2^24, so each product is one
// 32 x 32 -> 64 bit multiply-add.
__device__ __forceinline__ int64_t row_at(int id, int64_t page_stride, int slot, int64_t slot_stride) {
  const uint64_t page = uint64_t(uint32_t(id >= 0 ? id : 0)) * uint32_t(page_stride);
  return int64_t(page + uint64_t(uint32_t(slot)) * uint32_t(slot_stride));
}

// The 4 scales of slots s .. s + 3 of a page.
__device__ __forceinline__ v4f scales4(const float* p, int64_t stride) {
  if (stride == 1) return *reinterpret_cast<const v4f_u*>(p);
  return v4f{p[0], p[stride], p[2 * stride], p[3 * stride]};
}

// One finished row: o (8 channels of each of its D / 8 lanes), sum l, maximum
// m: normalized, unrotated, rounded and stored.
template <int D>
__device__ __forceinline__ void finish_row(const AttnArgs& a, int q0, int qn, int head, int row, float (&o)[8], float m,
                                           float l, int lane) {
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
  for (int e = 0; e < 8; ++e) o[e] *= inv;
  if (a.unrotate) {
    row_hadamard<D / 8>(o, lane);
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] *= kHeadPost<D>;
  }
  if (row >= qn * a.group) return;
  const int64_t t = q0 + row / a.group;
  const int h = head * a.group + row % a.group, c8 = lane & (D / 8 - 1);
  store_row8(a.out, a.out_bf16, t * a.out_token + h * a.out_head + 8 * c8, o);
  if (a.lse && c8 == 0) a.lse[t * a.heads + h] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// ---------------------------------------------------------------------------
// Few query rows (decoding, drafts): 16 rows a unit, the keys of an item over
// the block's 4 waves in tiles of 32, merged at the end.
//
// Scores are formed transposed, S^T = K Q^T (16 keys x 16 rows), the codes as
// the row operand: lane l = 16 g + n holds 8 channels of key n, which are a
// quarter of the 16-byte chunk it loaded (the order of the channels is free
// as long as the queries use the same).  The result leaves rows along lanes
// and keys 4 g + i in registers, which is the column operand of O^T = V^T P^T
// without a move, with keys ordered (4 g + 0..3, 16 + 4 g + 0..3) per lane
// group.  V^T needs the transpose of what is stored, so the values go through
// LDS as bf16, a wave's own 32 rows, read back by the transposing loads (16
// lanes read 4 rows of 16 channels and get 4 keys of one channel each).
// The maximum is raised only when a score exceeds it by 2^8: until then
// probabilities of up to 2^8 are harmless in fp32 and the rescaling of o (and
// the exchange across lanes that finds the maximum) is left out.
//
// Bound by memory: 64 requests of up to 16384 keys (8 KV heads of 128, 571 MB)
// take 132-147 us on different cards, 3.9-4.3 TB/s; the same loads without any
// arithmetic 114 us.
// 128-key steps with each wave's own 32 keys need no barrier, so loads of the
// next tile fly over all of a tile's work; 3 blocks a CU by registers and LDS (4
// spill: 275 us).
// ---------------------------------------------------------------------------
template <int D>
struct NarrowLds {
  static constexpr int kRow = 2 * D + 32;  // bytes of a V row; +32: 8 consecutive rows hit 8 bank groups
  static constexpr int kWaveBytes = 32 * kRow;
  static constexpr int kOutRow = D + 4;  // floats of an output row in the merge
  static_assert(kNarrowRows * kOutRow * 4 <= kWaveBytes, "merge rows fit the V rows");
};

// Blocks a CU holds by registers (168 for bf16 at D = 128; 4 blocks would spill).
template <int D, bool PRECISE>
constexpr int kNarrowBlocks = D == 256 ? (PRECISE ? 1 : 2) : (PRECISE ? 2 : 3);

// Units from which on whole ones are considered with sinks and more than 64 requests
// (whole_few): one a CU.
constexpr int kWholeFew = kCUs;

template <int D, bool PRECISE, bool SINKS>
__global__ __launch_bounds__(256, (kNarrowBlocks<D, PRECISE>)) void kv_attention_narrow_kernel(AttnArgs a) {
  constexpr int N = PRECISE ? 3 : 1;        // parts of the queries
  constexpr int NP = PRECISE ? 3 : 2;       // parts of the probabilities
  constexpr int NL = D / 64;                 // 16-byte loads a lane makes for 32 rows of codes
  constexpr int NK = D == 64 ? 4 : D / 32;   // query operands
  using L = NarrowLds<D>;
  __shared__ __align__(16) char lds[4 * L::kWaveBytes];
  __shared__ float wave_m[4][kNarrowRows], wave_l[4][kNarrowRows];

  const int tid = threadIdx.x, lane = tid & (kWave - 1), n = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  char* vbuf = lds + wave * L::kWaveBytes;
  const KvCache& kv = a.cache;
  __shared__ Line line;
  const Cut cut{kNarrowRows, kNarrowStep, int(gridDim.x), SINKS ? kWholeFew : 0, SINKS};
  line_build(a, cut, line);
  const bool by_units = SINKS && uniform(int(line.by_units));
  const int even = SINKS ? uniform(line.even) : 0;
  const int64_t total = line_total(line), share = by_units ? 1 : even > 0 ? even : line_share(total, cut.blocks);
  const int64_t begin_pos = share * blockIdx.x;
  const int64_t end_pos = begin_pos + share < total ? begin_pos + share : total;
  if (begin_pos >= end_pos) write_border(a, blockIdx.x, false, Piece{}, share);
  for (int64_t pos = begin_pos; pos < end_pos;) {
    const Piece it = line_find(a, cut, line, pos);
    const int steps = end_pos - pos < it.steps - it.at ? int(end_pos - pos) : it.steps - it.at;
    const bool complete = steps == it.steps;
    const int64_t slot = piece_slot(blockIdx.x, pos == begin_pos);
    if (pos == begin_pos) write_border(a, blockIdx.x, true, it, share);
    pos += even > 0 ? share : steps;  // even shares are of one unit

    const int row = it.tile * kNarrowRows + n;
    const bool live = row < it.r.qn * a.group;
    const int tok = live ? row / a.group : 0, head = it.head * a.group + (live ? row % a.group : 0);

    // operands of the queries
    v8bf q[NK][N];
    {
      const int64_t base = (it.r.q0 + tok) * a.q_token + head * a.q_head;
#pragma unroll
      for (int i = 0; i < NK; ++i) {
        const int chunk = D == 64 ? (g & 1) : 4 * (i >> 2) + g;
        query_operand<N>(a, base + 32 * chunk + 8 * pair_order(i & 3), live, q[i]);
      }
    }
    const float scale2 = a.scale * kLog2e;
    // keys: of the lane's row, of the tile's first and last rows
    int begin, end, lo, hi;
    row_range(a, it.r, tok, begin, end);
    const int first_tok = it.tile * kNarrowRows / a.group;
    int last_row = (it.tile + 1) * kNarrowRows - 1;
    if (last_row >= it.r.qn * a.group) last_row = it.r.qn * a.group - 1;
    const int last_tok = last_row / a.group;
    int full_lo, full_hi;  // keys that every row sees
    row_range(a, it.r, first_tok, lo, full_hi);
    row_range(a, it.r, last_tok, full_lo, hi);
    // from here on positions (keys, without sinks)
    const Places<SINKS, 16> places(a, lo);
    const int chunk0 = it.r.lo + it.at * kNarrowStep;  // whole units: at is 0
    const int64_t stop = by_units ? it.r.kv : int64_t(chunk0) + int64_t(steps) * kNarrowStep;
    if constexpr (SINKS) {
      lo = chunk0;
      hi = places.place(hi) < stop ? places.place(hi) : int(stop);
      begin = places.place(begin);
      end = places.place(end);
      full_lo = places.place(full_lo);
      full_hi = places.place(full_hi);
    } else {
      const int chunk1 = stop < it.r.kv ? int(stop) : it.r.kv;
      lo = lo > chunk0 ? lo : chunk0;
      hi = hi < chunk1 ? hi : chunk1;
      begin = begin > chunk0 ? begin : chunk0;
      end = end < chunk1 ? end : chunk1;
      lo &= ~31;
    }

    v4f o[D / 16];
#pragma unroll
    for (int c = 0; c < D / 16; ++c) o[c] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    float m = -INFINITY, l = 0.0f;

    // Page ids of 32 tiles at a time (two 16-key halves each), one per lane; -1: no key of the half is visible.
    int ids = -1;
    auto load_ids = [&](int j) {
      j += ids_ahead(lane);  // j < hi <= kMostKeys: the sum stays in 32 bits
      ids = -1;
      if (j < hi) {
        ids = a.block_table[it.b * a.table_width + (places.key(j) >> kv.log2_page)];
        if (ids >= kv.pages) ids = -1;
      }
    };
    // A tile's codes and scales; each is loaded for the next tile as soon as
    // the current tile's registers are used up.
    v4u kraw[NL], vraw[NL];
    v4f sk[2], sv[2];
    bool next_seen[2];
    int64_t code_at[2], scale_at[2];  // of the halves' first rows
    const int64_t code_lane = n * kv.code_slot + 16 * (D == 64 ? (g & 1) : g);
    const int64_t scale_lane = 4 * g * kv.scale_slot;
    auto locate = [&](int j, int tile) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int id = __builtin_amdgcn_readlane(ids, 2 * (tile & 31) + h);
        const int slot = places.key(j + 16 * h) & ((1 << kv.log2_page) - 1);
        next_seen[h] = id >= 0;
        const int64_t page = id >= 0 ? id : 0;  // a half without keys reads page 0, unused
        code_at[h] = page * kv.code_page + it.head * kv.code_head + slot * kv.code_slot;
        scale_at[h] = page * kv.scale_page + it.head * kv.scale_head + slot * kv.scale_slot;
      }
    };
    auto load_codes = [&](const uint8_t* codes, v4u(&raw)[NL]) {
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        const int64_t at = D == 64 ? (g >> 1 ? code_at[1] : code_at[0]) : D == 128 ? code_at[i] : code_at[i >> 1];
        raw[i] = *reinterpret_cast<const v4u*>(codes + at + code_lane + (D == 256 ? 64 * (i & 1) : 0));
      }
    };
    auto load_scales = [&](const float* scales, v4f(&to)[2]) {
#pragma unroll
      for (int h = 0; h < 2; ++h) to[h] = scales4(scales + scale_at[h] + scale_lane, kv.scale_slot);
    };

    int j0 = lo + 32 * wave, tile = 0;
    load_ids(j0);
    if (j0 < hi) {
      locate(j0, 0);
      load_codes(kv.k_codes, kraw);
      load_codes(kv.v_codes, vraw);
      load_scales(kv.k_scales, sk);
      load_scales(kv.v_scales, sv);
    }
    for (; j0 < hi; j0 += 128, ++tile) {
      const bool seen[2] = {next_seen[0], next_seen[1]};
      const int jn = j0 + 128;
      const bool more = jn < hi;
      if (more) {
        if (((tile + 1) & 31) == 0) load_ids(jn);
        locate(jn, tile + 1);
      }
      // scores
      v4f sc[2] = {v4f{0.0f, 0.0f, 0.0f, 0.0f}, v4f{0.0f, 0.0f, 0.0f, 0.0f}};
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        const v32bf k32 = open_chunk(kraw[i]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const v8bf k8 = part8(k32, e);
#pragma unroll
          for (int p = 0; p < N; ++p) {
            if constexpr (D == 64) {
              // lane groups 0, 1 hold keys 0-15, groups 2, 3 keys 16-31: the
              // queries are zeroed for the other half
              sc[0] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k8, g < 2 ? q[e][p] : v8bf{}, sc[0], 0, 0, 0);
              sc[1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k8, g < 2 ? v8bf{} : q[e][p], sc[1], 0, 0, 0);
            } else {
              const int h = D == 128 ? i : i >> 1, step = D == 128 ? e : 4 * (i & 1) + e;
              sc[h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k8, q[step][p], sc[h], 0, 0, 0);
            }
          }
        }
      }
      if (more) load_codes(kv.k_codes, kraw);
      // values to LDS
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        const int h = D == 64 ? (g >> 1) : D == 128 ? i : i >> 1;
        const int chunk = D == 64 ? (g & 1) : D == 128 ? g : 4 * (i & 1) + g;
        const v32bf v32 = open_chunk(vraw[i]);
        char* dst = vbuf + (16 * h + n) * L::kRow + 64 * chunk;
#pragma unroll
        for (int e = 0; e < 4; ++e) *reinterpret_cast<v8bf*>(dst + 16 * pair_order(e)) = part8(v32, e);
      }
      if (more) load_codes(kv.v_codes, vraw);
      // softmax
      float x[8];
      const bool whole = seen[0] && seen[1] && (j0 >= full_lo || (SINKS && (full_lo <= a.sinks || j0 + 32 <= a.sinks))) &&
                         j0 + 32 <= full_hi && j0 + 32 <= hi;
      // relative to the running maximum; 0 sk makes NaN of a key whose scale is
      // infinite, which could otherwise have a score of -infinity and be lost
      float ref = m == -INFINITY ? 0.0f : m;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        x[e] = fmaf(sc[e >> 2][e & 3], sk[e >> 2][e & 3] * scale2, fmaf(sk[e >> 2][e & 3], 0.0f, -ref));
      if (more) load_scales(kv.k_scales, sk);
      if (!whole) {
        keep_branch();
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int j = j0 + 16 * (e >> 2) + 4 * g + (e & 3);
          const bool vis = seen[e >> 2] && (j >= begin || (SINKS && j < a.sinks)) && j < end;
          x[e] = vis ? x[e] : -INFINITY;  // probability 0
          sv[e >> 2][e & 3] = vis ? sv[e >> 2][e & 3] : 0.0f;  // whatever lies behind the last key
        }
      }
      float top = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
      const float limit = m == -INFINITY ? -INFINITY : kSlack;
      if (__ballot(top > limit)) {
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        if (top > limit) {  // by rows: a row's results do not depend on its neighbours'
          const float alpha = m == -INFINITY ? 0.0f : exp2f(-top);
          m = ref + top;
          l *= alpha;
#pragma unroll
          for (int c = 0; c < D / 16; ++c) o[c] *= alpha;
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] -= top;
        }
      }
      v8bf pr[NP];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float p = __builtin_amdgcn_exp2f(x[e]);
        l += p;
        __bf16 part[NP];
        split_bf16<NP>(p * sv[e >> 2][e & 3], part);
#pragma unroll
        for (int i = 0; i < NP; ++i) pr[i][e] = part[i];
      }
      if (more) load_scales(kv.v_scales, sv);
      // output: keys of lane group g: 4 g + 0..3 and 16 + 4 g + 0..3
      wave_lds_order();
      const char* vsrc = vbuf + (4 * g + (n >> 2)) * L::kRow + 8 * (n & 3);
#pragma unroll
      for (int c = 0; c < D / 16; ++c) {
        const v8bf vt = lds_transposed(vsrc + 32 * c, vsrc + 32 * c + 16 * L::kRow);
#pragma unroll
        for (int i = 0; i < NP; ++i) o[c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vt, pr[i], o[c], 0, 0, 0);
      }
      wave_lds_order();
    }

    // merge of the 4 waves
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    if (g == 0) {
      wave_m[wave][n] = m;
      wave_l[wave][n] = l;
    }
    __syncthreads();
    {
      const float top = fmaxf(fmaxf(wave_m[0][n], wave_m[1][n]), fmaxf(wave_m[2][n], wave_m[3][n]));
      const float w = m == -INFINITY ? 0.0f : exp2f(m - top);
      float* dst = reinterpret_cast<float*>(vbuf) + n * L::kOutRow + 4 * g;
#pragma unroll
      for (int c = 0; c < D / 16; ++c) *reinterpret_cast<v4f*>(dst + 16 * c) = o[c] * w;
    }
    __syncthreads();
    constexpr int LR = D / 8, PASS = 256 / LR;  // lanes of a row, rows of a pass
#pragma unroll
    for (int r0 = 0; r0 < kNarrowRows; r0 += PASS) {
      const int r = r0 + tid / LR;
      if (r < kNarrowRows) {  // whole waves
        float top = -INFINITY, sum = 0.0f, acc[8] = {};
#pragma unroll
        for (int w = 0; w < 4; ++w) top = fmaxf(top, wave_m[w][r]);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          sum += wave_m[w][r] == -INFINITY ? 0.0f : wave_l[w][r] * exp2f(wave_m[w][r] - top);
          const float* src = reinterpret_cast<const float*>(lds + w * L::kWaveBytes) + r * L::kOutRow + 8 * (tid & (LR - 1));
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[e] += src[e];
        }
        if (complete) {
          finish_row<D>(a, it.r.q0, it.r.qn, it.head, it.tile * kNarrowRows + r, acc, top, sum, lane);
        } else {
          float* part = partials(a) + slot * (kNarrowRows * (D + 2));
          store_row8(part, false, r * D + 8 * (tid & (LR - 1)), acc);
          if ((tid & (LR - 1)) == 0) {
            part[kNarrowRows * D + r] = top;
            part[kNarrowRows * (D + 1) + r] = sum;
          }
        }
      }
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// Many query rows (prompts, chunks): 32 rows for each of a block's 4 waves,
// 64 keys a step.  The block opens a step's codes once, into two LDS buffers
// (rows of bf16 codes, keys and values alike, and the keys' scales, sk already
// times scale log2(e)), while it computes on the step before; one barrier a
// step.  The products are those of the narrow kernel in 32 x 32 tiles: S^T =
// K Q^T leaves a query row in lanes n and n + 32, keys 8 b + 4 h + i in
// registers (h the lane's half), which is the column operand of O^T = V^T P^T
// with keys ordered (16 b + 4 h + 0..3, 16 b + 8 + 4 h + 0..3) per half.
//
// Bound by the softmax's vector work beside the products (a step of 32 x 64
// scores at D = 128: 32 products of 32 cycles, 32 exponentials of 16 and about
// 200 other vector instructions of 4) and by the start and end of units: 4
// prompts of 1500-2048 tokens (32 heads of 128) 154 us, 668 TFLOP/s of what is
// visible; at D = 64, 6 chunks on up to 12000 keys, 73 us, 424 TFLOP/s (3 blocks a
// CU spill 35 registers, hardly in the loop; 2, without, 91 us where 3 take 85).  64
// rows a wave (1 wave a SIMD) took 287 us where this took 205; blocks of 8 waves
// whose halves take turns at products and softmax 157 us against 154, as one
// block a CU leaves the starts and ends of its units uncovered.
// ---------------------------------------------------------------------------
typedef float v16f __attribute__((ext_vector_type(16)));

// Blocks of the grid for each CU, and with how many units whole ones are taken.
template <int D, bool PRECISE>
constexpr int kWideBlocks = (D == 256 || PRECISE) ? 1 : D == 64 ? 3 : 2;
template <int D, bool PRECISE>
constexpr int kWhole = 2 * kCUs * kWideBlocks<D, PRECISE>;

template <int D>
struct WideLds {
  // Keys: rows of 2 D + 16 bytes, so that 16 lanes reading 16 bytes of 16 rows
  // hit every bank once, like 16 lanes writing 4 chunks of 4 rows (2 of 8).
  static constexpr int kKeyRow = 2 * D + 16;
  // Values: rows of 2 D bytes, their 16-byte units exchanged by a swizzle of
  // the row, for the same of 32 lanes reading 64 bytes of 4 rows.
  static constexpr int kValueRow = 2 * D;
  static constexpr int kValues = kWideStep * kKeyRow;  // where the values start
  static constexpr int kBuffer = kValues + kWideStep * kValueRow;
  static constexpr int kBytes = 2 * kBuffer;
  __device__ static constexpr int swizzle(int row) {
    return D == 64 ? ((row >> 1) & 3) + 4 * ((row >> 1) & 1) : 5 * (row & 3);
  }
};

// Exchanges the upper 32 lanes of a with the lower 32 lanes of b.
__device__ __forceinline__ void swap_halves(uint32_t& a, uint32_t& b) {
  const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}
__device__ __forceinline__ void swap_halves(float& a, float& b) {
  uint32_t x = __float_as_uint(a), y = __float_as_uint(b);
  swap_halves(x, y);
  a = __uint_as_float(x);
  b = __uint_as_float(y);
}

// y H_D of rows in the layout of the wide kernel's output (channel 32 c + 8 b +
// 4 h + i: c, b, i in registers, h the lane's half): all butterflies but the
// one over h are between registers; that one works on two registers at a time,
// whose halves are exchanged before and after it.
template <int D>
__device__ __forceinline__ void wide_hadamard(v16f (&o)[D / 32]) {
#pragma unroll
  for (int c = 0; c < D / 32; ++c) {
#pragma unroll
    for (int st = 1; st < 16; st <<= 1) {
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        if ((e & st) == 0) {
          const float x = o[c][e], y = o[c][e | st];
          o[c][e] = x + y;
          o[c][e | st] = x - y;
        }
      }
    }
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
      float x = o[c][e], y = o[c][e + 1];
      swap_halves(x, y);
      float u = x + y, v = x - y;
      swap_halves(u, v);
      o[c][e] = u;
      o[c][e + 1] = v;
    }
  }
#pragma unroll
  for (int st = 1; st < D / 32; st <<= 1) {
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
      if ((c & st) == 0) {
        const v16f x = o[c], y = o[c | st];
        o[c] = x + y;
        o[c | st] = x - y;
      }
    }
  }
}

// The rows of that layout, rounded and stored 16 bytes a lane: bf16 pairs of
// blocks b and b + 1 are exchanged between the halves, so that a lane holds 8
// consecutive channels.
template <int D, class It>
__device__ __forceinline__ void wide_store(const AttnArgs& a, const It& it, const v16f (&o)[D / 32], int row, bool live,
                                           int h) {
  const int tok = row / a.group;
  const int64_t at = (it.r.q0 + tok) * a.out_token + (it.head * a.group + row - tok * a.group) * a.out_head;
#pragma unroll
  for (int c = 0; c < D / 32; ++c) {
    if (a.out_bf16) {
#pragma unroll
      for (int b = 0; b < 4; b += 2) {
        v8bf p;
#pragma unroll
        for (int e = 0; e < 8; ++e) p[e] = static_cast<__bf16>(o[c][4 * b + e]);  // round to nearest even
        v4u w = __builtin_bit_cast(v4u, p);
        uint32_t w0 = w[0], w1 = w[1], w2 = w[2], w3 = w[3];
        swap_halves(w0, w2);
        swap_halves(w1, w3);
        if (live)
          *reinterpret_cast<v4u*>(reinterpret_cast<__bf16*>(a.out) + at + 32 * c + 8 * (b + h)) = v4u{w0, w1, w2, w3};
      }
    } else if (live) {
#pragma unroll
      for (int b = 0; b < 4; ++b)
        *reinterpret_cast<v4f*>(reinterpret_cast<float*>(a.out) + at + 32 * c + 8 * b + 4 * h) =
            v4f{o[c][4 * b], o[c][4 * b + 1], o[c][4 * b + 2], o[c][4 * b + 3]};
    }
  }
}

// The keys (positions, with sinks) of a piece that any of the unit's rows sees, [lo, hi)
// with lo on a step, what the rows of a wave (32 from row0) see, and what all of them see.
struct Reach {
  int lo, hi, wave_hi, full_lo, full_hi;
};
// Also cuts the lane's own [begin, end) to the piece (makes them positions).
template <bool SINKS>
__device__ __forceinline__ Reach wide_reach(const AttnArgs& a, const Piece& it, bool by_units, int steps, int row0, int& begin,
                                            int& end, Places<SINKS, 1>& places) {
  const int rows = it.r.qn * a.group;
  Reach u{0, 0, 0, 0, 0};
  int skip;
  const int last = (it.tile + 1) * kWideRows < rows ? (it.tile + 1) * kWideRows - 1 : rows - 1;
  row_range(a, it.r, it.tile * kWideRows / a.group, u.lo, skip);
  row_range(a, it.r, last / a.group, skip, u.hi);
  if (row0 < rows) {
    const int wave_last = row0 + 32 < rows ? row0 + 31 : rows - 1;
    row_range(a, it.r, row0 / a.group, skip, u.full_hi);
    row_range(a, it.r, wave_last / a.group, u.full_lo, u.wave_hi);
  }
  const int chunk0 = it.r.lo + (by_units ? 0 : it.at * kWideStep);
  const int64_t stop = by_units ? it.r.kv : int64_t(chunk0) + int64_t(steps) * kWideStep;
  if constexpr (SINKS) {
    places = Places<SINKS, 1>(a, u.lo);
    u.lo = chunk0;
    u.hi = places.place(u.hi) < stop ? places.place(u.hi) : int(stop);
    u.wave_hi = row0 < rows ? places.place(u.wave_hi) : 0;
    u.full_lo = places.place(u.full_lo);
    u.full_hi = places.place(u.full_hi);
    begin = places.place(begin);
    end = places.place(end);
    return u;
  }
  const int chunk1 = stop < it.r.kv ? int(stop) : it.r.kv;
  u.lo = u.lo > chunk0 ? u.lo : chunk0;
  u.hi = u.hi < chunk1 ? u.hi : chunk1;
  u.wave_hi = u.wave_hi < chunk1 ? u.wave_hi : chunk1;
  u.full_hi = u.full_hi < chunk1 ? u.full_hi : chunk1;
  u.lo = chunk0 + ((u.lo - chunk0) & ~(kWideStep - 1));
  begin = begin > chunk0 ? begin : chunk0;
  end = end < chunk1 ? end : chunk1;
  return u;
}

// o 2^unit.
template <int D>
__device__ __forceinline__ void wide_unit(v16f (&o)[D / 32], int unit) {
#pragma unroll
  for (int c = 0; c < D / 32; ++c)
#pragma unroll
    for (int e = 0; e < 16; ++e) o[c][e] = ldexpf(o[c][e], unit);
}

// A wave's rows after their last key: lane n, h holds channels 32 c + 8 b + 4 h
// + i of row n.  Written out, or left in the workspace for the combine kernel.
template <int D, bool HALF>
__device__ __forceinline__ void wide_finish(const AttnArgs& a, const Piece& it, v16f (&o)[D / 32], float m, float l,
                                            int unit, bool complete, int64_t slot, int wave, int n, int h) {
  l += __shfl_xor(l, 32);
  const int at = wave * 32 + n, row = it.tile * kWideRows + at, rows = it.r.qn * a.group;
  if (complete) {
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
    for (int c = 0; c < D / 32; ++c) o[c] *= a.unrotate ? inv * kHeadPost<D> : inv;
    if constexpr (HALF) wide_unit<D>(o, unit);
    if (a.unrotate) wide_hadamard<D>(o);
    wide_store<D>(a, it, o, row, row < rows, h);
    if (a.lse && h == 0 && row < rows)
      a.lse[(it.r.q0 + row / a.group) * int64_t(a.heads) + it.head * a.group + row % a.group] =
          l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
  } else if (row < rows) {
    if constexpr (HALF) wide_unit<D>(o, unit);
    float* part = partials(a) + slot * (kWideRows * (D + 2));
#pragma unroll
    for (int c = 0; c < D / 32; ++c)
#pragma unroll
      for (int b = 0; b < 4; ++b)
        *reinterpret_cast<v4f*>(part + at * D + 32 * c + 8 * b + 4 * h) =
            v4f{o[c][4 * b], o[c][4 * b + 1], o[c][4 * b + 2], o[c][4 * b + 3]};
    if (h == 0) {
      part[kWideRows * D + at] = m;
      part[kWideRows * (D + 1) + at] = l;
    }
  }
}

// ---------------------------------------------------------------------------
// Weights of the kernel for many rows.  Where queries and output are bf16, a
// probability times its value's scale, w = p sv, enters the product as one fp16
// number: half a step is 2^-11, an eighth of the output's.  (One bf16 part, 2^-8,
// makes the output's error 1.4 times as large as its own rounding; two take a
// quarter more time, 182 us for 147 on the prompt case, where fp16 takes 152.)
//   fp16 has 11 bits from 2^-14 to 2^16 and loses at most 2^-25 of what is smaller,
// so a piece's scales are multiplied by a power of two, which is exact: 2^-unit puts
// the largest of its first step into [2^5, 2^6).  If all of the piece's n keys then
// have a scale in [max(n 2^-16, 2^-14), 2^8), no weight passes 2^15 (p <=
// 2^kHalfSlack), each row has one of that much or more (its largest p is at least
// 1), and what n keys lose, 2^-25 each, is at most 2^-9 of it, and that only if all
// others lie below fp16's normal range.  At the first step with a key outside of the
// range (a value of zeros, say) the piece starts again with weights of two bf16
// parts, which need none; a prompt of such keys alone takes 194 us.
// ---------------------------------------------------------------------------
struct Unit {
  int exp;
  float least;  // n 2^-16, 2^-14 at least
};

// The largest v >= 0 of a wave's lanes.
__device__ __forceinline__ float wave_max(float v) {
  for (int d = 1; d < kWave; d <<= 1) v = fmaxf(v, __shfl_xor(v, d));
  return v;
}

// The power of two of a piece whose first step has this scale in the lane (0: none).
__device__ __forceinline__ int unit_exponent(float sv) {
  const float most = wave_max(fabsf(sv));
  return most > 0.0f ? uniform(__builtin_amdgcn_frexp_expf(most)) - 6 : 0;
}

// Products whose operands are read from LDS kAhead ahead (left to itself the
// compiler reads each right before its product); `meanwhile` is work in the
// shadow of the matrix unit.  The wave goes first meanwhile, so that the
// others of its SIMD do their softmax behind its products and not beside its.
constexpr int kAhead = 4;
template <int COUNT, class Load, class Product, class Meanwhile>
__device__ __forceinline__ void products(Load load, Product product, Meanwhile meanwhile) {
  v8bf operand[kAhead];
  __builtin_amdgcn_s_setprio(1);
#pragma unroll
  for (int at = 0; at < kAhead; ++at) operand[at] = load(at);
#pragma unroll
  for (int at = 0; at < COUNT; ++at) {
    __builtin_amdgcn_sched_barrier(0);
    product(at, operand[at % kAhead]);
    if (at + kAhead < COUNT) operand[at % kAhead] = load(at + kAhead);
    meanwhile(at);
  }
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_setprio(0);
}

template <int D, bool PRECISE, bool SINKS>
__global__ __launch_bounds__(256, (kWideBlocks<D, PRECISE>)) void kv_attention_wide_kernel(AttnArgs a, int blocks) {
  constexpr int N = PRECISE ? 3 : 1;                  // parts of the queries
  constexpr int NP = PRECISE ? 3 : 2;                 // bf16 parts of the weights
  constexpr int CH = D / 32;                          // chunks of a row
  constexpr int NS = (2 * kWideStep * CH) / 256;      // chunks a thread opens a step (1: keys or values)
  constexpr int NH = NS > 1 ? NS / 2 : 1;             // of one kind
  constexpr int kPer = D == 64 ? 2 : 1;               // scales read a product
  using L = WideLds<D>;
  extern __shared__ __align__(16) char lds[];
  __shared__ float scale_s[2][2][kWideStep];
  __shared__ int unit_s;                // the piece's power of two
  __shared__ int seen_s[2][kWideStep];  // bit 0: the key is visible; bit 1: fp16 weights do not do for the piece
  __shared__ Line line;

  const KvCache& kv = a.cache;
  const Cut cut{kWideRows, kWideStep, blocks, kWhole<D, PRECISE>};
  line_build(a, cut, line);
  const int64_t total = line_total(line);
  const bool by_units = uniform(int(line.by_units));
  const int64_t share = by_units ? 1 : line_share(total, cut.blocks);
  const int64_t begin_pos = share * blockIdx.x;
  const int64_t end_pos = begin_pos + share < total ? begin_pos + share : total;
  if (begin_pos >= end_pos && int(blockIdx.x) < cut.blocks) write_border(a, blockIdx.x, false, Piece{}, share);
  // The piece at pos, with weights in fp16 (false: they do not do for it) or in NP
  // bf16 parts; moves pos on.
  auto run = [&](auto half_weights, int64_t& pos) {
    constexpr bool HALF = decltype(half_weights)::value;
    // lane numbers of its own for each form, or the compiler computes both forms'
    // addresses ahead of the loop over pieces and spills them
    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));
    const int lane = tid & (kWave - 1), n = lane & 31, h = lane >> 5;
    const int wave = uniform(tid / kWave);
    const Piece it = line_find(a, cut, line, pos);
    const int steps = end_pos - pos < it.steps - it.at ? int(end_pos - pos) : it.steps - it.at;
    const bool complete = steps == it.steps;
    const int64_t slot = piece_slot(blockIdx.x, pos == begin_pos);
    if (pos == begin_pos && int(blockIdx.x) < cut.blocks) write_border(a, blockIdx.x, true, it, share);

    const int rows = it.r.qn * a.group, row0 = it.tile * kWideRows + wave * 32;
    v8bf q[D / 16][N];
    int begin, end;
    {
      const int row = row0 + n;
      const bool live = row < rows;
      const int tok = live ? row / a.group : 0, head = it.head * a.group + (live ? row % a.group : 0);
      const int64_t base = (it.r.q0 + tok) * a.q_token + head * a.q_head;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) query_operand<N>(a, base + 16 * i + 8 * h, live, q[i]);
      row_range(a, it.r, tok, begin, end);
    }
    Places<SINKS, 1> places(a, 0);
    const Reach reach = wide_reach<SINKS>(a, it, by_units, steps, row0, begin, end, places);
    const int lo = reach.lo, hi = reach.hi, wave_hi = reach.wave_hi;

    // staging: the thread's chunks of a step (row my_row + i * rows_apart, chunk my_chunk)
    constexpr int kApart = 256 / CH;
    const bool half_v = NS == 1 && wave >= 2;  // D = 64: one half of the threads takes keys, the other values
    const int my_row = NS == 1 ? (tid & 127) / CH : tid / CH, my_chunk = tid % CH;
    const float scale2 = a.scale * kLog2e;
    // page ids as they are read, checked where they are used: a check here would wait for them
    const uint32_t pages = kv.pages < 0x7FFFFFFF ? uint32_t(kv.pages) : 0x7FFFFFFFu;
    const int* table = a.block_table + it.b * a.table_width;
    int ids[NH], scale_id = 0;
    auto load_ids = [&](int j0) {
#pragma unroll
      for (int i = 0; i < NH; ++i) {
        const int j = j0 + my_row + i * kApart;
        ids[i] = table[places.key(j < hi ? j : hi - 1) >> kv.log2_page];
      }
      if (tid < kWideStep) scale_id = table[places.key(j0 + tid < hi ? j0 + tid : hi - 1) >> kv.log2_page];
    };
    v4u raw[NS];
    float scales[2];
    int seen = 0;
    const int64_t head_codes = it.head * kv.code_head, head_scales = it.head * kv.scale_head;
    auto load_step = [&](int j0) {
#pragma unroll
      for (int i = 0; i < NH; ++i) {
        const int j = places.key(j0 + my_row + i * kApart), at = j & ((1 << kv.log2_page) - 1);
        const int64_t off = head_codes + row_at(uint32_t(ids[i]) < pages ? ids[i] : 0, kv.code_page, at, kv.code_slot) + 16 * my_chunk;
        if constexpr (NS == 1) {
          raw[0] = *reinterpret_cast<const v4u*>((half_v ? kv.v_codes : kv.k_codes) + off);
        } else {
          raw[i] = *reinterpret_cast<const v4u*>(kv.k_codes + off);
          raw[NH + i] = *reinterpret_cast<const v4u*>(kv.v_codes + off);
        }
      }
      if (tid < kWideStep) {  // the keys' scales, from the first wave
        const int at = places.key(j0 + tid) & ((1 << kv.log2_page) - 1);
        const bool known = uint32_t(scale_id) < pages;
        seen = known && j0 + tid < hi;
        const int64_t off = head_scales + row_at(known ? scale_id : 0, kv.scale_page, at, kv.scale_slot);
        scales[0] = kv.k_scales[off];
        scales[1] = kv.v_scales[off];
      }
    };
    v16f o[D / 32];
#pragma unroll
    for (int c = 0; c < D / 32; ++c) o[c] = v16f{};
    float m = -INFINITY, l = 0.0f;

    Unit unit{0, fmaxf(float(hi - lo) * 0x1p-16f, 0x1p-14f)};
    auto store_step = [&](int buf, bool first) {
      char* base = lds + buf * L::kBuffer;
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        const bool v = NS == 1 ? half_v : i >= NH;
        const int row = my_row + (i % NH) * kApart;
        char* dst = base + (v ? L::kValues + row * L::kValueRow : row * L::kKeyRow);
        const int mix = v ? L::swizzle(row) : 0;
        auto store_chunk = [&](const auto& x) {
#pragma unroll
          for (int e = 0; e < 4; ++e) *reinterpret_cast<v8bf*>(dst + 16 * ((4 * my_chunk + pair_order(e)) ^ mix)) = part8(x, e);
        };
        if (HALF && v) store_chunk(open_chunk_half(raw[i]));
        else store_chunk(open_chunk(raw[i]));
      }
      if (tid < kWideStep) {
        // a scale that is not finite makes the key's score NaN (an infinite one
        // could otherwise make it -infinity, and the key would be lost); that of a
        // value is itself kept from the rows that do not see the key
        const bool fine = fabsf(scales[0]) < __builtin_huge_valf() && fabsf(scales[1]) < __builtin_huge_valf();
        scale_s[buf][0][tid] = fine ? scales[0] * scale2 : __builtin_nanf("");
        float sv = fine ? scales[1] : 0.0f;
        int word = seen;
        if constexpr (HALF) {
          if (first) {
            unit.exp = unit_exponent(seen ? sv : 0.0f);
            if (tid == 0) unit_s = unit.exp;
          }
          sv = seen ? ldexpf(sv, -unit.exp) : 0.0f;
          if (__ballot(seen && fine && !(fabsf(sv) >= unit.least && fabsf(sv) < 0x1p8f))) word |= 2;
        }
        scale_s[buf][1][tid] = sv;
        seen_s[buf][tid] = word;
      }
    };

    if (lo < hi) {
      load_ids(lo);
      load_step(lo);
      load_ids(lo + kWideStep);
      store_step(0, true);
    }
    int buf = 0;
    for (int j0 = lo; j0 < hi; j0 += kWideStep, buf ^= 1) {
      __syncthreads();
      const bool more = j0 + kWideStep < hi;
      if (more) {
        load_step(j0 + kWideStep);
        load_ids(j0 + 2 * kWideStep);
      }
      const int word = seen_s[buf][lane];
      if (j0 < wave_hi) {
        const char* kbase = lds + buf * L::kBuffer;
        const char* vbase = kbase + L::kValues;
        const uint64_t vis = __ballot((word & 1) != 0);
        const bool whole = vis == ~uint64_t(0) &&
                           (j0 >= reach.full_lo || (SINKS && (reach.full_lo <= a.sinks || j0 + kWideStep <= a.sinks))) &&
                           j0 + kWideStep <= reach.full_hi;
        // scores of the step's two 32-key halves
        v16f x[2] = {v16f{}, v16f{}};
        const char* krow = kbase + n * L::kKeyRow + 16 * h;
        v4f scale[8];
        products<D / 8>(
            [&](int at) { return *reinterpret_cast<const v8bf*>(krow + 32 * (at & 1) * L::kKeyRow + 32 * (at >> 1)); },
            [&](int at, const v8bf& k8) {
#pragma unroll
              for (int p = 0; p < N; ++p)
                x[at & 1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k8, q[at >> 1][p], x[at & 1], 0, 0, 0);
            },
            [&](int at) {  // the keys' scales
              if (at >= D / 8 - 8 / kPer) {
#pragma unroll
                for (int e = 0; e < kPer; ++e) {
                  const int k = (at - (D / 8 - 8 / kPer)) * kPer + e;
                  scale[k] = *reinterpret_cast<const v4f*>(&scale_s[buf][0][8 * k + 4 * h]);
                }
              }
            });
        const float ref = m == -INFINITY ? 0.0f : m;
#pragma unroll
        for (int e = 0; e < 32; ++e) x[e >> 4][e & 15] = fmaf(x[e >> 4][e & 15], scale[e >> 2][e & 3], -ref);
        // the values' scales
#pragma unroll
        for (int e = 0; e < 8; ++e) scale[e] = *reinterpret_cast<const v4f*>(&scale_s[buf][1][8 * e + 4 * h]);
        __builtin_amdgcn_sched_barrier(0);
        if (!whole) {
          keep_branch();
#pragma unroll
          for (int kb = 0; kb < 2; ++kb) {
            // bit 8 b + i: key 32 kb + 8 b + 4 h + i of the step
            const int j = j0 + 32 * kb + 4 * h;
            uint32_t bits = ~bits_below(begin - j);
            if constexpr (SINKS) bits |= bits_below(a.sinks - j);
            bits &= (uint32_t(vis >> (32 * kb)) >> (4 * h)) & bits_below(end - j);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const bool on = bits & (1u << (8 * (e >> 2) + (e & 3)));
              x[kb][e] = on ? x[kb][e] : -INFINITY;  // probability 0
            }
          }
        }
        float top = x[0][0];
#pragma unroll
        for (int e = 1; e < 32; ++e) top = fmaxf(top, x[e >> 4][e & 15]);
        const float limit = m == -INFINITY ? -INFINITY : HALF ? kHalfSlack : kSlack;
        if (__ballot(top > limit)) {
          top = fmaxf(top, __shfl_xor(top, 32));
          if (top > limit) {
            const float alpha = m == -INFINITY ? 0.0f : exp2f(-top);
            m = ref + top;
            l *= alpha;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) o[c] *= alpha;
#pragma unroll
            for (int e = 0; e < 32; ++e) x[e >> 4][e & 15] -= top;
          }
        }
        v8bf pr[4][NP];
        v8h half[4];
        auto probability = [&](int e) {
          const float p = __builtin_amdgcn_exp2f(x[e >> 4][e & 15]);
          l += p;
          if constexpr (HALF) {
            half[e >> 3][e & 7] = static_cast<_Float16>(p * scale[e >> 2][e & 3]);  // round to nearest even
          } else {
            __bf16 part[NP];
            split_bf16<NP>(p * scale[e >> 2][e & 3], part);
#pragma unroll
            for (int i = 0; i < NP; ++i) pr[e >> 3][i][e & 7] = part[i];
          }
        };
#pragma unroll
        for (int e = 0; e < 16; ++e) probability(e);
        // values: 8 bytes of row 32 kb + 16 b + 4 h + (l % 16) / 4 (and 8 rows on), 32-channel tile c
        const int vr = 4 * h + ((lane & 15) >> 2), vu = 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
        const char* vrow = vbase + vr * L::kValueRow + 8 * (lane & 1);
        products<4 * CH>(
            [&](int at) {
              const char* v0 = vrow + 16 * (at / CH) * L::kValueRow + 16 * ((4 * (at % CH) + vu) ^ L::swizzle(vr));
              return lds_transposed(v0, v0 + 8 * L::kValueRow);
            },
            [&](int at, const v8bf& v8) {
              if constexpr (HALF) {
                o[at % CH] = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(v8h, v8), half[at / CH], o[at % CH],
                                                                    0, 0, 0);
              } else {
#pragma unroll
                for (int i = 0; i < NP; ++i)
                  o[at % CH] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v8, pr[at / CH][i], o[at % CH], 0, 0, 0);
              }
            },
            [&](int at) {  // the second half's probabilities
              if (at < 2 * CH) {
#pragma unroll
                for (int e = 0; e < 8 / CH; ++e) probability(16 + at * (8 / CH) + e);
              }
            });
      }
      if (HALF && (uniform(word) & 2)) return false;
      if (more) store_step(buf ^ 1, false);
    }

    wide_finish<D, HALF>(a, it, o, m, l, HALF ? unit_s : 0, complete, slot, wave, n, h);
    pos += steps;
    return true;
  };
  bool half = true;
  for (int64_t pos = begin_pos; pos < end_pos;) {
    if constexpr (PRECISE) {
      run(std::false_type{}, pos);
    } else if (half) {
      half = run(std::true_type{}, pos);
    } else {
      run(std::false_type{}, pos);
      half = true;
    }
    __syncthreads();  // the buffers are free for the next piece
  }
}

// ---------------------------------------------------------------------------
// The pieces of cut units put together.  Block (w, part) looks at the border
// between blocks w - 1 and w of the attention's grid: if that is the first
// border inside a unit (block w wrote down what it found), it merges rows of
// that unit, D / 8 lanes a row, eight pieces in flight.  SPLIT (few rows, many
// pieces): the 4 waves take every fourth piece of the same rows and merge
// through LDS; otherwise each wave has rows of its own.
// ---------------------------------------------------------------------------
template <int D, bool SPLIT>
__global__ __launch_bounds__(256) void kv_attention_combine_kernel(AttnArgs a, int rows, int parts) {
  constexpr int LR = D / 8, R = kWave / LR;
  __shared__ float acc_s[4][kWave][9];
  __shared__ float m_s[4][R], l_s[4][R];
  const int tid = threadIdx.x, lane = tid & (kWave - 1), l8 = lane & (LR - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int w = 1 + blockIdx.x / parts;
  const Border* d = borders(a) + w;
  const int pieces = uniform(d->pieces);
  if (pieces == 0) return;
  const int tile = uniform(d->tile), q0 = uniform(d->q0), qn = uniform(d->qn), head = uniform(d->head);
  const int part = blockIdx.x % parts;
  for (int r0 = (SPLIT ? part : part * 4 + wave) * R; r0 < rows; r0 += (SPLIT ? parts : 4 * parts) * R) {
    const int r = r0 + lane / LR;
    if (tile * rows + r0 >= qn * a.group) return;  // the whole block or (not SPLIT) wave
    const int size = rows * (D + 2);
    const float* head_part = partials(a) + int64_t(uniform(d->first)) * size;
    const float* rest = partials(a) + int64_t(piece_slot(w, true)) * size;
    float m = -INFINITY, l = 0.0f, acc[8] = {};
    constexpr int kNext = SPLIT ? 4 : 1;
    for (int c0 = SPLIT ? wave : 0; c0 < pieces; c0 += 8 * kNext) {
      float mc[8], lc[8], v[8][8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = c0 + kNext * i;
        if (c < pieces) {  // uniform
          const float* part = c == 0 ? head_part : rest + int64_t(c - 1) * (2 * size);
          mc[i] = part[rows * D + r];
          lc[i] = part[rows * (D + 1) + r];
          RowSrc<false>{part, 0}.load8(0, r * D + 8 * l8, v[i]);
        }
      }
      float top = m;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c0 + kNext * i < pieces) top = fmaxf(top, mc[i]);
      const float keep = m == -INFINITY ? 0.0f : exp2f(m - top);
      m = top;
      l *= keep;
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] *= keep;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (c0 + kNext * i < pieces) {
          const float x = mc[i] == -INFINITY ? 0.0f : exp2f(mc[i] - m);
          l = fmaf(lc[i], x, l);
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[e] = fmaf(v[i][e], x, acc[e]);
        }
      }
    }
    if constexpr (!SPLIT) {
      finish_row<D>(a, q0, qn, head, tile * rows + r, acc, m, l, lane);
      continue;
    }
    if (l8 == 0) {
      m_s[wave][lane / LR] = m;
      l_s[wave][lane / LR] = l;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) acc_s[wave][lane][e] = acc[e];
    __syncthreads();
    if (wave == 0) {
      float top = m, sum = 0.0f, o[8] = {};
#pragma unroll
      for (int i = 1; i < 4; ++i) top = fmaxf(top, m_s[i][lane / LR]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float mi = m_s[i][lane / LR], x = mi == -INFINITY ? 0.0f : exp2f(mi - top);
        sum = fmaf(l_s[i][lane / LR], x, sum);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = fmaf(acc_s[i][lane][e], x, o[e]);
      }
      finish_row<D>(a, q0, qn, head, tile * rows + r, o, top, sum, lane);
    }
    __syncthreads();
  }
}

constexpr int most_of(int a, int b) { return a > b ? a : b; }

// Units and steps a call can have at most, as far as the host knows.
int64_t units_max(const AttnArgs& a, int rows) {
  return a.cache.heads * (a.T * a.group / rows + (a.B < a.T ? a.B : a.T));
}
int64_t steps_max(const AttnArgs& a, int rows, int step) {
  const int64_t units = units_max(a, rows);
  const int64_t room = a.table_width << a.cache.log2_page, steps = room > step ? (room + step - 1) / step : 1;
  return units > (int64_t(1) << 40) / steps ? int64_t(1) << 40 : units * steps;
}

template <int D, bool SPLIT>
hipError_t launch_combine(const AttnArgs& a, int rows, int step, int blocks, int64_t whole, hipStream_t st) {
  if (blocks < 2 || (a.table_width << a.cache.log2_page) <= step) return hipSuccess;  // no unit can be cut
  // blocks for the rows that max_q_len lets expect (they go on to the others if it is wrong)
  constexpr int kBlockRows = kWave / (D / 8) * (SPLIT ? 1 : 4);
  const int64_t live = a.max_q_len < rows ? a.max_q_len * a.group : rows;
  // With `whole` units or more (0: never) none is cut, which the device lengths
  // decide; if the tokens are enough for that, blocks are left to find nothing.
  const bool few = whole > 0 && a.cache.heads * (a.T * a.group / rows) >= whole;
  const int parts = few ? 1 : int((live < 1 ? 1 : live < rows ? live : rows) + kBlockRows - 1) / kBlockRows;
  hipLaunchKernelGGL((kv_attention_combine_kernel<D, SPLIT>), dim3((blocks - 1) * parts), dim3(256), 0, st, a, rows,
                     parts);
  return hipGetLastError();
}

template <int D, bool PRECISE>
hipError_t launch_narrow(const AttnArgs& a, hipStream_t st) {
  const int64_t most = steps_max(a, kNarrowRows, kNarrowStep);
  static_assert(kNarrowBlocks<D, PRECISE> <= kNarrowBlocksMost, "borders and partial results have no room");
  const int full = kCUs * kNarrowBlocks<D, PRECISE>;
  const int blocks = most < full ? int(most) : full;
  if (a.sinks > 0)
    hipLaunchKernelGGL((kv_attention_narrow_kernel<D, PRECISE, true>), dim3(blocks), dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL((kv_attention_narrow_kernel<D, PRECISE, false>), dim3(blocks), dim3(256), 0, st, a);
  const hipError_t e = hipGetLastError();
  return e != hipSuccess ? e : launch_combine<D, true>(a, kNarrowRows, kNarrowStep, blocks, 0, st);
}

template <int D, bool PRECISE>
hipError_t launch_wide(const AttnArgs& a, hipStream_t st) {
  const int64_t most = steps_max(a, kWideRows, kWideStep), units = units_max(a, kWideRows);
  static_assert(kWideBlocks<D, PRECISE> <= kWideBlocksMost, "borders and partial results have no room");
  const int full = kCUs * kWideBlocks<D, PRECISE>;
  const int blocks = most < full ? int(most) : full;
  const auto kernel = a.sinks > 0 ? kv_attention_wide_kernel<D, PRECISE, true> : kv_attention_wide_kernel<D, PRECISE, false>;
  const hipError_t set = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, WideLds<D>::kBytes);
  if (set != hipSuccess) return set;
  hipLaunchKernelGGL(kernel, dim3(unsigned(wide_grid(units, blocks))), dim3(256), WideLds<D>::kBytes, st, a,
                     blocks);
  const hipError_t e = hipGetLastError();
  return e != hipSuccess ? e : launch_combine<D, false>(a, kWideRows, kWideStep, blocks, kWhole<D, PRECISE>, st);
}

template <int D>
hipError_t launch_head(const AttnArgs& a, hipStream_t st) {
  const bool precise = !(a.q_bf16 && a.out_bf16);
  const int64_t most = a.max_q_len < a.T ? a.max_q_len : a.T;
  const int64_t rows = most * a.group;
  if (precise) return rows <= kNarrowMost<D, true> ? launch_narrow<D, true>(a, st) : launch_wide<D, true>(a, st);
  return rows <= kNarrowMost<D, false> ? launch_narrow<D, false>(a, st) : launch_wide<D, false>(a, st);
}

}  // namespace

namespace {

// Borders, and two partial results for each block of the largest grid that such a
// call can get: launch_head takes the kernel for few rows whatever the types where a
// call has that few.
template <int D>
int64_t workspace_bytes(int64_t rows) {
  const int64_t narrow = int64_t(kCUs) * most_of(kNarrowBlocks<D, false>, kNarrowBlocks<D, true>) * kNarrowRows;
  const int64_t wide = int64_t(kCUs) * most_of(kWideBlocks<D, false>, kWideBlocks<D, true>) * kWideRows;
  const bool few = rows <= kNarrowMost<D, false> && rows <= kNarrowMost<D, true>;
  return kMaxBlocks * int64_t(sizeof(Border)) +
         2 * (few || narrow > wide ? narrow : wide) * (D + 2) * int64_t(sizeof(float));
}

}  // namespace

int64_t kv_attention_workspace_bytes(int64_t T, int64_t heads, int64_t kv_heads, int64_t head_dim) {
  const int64_t rows = T * (heads / kv_heads);
  return head_dim == 64 ? workspace_bytes<64>(rows) : head_dim == 128 ? workspace_bytes<128>(rows) : workspace_bytes<256>(rows);
}

hipError_t launch_kv_attention(const AttnArgs& a, hipStream_t st) {
  switch (a.head_dim) {
    case 64: return launch_head<64>(a, st);
    case 128: return launch_head<128>(a, st);
    default: return launch_head<256>(a, st);
  }
}

}  // namespace rw4
