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
// exact up to the fp32 accumulation; probabilities enter the second product
// as bf16 (bf16 output) or as three bf16 parts (fp32 output, PRECISE, where
// fp32 queries are split the same way).
//
// Work.  A unit is a tile of query rows (row = query token x query head of one
// KV head) of one request and KV head; a unit's keys are cut into chunks of C
// tokens, and a (unit, chunk) is an item.  C follows on the device from the
// lengths: as many items as the grid takes at once, at least kMinChunk keys
// each.  Every wave works the schedule out by itself from kv_len and cu_q (64
// requests at a time, one per lane), so ragged batches need no plan and a
// captured graph follows its lengths.  A unit of one chunk writes its output;
// the others leave unnormalized partial results (o, m, l) in the workspace
// for the combine kernel.
#include "kv_device.h"
#include "kv_internal.h"

namespace rw4 {

namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v4f_u __attribute__((ext_vector_type(4), aligned(4)));
typedef int v6i __attribute__((ext_vector_type(6)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __bf16 v4bf __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef __bf16 v32bf __attribute__((ext_vector_type(32)));
typedef unsigned int v4u __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kMinChunk = 128;
constexpr int kNarrowRows = 16;
constexpr int kNarrowTarget = 1024;           // items aimed at: 4 blocks on each of 256 CUs
constexpr int kNarrowWhole = 4 * kNarrowTarget;  // from this many units on, requests are not split

struct Sched {
  int rows;            // query rows of a unit
  int64_t target;      // items aimed at
  int64_t whole;       // with this many units or more, one chunk each
};

// ---------------------------------------------------------------------------
// The schedule.
// ---------------------------------------------------------------------------
struct Req {
  int q0, qn, kv;   // first query token, query tokens, keys
  int tiles;        // row tiles
  int lo, span;     // first key any row sees (a multiple of 64) and keys from there on
};

__device__ __forceinline__ int clamp_int(int64_t v, int64_t hi) { return int(v < 0 ? 0 : v > hi ? hi : v); }

__device__ __forceinline__ Req request(const AttnArgs& a, int64_t b, int rows) {
  Req r{0, 0, 0, 0, 0, 0};
  if (b >= a.B) return r;
  const int q1 = clamp_int(a.cu_q[b + 1], a.T);
  r.q0 = clamp_int(a.cu_q[b], a.T);
  r.qn = q1 > r.q0 ? q1 - r.q0 : 0;
  const int64_t room = a.table_width << a.cache.log2_page;
  r.kv = clamp_int(a.kv_len[b], room < 0x7FFFFF00 ? room : 0x7FFFFF00);
  r.tiles = int((int64_t(r.qn) * a.group + rows - 1) / rows);
  if (a.window > 0) {
    const int64_t first = int64_t(r.kv) - r.qn + 1 - a.window;
    r.lo = first > 0 ? int(first) & ~63 : 0;
  }
  r.span = r.kv - r.lo;
  return r;
}

__device__ __forceinline__ int64_t wave_sum64(int64_t v) {
  for (int d = 32; d; d >>= 1) v += __shfl_xor(static_cast<long long>(v), d);
  return v;
}
__device__ __forceinline__ int64_t wave_prefix64(int64_t v, int lane) {
  for (int d = 1; d < kWave; d <<= 1) {
    const int64_t o = __shfl_up(static_cast<long long>(v), d);
    if (lane >= d) v += o;
  }
  return v;
}
__device__ __forceinline__ int lane_int(int v, int lane) { return __builtin_amdgcn_readlane(v, lane); }
__device__ __forceinline__ int64_t lane_int64(int64_t v, int lane) {
  return int64_t(uint32_t(lane_int(int(v), lane))) | (int64_t(lane_int(int(v >> 32), lane)) << 32);
}

// Keys of a chunk, the same on every wave of every kernel of a call.
__device__ __forceinline__ int chunk_keys(const AttnArgs& a, const Sched& s, int lane) {
  int64_t keys = 0, units = 0;
  for (int64_t b = lane; b - lane < a.B; b += kWave) {
    const Req r = request(a, b, s.rows);
    keys += int64_t(r.tiles) * r.span;
    units += r.tiles;
  }
  keys = wave_sum64(keys) * a.cache.heads;
  units = wave_sum64(units) * a.cache.heads;
  if (units >= s.whole) return 0x7FFFFF00;
  int64_t c = (keys + s.target - 1) / s.target;
  c = (c + 127) & ~int64_t(127);
  return int(c < kMinChunk ? kMinChunk : c > 0x7FFFFF00 ? 0x7FFFFF00 : c);
}

// Walks the items (or units) of the requests in order, 64 requests at a time.
struct Cursor {
  int64_t base;            // first request of the window
  int64_t items, units;    // before the window
  Req r;                   // the lane's request
  int chunks;
  int64_t upto_items, upto_units;  // inclusive sums over the window's lanes
};

__device__ __forceinline__ void cursor_load(const AttnArgs& a, const Sched& s, int C, Cursor& c, int lane) {
  c.r = request(a, c.base + lane, s.rows);
  c.chunks = c.r.span > C ? int((int64_t(c.r.span) + C - 1) / C) : 1;
  const int64_t units = int64_t(c.r.tiles) * a.cache.heads;
  c.upto_units = wave_prefix64(units, lane);
  c.upto_items = wave_prefix64(units * c.chunks, lane);
}

struct Item {
  Req r;
  int64_t b;
  int chunks, chunk, head, tile;  // head: KV head
  int64_t slot;                   // workspace slot of the unit's first chunk
};

// Item (by_units: unit, chunk 0) number n; false past the end.
__device__ __forceinline__ bool cursor_seek(const AttnArgs& a, const Sched& s, int C, Cursor& c, int64_t n,
                                            bool by_units, int lane, Item& it) {
  for (;;) {
    if (c.base >= a.B) return false;
    const int64_t last = lane_int64(by_units ? c.upto_units : c.upto_items, kWave - 1);
    const int64_t before = by_units ? c.units : c.items;
    if (n < before + last) break;
    c.items += lane_int64(c.upto_items, kWave - 1);
    c.units += lane_int64(c.upto_units, kWave - 1);
    c.base += kWave;
    if (c.base < a.B) cursor_load(a, s, C, c, lane);
  }
  const int64_t local = n - (by_units ? c.units : c.items);
  const uint64_t above = __ballot((by_units ? c.upto_units : c.upto_items) > local);
  const int src = __builtin_ctzll(above);
  it.r = Req{lane_int(c.r.q0, src), lane_int(c.r.qn, src), lane_int(c.r.kv, src), lane_int(c.r.tiles, src),
             lane_int(c.r.lo, src), lane_int(c.r.span, src)};
  it.b = c.base + src;
  it.chunks = lane_int(c.chunks, src);
  const int64_t units = int64_t(it.r.tiles) * a.cache.heads;
  const int64_t units0 = lane_int64(c.upto_units, src) - units;
  const int64_t items0 = lane_int64(c.upto_items, src) - units * it.chunks;
  const int64_t in_req = local - (by_units ? units0 : items0);
  const int unit = int(by_units ? in_req : in_req / it.chunks);
  it.chunk = by_units ? 0 : int(in_req % it.chunks);
  it.head = unit % a.cache.heads;
  it.tile = it.r.tiles - 1 - unit / a.cache.heads;  // the longest rows first
  it.slot = c.items + items0 + int64_t(unit) * it.chunks;
  return true;
}

// Keys [begin, end) that query token i of a request sees.
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
// A 16-byte chunk's 32 codes as bf16, in the order of the stored pairs:
// elements 8 i .. 8 i + 7 are channels 8 kPairOrder[i] .. of the chunk.
__device__ __forceinline__ v32bf open_chunk(const v4u& w) {
  uint32_t d[6];
  open_pair<true>(w[0], w[3], d[0], d[1], d[2]);
  open_pair<true>(w[1], w[2], d[3], d[4], d[5]);
  const v6i p = {int(d[0]), int(d[1]), int(d[2]), int(d[3]), int(d[4]), int(d[5])};
  return __builtin_amdgcn_cvt_scalef32_pk32_bf16_fp6(p, 8.0f);  // E2M3 c / 8 times 8
}
__device__ __forceinline__ int pair_order(int i) { return i == 0 ? 0 : i == 1 ? 3 : i == 2 ? 1 : 2; }

__device__ __forceinline__ v8bf part8(const v32bf& x, int i) {
  v8bf r;
#pragma unroll
  for (int e = 0; e < 8; ++e) r[e] = x[8 * i + e];
  return r;
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

// Orders a wave's own LDS writes and reads for the compiler (the hardware
// executes a wave's LDS operations in order).
__device__ __forceinline__ void wave_lds_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// The 4 scales of slots s .. s + 3 of a page.
__device__ __forceinline__ v4f scales4(const float* p, int64_t stride) {
  if (stride == 1) return *reinterpret_cast<const v4f_u*>(p);
  return v4f{p[0], p[stride], p[2 * stride], p[3 * stride]};
}

// One finished row: o (8 channels of each of its D / 8 lanes), sum l, maximum
// m: normalized, unrotated, rounded and stored.
template <int D>
__device__ __forceinline__ void finish_row(const AttnArgs& a, const Req& r, int head, int row, float (&o)[8], float m,
                                           float l, int lane) {
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
  for (int e = 0; e < 8; ++e) o[e] *= inv;
  if (a.unrotate) {
    row_hadamard<float, D / 8>(o, lane);
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] *= kHeadPost<D>;
  }
  if (row >= r.qn * a.group) return;
  const int64_t t = r.q0 + row / a.group;
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
// ---------------------------------------------------------------------------
template <int D>
struct NarrowLds {
  static constexpr int kRow = 2 * D + 32;  // bytes of a V row; +32: 8 consecutive rows hit 8 bank groups
  static constexpr int kWaveBytes = 32 * kRow;
  static constexpr int kOutRow = D + 4;  // floats of an output row in the merge
  static_assert(kNarrowRows * kOutRow * 4 <= kWaveBytes, "merge rows fit the V rows");
};

template <int D, bool PRECISE>
__global__ __launch_bounds__(256) void kv_attention_narrow_kernel(AttnArgs a, Sched s) {
  constexpr int N = PRECISE ? 3 : 1;
  constexpr int NL = D / 64;                 // 16-byte loads a lane makes for 32 rows of codes
  constexpr int NK = D == 64 ? 4 : D / 32;   // query operands
  using L = NarrowLds<D>;
  __shared__ __align__(16) char lds[4 * L::kWaveBytes];
  __shared__ float wave_m[4][kNarrowRows], wave_l[4][kNarrowRows];

  const int tid = threadIdx.x, lane = tid & (kWave - 1), n = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  char* vbuf = lds + wave * L::kWaveBytes;
  const KvCache& kv = a.cache;
  const int C = chunk_keys(a, s, lane);
  Cursor cur{0, 0, 0};
  cursor_load(a, s, C, cur, lane);
  Item it;
  for (int64_t item = blockIdx.x; cursor_seek(a, s, C, cur, item, false, lane, it); item += gridDim.x) {
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
    const int chunk0 = it.r.lo + it.chunk * C;  // C = 2^31 - 2^8 has a single chunk
    const int64_t chunk1 = int64_t(chunk0) + C;
    lo = lo > chunk0 ? lo : chunk0;
    hi = hi < chunk1 ? hi : int(chunk1);
    lo &= ~31;

    v4f o[D / 16];
#pragma unroll
    for (int c = 0; c < D / 16; ++c) o[c] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    float m = -INFINITY, l = 0.0f;

    for (int j0 = lo + 32 * wave; j0 < hi; j0 += 128) {
      // pages of the two 16-key halves (a half behind hi repeats the last key's page)
      int page[2], slot[2];
      bool seen[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int j = j0 + 16 * h, jj = j < hi ? j : hi - 1;
        const int id = a.block_table[it.b * a.table_width + (jj >> kv.log2_page)];
        seen[h] = j < hi && id >= 0 && id < kv.pages;
        page[h] = seen[h] ? id : 0;
        slot[h] = j & ((1 << kv.log2_page) - 1);
      }
      v4u kraw[NL], vraw[NL];
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        const int h = D == 64 ? (g >> 1) : D == 128 ? i : i >> 1;
        const int chunk = D == 64 ? (g & 1) : D == 128 ? g : 4 * (i & 1) + g;
        const int64_t off = int64_t(h ? page[1] : page[0]) * kv.code_page + it.head * kv.code_head +
                            int64_t((h ? slot[1] : slot[0]) + n) * kv.code_slot + 16 * chunk;
        kraw[i] = *reinterpret_cast<const v4u*>(kv.k_codes + off);
        vraw[i] = *reinterpret_cast<const v4u*>(kv.v_codes + off);
      }
      v4f sk[2], sv[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t off = int64_t(page[h]) * kv.scale_page + it.head * kv.scale_head +
                            int64_t(slot[h] + 4 * g) * kv.scale_slot;
        sk[h] = scales4(kv.k_scales + off, kv.scale_slot);
        sv[h] = scales4(kv.v_scales + off, kv.scale_slot);
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
      // softmax
      float x[8];
      bool vis[8];
      const bool whole = seen[0] && seen[1] && j0 >= full_lo && j0 + 32 <= full_hi && j0 + 32 <= hi;
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = sc[e >> 2][e & 3] * (sk[e >> 2][e & 3] * (a.scale * kLog2e));
      if (!whole) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int j = j0 + 16 * (e >> 2) + 4 * g + (e & 3);
          vis[e] = seen[e >> 2] && j >= begin && j < end && j >= chunk0 && j < chunk1;
          x[e] = vis[e] ? x[e] : -INFINITY;
        }
      }
      float top = x[0];
#pragma unroll
      for (int e = 1; e < 8; ++e) top = fmaxf(top, x[e]);
      if (__ballot(top > m + 8.0f)) {
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        const float m_new = top > m + 8.0f ? top : m;  // a row's results do not depend on its neighbours'
        const float alpha = m == -INFINITY ? 0.0f : exp2f(m - m_new);
        m = m_new;
        l *= alpha;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) o[c] *= alpha;
      }
      const float ref = m == -INFINITY ? 0.0f : m;
      v8bf pr[N];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float p = __builtin_amdgcn_exp2f(x[e] - ref);
        float pv = p * sv[e >> 2][e & 3];
        if (!whole) {
          p = vis[e] ? p : 0.0f;
          pv = vis[e] ? pv : 0.0f;
        }
        l += p;
        __bf16 part[N];
        split_bf16<N>(pv, part);
#pragma unroll
        for (int i = 0; i < N; ++i) pr[i][e] = part[i];
      }
      // output: keys of lane group g: 4 g + 0..3 and 16 + 4 g + 0..3
      wave_lds_order();
      const char* vsrc = vbuf + (4 * g + (n >> 2)) * L::kRow + 8 * (n & 3);
#pragma unroll
      for (int c = 0; c < D / 16; ++c) {
        const v8bf vt = lds_transposed(vsrc + 32 * c, vsrc + 32 * c + 16 * L::kRow);
#pragma unroll
        for (int i = 0; i < N; ++i) o[c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vt, pr[i], o[c], 0, 0, 0);
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
        if (it.chunks == 1) {
          finish_row<D>(a, it.r, it.head, it.tile * kNarrowRows + r, acc, top, sum, lane);
        } else {
          float* part = reinterpret_cast<float*>(a.workspace) + (it.slot + it.chunk) * (kNarrowRows * (D + 2));
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
// The partial results of split units put together: D / 8 lanes a row.
// ---------------------------------------------------------------------------
template <int D>
__global__ __launch_bounds__(256) void kv_attention_combine_kernel(AttnArgs a, Sched s) {
  constexpr int LR = D / 8, PASS = 256 / LR;
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int C = chunk_keys(a, s, lane);
  Cursor cur{0, 0, 0};
  cursor_load(a, s, C, cur, lane);
  Item it;
  for (int64_t unit = blockIdx.x; cursor_seek(a, s, C, cur, unit, true, lane, it); unit += gridDim.x) {
    if (it.chunks == 1) continue;
    const int size = s.rows * (D + 2);
    const float* first = reinterpret_cast<const float*>(a.workspace) + it.slot * size;
    for (int r0 = 0; r0 < s.rows; r0 += PASS) {
      const int r = r0 + tid / LR, row = it.tile * s.rows + r;
      if (r0 + (tid & ~(kWave - 1)) / LR >= s.rows) break;  // whole waves
      if (row - (lane / LR) >= it.r.qn * a.group) break;
      float top = -INFINITY, sum = 0.0f, acc[8] = {};
      for (int c = 0; c < it.chunks; ++c) top = fmaxf(top, first[int64_t(c) * size + s.rows * D + r]);
      for (int c = 0; c < it.chunks; ++c) {
        const float* part = first + int64_t(c) * size;
        const float m = part[s.rows * D + r], w = m == -INFINITY ? 0.0f : exp2f(m - top);
        float v[8];
        RowSrc<false>{part, 0}.load8(0, r * D + 8 * (tid & (LR - 1)), v);
        sum += m == -INFINITY ? 0.0f : part[s.rows * (D + 1) + r] * w;
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = fmaf(v[e], w, acc[e]);
      }
      finish_row<D>(a, it.r, it.head, row, acc, top, sum, lane);
    }
  }
}

// Units a call can have, and the workspace slots of its chunks: at most
// target items and one partial chunk for each unit, and nothing is split from
// `whole` units on.
int64_t units_max(int64_t T, int64_t B, int64_t group, int64_t kv_heads, int rows) {
  return kv_heads * (T * group / rows + (B < T ? B : T));
}
int64_t narrow_slots(int64_t T, int64_t B, int64_t group, int64_t kv_heads) {
  const int64_t units = units_max(T, B, group, kv_heads, kNarrowRows);
  return kNarrowTarget + (units < kNarrowWhole ? units : kNarrowWhole);
}

template <int D, bool PRECISE>
hipError_t launch_narrow(const AttnArgs& a, hipStream_t st) {
  const Sched s{kNarrowRows, kNarrowTarget, kNarrowWhole};
  const int64_t slots = narrow_slots(a.T, a.B, a.group, a.cache.heads);
  const int64_t units = units_max(a.T, a.B, a.group, a.cache.heads, kNarrowRows);
  const int64_t most = units > slots ? units : slots;
  const unsigned blocks = unsigned(most < kNarrowTarget ? most : kNarrowTarget);
  hipLaunchKernelGGL((kv_attention_narrow_kernel<D, PRECISE>), dim3(blocks), dim3(256), 0, st, a, s);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || (a.table_width << a.cache.log2_page) <= kMinChunk) return e;  // nothing can be split
  const unsigned again = unsigned(units < 1024 ? units : 1024);
  hipLaunchKernelGGL((kv_attention_combine_kernel<D>), dim3(again), dim3(256), 0, st, a, s);
  return hipGetLastError();
}

}  // namespace

int64_t kv_attention_workspace_bytes(int64_t T, int64_t B, int64_t heads, int64_t kv_heads, int64_t head_dim) {
  const int64_t slots = narrow_slots(T, B, heads / kv_heads, kv_heads);
  return slots * kNarrowRows * (head_dim + 2) * int64_t(sizeof(float));
}

hipError_t launch_kv_attention(const AttnArgs& a, hipStream_t st) {
  const bool precise = !(a.q_bf16 && a.out_bf16);
  switch (a.head_dim) {
    case 64: return precise ? launch_narrow<64, true>(a, st) : launch_narrow<64, false>(a, st);
    case 128: return precise ? launch_narrow<128, true>(a, st) : launch_narrow<128, false>(a, st);
    default: return precise ? launch_narrow<256, true>(a, st) : launch_narrow<256, false>(a, st);
  }
}

}  // namespace rw4
