// Serving with an INT4 KV cache, the token side: pages and slots from request
// lengths (kv_slots), and the per-head rows of a step's new tokens -- RMS
// norm, rotary positions, Hadamard rotation, INT4 quantization and the store
// into the cache's pages (qk_norm_rope, kv_append).
#include "kv_device.h"
#include "kv_index.h"
#include "kv_internal.h"

#include <type_traits>

namespace rw4 {

// ---------------------------------------------------------------------------
// kv_slots.  Three running sums over the requests give everything: the starts
// of the new tokens, the pages each request takes off the free list (need_b =
// ceil((ctx + new) / P) - ceil(ctx / P)) and the pages finished requests give
// back.  A request is served when its inclusive page sum fits in the list's
// count (sums rise, so from the first one that does not fit all later ones
// that need pages are refused too).  Every block forms the sums itself (one
// pass over 2 B integers) and keeps them in LDS, then tokens, taken pages and
// returned pages are independent entries found by binary search.  Pops read
// ring entries [head, head + count), pushes write behind them, so the phases
// need no order between blocks.  8.5 us for 48 requests of one token, 11.4 us
// for 65536 tokens of 700 requests: the latency of dependent loads and of the
// scan, not bytes.
// ---------------------------------------------------------------------------
constexpr int kSlotsThreads = 256;

struct SlotsLens {
  int64_t ctx, add;  // tokens held, tokens to add (< 0: finished)
  int64_t have, need, back;
  bool fits;
};

__device__ __forceinline__ SlotsLens slots_lens(const SlotsArgs& a, int64_t b) {
  SlotsLens r;
  const int64_t page = int64_t(1) << a.log2_page;
  r.ctx = a.ctx_len[b] > 0 ? a.ctx_len[b] : 0;
  r.add = a.new_len[b];
  r.have = (r.ctx + page - 1) >> a.log2_page;
  const int64_t all = r.ctx + (r.add > 0 ? r.add : 0), want = (all + page - 1) >> a.log2_page;
  r.fits = want <= a.table_width && all <= kMostKeys;
  r.need = r.add >= 0 && r.fits ? want - r.have : 0;
  r.back = r.add >= 0 ? 0 : r.have < a.table_width ? r.have : a.table_width;
  return r;
}

__device__ __forceinline__ int32_t sat32(int64_t v) { return v > 0x7FFFFFFF ? 0x7FFFFFFF : int32_t(v); }

// The last b in [0, n) with start[b] <= j (start[0] = 0 <= j).
__device__ __forceinline__ int slots_find(const int32_t* start, int n, int64_t j) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (start[mid] <= j) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// wide: tokens and pages; finish: lengths, starts, flags and the new state
// (which may be the arrays the wide part reads, hence after it).
__global__ __launch_bounds__(kSlotsThreads) void kv_slots_kernel(SlotsArgs a, bool wide, bool finish) {
  extern __shared__ int32_t sums[];  // [3][B + 1]
  const int B = int(a.B), tid = threadIdx.x;
  int32_t* tok0 = sums;
  int32_t* need0 = sums + (B + 1);
  int32_t* back0 = sums + 2 * (B + 1);
  __shared__ int64_t wave_sum[kSlotsThreads / kWave][3];
  __shared__ int32_t taken_s;

  const int64_t cap = a.capacity;
  int64_t head = a.free_state[0] % cap, count = a.free_state[1];
  if (head < 0) head += cap;
  count = count < 0 ? 0 : count > cap ? cap : count;
  if (tid == 0) taken_s = 0;

  const int per = (B + kSlotsThreads - 1) / kSlotsThreads;
  const int b0 = tid * per < B ? tid * per : B, b1 = b0 + per < B ? b0 + per : B;
  int64_t run[3] = {0, 0, 0};
  for (int b = b0; b < b1; ++b) {
    const SlotsLens r = slots_lens(a, b);
    run[0] += r.add > 0 ? r.add : 0;
    run[1] += r.need;
    run[2] += r.back;
  }
  const int lane = tid & (kWave - 1), wave = tid / kWave;
  int64_t upto[3];
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    upto[i] = run[i];
    for (int d = 1; d < kWave; d <<= 1) {
      const int64_t o = __shfl_up(static_cast<long long>(upto[i]), d);
      if (lane >= d) upto[i] += o;
    }
    if (lane == kWave - 1) wave_sum[wave][i] = upto[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    int64_t before = upto[i] - run[i];
    for (int w = 0; w < wave; ++w) before += wave_sum[w][i];
    run[i] = before;
  }
  int32_t most = 0;
  for (int b = b0; b < b1; ++b) {
    const SlotsLens r = slots_lens(a, b);
    tok0[b] = sat32(run[0]);
    need0[b] = sat32(run[1]);
    back0[b] = sat32(run[2]);
    run[0] += r.add > 0 ? r.add : 0;
    run[1] += r.need;
    run[2] += r.back;
    if (run[1] <= count) most = int32_t(run[1]);
  }
  if (b1 == B && (b0 < B || (B == 0 && tid == 0))) {
    tok0[B] = sat32(run[0]);
    need0[B] = sat32(run[1]);
    back0[B] = sat32(run[2]);
  }
  atomicMax(&taken_s, most);
  __syncthreads();
  const int64_t taken = taken_s;
  const int64_t given = back0[B] < cap - count ? back0[B] : cap - count;

  if (wide) {
    const int64_t first = int64_t(blockIdx.x) * kSlotsThreads + tid, step = int64_t(gridDim.x) * kSlotsThreads;
    const int64_t page = int64_t(1) << a.log2_page;
    for (int64_t t = first; t < a.tokens; t += step) {
      int64_t slot = -1;
      int32_t pos = -1;
      if (t < tok0[B]) {
        const int b = slots_find(tok0, B, t);
        const SlotsLens r = slots_lens(a, b);
        if (r.fits && (need0[b + 1] == need0[b] || need0[b + 1] <= count)) {
          const int64_t p = r.ctx + t - tok0[b], nth = p >> a.log2_page;
          const int32_t id = nth < r.have ? a.block_table[b * a.table_width + nth]
                                          : a.free_pages[(head + need0[b] + nth - r.have) % cap];
          if (id >= 0) slot = int64_t(id) * page + (p & (page - 1));
          pos = int32_t(p);
        }
      }
      a.slot_map[t] = slot;
      a.positions[t] = pos;
    }
    for (int64_t j = first; j < taken; j += step) {
      const int b = slots_find(need0, B, j);
      const SlotsLens r = slots_lens(a, b);
      a.block_table[b * a.table_width + r.have + j - need0[b]] = a.free_pages[(head + j) % cap];
    }
    for (int64_t j = first; j < given; j += step) {
      const int b = slots_find(back0, B, j);
      a.free_pages[(head + count + j) % cap] = a.block_table[b * a.table_width + j - back0[b]];
    }
  }
  if (finish && blockIdx.x == 0) {
    __syncthreads();  // the wide part's reads of lengths and state come first
    for (int b = tid; b < B; b += kSlotsThreads) {
      const SlotsLens r = slots_lens(a, b);
      const bool ok = r.add < 0 || (r.fits && (need0[b + 1] == need0[b] || need0[b + 1] <= count));
      a.kv_len[b] = r.add < 0 ? 0 : sat32(ok ? r.ctx + r.add : r.ctx);
      a.served[b] = ok ? 1 : 0;
      a.cu_new[b] = tok0[b];
    }
    if (tid == 0) {
      a.cu_new[B] = tok0[B];
      a.free_state_out[0] = int32_t((head + taken) % cap);
      a.free_state_out[1] = int32_t(count - taken + given);
    }
  }
}

hipError_t launch_kv_slots(const SlotsArgs& a, hipStream_t st) {
  const size_t lds = 3 * size_t(a.B + 1) * sizeof(int32_t);
  int64_t blocks = (a.tokens + 511) / 512;
  blocks = blocks < 1 ? 1 : blocks > 256 ? 256 : blocks;
  const bool alias = a.kv_len == a.ctx_len || a.free_state_out == a.free_state;
  const bool two = alias && blocks > 1;  // other blocks may still read what the finish part writes
  hipLaunchKernelGGL(kv_slots_kernel, dim3(unsigned(blocks)), dim3(kSlotsThreads), lds, st, a, true, !two);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !two) return e;
  hipLaunchKernelGGL(kv_slots_kernel, dim3(1), dim3(kSlotsThreads), lds, st, a, false, true);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Head rows.  A head row (D channels) lies in L = D / 8 lanes, 8 consecutive
// channels each, so a wave holds 64 / L rows; channel index = 8 lane + e, and
// the Sylvester butterflies run over e in registers and over the lane bits
// across lanes.  Dense rows (queries; keys without a cache) are evaluated in
// fp32 and bound by memory.
//
// Rows that are quantized get the codes of the exact quotients 7 u / m of the
// rotated row u, ties to even.  They are evaluated in fp32 first, together with
// a bound of the error: every u_j is a signed sum of D terms that passes
// through n roundings (the products with norm weight and rotary factors, log2 D
// additions), so it and m are off by at most n 2^-24 S, S the sum of the terms'
// magnitudes, and a quotient by (7 / m) 2 n 2^-24 S and the 5 roundings of its
// own (of at most 7).  Where a quotient lies that close to a half (1 % of the
// rows of 128 Gaussian values), the wave evaluates its rows again in fp64, in
// which the sums of bf16 values are exact.  8191 tokens (32 + 8 + 8 heads of 128)
// take 60 us, bound by vector arithmetic (71 % busy, about 170 instructions for
// a lane's 8 channels) and the waits for a group of heads that is loaded when the
// one before is stored; 80 us with every row in fp64.  Dense rows of 12001 tokens
// take 45 us, 5.6 TB/s.
// ---------------------------------------------------------------------------
__device__ __forceinline__ float lane_get(float v, int src) {
  return __int_as_float(__builtin_amdgcn_ds_bpermute(src << 2, __float_as_int(v)));
}
// 1 / sqrt(x): the hardware estimate (1 ulp) and a Newton step; 0 and infinity
// give infinity and 0.
__device__ __forceinline__ float inv_root(float x) {
  const float y = __builtin_amdgcn_rsqf(x);
  const float r = fmaf(-x * y, y, 1.0f);
  return x > 0.0f && x < __builtin_huge_valf() ? fmaf(0.5f * y, r, y) : y;
}
// Sum over the 16 lanes of a DPP row (lane masks 1, 2, 7 and 8 span them), as
// row16_max_dpp.
__device__ __forceinline__ float row16_sum_dpp(float s) {
  asm volatile(
      "s_nop 1\n"
      "v_add_f32_dpp %0, %0, %0 quad_perm:[1,0,3,2] row_mask:0xf bank_mask:0xf\n"
      "s_nop 1\n"
      "v_add_f32_dpp %0, %0, %0 quad_perm:[2,3,0,1] row_mask:0xf bank_mask:0xf\n"
      "s_nop 1\n"
      "v_add_f32_dpp %0, %0, %0 row_half_mirror row_mask:0xf bank_mask:0xf\n"
      "s_nop 1\n"
      "v_add_f32_dpp %0, %0, %0 row_ror:8 row_mask:0xf bank_mask:0xf\n"
      : "+v"(s));
  return s;
}

template <int L>
__device__ __forceinline__ float row_sum(float s) {
  if constexpr (L == 16) return row16_sum_dpp(s);
  s += lane_xor<1>(s);
  s += lane_xor<2>(s);
  s += lane_xor<4>(s);
  if constexpr (L > 8) s += lane_xor<8>(s);
  if constexpr (L > 16) s += lane_xor<16>(s);
  return s;
}
template <int L>
__device__ __forceinline__ float row_max(float m) {
  if constexpr (L == 16) return row16_max_dpp(m);
  m = fmax(m, lane_xor<1>(m));
  m = fmax(m, lane_xor<2>(m));
  m = fmax(m, lane_xor<4>(m));
  if constexpr (L > 8) m = fmax(m, lane_xor<8>(m));
  if constexpr (L > 16) m = fmax(m, lane_xor<16>(m));
  return m;
}

// The rotary factors of a lane's 8 channels: y'_e = c_e y_e + s_e y_partner(e).
struct RopeLane {
  float c[8], s[8];
  int partner;  // lane of the partner channels (halves form)
  bool on;      // the lane's channels are rotated
};

__device__ __forceinline__ RopeLane rope_lane(const RowsArgs& a, int64_t pos, int lane, int l) {
  RopeLane r;
  const int e0 = 8 * l, half = a.rot >> 1;
  r.on = e0 < a.rot;
  r.partner = lane;
  if (!r.on) return r;
  const float* row = a.cos_sin + pos * a.rot;
  if (a.interleaved) {
    const float4 c = *reinterpret_cast<const float4*>(row + e0 / 2);
    const float4 s = *reinterpret_cast<const float4*>(row + half + e0 / 2);
    const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r.c[2 * i] = r.c[2 * i + 1] = cc[i];
      r.s[2 * i] = -ss[i];
      r.s[2 * i + 1] = ss[i];
    }
  } else {
    const bool low = e0 < half;
    const int i0 = low ? e0 : e0 - half;
    r.partner = low ? lane + half / 8 : lane - half / 8;
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
      const float4 c = *reinterpret_cast<const float4*>(row + i0 + i);
      const float4 s = *reinterpret_cast<const float4*>(row + half + i0 + i);
      r.c[i] = c.x; r.c[i + 1] = c.y; r.c[i + 2] = c.z; r.c[i + 3] = c.w;
      r.s[i] = low ? -s.x : s.x;
      r.s[i + 1] = low ? -s.y : s.y;
      r.s[i + 2] = low ? -s.z : s.z;
      r.s[i + 3] = low ? -s.w : s.w;
    }
  }
  return r;
}

template <int L>
__device__ __forceinline__ void rope_apply(const RowsArgs& a, const RopeLane& r, float (&v)[8]) {
  if (a.interleaved) {
    if (r.on) {
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const float x = v[e], y = v[e + 1];
        v[e] = x * r.c[e] + y * r.s[e];
        v[e + 1] = y * r.c[e + 1] + x * r.s[e + 1];
      }
    }
  } else if (a.rot == 8 * L) {  // the whole head: the partner is half the lanes away
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float p = lane_xor<L / 2>(v[e]);
      v[e] = v[e] * r.c[e] + p * r.s[e];
    }
  } else {
    float p[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) p[e] = lane_get(v[e], r.partner);
    if (r.on) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = v[e] * r.c[e] + p[e] * r.s[e];
    }
  }
}

template <bool BF16>
__device__ __forceinline__ void load_row8(const void* base, int64_t off, float (&v)[8]) {
  RowSrc<BF16>{base, 0}.load8(0, off, v);
}

// Lane constants of the fp32 Hadamard.  D = 128 takes the 16-lane stages fused
// into multiply-adds, which leave lane l with (-1)^popcount(l) times the outputs of
// Sylvester lane h128_lane_word(l); the other sizes leave them in place.
struct QuantLane {
  float c1, c2, c7, c8, sign;
  int word;
};
template <int D>
__device__ __forceinline__ QuantLane quant_lane(int l) {
  if constexpr (D == 128)
    return QuantLane{parity_sign(l & 5), parity_sign(l & 6), parity_sign(l & 4), parity_sign(l & 8), parity_sign(l),
                     h128_lane_word(l)};
  else
    return QuantLane{0.0f, 0.0f, 0.0f, 0.0f, 1.0f, l};
}

// y H_D in fp32: lane l holds ql.sign times the outputs of word ql.word.
template <int D>
__device__ __forceinline__ void fast_hadamard(float (&v)[8], const QuantLane& ql, int lane) {
  if constexpr (D == 128) {
    fwht8(v);
    lane_stages_dpp(v, ql.c1, ql.c2, ql.c7, ql.c8);
  } else {
    row_hadamard<D / 8>(v, lane);
  }
}

// Whether a row's mean square + eps can be formed from this fp32 sum of squares.
__device__ __forceinline__ bool squares_fit(float ss, float eps) {
  return ss <= 0x1p120f && (ss >= 0x1p-100f || eps >= 0x1p-90f);
}

// The power of two 2^-k that brings a row's largest magnitude into [1/2, 1) (k >=
// -100, so that eps 4^-k stays in range where squares_fit fails); 0 for rows of
// zeros, with infinities or NaN.
template <int L>
__device__ __forceinline__ int row_exponent(const float (&v)[8]) {
  float most = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) most = fabsf(v[e]) < __builtin_huge_valf() ? fmaxf(most, fabsf(v[e])) : __builtin_huge_valf();
  most = row_max<L>(most);
  const int k = __builtin_amdgcn_frexp_expf(most);
  return most > 0.0f && most < __builtin_huge_valf() ? (k > -100 ? k : -100) : 0;
}

// 1 / sqrt(mean square + eps) of a row, times 2^k, from its values times 2^-k.
template <int L>
__device__ __forceinline__ float norm_factor(float ss, float eps, int k) {
  const float x = ss * (1.0f / (8 * L)) + ldexpf(ldexpf(eps, -k), -k);
  const bool tiny = x < 0x1p-100f;  // below the normal numbers the hardware's estimate is infinite
  const float y = inv_root(tiny ? x * 0x1p120f : x);
  return tiny ? y * 0x1p60f : y;
}

// One dense row (queries; keys without a cache).  The norm's factor is common to
// the row and enters at the end.  A row whose squares, or sums under the Hadamard,
// leave fp32's range is left to the RESCALED form, which takes its values times a
// power of two: returns whether the lane's row is one.
template <int D, bool BF16, bool RESCALED = false>
__device__ __forceinline__ bool dense_row(const RowsArgs& a, const DenseRows& r, const float* weight, int64_t t, int h,
                                          bool live, const RopeLane& rope, const QuantLane& ql, int lane, int l) {
  constexpr int L = D / 8;
  float v[8];
  load_row8<BF16>(r.in, t * r.in_token + h * r.in_head + 8 * l, v);
  float post = 1.0f;
  bool fits = true;
  int k = 0;
  if constexpr (RESCALED) {
    k = row_exponent<L>(v);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = ldexpf(v[e], -k);
  }
  if (weight) {
    float ss = 0.0f, w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(v[e], v[e], ss);
    ss = row_sum<L>(ss);
    if constexpr (RESCALED) {
      post = norm_factor<L>(ss, a.eps, k);
    } else {
      fits = squares_fit(ss, a.eps);
      post = inv_root(ss * (1.0f / D) + a.eps);
    }
    load_row8<false>(weight, 8 * l, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= w[e];
  }
  if (a.cos_sin) rope_apply<L>(a, rope, v);
  int word = l;
  if (a.rotate) {
    fast_hadamard<D>(v, ql, lane);
    if (!RESCALED && !weight) {
      float most = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) most = fmaxf(most, fabsf(v[e]));
      fits = row_max<L>(most) < __builtin_huge_valf();
    }
    post *= kHeadPost<D> * ql.sign;
    word = ql.word;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] *= post;
  if constexpr (RESCALED) {
    if (!weight) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = ldexpf(v[e], k);
    }
  }
  if (live && fits) store_row8(r.out, a.out_bf16, t * r.out_token + h * r.out_head + 8 * word, v);
  return live && !fits;
}

// The exact codes of one row, in fp64, by the whole wave: lane n has channels
// E n .. E n + E - 1 (E = D / 64) and gets their codes (c[e]); returns the row's
// maximum (infinite for infinities and NaN).  row: offset of the row's first
// channel; cos_sin: its rotary factors or null.  All lanes take the same row.
template <int D, bool BF16>
__device__ __forceinline__ double exact_row(const RowsArgs& a, const void* in, int64_t row, const float* weight,
                                            const float* cos_sin, int lane, int (&c)[D / 64]) {
  constexpr int E = D / 64;
  auto term = [&](int k) {  // channel k with its weight
    const double x = BF16 ? double(__uint_as_float(uint32_t(reinterpret_cast<const uint16_t*>(in)[row + k]) << 16))
                          : double(reinterpret_cast<const float*>(in)[row + k]);
    return weight ? x * double(weight[k]) : x;
  };
  double u[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int k = E * lane + e, half = a.rot >> 1;
    u[e] = term(k);
    if (cos_sin && k < a.rot) {
      const bool low = a.interleaved ? !(k & 1) : k < half;
      const int i = a.interleaved ? k >> 1 : low ? k : k - half;
      const int partner = a.interleaved ? k ^ 1 : low ? k + half : k - half;
      const double s = cos_sin[half + i];
      u[e] = u[e] * double(cos_sin[i]) + term(partner) * (low ? -s : s);
    }
  }
  if (a.rotate) {
#pragma unroll
    for (int st = 1; st < E; st <<= 1) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        if ((e & st) == 0) {
          const double x = u[e], y = u[e | st];
          u[e] = x + y;
          u[e | st] = x - y;
        }
      }
    }
    for (int st = 1; st < kWave; st <<= 1) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const double y = __shfl_xor(u[e], st);
        u[e] = (lane & st) ? y - u[e] : u[e] + y;
      }
    }
  }
  double top = 0.0;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const double p = fabs(u[e]);
    top = p < __builtin_huge_val() ? fmax(top, p) : __builtin_huge_val();  // NaN counts as infinite
  }
  for (int st = 1; st < kWave; st <<= 1) top = fmax(top, __shfl_xor(top, st));
  const bool bad = !(top < __builtin_huge_val());
  const double r7 = bad || !(top > 0.0) ? 0.0 : 7.0 / top;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    // the rounded product, put right by the exact remainder
    double q = bad ? 0.0 : rint(u[e] * r7);
    const double rem = fma(-q, top, 7.0 * u[e]), twice = 2.0 * fabs(rem);
    if (!bad && (twice > top || (twice == top && (int(q) & 1)))) q += rem > 0.0 ? 1.0 : -1.0;
    c[e] = int(q);
  }
  return top;
}

// One quantized row into the cache.
//   A key whose squares leave fp32's range is left to the RESCALED form, which takes
// its values times a power of two: returns whether the lane's row is one.
template <int D, bool BF16, bool KEY, bool RESCALED = false>
__device__ __forceinline__ bool cache_row(const RowsArgs& a, int64_t t, int h, bool live, int64_t slot, int64_t pos,
                                          const RopeLane& rope, const QuantLane& ql, int lane, int l) {
  constexpr int L = D / 8;
  const void* in = KEY ? a.k.in : a.v;
  const int64_t at = KEY ? t * a.k.in_token + h * a.k.in_head + 8 * l : t * a.v_token + h * a.v_head + 8 * l;
  const float* weight = KEY ? a.k_weight : nullptr;
  const bool roped = KEY && a.cos_sin;
  float v[8], inv = 1.0f;
  bool fits = true;
  int k = 0;
  load_row8<BF16>(in, at, v);
  if constexpr (RESCALED) {
    k = row_exponent<L>(v);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = ldexpf(v[e], -k);
  }
  if (KEY && weight) {
    // the norm's factor is common to the row: it does not move the codes, so
    // it enters the scale alone
    float ss = 0.0f, w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(v[e], v[e], ss);
    ss = row_sum<L>(ss);
    if constexpr (RESCALED) {
      inv = norm_factor<L>(ss, a.eps, k);
    } else {
      fits = squares_fit(ss, a.eps);
      inv = inv_root(ss * (1.0f / D) + a.eps);
    }
    load_row8<false>(weight, 8 * l, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= w[e];
  }
  // S: a rotary pair's terms are at most |x| (|c| + |s|) each, summed over the pair
  float size = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e)
    size += KEY && roped && rope.on ? fabsf(v[e]) * (fabsf(rope.c[e]) + fabsf(rope.s[e])) : fabsf(v[e]);
  if (roped) rope_apply<L>(a, rope, v);
  float sign = 1.0f;
  int word = l;
  if (a.rotate) {
    fast_hadamard<D>(v, ql, lane);
    sign = ql.sign;
    word = ql.word;
  }
  size = row_sum<L>(size);
  float m = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(v[e]));
  m = row_max<L>(m);
  const float post = inv * (a.rotate ? kHeadPost<D> / 7.0f : 1.0f / 7.0f);
  const float r7 = m > 0.0f ? __builtin_amdgcn_rcpf(m * (1.0f / 7.0f)) : 0.0f, rs = r7 * sign;
  float scale = m > 0.0f ? m * post : 0.0f, far = 0.0f;
  uint32_t b[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float r = fmaf(v[e], rs, kRoundMagic);
    b[e] = __float_as_uint(r);
    far = fmaxf(far, fabsf(fmaf(v[e], rs, kRoundMagic - r)));
  }
  // 2 n 2^-24 with n = 8 additions, 3 products and some room for S itself: 2^-20 (values), 2^-19 (keys)
  const float margin = fmaf(size * r7, KEY ? 0x1p-19f : 0x1p-20f, 0x1p-18f);
  // also where the range of the fp32 steps does not do (zeros are fine), for infinities and NaN
  uint64_t near = __ballot(!(far < 0.5f - margin) || !(size < 0x1p120f) || (size > 0.0f && (RESCALED || m < kTinyMax)));
  while (near) {  // a row at a time
    constexpr int E = D / 64;
    const int first = (__builtin_ctzll(near) / L) * L;
    near &= ~(((uint64_t(1) << (L - 1) << 1) - 1) << first);
    const int64_t row = int64_t(uint32_t(__builtin_amdgcn_readlane(int(at), first))) |
                        (int64_t(__builtin_amdgcn_readlane(int(at >> 32), first)) << 32);
    int c[E], lane_here = lane;
    asm volatile("" : "+v"(lane_here));  // keeps this rare path's addresses out of the registers of the common one
    const double top = exact_row<D, BF16>(a, in, row, weight, roped ? a.cos_sin + pos * a.rot : nullptr, lane_here, c);
    uint32_t packed = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) packed |= (uint32_t(c[e]) & 0xFFu) << (8 * e);
    const bool mine = lane - l == first;
    uint32_t got[8 / E];
#pragma unroll
    for (int i = 0; i < 8 / E; ++i)
      got[i] = uint32_t(__builtin_amdgcn_ds_bpermute((8 / E * (lane_here & (L - 1)) + i) << 2, int(packed)));
    if (mine) {
#pragma unroll
      for (int e = 0; e < 8; ++e) b[e] = kRoundMagicBits + uint32_t(int(int8_t(got[e / E] >> (8 * (e % E)))));
      word = l;
      scale = !(top < __builtin_huge_val()) ? __int_as_float(0x7FC00000) : top > 0.0 ? float(ldexp(top * double(post), -k)) : 0.0f;
    }
  }
  const uint32_t bits = pack8_bits(b, (word & 2) != 0);
  if (!live || !fits) return live;
  const KvCache& c = a.cache;
  const int64_t page = slot >> c.log2_page, off = slot & ((int64_t(1) << c.log2_page) - 1);
  *reinterpret_cast<uint32_t*>((KEY ? c.k_codes : c.v_codes) + page * c.code_page + h * c.code_head + off * c.code_slot +
                               4 * word) = bits;
  if (l == 0)
    (KEY ? c.k_scales : c.v_scales)[page * c.scale_page + h * c.scale_head + off * c.scale_slot] = scale;
  return false;
}

// A wave takes one token's head groups (64 / L heads of one kind: queries,
// keys, values) part, part + parts, ...; the rotary factors stay in registers
// across them.  Registers for 8 blocks a CU for dense rows, 5 for appends of 128: left
// to itself the compiler takes more for the rare paths, and 8191 tokens into a cache
// 68 us for 60, dense rows of 12001 tokens 58 for 54.
template <int D, bool BF16, bool APPEND>
__global__ __launch_bounds__(256, APPEND ? (D == 128 ? 5 : 1) : 8) void kv_rows_kernel(RowsArgs a, int parts) {
  constexpr int L = D / 8, R = kWave / L;
  const int lane = threadIdx.x & (kWave - 1), l = lane & (L - 1);
  const int64_t w =
      __builtin_amdgcn_readfirstlane(int(blockIdx.x * (blockDim.x / kWave) + threadIdx.x / kWave));
  const int64_t t = w / parts;
  if (t >= a.T) return;
  const int part = int(w % parts);
  int64_t pos = 0;
  RopeLane rope;
  if (a.cos_sin) {
    pos = a.positions[t];
    if (pos < 0 || pos >= a.max_pos) return;
    rope = rope_lane(a, pos, lane, l);
  }
  int64_t slot = -1;
  if constexpr (APPEND) slot = a.slot_map[t];
  const bool stored = APPEND && slot >= 0 && slot < a.cache.slots;
  const QuantLane ql = quant_lane<D>(l);
  const int gq = (a.q.heads + R - 1) / R, gk = (a.k.heads + R - 1) / R;
  const int groups = gq + gk + (APPEND ? gk : 0);
  for (int g = part; g < groups; g += parts) {
    const int kind = g < gq ? 0 : g < gq + gk ? 1 : 2;
    const int heads = kind == 0 ? a.q.heads : a.k.heads;
    int h = (kind == 0 ? g : kind == 1 ? g - gq : g - gq - gk) * R + lane / L;
    const bool live = h < heads;
    h = live ? h : heads - 1;
    auto dense = [&](const DenseRows& r, const float* weight) {
      const bool left = dense_row<D, BF16>(a, r, weight, t, h, live, rope, ql, lane, l);
      if (__builtin_expect(__ballot(left) != 0, 0)) {
        int lane2 = lane;
        asm volatile("" : "+v"(lane2));  // keeps the rare form's lane constants out of the common one's registers
        const int l2 = lane2 & (L - 1);
        dense_row<D, BF16, true>(a, r, weight, t, h, left, rope, quant_lane<D>(l2), lane2, l2);
      }
    };
    if (kind == 0) {
      dense(a.q, a.q_weight);
    } else if (!APPEND) {
      dense(a.k, a.k_weight);
    } else if (!stored) {
      continue;
    } else if (kind == 1) {
      const bool left = cache_row<D, BF16, true>(a, t, h, live, slot, pos, rope, ql, lane, l);
      if (__builtin_expect(__ballot(left) != 0, 0)) cache_row<D, BF16, true, true>(a, t, h, left, slot, pos, rope, ql, lane, l);
    } else {
      cache_row<D, BF16, false>(a, t, h, live, slot, pos, rope, ql, lane, l);
    }
  }
}

// Tokens of one launch, at most: a grid has fewer than 2^32 threads.
constexpr int64_t kMostTokens = int64_t(1) << 25;

// n tokens from token t on.
template <bool BF16>
static RowsArgs rows_from(const RowsArgs& a, int64_t t, int64_t n) {
  const int64_t in = BF16 ? 2 : 4, out = a.out_bf16 ? 2 : 4;
  RowsArgs r = a;
  auto on = [](auto*& p, int64_t bytes) {
    if (p) p = reinterpret_cast<std::remove_reference_t<decltype(p)>>(reinterpret_cast<uintptr_t>(p) + bytes);
  };
  on(r.q.in, t * a.q.in_token * in);
  on(r.q.out, t * a.q.out_token * out);
  on(r.k.in, t * a.k.in_token * in);
  on(r.k.out, t * a.k.out_token * out);
  on(r.v, t * a.v_token * in);
  on(r.slot_map, t * int64_t(sizeof(*r.slot_map)));
  on(r.positions, t * int64_t(sizeof(*r.positions)));
  r.T = n;
  return r;
}

template <int D, bool BF16, bool APPEND>
static hipError_t launch_rows(const RowsArgs& a, hipStream_t st) {
  constexpr int R = kWave / (D / 8);
  const int64_t gq = (a.q.heads + R - 1) / R, gk = (a.k.heads + R - 1) / R;
  const int64_t groups = gq + gk * (APPEND ? 2 : 1);
  // few tokens: a wave per head group; many: a wave keeps a token's rotary
  // factors for several groups, with at least 16384 waves in the grid
  int64_t parts = (16384 + a.T - 1) / a.T;
  parts = parts < 1 ? 1 : parts > groups ? groups : parts;
  for (int64_t t = 0; t < a.T; t += kMostTokens) {
    const RowsArgs some = rows_from<BF16>(a, t, a.T - t < kMostTokens ? a.T - t : kMostTokens);
    const int64_t blocks = (some.T * parts + 3) / 4;
    hipLaunchKernelGGL((kv_rows_kernel<D, BF16, APPEND>), dim3(unsigned(blocks)), dim3(256), 0, st, some, int(parts));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <bool APPEND>
static hipError_t launch_rows_any(const RowsArgs& a, bool x_bf16, hipStream_t st) {
  switch (a.head_dim) {
    case 64: return x_bf16 ? launch_rows<64, true, APPEND>(a, st) : launch_rows<64, false, APPEND>(a, st);
    case 128: return x_bf16 ? launch_rows<128, true, APPEND>(a, st) : launch_rows<128, false, APPEND>(a, st);
    default: return x_bf16 ? launch_rows<256, true, APPEND>(a, st) : launch_rows<256, false, APPEND>(a, st);
  }
}

hipError_t launch_qk_norm_rope(const RowsArgs& a, bool x_bf16, hipStream_t st) {
  return launch_rows_any<false>(a, x_bf16, st);
}
hipError_t launch_kv_append(const RowsArgs& a, bool x_bf16, hipStream_t st) {
  return launch_rows_any<true>(a, x_bf16, st);
}

}  // namespace rw4
