// Attention over the paged INT4 KV cache.
//
//   s_j = scale sk_j (q . ck_j),  out = sum_j softmax(s)_j sv_j cv_j
//
// with the stored codes ck, cv and one scale per cached row.  One block per
// (query token, query head): tiles of 256 keys, one key's score per thread
// (fp32 products of the opened codes), then the running maximum and sum of
// the softmax over the block, then the tile's values, each thread one stored
// word (8 channels) of every n-th key.
#include "kv_internal.h"
#include "rw4_device.h"

namespace rw4 {

namespace {

constexpr int kTile = 256;

// 8 signed codes of stored word w (of its row) as floats.
__device__ __forceinline__ void open_word(const uint32_t* row, int w, float (&c)[8]) {
  uint32_t lo, hi;
  pair_fields<true>(row[w], row[w ^ 3], (w & 2) != 0, lo, hi);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t f = field6(lo, hi, e);
    const float mag = float(f & 7u);
    c[e] = (f & 32u) ? -mag : mag;
  }
}

__device__ __forceinline__ float wave_max(float v) {
  for (int d = 32; d; d >>= 1) v = fmaxf(v, __shfl_xor(v, d));
  return v;
}
__device__ __forceinline__ float wave_sum(float v) {
  for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

template <int D>
__global__ __launch_bounds__(256) void kv_attention_kernel(AttnArgs a) {
  constexpr int W = D / 8, SUB = 256 / W;
  const int tid = threadIdx.x;
  const int64_t t = blockIdx.x / a.heads;
  const int h = int(blockIdx.x % a.heads), kh = h / (a.heads / a.cache.heads);
  const KvCache& c = a.cache;

  // the request of token t: the last b with cu_q[b] <= t
  int64_t lo_b = 0, hi_b = a.B - 1;
  while (lo_b < hi_b) {
    const int64_t mid = (lo_b + hi_b + 1) >> 1;
    if (a.cu_q[mid] <= t) lo_b = mid;
    else hi_b = mid - 1;
  }
  const int64_t b = lo_b;
  if (t < a.cu_q[b] || t >= a.cu_q[b + 1]) return;
  const int64_t room = a.table_width << c.log2_page;
  int64_t kv = a.kv_len[b];
  kv = kv < 0 ? 0 : kv > room ? room : kv;
  const int64_t place = kv - (a.cu_q[b + 1] - t);
  int64_t end = a.causal ? place + 1 : kv, begin = 0;
  if (end > kv) end = kv;
  if (a.window > 0 && place - a.window + 1 > 0) begin = place - a.window + 1;

  __shared__ float qs[D];
  __shared__ float prob[kTile];
  __shared__ int64_t vrow[kTile];
  __shared__ float acc_s[SUB][D];
  __shared__ float red[8];
  for (int d = tid; d < D; d += 256) {
    const int64_t off = t * a.q_token + h * a.q_head + d;
    qs[d] = a.q_bf16 ? __uint_as_float(uint32_t(reinterpret_cast<const uint16_t*>(a.q)[off]) << 16)
                     : reinterpret_cast<const float*>(a.q)[off];
  }
  __syncthreads();

  float m = -INFINITY, l = 0.0f, acc[8] = {};
  const int w = tid % W, sub = tid / W;
  for (int64_t j0 = begin & ~int64_t(kTile - 1); j0 < end; j0 += kTile) {
    const int64_t j = j0 + tid;
    float s = -INFINITY, sv = 0.0f;
    int64_t off_v = -1;
    if (j >= begin && j < end) {
      const int64_t page = a.block_table[b * a.table_width + (j >> c.log2_page)];
      if (page >= 0 && page < c.pages) {
        const int64_t slot = j & ((int64_t(1) << c.log2_page) - 1);
        off_v = page * c.code_page + kh * c.code_head + slot * c.code_slot;
        const int64_t sc = page * c.scale_page + kh * c.scale_head + slot * c.scale_slot;
        const uint32_t* row = reinterpret_cast<const uint32_t*>(c.k_codes + off_v);
        float dot = 0.0f;
        for (int i = 0; i < W; ++i) {
          float k8[8];
          open_word(row, i, k8);
#pragma unroll
          for (int e = 0; e < 8; ++e) dot = fmaf(qs[8 * i + e], k8[e], dot);
        }
        s = dot * c.k_scales[sc] * a.scale;
        sv = c.v_scales[sc];
      }
    }
    const float top = wave_max(s);
    if ((tid & 63) == 0) red[tid >> 6] = top;
    __syncthreads();
    const float m_new = fmaxf(fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])), m);
    const float m_ref = m_new == -INFINITY ? 0.0f : m_new;
    const float p = off_v < 0 ? 0.0f : expf(s - m_ref);
    prob[tid] = off_v < 0 ? 0.0f : p * sv;
    vrow[tid] = off_v;
    const float part = wave_sum(p);
    if ((tid & 63) == 0) red[4 + (tid >> 6)] = part;
    __syncthreads();
    const float alpha = m == -INFINITY ? 0.0f : expf(m - m_ref);
    m = m_new;
    l = l * alpha + red[4] + red[5] + red[6] + red[7];
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] *= alpha;
    for (int i = sub; i < kTile; i += SUB) {
      if (vrow[i] < 0) continue;
      float v8[8];
      open_word(reinterpret_cast<const uint32_t*>(c.v_codes + vrow[i]), w, v8);
      const float pi = prob[i];
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] = fmaf(pi, v8[e], acc[e]);
    }
    __syncthreads();
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) acc_s[sub][8 * w + e] = acc[e];
  __syncthreads();
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  if (tid < D) {
    float o = 0.0f;
    for (int i = 0; i < SUB; ++i) o += acc_s[i][tid];
    qs[tid] = o * inv;
  }
  __syncthreads();
  if (tid < D) {
    float o = qs[tid];
    if (a.unrotate) {
      o = 0.0f;
      for (int d = 0; d < D; ++d) o += (__builtin_popcount(d & tid) & 1) ? -qs[d] : qs[d];
      o *= D == 64 ? 0.125f : D == 256 ? 0.0625f : 0.08838834764831845f;
    }
    const int64_t off = t * a.out_token + h * a.out_head + tid;
    if (a.out_bf16)
      reinterpret_cast<__bf16*>(a.out)[off] = static_cast<__bf16>(o);
    else
      reinterpret_cast<float*>(a.out)[off] = o;
  }
  if (a.lse && tid == 0) a.lse[t * a.heads + h] = l == 0.0f ? -INFINITY : m + logf(l);
}

}  // namespace

int64_t kv_attention_workspace_bytes(int64_t, int64_t, int64_t, int64_t, int64_t) { return 16; }

hipError_t launch_kv_attention(const AttnArgs& a, hipStream_t st) {
  const int64_t blocks = a.T * a.heads;
  if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
  const dim3 grid{unsigned(blocks)};
  if (a.head_dim == 64)
    hipLaunchKernelGGL(kv_attention_kernel<64>, grid, dim3(256), 0, st, a);
  else if (a.head_dim == 128)
    hipLaunchKernelGGL(kv_attention_kernel<128>, grid, dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL(kv_attention_kernel<256>, grid, dim3(256), 0, st, a);
  return hipGetLastError();
}

}  // namespace rw4
