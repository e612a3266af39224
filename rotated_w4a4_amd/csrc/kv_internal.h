// Host-side interface of the KV cache kernels (kvcache.hip, kvattn.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace rw4 {

// The caller's cache (include/rw4.h) with what the kernels derive from it.
struct KvCache {
  uint8_t* k_codes;
  float* k_scales;
  uint8_t* v_codes;
  float* v_scales;
  int64_t pages, slots;  // slots = pages << log2_page
  int log2_page, heads;
  int64_t code_page, code_head, code_slot;     // bytes
  int64_t scale_page, scale_head, scale_slot;  // floats
};

struct SlotsArgs {
  const int32_t* ctx_len;
  const int32_t* new_len;
  int64_t B;
  int log2_page;
  int32_t* block_table;
  int64_t table_width;
  int32_t* free_pages;
  int64_t capacity;
  const int32_t* free_state;
  int32_t* free_state_out;
  int32_t* kv_len;
  int32_t* cu_new;
  int32_t* served;
  int64_t* slot_map;
  int32_t* positions;
  int64_t tokens;
};

struct DenseRows {
  const void* in;
  int64_t in_token, in_head;
  void* out;
  int64_t out_token, out_head;
  int heads;
};

struct RowsArgs {
  DenseRows q, k;  // kv_append: k.out unused
  const void* v;
  int64_t v_token, v_head;
  const int64_t* slot_map;
  KvCache cache;
  int64_t T;
  int head_dim;
  const float* q_weight;
  const float* k_weight;
  float eps;
  const float* cos_sin;
  int64_t max_pos;
  int rot;
  int interleaved, rotate, out_bf16;
  const int32_t* positions;
};

struct AttnArgs {
  KvCache cache;
  const void* q;
  int64_t q_token, q_head;
  int64_t T;
  int heads, head_dim, group;  // group: query heads of a KV head
  int q_bf16, out_bf16;
  const int32_t* block_table;
  int64_t table_width;
  const int32_t* kv_len;
  const int32_t* cu_q;
  int64_t B, max_q_len;
  float scale;
  int causal, unrotate;
  int64_t window;
  int sinks;  // first keys that stay visible; 0 where window is 0
  void* out;
  int64_t out_token, out_head;
  float* lse;
  void* workspace;
};

hipError_t launch_kv_slots(const SlotsArgs& a, hipStream_t st);
hipError_t launch_qk_norm_rope(const RowsArgs& a, bool x_bf16, hipStream_t st);
hipError_t launch_kv_append(const RowsArgs& a, bool x_bf16, hipStream_t st);

int64_t kv_attention_workspace_bytes(int64_t T, int64_t heads, int64_t kv_heads, int64_t head_dim);
hipError_t launch_kv_attention(const AttnArgs& a, hipStream_t st);

}  // namespace rw4
