// Host-side internals of the paged key-value cache operators: what the C ABI hands the launchers.
#pragma once

#include "nvfp4_internal.h"

namespace nvfp4 {

// Head vectors with their strides in elements; heads == 0: absent.
struct HeadsView {
  void* data;
  int64_t tok, head;
  int32_t heads;
};

// Kernel arguments of qk_norm_rope and kv_append (rope_append.hip).
struct RopeAppendArgs {
  HeadsView q, k, v;             // inputs; v only when appending
  HeadsView q_out, k_out;        // k_out unused when appending
  const float *q_weight, *k_weight;
  const float* table;            // nullptr: no rotation
  const int32_t* positions;      // nullptr (append only): the token's place in its sequence
  int64_t table_rows;
  float eps;
  int32_t dim, rot, interleaved;
  int32_t tokens;
  int32_t out_bf16;
  // cache
  uint8_t *k_cache, *v_cache;
  int64_t k_page, v_page;        // bytes between pages
  const int32_t* page_table;
  int64_t table_stride;
  const float *k_scale, *v_scale;
  const int32_t *cu_q, *kv_len;
  int32_t num_pages, page_shift, num_seqs, table_width, scale_stride, fp8;
  int32_t groups, jobs;          // groups of head vectors and wavefronts per token
};

int launch_rope_append(const RopeAppendArgs& a, int x_dtype, bool append, hipStream_t stream);

// Kernel arguments of paged_attention (paged_attention.hip).
struct AttentionArgs {
  const uint16_t* q;
  uint16_t* out;
  float* lse;
  int64_t q_tok, q_head, o_tok, o_head;
  const uint8_t *k, *v;
  int64_t k_page, v_page;        // bytes between pages
  const int32_t* page_table;
  int64_t table_stride;
  const float *k_scale, *v_scale;   // nullptr: bf16 cache
  const int32_t *cu_q, *kv_len;
  int32_t num_pages, page_shift, num_seqs, table_width, scale_stride;
  int32_t tokens, q_heads, kv_heads, group;
  FastDivU32 div_group;
  float scale_log2;              // softmax scale * log2(e)
  int32_t causal, window;        // window 0: none
};

// Whether the blocks of a head that a split launch can plan, and a share of all heads' blocks, stay below 2^31
// whatever cu_q holds on the device.  In order, its sequences have at most `slots` row tiles of at most `cap` blocks each;
// where it is not (a caller's mistake, which must not lead to accesses out of range), every one of them may have
// all `tokens * group` rows, or the `rows_hi` that a launch takes at most.  per_sequence: the plan adds up sequences, else
// slots, each counted once.
inline bool plan_fits(bool per_sequence, int64_t slots, int64_t num_seqs, int64_t rows, int64_t rows_hi, int64_t bm,
                      int64_t cap, int64_t kv_heads, int64_t workgroups) {
  const int64_t most = rows < rows_hi ? rows : rows_hi;
  int64_t tiles = per_sequence ? num_seqs * ((most + bm - 1) / bm) : 0;
  if (tiles < slots) tiles = slots;
  return tiles * cap < INT32_MAX && tiles * cap / workgroups * kv_heads < INT32_MAX / 2;
}

int launch_paged_attention(const AttentionArgs& a, int64_t max_q, int head_dim, void* workspace, hipStream_t stream);
size_t paged_attention_workspace_bytes(int64_t tokens, int64_t max_q, int64_t num_seqs, int64_t q_heads,
                                       int64_t kv_heads, int head_dim);

}  // namespace nvfp4
