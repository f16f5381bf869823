// Host-side internals of the Gated DeltaNet layer's operators and of the norms with quantized outputs: what the C ABI
// hands the launchers.
#pragma once

#include "paged_internal.h"

namespace nvfp4 {

// Kernel arguments of add_rms_norm and gated_rms_norm (rms_norm.hip).  Rows of `blocks` 16-element blocks.
struct NormArgs {
  const void *x, *aux;             // aux: the residual, or the gates z
  int64_t x_row, aux_row;          // elements between rows
  int64_t x_head, aux_head;        // gated: elements between heads
  void* residual_out;              // nullptr: none
  int64_t residual_out_row;
  const float* weight;             // [cols], gated: [head dim]
  float eps;
  int32_t rows, blocks;
  int32_t head_blocks;             // gated: 16-element blocks per head (a power of two)
  int32_t row_lanes_log;           // rows that share a workgroup: log2 of a row's threads
  // outputs
  void* y;                         // nullptr: none
  int64_t y_row;
  int32_t y_bf16;
  uint8_t *codes, *scales;         // scales: NVFP4 only
  float* global;                   // [rows] written, or [1] read
  int32_t given;
};

int launch_rms_norm(const NormArgs& a, bool gated, int x_dtype, int aux_dtype, int format, hipStream_t stream);

// A pool of per-sequence states and the batch that uses it.
struct SeqState {
  void* state;
  int64_t slot;                    // elements between slots
  const int32_t *slots, *cu_q, *kv_len;
  int32_t num_slots, num_seqs, tokens;
};

// Kernel arguments of gdn_conv (gdn_conv.hip).
struct ConvArgs {
  SeqState s;
  const void* x;
  void* y;
  int64_t x_row, y_row;
  const float *weight, *bias;
  int32_t channels;
  int32_t out_bf16;
  int32_t run, tiles;              // tokens of a tile, tiles of 512 channels
};

int launch_gdn_conv(const ConvArgs& a, int x_dtype, int width, hipStream_t stream);

// Kernel arguments of gated_delta_rule (gdn_step.hip).
struct DeltaArgs {
  SeqState s;
  const uint16_t *q, *k, *v;
  int64_t q_tok, q_head, k_tok, k_head, v_tok, v_head, o_tok, o_head;
  const float *g, *beta;
  uint16_t* out;
  float scale;
  int32_t k_heads, v_heads, v_dim;
  FastDivU32 div_group;            // value heads per key head
};

int launch_gated_delta_rule(const DeltaArgs& a, int64_t max_q, int k_dim, void* workspace, hipStream_t stream);
size_t gated_delta_rule_workspace_bytes(int64_t tokens, int64_t max_q, int64_t num_seqs, int64_t k_heads,
                                        int64_t v_heads, int k_dim, int v_dim);

}  // namespace nvfp4
