// The blockwise kernels of the gated delta rule (gdn_chunk.hip) as the operator's dispatch (gdn_step.hip) sees them.
#pragma once

#include "gdn_internal.h"

namespace nvfp4 {

struct ChunkWork {
  _Float16 *k, *q, *t, *a;         // fragments of every block
  float* factors;
  uint8_t* flags;                  // [sequence][value head][16 columns]: left to the token-by-token kernel
  int64_t blocks;                  // slots for blocks of 64 tokens
  int32_t short_len;               // sequences up to this length are the token-by-token kernel's
};

// Lays the workspace out from `base` on and returns its size.
size_t chunk_workspace(int64_t tokens, int64_t num_seqs, int64_t k_heads, int64_t v_heads, int k_dim, int v_dim, void* base,
                       ChunkWork& ws);
int launch_chunks(const DeltaArgs& a, const ChunkWork& ws, int64_t max_q, int k_dim, hipStream_t stream);

}  // namespace nvfp4
