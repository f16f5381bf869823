// Device helpers of the operators that carry a state along each sequence (gdn_conv.hip, gdn_step.hip, gdn_chunk.hip).
#pragma once

#include "gdn_internal.h"
#include "paged_device.h"

namespace nvfp4 {

// The new tokens of sequence s as rows [first, end) of the call, inside [0, tokens] whatever cu_q holds.
struct SeqRows {
  int first, end;
};

__device__ __forceinline__ SeqRows seq_rows(const SeqState& s, int seq) {
  const int first = clamp_int(scalar_load(s.cu_q + seq), 0, s.tokens);
  return SeqRows{first, clamp_int(scalar_load(s.cu_q + seq + 1), first, s.tokens)};
}

// The slot of a sequence's state, or -1 where it has none.
__device__ __forceinline__ int seq_slot(const SeqState& s, int seq) {
  const int slot = s.slots ? scalar_load(s.slots + seq) : seq;
  return slot >= 0 && slot < s.num_slots ? slot : -1;
}

}  // namespace nvfp4
