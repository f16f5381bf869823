// Argument checks shared by the C ABI's files of head-vector operators.
#pragma once

#include "paged_internal.h"

namespace nvfp4 {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// A strided [tokens, heads, dim] operand of `esize`-byte elements.
inline int check_heads(const nvfp4_heads* x, int64_t tokens, int64_t dim, int64_t esize, HeadsView& v) {
  if (!x || !x->data || !aligned(x->data, 16) || x->heads <= 0) return NVFP4_ERR_INVALID_ARG;
  if (x->heads > 65536) return NVFP4_ERR_UNSUPPORTED;
  if (tokens > 1 && (x->token_stride < 0 || (x->token_stride * esize) % 16 != 0)) return NVFP4_ERR_INVALID_ARG;
  if (x->heads > 1 && (x->head_stride < dim || (x->head_stride * esize) % 16 != 0)) return NVFP4_ERR_INVALID_ARG;
  v = HeadsView{x->data, tokens > 1 ? x->token_stride : 0, x->heads > 1 ? x->head_stride : 0, (int32_t)x->heads};
  return NVFP4_OK;
}

// Rows written by several tokens at once would race: an output's tokens and heads must not overlap.
inline bool disjoint(const HeadsView& o, int64_t tokens, int64_t dim) {
  if (tokens <= 1 || o.heads <= 0) return true;
  const int64_t row = (int64_t)(o.heads - 1) * o.head + dim;
  // token rows apart, or heads apart with the tokens inside one head's pitch
  return o.tok >= row || (o.heads > 1 && o.tok >= dim && o.head >= (tokens - 1) * o.tok + dim) || (o.heads == 1 && o.tok >= dim);
}

inline int elem_size(int dtype) { return dtype == NVFP4_F32 ? 4 : 2; }

inline bool in_or_out_dtype(int d) { return d == NVFP4_F32 || d == NVFP4_BF16; }

}  // namespace nvfp4
