// C ABI of the paged key-value cache operators: argument validation and dispatch.  Every argument
// error is detected here, on the host, before anything is enqueued; what lies on the device (cu_q,
// kv_len, the page table, positions) is bounds-checked by the kernels.
#include <math.h>

#include "paged_internal.h"

using namespace nvfp4;

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// A strided [tokens, heads, dim] operand of `esize`-byte elements.
int check_heads(const nvfp4_heads* x, int64_t tokens, int64_t dim, int64_t esize, HeadsView& v) {
  if (!x || !x->data || !aligned(x->data, 16) || x->heads <= 0) return NVFP4_ERR_INVALID_ARG;
  if (x->heads > 65536) return NVFP4_ERR_UNSUPPORTED;
  if (tokens > 1 && (x->token_stride < 0 || (x->token_stride * esize) % 16 != 0)) return NVFP4_ERR_INVALID_ARG;
  if (x->heads > 1 && (x->head_stride < dim || (x->head_stride * esize) % 16 != 0)) return NVFP4_ERR_INVALID_ARG;
  v = HeadsView{x->data, tokens > 1 ? x->token_stride : 0, x->heads > 1 ? x->head_stride : 0, (int32_t)x->heads};
  return NVFP4_OK;
}

// Rows written by several tokens at once would race: an output's tokens and heads must not overlap.
bool disjoint(const HeadsView& o, int64_t tokens, int64_t dim) {
  if (tokens <= 1 || o.heads <= 0) return true;
  const int64_t row = (int64_t)(o.heads - 1) * o.head + dim;
  // token rows apart, or heads apart with the tokens inside one head's pitch
  return o.tok >= row || (o.heads > 1 && o.tok >= dim && o.head >= (tokens - 1) * o.tok + dim) || (o.heads == 1 && o.tok >= dim);
}

int check_rope(const nvfp4_rope* r, int64_t dim, bool need_positions, RopeAppendArgs& a) {
  if (!r) return NVFP4_OK;
  if (!r->table || !aligned(r->table, 16) || r->rows < 0 || r->dim <= 0 || r->dim % 16 != 0 || r->dim > dim)
    return NVFP4_ERR_INVALID_ARG;
  if (r->interleaved != 0 && r->interleaved != 1) return NVFP4_ERR_INVALID_ARG;
  if (!aligned(r->positions, 4) || (need_positions && !r->positions)) return NVFP4_ERR_INVALID_ARG;
  a.table = r->table;
  a.table_rows = r->rows;
  a.positions = r->positions;
  a.rot = r->dim;
  a.interleaved = r->interleaved;
  return NVFP4_OK;
}

int elem_size(int dtype) { return dtype == NVFP4_F32 ? 4 : 2; }

bool in_or_out_dtype(int d) { return d == NVFP4_F32 || d == NVFP4_BF16; }

int check_cache(const nvfp4_paged_kv* c, int64_t tokens) {
  if (!c) return NVFP4_ERR_INVALID_ARG;
  if (c->dtype != NVFP4_E4M3 && c->dtype != NVFP4_BF16) return NVFP4_ERR_INVALID_ARG;
  if (c->kv_heads <= 0 || c->head_dim <= 0 || c->num_seqs < 0 || c->table_width < 0 || c->num_pages < 0)
    return NVFP4_ERR_INVALID_ARG;
  if (c->page_size <= 0 || (c->page_size & (c->page_size - 1)) != 0) return NVFP4_ERR_INVALID_ARG;
  if (c->page_size < 16 || c->page_size > 1024 || c->num_pages > INT32_MAX || c->kv_heads > 65536)
    return NVFP4_ERR_UNSUPPORTED;
  if ((int64_t)c->table_width * c->page_size > INT32_MAX) return NVFP4_ERR_UNSUPPORTED;
  if (tokens == 0 || c->num_seqs == 0) return NVFP4_OK;
  if (c->num_pages == 0 || !c->k || !c->v || !aligned(c->k, 16) || !aligned(c->v, 16)) return NVFP4_ERR_INVALID_ARG;
  const int64_t esize = c->dtype == NVFP4_E4M3 ? 1 : 2;
  const int64_t page = (int64_t)c->kv_heads * c->page_size * c->head_dim;
  if (page > INT32_MAX) return NVFP4_ERR_UNSUPPORTED;
  if (c->num_pages > 1 && (c->k_page_stride < page || c->v_page_stride < page || (c->k_page_stride * esize) % 16 != 0 ||
                           (c->v_page_stride * esize) % 16 != 0))
    return NVFP4_ERR_INVALID_ARG;
  if (!c->cu_q || !c->kv_len || !aligned(c->cu_q, 4) || !aligned(c->kv_len, 4)) return NVFP4_ERR_INVALID_ARG;
  if (c->table_width > 0 && (!c->page_table || !aligned(c->page_table, 4) ||
                             (c->num_seqs > 1 && c->table_stride < c->table_width)))
    return NVFP4_ERR_INVALID_ARG;
  if (c->dtype == NVFP4_E4M3) {
    if (c->scale_count != 1 && c->scale_count != c->kv_heads) return NVFP4_ERR_INVALID_ARG;
    if (!c->k_scale || !c->v_scale || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4)) return NVFP4_ERR_INVALID_ARG;
  }
  return NVFP4_OK;
}

int log2_of(int v) {
  int s = 0;
  while ((1 << s) < v) ++s;
  return s;
}

}  // namespace

extern "C" {

int nvfp4_qk_norm_rope(int64_t tokens, int64_t head_dim, int x_dtype, const nvfp4_heads* q, const nvfp4_heads* k,
                       const float* q_weight, const float* k_weight, float eps, const nvfp4_rope* rope, int out_dtype,
                       const nvfp4_heads* q_out, const nvfp4_heads* k_out, void* stream) {
  if (tokens < 0 || head_dim <= 0 || head_dim % 16 != 0 || !in_or_out_dtype(x_dtype) || !in_or_out_dtype(out_dtype))
    return NVFP4_ERR_INVALID_ARG;
  if (head_dim > 512 || tokens > INT32_MAX) return NVFP4_ERR_UNSUPPORTED;
  if (!q || !q_out || !k != !k_out || !(eps >= 0.0f)) return NVFP4_ERR_INVALID_ARG;
  if (tokens == 0) return NVFP4_OK;
  RopeAppendArgs a{};
  int st = check_heads(q, tokens, head_dim, elem_size(x_dtype), a.q);
  if (st == NVFP4_OK) st = check_heads(q_out, tokens, head_dim, elem_size(out_dtype), a.q_out);
  if (st == NVFP4_OK && k) st = check_heads(k, tokens, head_dim, elem_size(x_dtype), a.k);
  if (st == NVFP4_OK && k) st = check_heads(k_out, tokens, head_dim, elem_size(out_dtype), a.k_out);
  if (st == NVFP4_OK) st = check_rope(rope, head_dim, true, a);
  if (st != NVFP4_OK) return st;
  if (a.q.heads != a.q_out.heads || a.k.heads != a.k_out.heads) return NVFP4_ERR_INVALID_ARG;
  if (!disjoint(a.q_out, tokens, head_dim) || !disjoint(a.k_out, tokens, head_dim)) return NVFP4_ERR_INVALID_ARG;
  if (!aligned(q_weight, 16) || !aligned(k_weight, 16)) return NVFP4_ERR_INVALID_ARG;
  a.q_weight = q_weight;
  a.k_weight = k_weight;
  a.eps = eps;
  a.dim = (int32_t)head_dim;
  a.tokens = (int32_t)tokens;
  a.out_bf16 = out_dtype == NVFP4_BF16;
  return launch_rope_append(a, x_dtype, false, static_cast<hipStream_t>(stream));
}

int nvfp4_kv_append(const nvfp4_paged_kv* kv, int64_t tokens, int x_dtype, const nvfp4_heads* k, const nvfp4_heads* v,
                    const float* k_weight, float eps, const nvfp4_rope* rope, const nvfp4_heads* q,
                    const float* q_weight, int q_out_dtype, const nvfp4_heads* q_out, void* stream) {
  if (tokens < 0 || !in_or_out_dtype(x_dtype) || !(eps >= 0.0f)) return NVFP4_ERR_INVALID_ARG;
  if (tokens > INT32_MAX) return NVFP4_ERR_UNSUPPORTED;
  int st = check_cache(kv, tokens);
  if (st != NVFP4_OK) return st;
  const int64_t dim = kv->head_dim;
  if (dim % 16 != 0) return NVFP4_ERR_INVALID_ARG;
  if (dim > 512) return NVFP4_ERR_UNSUPPORTED;
  if (!k || !v || !q != !q_out || (q && !in_or_out_dtype(q_out_dtype))) return NVFP4_ERR_INVALID_ARG;
  if (tokens == 0 || kv->num_seqs == 0) return NVFP4_OK;
  RopeAppendArgs a{};
  st = check_heads(k, tokens, dim, elem_size(x_dtype), a.k);
  if (st == NVFP4_OK) st = check_heads(v, tokens, dim, elem_size(x_dtype), a.v);
  if (st == NVFP4_OK && q) st = check_heads(q, tokens, dim, elem_size(x_dtype), a.q);
  if (st == NVFP4_OK && q) st = check_heads(q_out, tokens, dim, elem_size(q_out_dtype), a.q_out);
  if (st == NVFP4_OK) st = check_rope(rope, dim, false, a);
  if (st != NVFP4_OK) return st;
  if (a.k.heads != kv->kv_heads || a.v.heads != kv->kv_heads || a.q.heads != a.q_out.heads) return NVFP4_ERR_INVALID_ARG;
  if (!disjoint(a.q_out, tokens, dim)) return NVFP4_ERR_INVALID_ARG;
  if (!aligned(q_weight, 16) || !aligned(k_weight, 16)) return NVFP4_ERR_INVALID_ARG;
  const int64_t esize = kv->dtype == NVFP4_E4M3 ? 1 : 2;
  a.q_weight = q_weight;
  a.k_weight = k_weight;
  a.eps = eps;
  a.dim = (int32_t)dim;
  a.tokens = (int32_t)tokens;
  a.out_bf16 = q_out_dtype == NVFP4_BF16;
  a.k_cache = static_cast<uint8_t*>(kv->k);
  a.v_cache = static_cast<uint8_t*>(kv->v);
  a.k_page = kv->num_pages > 1 ? kv->k_page_stride * esize : 0;
  a.v_page = kv->num_pages > 1 ? kv->v_page_stride * esize : 0;
  a.page_table = kv->page_table;
  a.table_stride = kv->num_seqs > 1 ? kv->table_stride : 0;
  a.k_scale = kv->k_scale;
  a.v_scale = kv->v_scale;
  a.cu_q = kv->cu_q;
  a.kv_len = kv->kv_len;
  a.num_pages = (int32_t)kv->num_pages;
  a.page_shift = log2_of(kv->page_size);
  a.num_seqs = kv->num_seqs;
  a.table_width = kv->table_width;
  a.scale_stride = kv->scale_count > 1 ? 1 : 0;
  a.fp8 = kv->dtype == NVFP4_E4M3;
  return launch_rope_append(a, x_dtype, true, static_cast<hipStream_t>(stream));
}

size_t nvfp4_paged_attention_workspace_size(int64_t tokens, int64_t max_q, int64_t num_seqs, int64_t q_heads,
                                            int64_t kv_heads, int64_t head_dim, int dtype) {
  if (tokens <= 0 || max_q < 0 || num_seqs <= 0 || q_heads <= 0 || kv_heads <= 0 || q_heads % kv_heads != 0 ||
      (head_dim != 64 && head_dim != 128 && head_dim != 256) || (dtype != NVFP4_E4M3 && dtype != NVFP4_BF16))
    return 0;
  return paged_attention_workspace_bytes(tokens, max_q, num_seqs, q_heads, kv_heads, (int)head_dim);
}

int nvfp4_paged_attention(const nvfp4_paged_kv* kv, int64_t tokens, int64_t max_q, const nvfp4_heads* q, float scale,
                          int causal, int64_t window, const nvfp4_heads* out, float* lse, void* workspace,
                          size_t workspace_bytes, void* stream) {
  if (tokens < 0 || max_q < 0 || window < 0 || (causal != 0 && causal != 1) || (window > 0 && !causal))
    return NVFP4_ERR_INVALID_ARG;
  if (!(scale > 0.0f) || !isfinite(scale)) return NVFP4_ERR_INVALID_ARG;
  int st = check_cache(kv, tokens);
  if (st != NVFP4_OK) return st;
  const int64_t dim = kv->head_dim;
  if (dim != 64 && dim != 128 && dim != 256) return NVFP4_ERR_UNSUPPORTED;
  // key numbers stay in 32 bits, also a block past the end, and where cu_q is not ordered and a tile is given the
  // blocks of another
  if ((int64_t)kv->table_width * kv->page_size > (int64_t)1 << 30) return NVFP4_ERR_UNSUPPORTED;
  if (!q || !out) return NVFP4_ERR_INVALID_ARG;
  if (tokens == 0 || kv->num_seqs == 0) return NVFP4_OK;
  HeadsView qv, ov;
  st = check_heads(q, tokens, dim, 2, qv);
  if (st == NVFP4_OK) st = check_heads(out, tokens, dim, 2, ov);
  if (st != NVFP4_OK) return st;
  if (qv.heads != ov.heads || qv.heads % kv->kv_heads != 0 || !disjoint(ov, tokens, dim) || !aligned(lse, 4))
    return NVFP4_ERR_INVALID_ARG;
  const int64_t group = qv.heads / kv->kv_heads;
  if (group > 256 || tokens * qv.heads + kv->num_seqs > (int64_t)INT32_MAX / 2) return NVFP4_ERR_UNSUPPORTED;
  const size_t need = paged_attention_workspace_bytes(tokens, max_q, kv->num_seqs, qv.heads, kv->kv_heads, (int)dim);
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 16))) return NVFP4_ERR_WORKSPACE;
  const int64_t esize = kv->dtype == NVFP4_E4M3 ? 1 : 2;
  AttentionArgs a{};
  a.q = static_cast<const uint16_t*>(qv.data);
  a.out = static_cast<uint16_t*>(ov.data);
  a.lse = lse;
  a.q_tok = qv.tok;
  a.q_head = qv.head;
  a.o_tok = ov.tok;
  a.o_head = ov.head;
  a.k = static_cast<const uint8_t*>(kv->k);
  a.v = static_cast<const uint8_t*>(kv->v);
  a.k_page = kv->num_pages > 1 ? kv->k_page_stride * esize : 0;
  a.v_page = kv->num_pages > 1 ? kv->v_page_stride * esize : 0;
  a.page_table = kv->page_table;
  a.table_stride = kv->num_seqs > 1 ? kv->table_stride : 0;
  a.k_scale = kv->dtype == NVFP4_E4M3 ? kv->k_scale : nullptr;
  a.v_scale = kv->dtype == NVFP4_E4M3 ? kv->v_scale : nullptr;
  a.cu_q = kv->cu_q;
  a.kv_len = kv->kv_len;
  a.num_pages = (int32_t)kv->num_pages;
  a.page_shift = log2_of(kv->page_size);
  a.num_seqs = kv->num_seqs;
  a.table_width = kv->table_width;
  a.scale_stride = kv->scale_count > 1 ? 1 : 0;
  a.tokens = (int32_t)tokens;
  a.q_heads = qv.heads;
  a.kv_heads = kv->kv_heads;
  a.group = (int32_t)group;
  a.div_group = make_fastdiv((uint32_t)group);
  a.scale_log2 = scale * 1.44269504088896340736f;
  a.causal = causal;
  a.window = window > INT32_MAX ? 0 : (int32_t)window;
  return launch_paged_attention(a, max_q, (int)dim, workspace, static_cast<hipStream_t>(stream));
}

}  // extern "C"
