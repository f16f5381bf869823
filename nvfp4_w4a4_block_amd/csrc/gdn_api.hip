// C ABI of the Gated DeltaNet layer's operators and of the norms with quantized outputs: argument validation and
// dispatch.  Every argument error is detected here, on the host, before anything is enqueued; what lies on the device
// (cu_q, kv_len, slots) is bounds-checked by the kernels.
#include <math.h>

#include "abi_checks.h"
#include "gdn_internal.h"

using namespace nvfp4;

namespace {

constexpr int64_t kMaxNormCols = 32768;        // 1024 threads of two 16-element blocks

// The outputs of a norm over rows of `cols` columns.
int check_norm_out(const nvfp4_norm_out* o, int64_t rows, int64_t cols, NormArgs& a) {
  if (!o || o->format < NVFP4_NORM_PLAIN || o->format > NVFP4_NORM_FP8) return NVFP4_ERR_INVALID_ARG;
  if (!o->y && o->format == NVFP4_NORM_PLAIN) return NVFP4_ERR_INVALID_ARG;
  if (o->y) {
    if (!in_or_out_dtype(o->y_dtype) || !aligned(o->y, 16)) return NVFP4_ERR_INVALID_ARG;
    if (rows > 1 && (o->ldy < cols || (o->ldy * elem_size(o->y_dtype)) % 16 != 0)) return NVFP4_ERR_INVALID_ARG;
  }
  if (o->format != NVFP4_NORM_PLAIN) {
    if (o->mode != NVFP4_SCALE_PER_ROW && o->mode != NVFP4_SCALE_GIVEN) return NVFP4_ERR_INVALID_ARG;
    if (!o->codes || !aligned(o->codes, 16) || !o->scale || !aligned(o->scale, 4)) return NVFP4_ERR_INVALID_ARG;
    if (o->format == NVFP4_NORM_NVFP4 && !o->block_scales) return NVFP4_ERR_INVALID_ARG;
  }
  a.y = o->y;
  a.y_row = rows > 1 ? o->ldy : 0;
  a.y_bf16 = o->y_dtype == NVFP4_BF16;
  a.codes = o->codes;
  a.scales = o->block_scales;
  a.global = o->scale;
  a.given = o->mode == NVFP4_SCALE_GIVEN;
  return NVFP4_OK;
}

// A pool of states with `per_slot` contiguous elements of `esize` bytes each.
int check_states(const nvfp4_seq_states* p, int64_t tokens, int64_t per_slot, int64_t esize, SeqState& s) {
  if (!p || p->num_seqs < 0 || p->num_slots < 0) return NVFP4_ERR_INVALID_ARG;
  if (p->num_slots > INT32_MAX || p->num_seqs > INT32_MAX / 2) return NVFP4_ERR_UNSUPPORTED;
  if (tokens == 0 || p->num_seqs == 0) return NVFP4_OK;
  if (!p->cu_q || !p->kv_len || !aligned(p->cu_q, 4) || !aligned(p->kv_len, 4) || !aligned(p->slots, 4))
    return NVFP4_ERR_INVALID_ARG;
  if (p->num_slots > 0 && (!p->data || !aligned(p->data, 16))) return NVFP4_ERR_INVALID_ARG;
  if (p->num_slots > 1 && (p->slot_stride < per_slot || (p->slot_stride * esize) % 16 != 0)) return NVFP4_ERR_INVALID_ARG;
  s.state = p->data;
  s.slot = p->num_slots > 1 ? p->slot_stride : 0;
  s.slots = p->slots;
  s.cu_q = p->cu_q;
  s.kv_len = p->kv_len;
  s.num_slots = (int32_t)p->num_slots;
  s.num_seqs = p->num_seqs;
  s.tokens = (int32_t)tokens;
  return NVFP4_OK;
}

}  // namespace

extern "C" {

int nvfp4_add_rms_norm(int64_t rows, int64_t cols, const void* x, int x_dtype, int64_t ldx, const void* residual,
                       int residual_dtype, int64_t ldr, const float* weight, float eps, void* residual_out, int64_t ldro,
                       const nvfp4_norm_out* out, void* stream) {
  if (rows < 0 || cols <= 0 || cols % 16 != 0 || !in_or_out_dtype(x_dtype) || !(eps >= 0.0f)) return NVFP4_ERR_INVALID_ARG;
  if (residual && !in_or_out_dtype(residual_dtype)) return NVFP4_ERR_INVALID_ARG;
  if (!residual && residual_out) return NVFP4_ERR_INVALID_ARG;
  if (cols > kMaxNormCols || rows > INT32_MAX / 1024) return NVFP4_ERR_UNSUPPORTED;       // threads of a launch below 2^32
  NormArgs a{};
  if (rows == 0) return NVFP4_OK;
  const int st = check_norm_out(out, rows, cols, a);
  if (st != NVFP4_OK) return st;
  if (!x || !weight || !aligned(x, 16) || !aligned(weight, 16) || !aligned(residual, 16) || !aligned(residual_out, 16))
    return NVFP4_ERR_INVALID_ARG;
  if (rows > 1) {
    if (ldx < cols || (ldx * elem_size(x_dtype)) % 16 != 0) return NVFP4_ERR_INVALID_ARG;
    if (residual && (ldr < cols || (ldr * elem_size(residual_dtype)) % 16 != 0)) return NVFP4_ERR_INVALID_ARG;
    if (residual_out && (ldro < cols || (ldro * elem_size(residual_dtype)) % 16 != 0)) return NVFP4_ERR_INVALID_ARG;
  }
  a.x = x;
  a.x_row = rows > 1 ? ldx : 0;
  a.aux = residual;
  a.aux_row = rows > 1 ? ldr : 0;
  a.residual_out = residual_out;
  a.residual_out_row = rows > 1 ? ldro : 0;
  a.weight = weight;
  a.eps = eps;
  a.rows = (int32_t)rows;
  a.blocks = (int32_t)(cols / 16);
  return launch_rms_norm(a, false, x_dtype, residual ? residual_dtype : x_dtype, out->format, static_cast<hipStream_t>(stream));
}

int nvfp4_gated_rms_norm(int64_t tokens, int64_t head_dim, const nvfp4_heads* x, int x_dtype, const nvfp4_heads* z, int z_dtype,
                         const float* weight, float eps, const nvfp4_norm_out* out, void* stream) {
  if (tokens < 0 || head_dim < 16 || (head_dim & (head_dim - 1)) != 0 || !in_or_out_dtype(x_dtype) || !in_or_out_dtype(z_dtype) ||
      !(eps >= 0.0f))
    return NVFP4_ERR_INVALID_ARG;
  if (head_dim > 1024 || tokens > INT32_MAX / 1024) return NVFP4_ERR_UNSUPPORTED;
  if (!x || !z || x->heads <= 0 || x->heads != z->heads) return NVFP4_ERR_INVALID_ARG;
  if (x->heads > kMaxNormCols / head_dim) return NVFP4_ERR_UNSUPPORTED;
  if (tokens == 0) return NVFP4_OK;
  HeadsView xv, zv;
  int st = check_heads(x, tokens, head_dim, elem_size(x_dtype), xv);
  if (st == NVFP4_OK) st = check_heads(z, tokens, head_dim, elem_size(z_dtype), zv);
  NormArgs a{};
  if (st == NVFP4_OK) st = check_norm_out(out, tokens, xv.heads * head_dim, a);
  if (st != NVFP4_OK) return st;
  if (!weight || !aligned(weight, 16)) return NVFP4_ERR_INVALID_ARG;
  a.x = xv.data;
  a.x_row = xv.tok;
  a.x_head = xv.head;
  a.aux = zv.data;
  a.aux_row = zv.tok;
  a.aux_head = zv.head;
  a.weight = weight;
  a.eps = eps;
  a.rows = (int32_t)tokens;
  a.head_blocks = (int32_t)(head_dim / 16);
  a.blocks = xv.heads * a.head_blocks;
  return launch_rms_norm(a, true, x_dtype, z_dtype, out->format, static_cast<hipStream_t>(stream));
}

int nvfp4_gdn_conv(const nvfp4_seq_states* states, int64_t tokens, int64_t channels, int width, const void* x, int x_dtype,
                   int64_t ldx, const float* weight, const float* bias, void* y, int y_dtype, int64_t ldy, void* stream) {
  if (tokens < 0 || channels <= 0 || channels % 8 != 0 || !in_or_out_dtype(x_dtype) || !in_or_out_dtype(y_dtype))
    return NVFP4_ERR_INVALID_ARG;
  if (width < 2 || width > 4 || tokens > INT32_MAX / 2 || channels > (1 << 24)) return NVFP4_ERR_UNSUPPORTED;
  ConvArgs a{};
  const int st = check_states(states, tokens, (width - 1) * channels, elem_size(x_dtype), a.s);
  if (st != NVFP4_OK || tokens == 0 || states->num_seqs == 0) return st;
  if (!x || !y || !weight || !aligned(x, 16) || !aligned(y, 16) || !aligned(weight, 16) || !aligned(bias, 16))
    return NVFP4_ERR_INVALID_ARG;
  if (tokens > 1 && (ldx < channels || ldy < channels || (ldx * elem_size(x_dtype)) % 16 != 0 || (ldy * elem_size(y_dtype)) % 16 != 0))
    return NVFP4_ERR_INVALID_ARG;
  a.x = x;
  a.x_row = tokens > 1 ? ldx : 0;
  a.y = y;
  a.y_row = tokens > 1 ? ldy : 0;
  a.weight = weight;
  a.bias = bias;
  a.channels = (int32_t)channels;
  a.out_bf16 = y_dtype == NVFP4_BF16;
  return launch_gdn_conv(a, x_dtype, width, static_cast<hipStream_t>(stream));
}

size_t nvfp4_gated_delta_rule_workspace_size(int64_t tokens, int64_t max_q, int64_t num_seqs, int64_t k_heads, int64_t v_heads,
                                             int64_t k_dim, int64_t v_dim) {
  if (tokens <= 0 || max_q < 0 || num_seqs <= 0 || k_heads <= 0 || v_heads <= 0 || v_heads % k_heads != 0 ||
      (k_dim != 64 && k_dim != 128) || v_dim <= 0 || v_dim % 32 != 0 || v_dim > 512 || tokens > INT32_MAX / 2 ||
      num_seqs > INT32_MAX || v_heads > 65536)
    return 0;
  return gated_delta_rule_workspace_bytes(tokens, max_q, num_seqs, k_heads, v_heads, (int)k_dim, (int)v_dim);
}

int nvfp4_gated_delta_rule(const nvfp4_seq_states* states, int64_t tokens, int64_t max_q, int64_t k_dim, int64_t v_dim,
                           const nvfp4_heads* q, const nvfp4_heads* k, const nvfp4_heads* v, const float* g, const float* beta,
                           float scale, const nvfp4_heads* out, void* workspace, size_t workspace_bytes, void* stream) {
  if (tokens < 0 || max_q < 0 || k_dim <= 0 || v_dim <= 0 || !isfinite(scale)) return NVFP4_ERR_INVALID_ARG;
  if ((k_dim != 64 && k_dim != 128) || v_dim % 32 != 0 || v_dim > 512 || tokens > INT32_MAX / 2) return NVFP4_ERR_UNSUPPORTED;
  if (!q || !k || !v || !out || q->heads <= 0 || k->heads != q->heads || v->heads != out->heads || v->heads % q->heads != 0)
    return NVFP4_ERR_INVALID_ARG;
  if (v->heads > 65536) return NVFP4_ERR_UNSUPPORTED;
  DeltaArgs a{};
  int st = check_states(states, tokens, v->heads * k_dim * v_dim, 4, a.s);
  if (st != NVFP4_OK || tokens == 0 || states->num_seqs == 0) return st;
  HeadsView qv, kv, vv, ov;
  st = check_heads(q, tokens, k_dim, 2, qv);
  if (st == NVFP4_OK) st = check_heads(k, tokens, k_dim, 2, kv);
  if (st == NVFP4_OK) st = check_heads(v, tokens, v_dim, 2, vv);
  if (st == NVFP4_OK) st = check_heads(out, tokens, v_dim, 2, ov);
  if (st != NVFP4_OK) return st;
  if (vv.tok >= 1 << 24 || ov.tok >= 1 << 24) return NVFP4_ERR_UNSUPPORTED;      // 64 rows within 2^31 bytes
  if (!disjoint(ov, tokens, v_dim) || !g || !beta || !aligned(g, 4) || !aligned(beta, 4)) return NVFP4_ERR_INVALID_ARG;
  const size_t need = gated_delta_rule_workspace_bytes(tokens, max_q, states->num_seqs, qv.heads, vv.heads, (int)k_dim, (int)v_dim);
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 16))) return NVFP4_ERR_WORKSPACE;
  a.q = static_cast<const uint16_t*>(qv.data);
  a.k = static_cast<const uint16_t*>(kv.data);
  a.v = static_cast<const uint16_t*>(vv.data);
  a.out = static_cast<uint16_t*>(ov.data);
  a.q_tok = qv.tok;
  a.q_head = qv.head;
  a.k_tok = kv.tok;
  a.k_head = kv.head;
  a.v_tok = vv.tok;
  a.v_head = vv.head;
  a.o_tok = ov.tok;
  a.o_head = ov.head;
  a.g = g;
  a.beta = beta;
  a.scale = scale;
  a.k_heads = qv.heads;
  a.v_heads = vv.heads;
  a.v_dim = (int32_t)v_dim;
  a.div_group = make_fastdiv((uint32_t)(vv.heads / qv.heads));
  return launch_gated_delta_rule(a, max_q, (int)k_dim, workspace, static_cast<hipStream_t>(stream));
}

}  // extern "C"
