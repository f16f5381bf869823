// The gated delta rule token by token (gfx950): single tokens, drafts, short sequences, and the dispatch of the
// operator.  Per value head, with the state S [Dk, Dv] in fp32, k^ = k / sqrt(k.k + 1e-6) and q^ likewise:
//   S <- e^g S,  u = beta (v - S^T k^),  S <- S + k^ u^T,  o = scale S^T q^
//
// The columns of S do not meet: a wavefront keeps 16 of them (a lane 4 columns of Dk / 16 consecutive rows) in
// registers over all the sequence's new tokens, with no barrier.  Both products with the old state are taken in
// one pass and one reduction, o = scale (e^g S^T q^ + (k^.q^) u).
// HBM-bound for single tokens: a state is read once and written once (64 sequences of 32 heads of 128 x 128, 270 MB: 62 us,
// 4.4 TB/s; 44 us with the states still in the 256 MB cache).
#include "gdn_chunk.h"
#include "seq_device.h"

namespace nvfp4 {

namespace {

constexpr int kThreads = 256;

// Sum over the 16 row groups: lanes 4 apart.
__device__ __forceinline__ float rows_sum(float v) {
#pragma unroll
  for (int m = 4; m < 64; m *= 2) v += __shfl_xor(v, m, 64);
  return v;
}

template <int N>
__device__ __forceinline__ void load_row(const uint16_t* p, float (&v)[N]) {
  if constexpr (N == 8) {
    widen(*reinterpret_cast<const uint4*>(p), v, static_cast<const uint16_t*>(nullptr));
  } else {
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    v[0] = __uint_as_float(w.x << 16);
    v[1] = __uint_as_float(w.x & 0xFFFF0000u);
    v[2] = __uint_as_float(w.y << 16);
    v[3] = __uint_as_float(w.y & 0xFFFF0000u);
  }
}

// x <- x / sqrt(x.x + 1e-6), a lane holding R of the row's values.  Ahead of the products with the state, so that
// those stay in range; a row whose squares do not is scaled by 2^-80 first, which makes 1e-6 less than 2^-179: nothing
// beside a scaled sum of 2^-60 and more.
template <int R>
__device__ __forceinline__ void unit_row(float (&x)[R]) {
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < R; ++i) s = __builtin_fmaf(x[i], x[i], s);
  s = rows_sum(s);
  float eps = 1e-6f;
  if (!(s < 0x1p100f)) {
    s = eps = 0.0f;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      x[i] *= 0x1p-80f;
      s = __builtin_fmaf(x[i], x[i], s);
    }
    s = rows_sum(s);
  }
  const float r = 1.0f / __builtin_sqrtf(s + eps);
#pragma unroll
  for (int i = 0; i < R; ++i) x[i] *= r;
}

template <int DK>
__global__ __launch_bounds__(kThreads) void delta_step_kernel(DeltaArgs a, int short_len, const uint8_t* flags) {
  constexpr int R = DK / 16;
  const int lane = threadIdx.x & 63;
  const int slices = a.v_dim / 16;
  const int64_t job = (int64_t)blockIdx.x * (kThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int slice = (int)(job % slices);
  const int64_t pair = job / slices;
  const int seq = (int)(pair / a.v_heads), head = (int)(pair - (int64_t)seq * a.v_heads);
  if (seq >= a.s.num_seqs) return;
  const SeqRows rows = seq_rows(a.s, seq);
  const int n = rows.end - rows.first;
  // longer sequences: only the slices that the blockwise kernel left
  if (n == 0 || (n > short_len && flags[pair * slices + slice] == 0)) return;
  const int slot = seq_slot(a.s, seq);
  const int k_head = (int)fastdiv((uint32_t)head, a.div_group);
  const int r0 = (lane >> 2) * R, c0 = slice * 16 + (lane & 3) * 4;
  float4 S[R];
  float* state = static_cast<float*>(a.s.state) + (slot >= 0 ? slot : 0) * a.s.slot + ((int64_t)head * DK + r0) * a.v_dim + c0;
  const bool old = slot >= 0 && scalar_load(a.s.kv_len + seq) > n;
#pragma unroll
  for (int i = 0; i < R; ++i)
    S[i] = old ? *reinterpret_cast<const float4*>(state + (int64_t)i * a.v_dim) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);

  for (int64_t t = rows.first; t < rows.end; ++t) {
    float k[R], q[R], v[4];
    load_row(a.k + t * a.k_tok + k_head * a.k_head + r0, k);
    load_row(a.q + t * a.q_tok + k_head * a.q_head + r0, q);
    load_row(a.v + t * a.v_tok + head * a.v_head + c0, v);
    const float decay = expf(a.g[t * a.v_heads + head]), beta = a.beta[t * a.v_heads + head];
    unit_row(k);
    unit_row(q);
    float kq = 0.0f;
    float p[4] = {0.0f, 0.0f, 0.0f, 0.0f}, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < R; ++i) {
      kq = __builtin_fmaf(k[i], q[i], kq);
      const float s[4] = {S[i].x, S[i].y, S[i].z, S[i].w};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        p[c] = __builtin_fmaf(s[c], k[i], p[c]);
        o[c] = __builtin_fmaf(s[c], q[i], o[c]);
      }
    }
    kq = rows_sum(kq);
    float u[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      u[c] = beta * (v[c] - decay * rows_sum(p[c]));
      o[c] = a.scale * (decay * rows_sum(o[c]) + kq * u[c]);
    }
#pragma unroll
    for (int i = 0; i < R; ++i)
      S[i] = make_float4(__builtin_fmaf(k[i], u[0], decay * S[i].x), __builtin_fmaf(k[i], u[1], decay * S[i].y),
                         __builtin_fmaf(k[i], u[2], decay * S[i].z), __builtin_fmaf(k[i], u[3], decay * S[i].w));
    if (lane < 4)
      *reinterpret_cast<uint2*>(a.out + t * a.o_tok + head * a.o_head + c0) = make_uint2(bf16_pair(o[0], o[1]), bf16_pair(o[2], o[3]));
  }
  if (slot >= 0) {
#pragma unroll
    for (int i = 0; i < R; ++i) *reinterpret_cast<float4*>(state + (int64_t)i * a.v_dim) = S[i];
  }
}

}  // namespace

// Sequences of at most this many new tokens go token by token, the whole call where the longest is known to be no longer.
// A token's step is 1.4 us where the states fill the machine once, a block about the same for one token as for 64.  Calls by
// steps against in blocks, us, with 32 heads of 128 x 128: one sequence of 8 tokens 15 / 21, of 12 21 / 21, of 17 27 / 21;
// eight of 16 34 / 37, of 20 41 / 37; 64 of 16 153 / 218, of 24 217 / 221.
constexpr int kShort = 16;

size_t gated_delta_rule_workspace_bytes(int64_t tokens, int64_t max_q, int64_t num_seqs, int64_t k_heads, int64_t v_heads,
                                        int k_dim, int v_dim) {
  if ((max_q > 0 && max_q <= kShort) || tokens <= kShort) return 0;
  ChunkWork ws;
  return chunk_workspace(tokens, num_seqs, k_heads, v_heads, k_dim, v_dim, nullptr, ws);
}

int launch_gated_delta_rule(const DeltaArgs& a, int64_t max_q, int k_dim, void* workspace, hipStream_t stream) {
  const int64_t jobs = (int64_t)a.s.num_seqs * a.v_heads * (a.v_dim / 16);
  const int64_t grid = (jobs + kThreads / 64 - 1) / (kThreads / 64);
  if (grid * kThreads > (int64_t)UINT32_MAX) return NVFP4_ERR_UNSUPPORTED;           // threads of a launch
  int short_len = INT32_MAX;
  const uint8_t* flags = nullptr;
  if (gated_delta_rule_workspace_bytes(a.s.tokens, max_q, a.s.num_seqs, a.k_heads, a.v_heads, k_dim, a.v_dim) > 0) {
    ChunkWork ws;
    chunk_workspace(a.s.tokens, a.s.num_seqs, a.k_heads, a.v_heads, k_dim, a.v_dim, workspace, ws);
    ws.short_len = short_len = kShort;
    flags = ws.flags;
    const int st = launch_chunks(a, ws, max_q, k_dim, stream);
    if (st != NVFP4_OK) return st;
  }
  if (k_dim == 128)
    delta_step_kernel<128><<<(unsigned)grid, kThreads, 0, stream>>>(a, short_len, flags);
  else
    delta_step_kernel<64><<<(unsigned)grid, kThreads, 0, stream>>>(a, short_len, flags);
  return hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP;
}

}  // namespace nvfp4
