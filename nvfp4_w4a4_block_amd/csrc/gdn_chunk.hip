// The gated delta rule over blocks of 64 tokens on matrix instructions (gfx950): chunks and prompts.
//
// Mathematics.  With G_i the sum of the log decays g_1 .. g_i of a block, S the state in front of it (k, q: unit
// rows), the updates u_i of the token-by-token rule solve
//   u_i + beta_i sum_{j<i} e^{G_i - G_j} (k_i.k_j) u_j = beta_i (v_i - e^{G_i} S^T k_i),      (1 + L) U = R
// so that, T = (1 + L)^-1 (unit lower triangular, |T_ij| <= beta_i since every step is a contraction),
//   U = T R,   O = scale (e^{G_i} Q S + A U),  A_ij = e^{G_i - G_j} q_i.k_j  (j <= i),   S <- e^{G_64} S + K^T (e^{G_64 - G_j} U)
// Two kernels: what does not depend on the state (T, A, row factors) for all blocks at once, then a scan along each
// sequence, one workgroup per value head and slice of state columns (the columns do not meet).
//
// Precision.  State, sums, T and statistics are fp32.  Matrix operands are fp16: k and q rows scaled by powers of two
// (exact but for elements below 2^-16 of a row's largest); S, R, T, U in two parts (2^-22), R and U and S in units of a
// power of two per column that keeps them in range; what only reaches the bf16 output (S and U there, A) in one (2^-11).
// That scale rests on the contraction (finite values, g <= 0, 0 <= beta <= 2): a column's 2-norm stays below the
// running sum B <- e^G B + sum |beta v|.  Where a block breaks that premise the scan gives up its slice with a flag, and
// the token-by-token kernel, which runs behind it, takes the slice from the sequence's start.
#include "gdn_chunk.h"
#include "seq_device.h"

namespace nvfp4 {

namespace {

constexpr int kThreads = 256;
constexpr int kTok = 64;           // tokens of a block

// Workspace of one block: K and Q fragments per key head, T (two parts) and A fragments and row factors per value
// head.  A fragment is the 64 lanes' 16 B of one matrix operand; of a lower triangular 64 x 64 operand only the six
// (row block, half) pairs that are not all zero are kept.
constexpr int kTriFrags = 6;
constexpr int kFactors = 4 * kTok + 16;

__device__ __forceinline__ int tri_frag(int w, int ks) { return w + (w == 3) + ks; }

__device__ __forceinline__ f32x4_t mfma(half8_t a, half8_t b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4_t mfma_f32(float a, float b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

// Barrier over LDS alone: loads from memory stay in flight.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

__device__ __forceinline__ half2_t to_half2(float a, float b) {
  typedef float f32x2_t __attribute__((ext_vector_type(2)));
  return __builtin_convertvector((f32x2_t){a, b}, half2_t);
}

// Four values in two fp16 parts.
__device__ __forceinline__ void split4(const f32x4_t x, half4_t& hi, half4_t& lo) {
  const half2_t a = to_half2(x[0], x[1]), b = to_half2(x[2], x[3]);
  hi = half4_t{a[0], a[1], b[0], b[1]};
  const half2_t c = to_half2(x[0] - (float)a[0], x[1] - (float)a[1]), d = to_half2(x[2] - (float)b[0], x[3] - (float)b[1]);
  lo = half4_t{c[0], c[1], d[0], d[1]};
}

// Sum over the four lanes 16 apart.
__device__ __forceinline__ float quad_sum(float v) {
  v += __shfl_xor(v, 16, 64);
  return v + __shfl_xor(v, 32, 64);
}

// One row of q or k as fp16 fragments, scaled by a power of two to a largest element in [2, 4): lane (row, part) holds
// elements ks * 32 + part * 8 .. + 7.  Returns the factor that makes the scaled row a unit row, 1 / (sc sqrt(x.x + 1e-6)).
template <int KS>
__device__ __forceinline__ float row_frags(const uint16_t* p, int part, bool live, half8_t (&f)[KS], bool& bad) {
  uint4 raw[KS];
#pragma unroll
  for (int ks = 0; ks < KS; ++ks)
    raw[ks] = live ? *reinterpret_cast<const uint4*>(p + ks * 32 + part * 8) : make_uint4(0, 0, 0, 0);
  uint32_t top = 0;
#pragma unroll
  for (int ks = 0; ks < KS; ++ks) top = max(top, max_abs_bits(raw[ks], static_cast<const uint16_t*>(nullptr)));
  top = max(top, (uint32_t)__shfl_xor((int)top, 16, 64));
  top = max(top, (uint32_t)__shfl_xor((int)top, 32, 64));
  bad |= top >= 0x7F800000u;
  const uint32_t e = top >> 23;
  const float sc = __uint_as_float((e == 0 ? 254u : (e >= 254u ? 1u : 255u - e)) << 23);
  float s = 0.0f;
#pragma unroll
  for (int ks = 0; ks < KS; ++ks) {
    float v[8];
    widen(raw[ks], v, static_cast<const uint16_t*>(nullptr));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] *= sc;
      s = __builtin_fmaf(v[i], v[i], s);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const half2_t h = to_half2(v[2 * i], v[2 * i + 1]);
      f[ks][2 * i] = h[0];
      f[ks][2 * i + 1] = h[1];
    }
  }
  s = quad_sum(s);
  if (!live) return 0.0f;
  // neither form overflows: the scaled eps for large rows, the unscaled sum for small ones
  if (sc < 1.0f) return 1.0f / __builtin_sqrtf(s + 1e-6f * sc * sc);
  const float inv = 1.0f / sc;
  return inv / __builtin_sqrtf(s * inv * inv + 1e-6f);
}

__device__ __forceinline__ double shfl_double(double v, int lane) { return __shfl(v, lane, 64); }

// T, A and the row factors of one block for the value heads of one key head.
template <int DK>
__global__ __launch_bounds__(kThreads) void chunk_prepare_kernel(DeltaArgs a, ChunkWork ws) {
  constexpr int KS = DK / 32;
  __shared__ half8_t Kf[4][KS][64];
  __shared__ float L[kTok][kTok + 4];          // L, then T
  __shared__ float D[4][16][20];               // inverses of the diagonal blocks
  __shared__ _Float16 At[kTok][kTok + 8];
  __shared__ float rk[kTok], rq[kTok];
  __shared__ int bads[4];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), c = lane & 15, g = lane >> 4;
  const int block = blockIdx.x / a.k_heads, k_head = blockIdx.x - block * a.k_heads;
  // blocks of a sequence start at slot first / 64 + seq, so that no sequence's slots meet another's
  const SeqState& st = a.s;
  const int seq = wave_search(st.num_seqs, [&](int j) {
    return clamp_int(st.cu_q[j], 0, st.tokens) / kTok + j <= block;
  });
  if (seq < 0) return;
  const SeqRows rows = seq_rows(st, seq);
  const int n = rows.end - rows.first, index = block - (rows.first / kTok + seq);
  if (n <= ws.short_len || index < 0 || index >= (n + kTok - 1) / kTok) return;
  const int m = n - index * kTok < kTok ? n - index * kTok : kTok;
  const int64_t row0 = rows.first + (int64_t)index * kTok;

  half8_t kf[KS], qf[KS];
  bool bad = false;
  {
    const int t = 16 * w + c;
    const int64_t row = row0 + (t < m ? t : 0);
    const float fk = row_frags<KS>(a.k + row * a.k_tok + k_head * a.k_head, g, t < m, kf, bad);
    const float fq = row_frags<KS>(a.q + row * a.q_tok + k_head * a.q_head, g, t < m, qf, bad);
    if (g == 0) {
      rk[t] = fk;
      rq[t] = fq;
    }
  }
  if (lane == 0) bads[w] = 0;
  if (__builtin_amdgcn_ballot_w64(bad) != 0 && lane == 0) bads[w] = 1;
  half8_t* wk = reinterpret_cast<half8_t*>(ws.k) + (((int64_t)block * a.k_heads + k_head) * 4 + w) * KS * 64 + lane;
  half8_t* wq = reinterpret_cast<half8_t*>(ws.q) + (((int64_t)block * a.k_heads + k_head) * 4 + w) * KS * 64 + lane;
#pragma unroll
  for (int ks = 0; ks < KS; ++ks) {
    Kf[w][ks][lane] = kf[ks];
    wk[ks * 64] = kf[ks];
    wq[ks * 64] = qf[ks];
  }
  __syncthreads();

  const f32x4_t zero = {0.0f, 0.0f, 0.0f, 0.0f};
  f32x4_t kk[4], qk[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    kk[j] = zero;
    qk[j] = zero;
    if (j <= w) {
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const half8_t b = Kf[j][ks][lane];
        kk[j] = mfma(kf[ks], b, kk[j]);
        qk[j] = mfma(qf[ks], b, qk[j]);
      }
    }
  }
  const bool bad_rows = (bads[0] | bads[1] | bads[2] | bads[3]) != 0;
  const int group = a.v_heads / a.k_heads;
  for (int h = 0; h < group; ++h) {
    const int head = k_head * group + h;
    // lane t: the sum of the log decays up to token t, in 64 bits: differences of far sums keep their last bits
    const int64_t at = (row0 + (lane < m ? lane : 0)) * a.v_heads + head;
    const float gt = lane < m ? a.g[at] : 0.0f, beta = lane < m ? a.beta[at] : 0.0f;
    const bool off = !(gt <= 0.0f && gt >= -3e38f) || !(beta >= 0.0f && beta <= 2.0f);
    const bool bad_head = bad_rows || __builtin_amdgcn_ballot_w64(off) != 0;
    double sum = gt;
#pragma unroll
    for (int s = 1; s < 64; s *= 2) {
      const double other = shfl_double(sum, lane - s);
      if (lane >= s) sum += other;
    }
    const double total = shfl_double(sum, 63);
    if (w == 0) {
      float* f = ws.factors + ((int64_t)block * a.v_heads + head) * kFactors;
      const float since = expf((float)sum);
      f[lane] = beta;
      f[kTok + lane] = beta * since * rk[lane];
      f[2 * kTok + lane] = expf((float)(total - sum)) * rk[lane];
      f[3 * kTok + lane] = since * rq[lane];
      if (lane == 0) {
        f[4 * kTok] = expf((float)total);
        f[4 * kTok + 1] = bad_head ? 1.0f : 0.0f;
      }
    }
    double row_sum[4];
    float row_k[4], row_q[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int i = 16 * w + 4 * g + r;
      row_sum[r] = shfl_double(sum, i);
      row_k[r] = __shfl(beta, i, 64) * rk[i];
      row_q[r] = rq[i];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j <= w) {
        const int col = 16 * j + c;
        const double col_sum = shfl_double(sum, col);
        const float col_k = rk[col];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int i = 16 * w + 4 * g + r;
          const float d = expf((float)(row_sum[r] - col_sum)) * col_k;
          L[i][col] = i > col ? kk[j][r] * row_k[r] * d : 0.0f;
          At[i][col] = (_Float16)(i >= col ? qk[j][r] * row_q[r] * d : 0.0f);
        }
      } else if (j == w + 1 && (w & 1) == 0) {
#pragma unroll
        for (int r = 0; r < 4; ++r) At[16 * w + 4 * g + r][16 * j + c] = (_Float16)0.0f;
      }
    }
    __syncthreads();
    {
      // forward substitution for column c of this wavefront's diagonal block
      float x[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float s = i == c ? 1.0f : 0.0f;
#pragma unroll
        for (int j = 0; j < i; ++j) s = __builtin_fmaf(-L[16 * w + i][16 * w + j], x[j], s);
        x[i] = s;
        if ((i >> 2) == g) D[w][i][c] = s;
      }
    }
    __syncthreads();
    // this wavefront's column of blocks: T_ij = -T_ii sum_k L_ik T_kj.  A product's result has rows 4 g + r in register r,
    // which is the next one's operand if its steps take the contracted index in that order.
    f32x4_t T[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) T[0][r] = D[w][4 * g + r][c];
#pragma unroll
    for (int d = 1; d < 4; ++d) {
      T[d] = zero;
      if (w + d < 4) {
        f32x4_t acc = zero;
#pragma unroll
        for (int e = 0; e < d; ++e) {
          const float4 l = *reinterpret_cast<const float4*>(&L[16 * (w + d) + c][16 * (w + e) + 4 * g]);
          acc = mfma_f32(l.x, T[e][0], acc);
          acc = mfma_f32(l.y, T[e][1], acc);
          acc = mfma_f32(l.z, T[e][2], acc);
          acc = mfma_f32(l.w, T[e][3], acc);
        }
        const float4 l = *reinterpret_cast<const float4*>(&D[w + d][c][4 * g]);
        T[d] = mfma_f32(-l.x, acc[0], T[d]);
        T[d] = mfma_f32(-l.y, acc[1], T[d]);
        T[d] = mfma_f32(-l.z, acc[2], T[d]);
        T[d] = mfma_f32(-l.w, acc[3], T[d]);
      }
    }
    __syncthreads();
#pragma unroll
    for (int d = 0; d < 4; ++d)
      if (w + d < 4) {
#pragma unroll
        for (int r = 0; r < 4; ++r) L[16 * (w + d) + 4 * g + r][16 * w + c] = T[d][r];
      }
    if (w & 1) {                               // the upper block beside an even diagonal block shares its fragment
#pragma unroll
      for (int r = 0; r < 4; ++r) L[16 * (w - 1) + 4 * g + r][16 * w + c] = 0.0f;
    }
    __syncthreads();
    const int64_t frag0 = ((int64_t)block * a.v_heads + head) * kTriFrags;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
      if (ks <= (w >> 1)) {
        half8_t hi, lo;
        const float* row = &L[16 * w + c][ks * 32 + g * 8];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          half4_t h, l;
          const float4 x = reinterpret_cast<const float4*>(row)[i];
          split4(f32x4_t{x.x, x.y, x.z, x.w}, h, l);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            hi[4 * i + j] = h[j];
            lo[4 * i + j] = l[j];
          }
        }
        const int64_t frag = frag0 + tri_frag(w, ks);
        reinterpret_cast<half8_t*>(ws.t)[(2 * frag) * 64 + lane] = hi;
        reinterpret_cast<half8_t*>(ws.t)[(2 * frag + 1) * 64 + lane] = lo;
        reinterpret_cast<half8_t*>(ws.a)[frag * 64 + lane] = *reinterpret_cast<const half8_t*>(&At[16 * w + c][ks * 32 + g * 8]);
      }
    __syncthreads();
  }
}

// What a wavefront needs of one block.
template <int KS, int NC>
struct Stage {
  half8_t k[KS], q[KS], t_hi[2], t_lo[2], a[2];
  float4 beta, c, d, e;            // factors of rows 4 g .. 4 g + 3 of its 16 tokens
  float decay, bad;
  uint32_t v[NC][2];               // bf16 values of those rows, two to a word
};

// The scan: one workgroup per sequence, value head and slice of 16 NC state columns.  Wavefront w takes tokens
// 16 w .. 16 w + 15 of each block in the products whose rows are tokens, and Dk / 4 rows of the state, which stay in its
// registers; S, R and U meet the other wavefronts in LDS, one barrier each.
template <int DK, int NC>
__global__ __launch_bounds__(kThreads, 2) void chunk_scan_kernel(DeltaArgs a, ChunkWork ws) {
  constexpr int KS = DK / 32, RT = DK / 64;
  __shared__ __attribute__((aligned(16))) _Float16 Ss[2][NC][16][DK + 8];
  __shared__ __attribute__((aligned(16))) _Float16 Rs[2][NC][16][kTok + 8];
  __shared__ __attribute__((aligned(16))) _Float16 Us[3][NC][16][kTok + 8];
  __shared__ __attribute__((aligned(16))) _Float16 Ks[2][kTok][DK + 16];
  __shared__ float Ms[2][4][NC * 16];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), c = lane & 15, g = lane >> 4;
  // a key head's workgroups share its K, Q and their value head's T, A: all on one XCD (workgroup i runs on XCD i mod 8)
  const int group = a.v_heads / a.k_heads, slices = a.v_dim / (16 * NC), per_unit = group * slices;
  const int j = blockIdx.x >> 3;
  const int unit = (j / per_unit) * 8 + (blockIdx.x & 7), part = j % per_unit;
  const int seq = unit / a.k_heads, k_head = unit - seq * a.k_heads;
  if (seq >= a.s.num_seqs) return;
  const int head = k_head * group + part / slices, slice = part % slices;
  const SeqRows rows = seq_rows(a.s, seq);
  const int n = rows.end - rows.first;
  if (n <= ws.short_len) return;
  const int blocks = (n + kTok - 1) / kTok, slot0 = rows.first / kTok + seq;
  const int slot = seq_slot(a.s, seq);
  const bool old = slot >= 0 && scalar_load(a.s.kv_len + seq) > n;
  const int c0 = slice * 16 * NC;
  uint8_t* flag = ws.flags + ((int64_t)seq * a.v_heads + head) * (a.v_dim / 16) + slice * NC;

  auto load = [&](Stage<KS, NC>& s, int b) {
    if (b >= blocks) return;
    const int64_t kq = (((int64_t)(slot0 + b) * a.k_heads + k_head) * 4 + w) * KS * 64 + lane;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      s.k[ks] = reinterpret_cast<const half8_t*>(ws.k)[kq + ks * 64];
      s.q[ks] = reinterpret_cast<const half8_t*>(ws.q)[kq + ks * 64];
    }
    const int64_t pair = (int64_t)(slot0 + b) * a.v_heads + head;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
      if (ks <= (w >> 1)) {
        const int64_t frag = pair * kTriFrags + tri_frag(w, ks);
        s.t_hi[ks] = reinterpret_cast<const half8_t*>(ws.t)[(2 * frag) * 64 + lane];
        s.t_lo[ks] = reinterpret_cast<const half8_t*>(ws.t)[(2 * frag + 1) * 64 + lane];
        s.a[ks] = reinterpret_cast<const half8_t*>(ws.a)[frag * 64 + lane];
      }
    const float* f = ws.factors + pair * kFactors;
    s.beta = *reinterpret_cast<const float4*>(f + 16 * w + 4 * g);
    s.c = *reinterpret_cast<const float4*>(f + kTok + 16 * w + 4 * g);
    s.d = *reinterpret_cast<const float4*>(f + 2 * kTok + 16 * w + 4 * g);
    s.e = *reinterpret_cast<const float4*>(f + 3 * kTok + 16 * w + 4 * g);
    s.decay = scalar_load(f + 4 * kTok);
    s.bad = scalar_load(f + 4 * kTok + 1);
#pragma unroll
    for (int nc = 0; nc < NC; ++nc) {
      uint32_t v[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int t = b * kTok + 16 * w + 4 * g + r;
        v[r] = t < n ? a.v[(int64_t)(rows.first + t) * a.v_tok + head * a.v_head + c0 + nc * 16 + c] : 0;
      }
      s.v[nc][0] = v[0] | v[1] << 16;
      s.v[nc][1] = v[2] | v[3] << 16;
    }
  };
  auto value = [&](const Stage<KS, NC>& s, int nc, int r) {
    const uint32_t x = s.v[nc][r >> 1];
    return __uint_as_float(r & 1 ? x & 0xFFFF0000u : x << 16);
  };
  // sum of |beta v| over the wavefront's tokens, by column, for the block's scale
  auto write_sums = [&](const Stage<KS, NC>& s, int buf) {
#pragma unroll
    for (int nc = 0; nc < NC; ++nc) {
      const float b[4] = {s.beta.x, s.beta.y, s.beta.z, s.beta.w};
      float m = 0.0f;
#pragma unroll
      for (int r = 0; r < 4; ++r) m = __builtin_fmaf(b[r], __builtin_fabsf(value(s, nc, r)), m);
      m = quad_sum(m);
      if (g == 0) Ms[buf][w][nc * 16 + c] = m;
    }
  };
  auto read_sums = [&](float (&m)[NC], int buf) {
#pragma unroll
    for (int nc = 0; nc < NC; ++nc) {
      const int i = nc * 16 + c;
      m[nc] = Ms[buf][0][i] + Ms[buf][1][i] + Ms[buf][2][i] + Ms[buf][3][i];
    }
  };

  Stage<KS, NC> s0, s1;
  load(s0, 0);
  load(s1, 1);
  // the state, rows (w RT + rt) 16 + 4 g + r of column c, in units of `unit_of` from here on
  f32x4_t S[RT][NC];
  float* state = static_cast<float*>(a.s.state) + (slot >= 0 ? slot : 0) * a.s.slot +
                 ((int64_t)head * DK + w * RT * 16 + 4 * g) * a.v_dim + c0 + c;
  float bound[NC], up[NC], down[NC];           // of a column: its norm's bound, 1 / unit, unit
#pragma unroll
  for (int nc = 0; nc < NC; ++nc) {
    float m = 0.0f;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        S[rt][nc][r] = old ? state[(int64_t)(rt * 16 + r) * a.v_dim + nc * 16] : 0.0f;
        m += __builtin_fabsf(S[rt][nc][r]);
      }
    m = quad_sum(m);
    if (g == 0) Ms[1][w][nc * 16 + c] = m;
  }
  write_sums(s0, 0);
  lds_barrier();
  read_sums(bound, 1);
  float sums[NC];
  read_sums(sums, 0);
  bool bad = s0.bad != 0.0f;
  // Units: the bound on everything of the block, below 2^13 of them; updates stay below three times that.
  auto set_unit = [&](int nc) {
    const float most = bound[nc] + sums[nc];
    bad |= !(most < 0x1p100f);
    const uint32_t e = max(__float_as_uint(most) >> 23, 20u);
    up[nc] = __uint_as_float((266u - e) << 23);
    down[nc] = __uint_as_float((e - 12u) << 23);
  };
  auto write_state = [&](const f32x4_t (&x)[RT][NC]) {
#pragma unroll
    for (int nc = 0; nc < NC; ++nc)
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        half4_t hi, lo;
        split4(x[rt][nc], hi, lo);
        *reinterpret_cast<half4_t*>(&Ss[0][nc][c][(w * RT + rt) * 16 + 4 * g]) = hi;
        *reinterpret_cast<half4_t*>(&Ss[1][nc][c][(w * RT + rt) * 16 + 4 * g]) = lo;
      }
  };
#pragma unroll
  for (int nc = 0; nc < NC; ++nc) {
    set_unit(nc);
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) S[rt][nc] *= up[nc];
  }
  if (__builtin_amdgcn_ballot_w64(bad) != 0) {
    if (threadIdx.x < NC) flag[threadIdx.x] = 1;
    return;
  }
  write_state(S);
  lds_barrier();

  const f32x4_t zero = {0.0f, 0.0f, 0.0f, 0.0f};
  // One block; false where the next one breaks the scale's premise.
  auto block_step = [&](Stage<KS, NC>& s, const Stage<KS, NC>& next, int b) -> bool {
    const int buf = b & 1;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) *reinterpret_cast<half8_t*>(&Ks[buf][16 * w + c][ks * 32 + g * 8]) = s.k[ks];
    f32x4_t Y[NC], R[NC];
#pragma unroll
    for (int nc = 0; nc < NC; ++nc) {
      f32x4_t x = zero, xl = zero;
      Y[nc] = zero;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const half8_t hi = *reinterpret_cast<const half8_t*>(&Ss[0][nc][c][ks * 32 + g * 8]);
        const half8_t lo = *reinterpret_cast<const half8_t*>(&Ss[1][nc][c][ks * 32 + g * 8]);
        x = mfma(s.k[ks], hi, x);
        xl = mfma(s.k[ks], lo, xl);
        Y[nc] = mfma(s.q[ks], hi, Y[nc]);
      }
      const float be[4] = {s.beta.x, s.beta.y, s.beta.z, s.beta.w}, cc[4] = {s.c.x, s.c.y, s.c.z, s.c.w};
#pragma unroll
      for (int r = 0; r < 4; ++r) R[nc][r] = be[r] * (value(s, nc, r) * up[nc]) - cc[r] * (x[r] + xl[r]);
      half4_t hi, lo;
      split4(R[nc], hi, lo);
      *reinterpret_cast<half4_t*>(&Rs[0][nc][c][16 * w + 4 * g]) = hi;
      *reinterpret_cast<half4_t*>(&Rs[1][nc][c][16 * w + 4 * g]) = lo;
    }
    if (b + 1 < blocks) write_sums(next, buf ^ 1);
    lds_barrier();
#pragma unroll
    for (int nc = 0; nc < NC; ++nc) {
      f32x4_t u = zero, ul = zero;
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
        if (ks <= (w >> 1)) {
          const half8_t hi = *reinterpret_cast<const half8_t*>(&Rs[0][nc][c][ks * 32 + g * 8]);
          const half8_t lo = *reinterpret_cast<const half8_t*>(&Rs[1][nc][c][ks * 32 + g * 8]);
          u = mfma(s.t_hi[ks], hi, u);
          ul = mfma(s.t_hi[ks], lo, ul);
          ul = mfma(s.t_lo[ks], hi, ul);
        }
      u += ul;
      const float d[4] = {s.d.x, s.d.y, s.d.z, s.d.w};
      const half2_t ua = to_half2(u[0], u[1]), ub = to_half2(u[2], u[3]);
      half4_t hi, lo;
      split4(f32x4_t{u[0] * d[0], u[1] * d[1], u[2] * d[2], u[3] * d[3]}, hi, lo);
      *reinterpret_cast<half4_t*>(&Us[0][nc][c][16 * w + 4 * g]) = half4_t{ua[0], ua[1], ub[0], ub[1]};
      *reinterpret_cast<half4_t*>(&Us[1][nc][c][16 * w + 4 * g]) = hi;
      *reinterpret_cast<half4_t*>(&Us[2][nc][c][16 * w + 4 * g]) = lo;
    }
    lds_barrier();
    // the state behind the block
#pragma unroll
    for (int nc = 0; nc < NC; ++nc) {
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) S[rt][nc] *= s.decay;
      bound[nc] = __builtin_fmaf(s.decay, bound[nc], sums[nc]) * 1.00001f;
    }
    typedef short s16x4_t __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) s16x4_t lds_s16x4_t;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      half8_t kt[RT];
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        // transposing read: lane i of 16 addresses 4 channels of token i / 4 and gets channel i of 4 tokens
        half4_t p[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
          p[i] = __builtin_bit_cast(half4_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
              (lds_s16x4_t*)&Ks[buf][ks * 32 + g * 8 + i * 4 + (c >> 2)][(w * RT + rt) * 16 + (c & 3) * 4]));
        kt[rt] = half8_t{p[0][0], p[0][1], p[0][2], p[0][3], p[1][0], p[1][1], p[1][2], p[1][3]};
      }
#pragma unroll
      for (int nc = 0; nc < NC; ++nc) {
        const half8_t hi = *reinterpret_cast<const half8_t*>(&Us[1][nc][c][ks * 32 + g * 8]);
        const half8_t lo = *reinterpret_cast<const half8_t*>(&Us[2][nc][c][ks * 32 + g * 8]);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          S[rt][nc] = mfma(kt[rt], hi, S[rt][nc]);
          S[rt][nc] = mfma(kt[rt], lo, S[rt][nc]);
        }
      }
    }
    float down_now[NC];
    bad = false;
#pragma unroll
    for (int nc = 0; nc < NC; ++nc) down_now[nc] = down[nc];
    if (b + 1 < blocks) {
      bad = next.bad != 0.0f;
      read_sums(sums, buf ^ 1);
#pragma unroll
      for (int nc = 0; nc < NC; ++nc) {
        set_unit(nc);
        const float ratio = down_now[nc] * up[nc];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) S[rt][nc] *= ratio;
      }
      write_state(S);
    }
    // the outputs
#pragma unroll
    for (int nc = 0; nc < NC; ++nc) {
      const float e[4] = {s.e.x, s.e.y, s.e.z, s.e.w};
      f32x4_t o;
#pragma unroll
      for (int r = 0; r < 4; ++r) o[r] = e[r] * Y[nc][r];
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
        if (ks <= (w >> 1)) o = mfma(s.a[ks], *reinterpret_cast<const half8_t*>(&Us[0][nc][c][ks * 32 + g * 8]), o);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int t = b * kTok + 16 * w + 4 * g + r;
        if (t < n)
          a.out[(int64_t)(rows.first + t) * a.o_tok + head * a.o_head + c0 + nc * 16 + c] =
              (uint16_t)bf16_pair(o[r] * down_now[nc] * a.scale, 0.0f);
      }
    }
    lds_barrier();
    return __builtin_amdgcn_ballot_w64(bad) == 0;
  };
  for (int b = 0; b < blocks; b += 2) {
    bool good = block_step(s0, s1, b);
    if (good && b + 1 < blocks) {
      load(s0, b + 2);
      good = block_step(s1, s0, b + 1);
      if (good) load(s1, b + 3);
    }
    if (!good) {
      if (threadIdx.x < NC) flag[threadIdx.x] = 1;
      return;
    }
  }
  if (threadIdx.x < NC) flag[threadIdx.x] = 0;
  if (slot < 0) return;
#pragma unroll
  for (int nc = 0; nc < NC; ++nc)
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int r = 0; r < 4; ++r) state[(int64_t)(rt * 16 + r) * a.v_dim + nc * 16] = S[rt][nc][r] * down[nc];
}

template <int DK>
int launch_dk(const DeltaArgs& a, const ChunkWork& ws, hipStream_t stream) {
  constexpr int NC = 2;
  const int64_t prepare = ws.blocks * a.k_heads;
  const int64_t units = (int64_t)a.s.num_seqs * a.k_heads;
  const int64_t scan = (units + 7) / 8 * 8 * (a.v_heads / a.k_heads) * (a.v_dim / (16 * NC));
  if (prepare * kThreads > (int64_t)UINT32_MAX || scan * kThreads > (int64_t)UINT32_MAX) return NVFP4_ERR_UNSUPPORTED;
  chunk_prepare_kernel<DK><<<(unsigned)prepare, kThreads, 0, stream>>>(a, ws);
  if (hipGetLastError() != hipSuccess) return NVFP4_ERR_HIP;
  chunk_scan_kernel<DK, NC><<<(unsigned)scan, kThreads, 0, stream>>>(a, ws);
  return hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP;
}

int64_t aligned_up(int64_t n) { return (n + 255) & ~(int64_t)255; }

}  // namespace

size_t chunk_workspace(int64_t tokens, int64_t num_seqs, int64_t k_heads, int64_t v_heads, int k_dim, int v_dim, void* base,
                       ChunkWork& ws) {
  ws.blocks = tokens / kTok + num_seqs;
  char* p = static_cast<char*>(base);
  auto take = [&](int64_t bytes) {
    char* at = p;
    p += aligned_up(bytes);
    return at;
  };
  ws.k = reinterpret_cast<_Float16*>(take(ws.blocks * k_heads * kTok * k_dim * 2));
  ws.q = reinterpret_cast<_Float16*>(take(ws.blocks * k_heads * kTok * k_dim * 2));
  ws.t = reinterpret_cast<_Float16*>(take(ws.blocks * v_heads * kTriFrags * 2 * 1024));
  ws.a = reinterpret_cast<_Float16*>(take(ws.blocks * v_heads * kTriFrags * 1024));
  ws.factors = reinterpret_cast<float*>(take(ws.blocks * v_heads * kFactors * 4));
  ws.flags = reinterpret_cast<uint8_t*>(take(num_seqs * v_heads * (v_dim / 16)));
  return (size_t)(p - static_cast<char*>(base));
}

int launch_chunks(const DeltaArgs& a, const ChunkWork& ws, int k_dim, hipStream_t stream) {
  return k_dim == 128 ? launch_dk<128>(a, ws, stream) : launch_dk<64>(a, ws, stream);
}

}  // namespace nvfp4
