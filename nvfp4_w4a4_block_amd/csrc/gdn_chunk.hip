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
#include <type_traits>

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

// Four values in two fp16 parts.  `one` is 1.0f where the compiler does not see it: x - (float)h is then one mixed
// multiply-add instead of a conversion and a difference.
__device__ __forceinline__ void split4(const f32x4_t x, half4_t& hi, half4_t& lo, float one) {
  const half2_t a = to_half2(x[0], x[1]), b = to_half2(x[2], x[3]);
  hi = half4_t{a[0], a[1], b[0], b[1]};
  const half2_t c = to_half2(__builtin_fmaf((float)a[0], -one, x[0]), __builtin_fmaf((float)a[1], -one, x[1]));
  const half2_t d = to_half2(__builtin_fmaf((float)b[0], -one, x[2]), __builtin_fmaf((float)b[1], -one, x[3]));
  lo = half4_t{c[0], c[1], d[0], d[1]};
}
__device__ __forceinline__ float hidden_one() {
  uint32_t bits = 0x3F800000u;
  asm("" : "+s"(bits));
  return __uint_as_float(bits);
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
      if (lane < 8) {
        f[4 * kTok + 2 * lane] = expf((float)total);
        f[4 * kTok + 2 * lane + 1] = bad_head ? 1.0f : 0.0f;
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
          split4(f32x4_t{x.x, x.y, x.z, x.w}, h, l, 1.0f);
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

constexpr int kScanThreads = 512;

// What a wavefront of the solving half needs of one block, and one of the output half.
template <int KS, int NC>
struct SolveStage {
  half8_t k[KS], t_hi[2], t_lo[2];
  float4 beta, c, d;               // factors of rows 4 g .. 4 g + 3 of its 16 tokens
  float2 whole;                    // the block's decay, and whether it is out of the scale's premise
  uint32_t v[NC][4];               // bf16 values of those rows
};
template <int KS>
struct OutStage {
  half8_t q[KS], a[2];
  float4 e;
  float2 whole;
};

typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4_t;

template <typename T>
__device__ __forceinline__ T load_at(const void* base, uint32_t bytes) {
  return *reinterpret_cast<const T*>(static_cast<const char*>(base) + bytes);
}

// The scan: one workgroup per sequence, value head and slice of 16 NC state columns; eight wavefronts that walk along
// the sequence together, three barriers a block.  Four solve for the updates (16 tokens each: X = K S, R, U = T R), four
// make the outputs (Q S while the others do K S, A U while those are at the next block); all update the state, 16 rows
// of it in the registers of each wavefront that has some.  S, R and U meet the others in LDS.
template <int DK, int NC>
struct Scan {
  static constexpr int KS = DK / 32, TILES = DK / 16;
  struct Lds {
    _Float16 S[2][NC][16][DK + 8];
    _Float16 R[2][NC][16][kTok + 8];
    _Float16 U[3][NC][16][kTok + 8];           // U, then its product with the decays to the block's end in two parts
    _Float16 K[2][kTok][DK + 16];
    float norm[8][NC * 16];
    uint32_t top[3][NC * 16];                  // largest |beta v| of a block, as bits
  };

  const DeltaArgs& a;
  const ChunkWork& ws;
  Lds& lds;
  const int lane, w, c, g, seq, head, k_head, c0;
  SeqRows rows;
  int n, blocks, slot0;
  f32x4_t S[NC];
  float bound[NC], down[NC];                   // of a column: its norm's bound, the block's unit
  float state_down[NC], to_state[NC];          // the unit of S between blocks, and the block's in terms of it
  bool bad = false;
  const float one = hidden_one();

  __device__ Scan(const DeltaArgs& args, const ChunkWork& work, Lds& shared, int seq_, int head_, int k_head_, int c0_)
      : a(args), ws(work), lds(shared), lane(threadIdx.x & 63), w(__builtin_amdgcn_readfirstlane(threadIdx.x >> 6)),
        c(lane & 15), g(lane >> 4), seq(seq_), head(head_), k_head(k_head_), c0(c0_) {}

  // The state's tile of this wavefront; the solving half has none if there are only four.
  __device__ __forceinline__ int tile() const { return TILES == 8 ? w : w - 4; }
  __device__ __forceinline__ bool owner() const { return tile() >= 0; }

  __device__ __forceinline__ const char* at(const void* base, int block, int heads, int h, int bytes) const {
    return static_cast<const char*>(base) + ((int64_t)(slot0 + block) * heads + h) * bytes;
  }
  __device__ __forceinline__ const char* factors(int block) const {
    return at(ws.factors, block, a.v_heads, head, kFactors * 4);
  }
  // Rows of a block as a buffer: reads past the sequence's end give 0, writes there go nowhere.
  __device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const uint16_t* x, int64_t tok, int64_t h, int block) const {
    const int row = block * kTok, m = min(n - row, kTok);
    const uint16_t* p = x + (int64_t)(rows.first + row) * tok + head * h + c0;
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(p), 0, (uint32_t)((m - 1) * (uint32_t)tok + 16 * NC) * 2,
                                             0x00027000);
  }

  // Loads are straight-line and the same every time (past the end: the last block again), so that the waits in the
  // loop count on exactly what was issued since.
  __device__ __forceinline__ void load(SolveStage<KS, NC>& s, int block, const uint32_t (&v_at)[4]) const {
    const int b = min(block, blocks - 1);
    const char* kp = at(ws.k, b, a.k_heads, k_head, 4 * KS * 1024);
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) s.k[ks] = load_at<half8_t>(kp, ((w * KS + ks) * 64 + lane) * 16);
    const char* tp = at(ws.t, b, a.v_heads, head, kTriFrags * 2048);
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      const uint32_t frag = tri_frag(w, min(ks, w >> 1)) * 2048 + lane * 16;
      s.t_hi[ks] = load_at<half8_t>(tp, frag);
      s.t_lo[ks] = load_at<half8_t>(tp, frag + 1024);
    }
    const char* f = factors(b);
    const uint32_t row = (16 * w + 4 * g) * 4;
    s.beta = load_at<float4>(f, row);
    s.c = load_at<float4>(f, row + kTok * 4);
    s.d = load_at<float4>(f, row + 2 * kTok * 4);
    // one copy for each of eight lanes: as a scalar load, every wait on LDS would wait for it
    s.whole = load_at<float2>(f, 4 * kTok * 4 + 8 * (lane & 7));
    const __amdgpu_buffer_rsrc_t v = buffer(a.v, a.v_tok, a.v_head, b);
#pragma unroll
    for (int nc = 0; nc < NC; ++nc)
#pragma unroll
      for (int r = 0; r < 4; ++r) s.v[nc][r] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(v, v_at[r], nc * 32, 0);
  }
  __device__ __forceinline__ void load(OutStage<KS>& s, int block) const {
    const int b = min(block, blocks - 1), o = w - 4;
    const char* qp = at(ws.q, b, a.k_heads, k_head, 4 * KS * 1024);
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) s.q[ks] = load_at<half8_t>(qp, ((o * KS + ks) * 64 + lane) * 16);
    const char* ap = at(ws.a, b, a.v_heads, head, kTriFrags * 1024);
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) s.a[ks] = load_at<half8_t>(ap, tri_frag(o, min(ks, o >> 1)) * 1024 + lane * 16);
    const char* f = factors(b);
    s.e = load_at<float4>(f, 3 * kTok * 4 + (16 * o + 4 * g) * 4);
    s.whole = load_at<float2>(f, 4 * kTok * 4 + 8 * (lane & 7));
  }

  __device__ __forceinline__ static float value(const SolveStage<KS, NC>& s, int nc, int r) {
    return __uint_as_float(s.v[nc][r] << 16);
  }
  // The largest |beta v| of the wavefront's tokens, by column, for the block's unit.
  __device__ __forceinline__ void write_top(const SolveStage<KS, NC>& s, int block) const {
    const float b[4] = {s.beta.x, s.beta.y, s.beta.z, s.beta.w};
#pragma unroll
    for (int nc = 0; nc < NC; ++nc) {
      uint32_t m = 0;                          // as bits, so that a NaN is the largest
#pragma unroll
      for (int r = 0; r < 4; ++r) m = max(m, __float_as_uint(b[r] * value(s, nc, r)) & 0x7FFFFFFFu);
      atomicMax(&lds.top[block % 3][nc * 16 + c], m);
    }
  }

  __device__ __forceinline__ void write_state() const {
    if (!owner()) return;
#pragma unroll
    for (int nc = 0; nc < NC; ++nc) {
      half4_t hi, lo;
      split4(S[nc], hi, lo, one);
      *reinterpret_cast<half4_t*>(&lds.S[0][nc][c][tile() * 16 + 4 * g]) = hi;
      *reinterpret_cast<half4_t*>(&lds.S[1][nc][c][tile() * 16 + 4 * g]) = lo;
    }
  }

  // The power of two that takes x < 2^100 below 2^13, and its inverse.
  __device__ __forceinline__ static void unit(float x, float& up, float& down) {
    const uint32_t e = max(min(__float_as_uint(x) >> 23, 226u), 20u);
    up = __uint_as_float((266u - e) << 23);
    down = __uint_as_float((e - 12u) << 23);
  }

  // The units of a block: everything in it is below bound + 64 max|beta v| of a column, updates below three times that.
  // Between blocks S has a unit of its own, by its bound alone, which follows strong decays.  ratio: from the state's unit
  // to the block's.
  __device__ __forceinline__ void open_block(int block, float2 whole, float (&up)[NC], float (&ratio)[NC]) {
    bad |= whole.y != 0.0f;
#pragma unroll
    for (int nc = 0; nc < NC; ++nc) {
      const float more = 64.0f * __uint_as_float(lds.top[block % 3][nc * 16 + c]);
      const float most = bound[nc] + more;
      bad |= !(most < 0x1p100f);
      unit(most, up[nc], down[nc]);
      ratio[nc] = state_down[nc] * up[nc];
      bound[nc] = __builtin_fmaf(whole.x, bound[nc], more) * 1.00001f;
      float state_up;
      unit(bound[nc], state_up, state_down[nc]);
      to_state[nc] = down[nc] * state_up;
    }
    if (threadIdx.x >= kScanThreads - NC * 16) lds.top[(block + 2) % 3][threadIdx.x - (kScanThreads - NC * 16)] = 0;
  }

  // Transposed K: lane i of 16 addresses 4 channels of token i / 4 and gets channel i of 4 tokens.
  __device__ __forceinline__ void read_kt(half8_t (&kt)[2], int block) const {
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      half4_t p[2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
        p[i] = __builtin_bit_cast(half4_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (lds_s16x4_t*)&lds.K[block & 1][ks * 32 + g * 8 + i * 4 + (c >> 2)][tile() * 16 + (c & 3) * 4]));
      kt[ks] = half8_t{p[0][0], p[0][1], p[0][2], p[0][3], p[1][0], p[1][1], p[1][2], p[1][3]};
    }
  }

  // S <- decay S + K^T U in the block's unit, then in the state's.
  __device__ __forceinline__ void update(const half8_t (&kt)[2], float decay, const float (&ratio)[NC]) {
    half8_t hi[NC][2], lo[NC][2];
#pragma unroll
    for (int nc = 0; nc < NC; ++nc)
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        hi[nc][ks] = *reinterpret_cast<const half8_t*>(&lds.U[1][nc][c][ks * 32 + g * 8]);
        lo[nc][ks] = *reinterpret_cast<const half8_t*>(&lds.U[2][nc][c][ks * 32 + g * 8]);
      }
#pragma unroll
    for (int nc = 0; nc < NC; ++nc) S[nc] *= decay * ratio[nc];
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
#pragma unroll
      for (int nc = 0; nc < NC; ++nc) S[nc] = mfma(kt[ks], lo[nc][ks], S[nc]);
#pragma unroll
      for (int nc = 0; nc < NC; ++nc) S[nc] = mfma(kt[ks], hi[nc][ks], S[nc]);
    }
#pragma unroll
    for (int nc = 0; nc < NC; ++nc) S[nc] *= to_state[nc];
  }

  __device__ __forceinline__ void solve_block(const SolveStage<KS, NC>& s, const SolveStage<KS, NC>& next, int b) {
    float up[NC], ratio[NC];
    open_block(b, s.whole, up, ratio);
    half8_t hi[NC][KS], lo[NC][KS];
#pragma unroll
    for (int nc = 0; nc < NC; ++nc)
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        lo[nc][ks] = *reinterpret_cast<const half8_t*>(&lds.S[1][nc][c][ks * 32 + g * 8]);
        hi[nc][ks] = *reinterpret_cast<const half8_t*>(&lds.S[0][nc][c][ks * 32 + g * 8]);
      }
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) *reinterpret_cast<half8_t*>(&lds.K[b & 1][16 * w + c][ks * 32 + g * 8]) = s.k[ks];
    const float be[4] = {s.beta.x, s.beta.y, s.beta.z, s.beta.w}, cc[4] = {s.c.x, s.c.y, s.c.z, s.c.w};
#pragma unroll
    for (int nc = 0; nc < NC; ++nc) {
      f32x4_t x = {0.0f, 0.0f, 0.0f, 0.0f}, r4;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) x = mfma(s.k[ks], lo[nc][ks], x);
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) x = mfma(s.k[ks], hi[nc][ks], x);
#pragma unroll
      for (int r = 0; r < 4; ++r) r4[r] = __builtin_fmaf(be[r] * value(s, nc, r), up[nc], -(cc[r] * ratio[nc]) * x[r]);
      half4_t rh, rl;
      split4(r4, rh, rl, one);
      *reinterpret_cast<half4_t*>(&lds.R[0][nc][c][16 * w + 4 * g]) = rh;
      *reinterpret_cast<half4_t*>(&lds.R[1][nc][c][16 * w + 4 * g]) = rl;
    }
    lds_barrier();
    half8_t kt[2];
    if (TILES == 8) read_kt(kt, b);
#pragma unroll
    for (int nc = 0; nc < NC; ++nc) {
      f32x4_t u = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
        if (ks <= (w >> 1)) {
          const half8_t rh = *reinterpret_cast<const half8_t*>(&lds.R[0][nc][c][ks * 32 + g * 8]);
          const half8_t rl = *reinterpret_cast<const half8_t*>(&lds.R[1][nc][c][ks * 32 + g * 8]);
          u = mfma(s.t_lo[ks], rh, u);
          u = mfma(s.t_hi[ks], rl, u);
          u = mfma(s.t_hi[ks], rh, u);
        }
      const float d[4] = {s.d.x, s.d.y, s.d.z, s.d.w};
      const half2_t ua = to_half2(u[0], u[1]), ub = to_half2(u[2], u[3]);
      half4_t uh, ul;
      split4(f32x4_t{u[0] * d[0], u[1] * d[1], u[2] * d[2], u[3] * d[3]}, uh, ul, one);
      *reinterpret_cast<half4_t*>(&lds.U[1][nc][c][16 * w + 4 * g]) = uh;
      *reinterpret_cast<half4_t*>(&lds.U[2][nc][c][16 * w + 4 * g]) = ul;
      *reinterpret_cast<half4_t*>(&lds.U[0][nc][c][16 * w + 4 * g]) = half4_t{ua[0], ua[1], ub[0], ub[1]};
    }
    lds_barrier();
    if (TILES == 8) {
      update(kt, s.whole.x, ratio);
      write_state();
    }
    write_top(next, b + 1);
    lds_barrier();
  }

  __device__ __forceinline__ void solve() {
    uint32_t v_at[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) v_at[r] = (uint32_t)((16 * w + 4 * g + r) * (uint32_t)a.v_tok + c) * 2;
    SolveStage<KS, NC> s0, s1, s2;
    load(s0, 0, v_at);
    load(s1, 1, v_at);
    load(s2, 2, v_at);
    open();
    write_top(s0, 0);
    lds_barrier();
    int b = 0;
    for (; b + 2 < blocks; b += 3) {
      solve_block(s0, s1, b);
      load(s0, b + 3, v_at);
      solve_block(s1, s2, b + 1);
      load(s1, b + 4, v_at);
      solve_block(s2, s0, b + 2);
      load(s2, b + 5, v_at);
    }
    if (b < blocks) solve_block(s0, s1, b);
    if (b + 1 < blocks) solve_block(s1, s1, b + 1);
  }

  // The outputs of a block from its Q S and the updates in LDS.
  __device__ __forceinline__ void store_out(const OutStage<KS>& s, const f32x4_t (&y)[NC], const float (&ratio)[NC], int b,
                                            const uint32_t (&o_at)[4]) const {
    const int o = w - 4;
    const float e[4] = {s.e.x, s.e.y, s.e.z, s.e.w};
    const __amdgpu_buffer_rsrc_t out = buffer(a.out, a.o_tok, a.o_head, b);
#pragma unroll
    for (int nc = 0; nc < NC; ++nc) {
      f32x4_t x;
#pragma unroll
      for (int r = 0; r < 4; ++r) x[r] = e[r] * ratio[nc] * y[nc][r];
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
        if (ks <= (o >> 1)) x = mfma(s.a[ks], *reinterpret_cast<const half8_t*>(&lds.U[0][nc][c][ks * 32 + g * 8]), x);
      const float f = down[nc] * a.scale;
#pragma unroll
      for (int r = 0; r < 4; r += 2) {
        const uint32_t two = bf16_pair(x[r] * f, x[r + 1] * f);
        __builtin_amdgcn_raw_buffer_store_b16((short)two, out, o_at[r], nc * 32, 0);
        __builtin_amdgcn_raw_buffer_store_b16((short)(two >> 16), out, o_at[r + 1], nc * 32, 0);
      }
    }
  }

  __device__ __forceinline__ void out_block(const OutStage<KS>& s, int b, const uint32_t (&o_at)[4]) {
    float up[NC], ratio[NC];
    open_block(b, s.whole, up, ratio);
    f32x4_t y[NC];
#pragma unroll
    for (int nc = 0; nc < NC; ++nc) {
      y[nc] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
        y[nc] = mfma(s.q[ks], *reinterpret_cast<const half8_t*>(&lds.S[0][nc][c][ks * 32 + g * 8]), y[nc]);
    }
    lds_barrier();
    half8_t kt[2];
    read_kt(kt, b);
    lds_barrier();
    update(kt, s.whole.x, ratio);
    write_state();
    lds_barrier();
    store_out(s, y, ratio, b, o_at);           // while the others are at the next block's K S
  }

  __device__ __forceinline__ void output() {
    uint32_t o_at[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) o_at[r] = (uint32_t)((16 * (w - 4) + 4 * g + r) * (uint32_t)a.o_tok + c) * 2;
    OutStage<KS> s0, s1, s2;
    load(s0, 0);
    load(s1, 1);
    load(s2, 2);
    open();
    lds_barrier();
    int b = 0;
    for (; b + 2 < blocks; b += 3) {
      out_block(s0, b, o_at);
      load(s0, b + 3);
      out_block(s1, b + 1, o_at);
      load(s1, b + 4);
      out_block(s2, b + 2, o_at);
      load(s2, b + 5);
    }
    if (b < blocks) out_block(s0, b, o_at);
    if (b + 1 < blocks) out_block(s1, b + 1, o_at);
  }

  // Reads the state in; one barrier inside, one is due behind it.
  __device__ __forceinline__ void open() {
    const int slot = seq_slot(a.s, seq);
    const bool old = slot >= 0 && scalar_load(a.s.kv_len + seq) > n;
    if (threadIdx.x < 3 * NC * 16) (&lds.top[0][0])[threadIdx.x] = 0;
    if (owner()) {
      const float* p = state(slot);
#pragma unroll
      for (int nc = 0; nc < NC; ++nc) {
        float m = 0.0f;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          S[nc][r] = old ? p[(int64_t)r * a.v_dim + nc * 16] : 0.0f;
          m += __builtin_fabsf(S[nc][r]);
        }
        m = quad_sum(m);
        if (g == 0) lds.norm[tile()][nc * 16 + c] = m;
      }
    }
    lds_barrier();
#pragma unroll
    for (int nc = 0; nc < NC; ++nc) {
      bound[nc] = 0.0f;
#pragma unroll
      for (int i = 0; i < TILES; ++i) bound[nc] += lds.norm[i][nc * 16 + c];
      float up;
      unit(bound[nc], up, state_down[nc]);
      S[nc] *= up;
    }
    write_state();
  }
  __device__ __forceinline__ float* state(int slot) const {
    return static_cast<float*>(a.s.state) + (slot >= 0 ? slot : 0) * a.s.slot +
           ((int64_t)head * DK + tile() * 16 + 4 * g) * a.v_dim + c0 + c;
  }
  __device__ __forceinline__ void close() const {
    const int slot = seq_slot(a.s, seq), slice = c0 / 16;
    const bool left = __builtin_amdgcn_ballot_w64(bad) != 0;
    uint8_t* flag = ws.flags + ((int64_t)seq * a.v_heads + head) * (a.v_dim / 16) + slice;
    if (threadIdx.x < NC) flag[threadIdx.x] = left;
    if (slot < 0 || left || !owner()) return;
    float* p = state(slot);
#pragma unroll
    for (int nc = 0; nc < NC; ++nc)
#pragma unroll
      for (int r = 0; r < 4; ++r) p[(int64_t)r * a.v_dim + nc * 16] = S[nc][r] * state_down[nc];
  }
};

template <int DK, int NC>
__global__ __launch_bounds__(kScanThreads) void chunk_scan_kernel(DeltaArgs a, ChunkWork ws) {
  __shared__ __attribute__((aligned(16))) typename Scan<DK, NC>::Lds lds;
  // a key head's workgroups share its K, Q and their value head's T, A: all on one XCD (workgroup i runs on XCD i mod 8)
  const int group = a.v_heads / a.k_heads, slices = a.v_dim / (16 * NC), per_pair = group * slices;
  const int j = blockIdx.x >> 3;
  const int pair = (j / per_pair) * 8 + (blockIdx.x & 7), part = j % per_pair;
  const int seq = pair / a.k_heads, k_head = pair - seq * a.k_heads;
  if (seq >= a.s.num_seqs) return;
  Scan<DK, NC> scan(a, ws, lds, seq, k_head * group + part / slices, k_head, part % slices * 16 * NC);
  scan.rows = seq_rows(a.s, seq);
  scan.n = scan.rows.end - scan.rows.first;
  if (scan.n <= ws.short_len) return;
  scan.blocks = (scan.n + kTok - 1) / kTok;
  scan.slot0 = scan.rows.first / kTok + seq;
  if (scan.w < 4)
    scan.solve();
  else
    scan.output();
  scan.close();
}

template <int DK>
int launch_dk(const DeltaArgs& a, const ChunkWork& ws, hipStream_t stream) {
  constexpr int NC = 1;
  const int64_t prepare = ws.blocks * a.k_heads;
  const int64_t units = (int64_t)a.s.num_seqs * a.k_heads;
  const int64_t scan = (units + 7) / 8 * 8 * (a.v_heads / a.k_heads) * (a.v_dim / (16 * NC));
  if (prepare * kThreads > (int64_t)UINT32_MAX || scan * kScanThreads > (int64_t)UINT32_MAX) return NVFP4_ERR_UNSUPPORTED;
  chunk_prepare_kernel<DK><<<(unsigned)prepare, kThreads, 0, stream>>>(a, ws);
  if (hipGetLastError() != hipSuccess) return NVFP4_ERR_HIP;
  chunk_scan_kernel<DK, NC><<<(unsigned)scan, kScanThreads, 0, stream>>>(a, ws);
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
