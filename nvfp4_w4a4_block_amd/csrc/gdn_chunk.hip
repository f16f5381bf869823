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
// (exact but for elements below 2^-16 of a row's largest); S, R, T, U, A in two parts (2^-22), R and U and S in units of a
// power of two per column that keeps them in range.  (With S, U and A in one part where they only reach the bf16 output the
// outputs were off by 2^-11 of what the state holds, many steps of an output far below that.)
// That scale rests on the contraction (finite values, g <= 0, 0 <= beta <= 2): a column's 2-norm stays below the
// running sum B <- e^G B + sum |beta v|.  A block's unit goes by the largest that its bound M can become in it, and leaves
// 2^-48 M of an element: a token that writes far less than M, or a small state before a large write, would lose its bits to
// what comes after it.  So where a token writes less than kRange M at most (its largest column of the slice), and what was
// there before, old state or the first token's write, has decayed below that by the block's end, or where a block breaks the
// premise, the scan gives up its slice with a flag, and the token-by-token kernel, which runs behind it, takes the slice from the
// sequence's start.  (Tokens that write nothing, padding for one, do not count: 2^-48 M is what their outputs are held to.)
#include <type_traits>

#include "gdn_chunk.h"
#include "seq_device.h"

namespace nvfp4 {

namespace {

constexpr int kTok = 64;           // tokens of a block

// Workspace of one block: K and Q fragments per key head, T and A fragments (two parts each) and row factors per value
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

// The second of two parts, times kPart: it is no larger than the first one then, and as small values keep their bits.
constexpr float kPart = 0x1p11f;
// T and A (at most 2) are multiplied by kTri: both parts of elements down to 2^-28 are normal numbers.
constexpr float kTri = 0x1p14f;

// Four values in two fp16 parts, x = hi + lo / kPart.  `one` is 1.0f where the compiler does not see it: x - (float)h is then
// one mixed multiply-add instead of a conversion and a difference.
__device__ __forceinline__ void split4(const f32x4_t x, half4_t& hi, half4_t& lo, float one) {
  const half2_t a = to_half2(x[0], x[1]), b = to_half2(x[2], x[3]);
  hi = half4_t{a[0], a[1], b[0], b[1]};
  const half2_t c = to_half2(kPart * __builtin_fmaf((float)a[0], -one, x[0]), kPart * __builtin_fmaf((float)a[1], -one, x[1]));
  const half2_t d = to_half2(kPart * __builtin_fmaf((float)b[0], -one, x[2]), kPart * __builtin_fmaf((float)b[1], -one, x[3]));
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

// The value of the lane 1 and 2 away (by xor), in the other quad of 8 and in the other half of 16: one instruction with
// what takes it, where a general exchange goes through LDS.
template <int CONTROL>
__device__ __forceinline__ uint32_t moved(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CONTROL, 0xF, 0xF, true);
}
// Sum and largest over the 8 or 16 neighbouring lanes that hold a row.
template <int LANES>
__device__ __forceinline__ float row_total(float v) {
  v += __uint_as_float(moved<0xB1>(__float_as_uint(v)));          // quad_perm 1 0 3 2
  v += __uint_as_float(moved<0x4E>(__float_as_uint(v)));          // quad_perm 2 3 0 1
  v += __uint_as_float(moved<0x141>(__float_as_uint(v)));         // mirrored in 8
  if (LANES == 16) v += __uint_as_float(moved<0x140>(__float_as_uint(v)));   // mirrored in 16
  return v;
}
template <int LANES>
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
  v = max(v, moved<0xB1>(v));
  v = max(v, moved<0x4E>(v));
  v = max(v, moved<0x141>(v));
  if (LANES == 16) v = max(v, moved<0x140>(v));
  return v;
}

// Smallest of a wavefront's values, in lane 63.
__device__ __forceinline__ uint32_t wave_min(uint32_t v) {
  v = min(v, moved<0xB1>(v));
  v = min(v, moved<0x4E>(v));
  v = min(v, moved<0x141>(v));
  v = min(v, moved<0x140>(v));
  v = min(v, (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, 0x142, 0xA, 0xF, false));     // rows 0, 2 to 1, 3
  return min(v, (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, 0x143, 0xC, 0xF, false));  // lane 31 to rows 2, 3
}

// 8 elements of a row of q or k as fp16, the row (DK / 8 neighbouring lanes) scaled by a power of two `sc` to a largest
// element in [2, 4).  Returns the scaled row's squares' sum.
template <int LANES>
__device__ __forceinline__ float scaled_row(const uint4& raw, half8_t& f, float& sc, bool& bad) {
  const uint32_t top = row_max<LANES>(max_abs_bits(raw, static_cast<const uint16_t*>(nullptr)));
  bad |= top >= 0x7F800000u;
  const uint32_t e = top >> 23;
  sc = __uint_as_float((e == 0 ? 254u : 255u - min(e, 254u)) << 23);
  float s = 0.0f, v[8];
  widen(raw, v, static_cast<const uint16_t*>(nullptr));
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] *= sc;
    s = __builtin_fmaf(v[i], v[i], s);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const half2_t h = to_half2(v[2 * i], v[2 * i + 1]);
    f[2 * i] = h[0];
    f[2 * i + 1] = h[1];
  }
  return row_total<LANES>(s);
}
// The factor that makes a scaled row a unit row, 1 / (sc sqrt(x.x + 1e-6)).  Neither form overflows: the scaled eps for
// large rows, the unscaled sum for small ones.
__device__ __forceinline__ float unit_factor(float s, float sc) {
  const float inv = 1.0f / sc;                 // a power of two
  return sc < 1.0f ? 1.0f / __builtin_sqrtf(s + 1e-6f * sc * sc) : inv / __builtin_sqrtf(s * inv * inv + 1e-6f);
}

// v + the value of a lane before it, in 64 bits, where CONTROL and ROWS have one.
template <int CONTROL, int ROWS>
__device__ __forceinline__ double plus_earlier(double v) {
  const uint64_t bits = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)bits, CONTROL, ROWS, 0xF, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(bits >> 32), CONTROL, ROWS, 0xF, false);
  return v + __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
// Lane l: the sum of lanes 0 .. l.
__device__ __forceinline__ double running_sum(double v) {
  v = plus_earlier<0x111, 0xF>(v);             // within rows of 16: the lane 1, 2, 4, 8 before
  v = plus_earlier<0x112, 0xF>(v);
  v = plus_earlier<0x114, 0xF>(v);
  v = plus_earlier<0x118, 0xF>(v);
  v = plus_earlier<0x142, 0xA>(v);             // a row's last lane to the next row, of rows 1 and 3
  return plus_earlier<0x143, 0xC>(v);          // lane 31 to rows 2 and 3
}
__device__ __forceinline__ double last_lane(double v) {
  const uint64_t bits = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)bits, 63), hi = __builtin_amdgcn_readlane((uint32_t)(bits >> 32), 63);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// 2^x for x <= 0 by the hardware's instruction: what one rounding of x costs, |x| 2^x 2^-25, stays below 2^-25.
__device__ __forceinline__ float power2(float x) { return __builtin_amdgcn_exp2f(x); }

// T, A and the row factors of one block for two value heads of one key head: eight wavefronts, four to a value head;
// wavefront w of four has rows 16 w .. 16 w + 15.  K K^T and Q K^T are both halves' own work, a tenth of
// what exchanging them would wait for.  Bound by its bytes (q, k in, fragments out) and the latency of the inverse: 8192
// tokens of 16 and 32 heads of 128, 240 MB, 59 us (4.1 TB/s).  One workgroup that takes block after block with the next
// one's rows on the way took 70 where this form took 58, before A had a second part.
constexpr int kPrepareThreads = 512;

template <int DK>
__global__ __launch_bounds__(kPrepareThreads, 4) void chunk_prepare_kernel(DeltaArgs a, ChunkWork ws) {
  constexpr int KS = DK / 32;
  // K and Q fragments, then A (rows of 72) of both heads
  __shared__ __attribute__((aligned(16))) char shared[2 * 4 * KS * 1024 > 2 * kTok * 144 ? 2 * 4 * KS * 1024 : 2 * kTok * 144];
  __shared__ __attribute__((aligned(16))) float Ls[2][kTok][kTok + 4];         // L, then T
  __shared__ __attribute__((aligned(16))) float Ds[2][4][16][20];              // inverses of the diagonal blocks
  __shared__ __attribute__((aligned(16))) float unit_k[kTok], unit_q[kTok], betas[2][kTok];
  __shared__ __attribute__((aligned(16))) float decay_hi[2][kTok], decay_lo[2][kTok];      // running sum of a head's log2 decays
  __shared__ float sums[8][16], scales[8][16];
  __shared__ int bads[8];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), c = lane & 15, g = lane >> 4;
  const int half = wave >> 2, w = wave & 3;
  half8_t(*Kf)[KS][64] = reinterpret_cast<half8_t(*)[KS][64]>(shared);
  half8_t(*Qf)[KS][64] = Kf + 4;
  const int group = a.v_heads / a.k_heads, twos = (group + 1) / 2;
  const int block = blockIdx.x / (a.k_heads * twos), part = blockIdx.x - block * a.k_heads * twos;
  const int k_head = part / twos, first_head = 2 * (part - k_head * twos);
  // an odd last head: the second half repeats it and writes the same
  const int head = k_head * group + min(first_head + half, group - 1);
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
  // decays and strengths come from far, too: out ahead of the rows, their sums taken before those are in
  const int64_t at = (row0 + (lane < m ? lane : 0)) * a.v_heads + head;
  const float g_load = a.g[at], beta_load = a.beta[at];
  double sum = 0.0;
  bool off = false;
  {
    // One half takes the rows of k, the other those of q, whole rows at a time.  Fragments, K's and Q's alike: lane (row,
    // part) of 16 x 4 holds channels 32 ks + 4 part .. + 3 and 32 ks + 16 + 4 part .. + 3, the rows that a lane holds of
    // two 16-row results, so that the state can be the other operand as it is.
    constexpr int LANES = DK / 8, ROWS = 64 / LANES, LOADS = 16 / ROWS;
    const uint16_t* x = half == 0 ? a.k + k_head * a.k_head : a.q + k_head * a.q_head;
    const int64_t pitch = half == 0 ? a.k_tok : a.q_tok;
    const int d = lane % LANES * 8;
    uint4 raw[LOADS];
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      const int t = 16 * w + i * ROWS + lane / LANES;
      raw[i] = *reinterpret_cast<const uint4*>(x + (row0 + min(t, m - 1)) * pitch + d);
    }
    if (w == 0) {
      // lane t: the sum of the log2 decays up to token t, in 64 bits: differences of far sums keep their last bits.  Decays
      // below 2^-1000, to 0, are as good as that one, and sums of it stay finite in fp32.
      const float gt = lane < m ? g_load : 0.0f, beta = lane < m ? beta_load : 0.0f;
      off = __builtin_amdgcn_ballot_w64(!(gt <= 0.0f) || !(beta >= 0.0f && beta <= 2.0f)) != 0;
      sum = running_sum(__builtin_fmax((double)gt * 1.4426950408889634074, -1000.0));
      const float hi = (float)sum;
      decay_hi[half][lane] = hi;
      decay_lo[half][lane] = (float)(sum - (double)hi);
      betas[half][lane] = beta;
    }
    bool bad = false;
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      const int r = i * ROWS + lane / LANES, t = 16 * w + r;
      half8_t f;
      float sc;
      const float s = scaled_row<LANES>(raw[i], f, sc, bad);
      if (t >= m) f = half8_t{};               // rows behind the end
      if (lane % LANES == 0) {
        sums[wave][r] = s;
        scales[wave][r] = sc;
      }
      // channels d .. d + 3 and d + 4 .. d + 7 are parts (d / 4) % 4 and the next of half (d / 16) % 2
      half4_t* to = reinterpret_cast<half4_t*>(&Kf[half * 4 + w][d / 32][r + d / 4 % 4 * 16]) + d / 16 % 2;
      to[0] = half4_t{f[0], f[1], f[2], f[3]};
      to[32] = half4_t{f[4], f[5], f[6], f[7]};
    }
    const bool any = __builtin_amdgcn_ballot_w64(bad) != 0;
    if (lane == 0) bads[wave] = any;
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    if (lane < 16) (half == 0 ? unit_k : unit_q)[16 * w + lane] = 16 * w + lane < m ? unit_factor(sums[wave][lane], scales[wave][lane]) : 0.0f;
  }
  lds_barrier();
  if (first_head == 0) {
    half8_t* out = reinterpret_cast<half8_t*>(half == 0 ? ws.k : ws.q) + (((int64_t)block * a.k_heads + k_head) * 4 + w) * KS * 64 + lane;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) out[ks * 64] = Kf[half * 4 + w][ks][lane];
  }

  f32x4_t kk[4], qk[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    kk[j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    qk[j] = kk[j];
  }
#pragma unroll
  for (int ks = 0; ks < KS; ++ks) {
    const half8_t kf = Kf[w][ks][lane], qf = Qf[w][ks][lane];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j <= w) {
        const half8_t b = Kf[j][ks][lane];
        kk[j] = mfma(kf, b, kk[j]);
        qk[j] = mfma(qf, b, qk[j]);
      }
  }
  bool bad_rows = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) bad_rows |= bads[i] != 0;
  lds_barrier();                               // K and Q are read, A may take their place
  float(*L)[kTok + 4] = Ls[half];
  float(*D)[16][20] = Ds[half];
  _Float16(*At)[kTok + 8] = reinterpret_cast<_Float16(*)[kTok + 8]>(shared) + half * kTok;

  {
    if (w == 0) {
      const double total = last_lane(sum);
      float* f = ws.factors + ((int64_t)block * a.v_heads + head) * kFactors;
      const float since = power2((float)sum), beta = betas[half][lane], uk = unit_k[lane];
      f[lane] = beta;
      f[kTok + lane] = beta * since * uk;
      f[2 * kTok + lane] = power2((float)(total - sum)) * uk;
      f[3 * kTok + lane] = since * unit_q[lane];
      if (lane < 16) f[4 * kTok + lane] = bad_rows || off ? __builtin_nanf("") : power2((float)total);
    }
    const int row = 16 * w + 4 * g;
    const f32x4_t row_hi = *reinterpret_cast<const f32x4_t*>(&decay_hi[half][row]), row_lo = *reinterpret_cast<const f32x4_t*>(&decay_lo[half][row]);
    const f32x4_t row_k = *reinterpret_cast<const f32x4_t*>(&betas[half][row]) * *reinterpret_cast<const f32x4_t*>(&unit_k[row]);
    const f32x4_t row_q = *reinterpret_cast<const f32x4_t*>(&unit_q[row]);
    half4_t a_low[4];                          // the second parts of A
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j <= w) {
        const int col = 16 * j + c;
        const float col_hi = decay_hi[half][col], col_lo = decay_lo[half][col], col_k = unit_k[col];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int i = 16 * w + 4 * g + r;
          const float d = power2((row_hi[r] - col_hi) + (row_lo[r] - col_lo)) * col_k;
          float l = kk[j][r] * row_k[r] * d, q = qk[j][r] * row_q[r] * d;
          if (j == w) {
            l = i > col ? l : 0.0f;
            q = i >= col ? q : 0.0f;
          }
          L[i][col] = l;
          q *= kTri;
          At[i][col] = (_Float16)q;
          a_low[j][r] = (_Float16)(kPart * (q - (float)(_Float16)q));
        }
      } else if (j == w + 1 && (w & 1) == 0) {
#pragma unroll
        for (int r = 0; r < 4; ++r) At[16 * w + 4 * g + r][16 * j + c] = (_Float16)0.0f;
      }
    }
    // the diagonal block and the rows of A are this wavefront's own: no barrier between them and their use
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    half8_t* a_out = reinterpret_cast<half8_t*>(ws.a) + 2 * ((int64_t)block * a.v_heads + head) * kTriFrags * 64 + lane;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
      if (ks <= (w >> 1)) a_out[2 * tri_frag(w, ks) * 64] = *reinterpret_cast<const half8_t*>(&At[16 * w + c][ks * 32 + g * 8]);
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    // they take the first ones' place
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j <= w) {
#pragma unroll
        for (int r = 0; r < 4; ++r) At[16 * w + 4 * g + r][16 * j + c] = a_low[j][r];
      }
    {
      // forward substitution for column c of the block, four known elements taken out of all later rows at once
      float x[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = i == c ? 1.0f : 0.0f;
#pragma unroll
      for (int jb = 0; jb < 4; ++jb) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          if (i <= 4 * jb) continue;
          const float4 l = *reinterpret_cast<const float4*>(&L[16 * w + i][16 * w + 4 * jb]);
          x[i] = __builtin_fmaf(-l.x, x[4 * jb], x[i]);
          if (i > 4 * jb + 1) x[i] = __builtin_fmaf(-l.y, x[4 * jb + 1], x[i]);
          if (i > 4 * jb + 2) x[i] = __builtin_fmaf(-l.z, x[4 * jb + 2], x[i]);
          if (i > 4 * jb + 3) x[i] = __builtin_fmaf(-l.w, x[4 * jb + 3], x[i]);
          if (i % 4 == 3) __builtin_amdgcn_sched_barrier(0);         // four rows in flight, not all of them
        }
      }
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if ((i >> 2) == g) D[w][i][c] = x[i];
    }
    lds_barrier();
    // this wavefront's column of blocks: T_ij = -T_ii sum_k L_ik T_kj.  A product's result has rows 4 g + r in register r,
    // which is the next one's operand if its steps take the contracted index in that order.
    const f32x4_t zero = {0.0f, 0.0f, 0.0f, 0.0f};
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
    lds_barrier();
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
    lds_barrier();
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
          split4(f32x4_t{kTri * x.x, kTri * x.y, kTri * x.z, kTri * x.w}, h, l, 1.0f);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            hi[4 * i + j] = h[j];
            lo[4 * i + j] = l[j];
          }
        }
        const int64_t frag = frag0 + tri_frag(w, ks);
        reinterpret_cast<half8_t*>(ws.t)[(2 * frag) * 64 + lane] = hi;
        reinterpret_cast<half8_t*>(ws.t)[(2 * frag + 1) * 64 + lane] = lo;
        reinterpret_cast<half8_t*>(ws.a)[(2 * frag + 1) * 64 + lane] = *reinterpret_cast<const half8_t*>(&At[16 * w + c][ks * 32 + g * 8]);
      }
  }
}

constexpr int kScanThreads = 512;

// Range of what a block's tokens write: 2^-48 M is 2^-20 of the smallest then.  Beside values of order 1 (M about 200) that
// takes a token's strength, in all columns, below 10^-6.
constexpr float kRange = 0x1p-28f;

// What a wavefront of the solving half needs of one block in registers, and one of the output half.
struct SolveStage {
  half8_t k[4], t_hi[2], t_lo[2];  // k: 32 channels of all 64 tokens
};
template <int KS>
struct OutStage {
  half8_t q[KS], a_hi[2], a_lo[2]; // 16 tokens
};

// Values and row factors wait in LDS from six blocks ahead on: they come from memory, not from other workgroups' reads.
constexpr int kAhead = 6, kRing = 8;
static_assert(kAhead == 6, "the first blocks' order and counts in out_block");

// Copies 16 B (4 B) a lane from memory to LDS, lane l's to dst + 16 l (4 l): base + off, base and dst (an LDS address) the
// same for all lanes.  From inline assembly, so that the compiler does not make every later LDS read wait for it; the copies write
// no registers, and the kernel orders them itself: they are issued behind a barrier that follows every read of what
// they overwrite, waited for by count and published with a barrier.  The s_nop is the wait state that a scalar write of M0
// needs before a load to LDS; the compiler inserts none inside inline assembly.  Nothing else in this file uses M0.  The
// build checks both on the generated assembly.
typedef __attribute__((address_space(3))) void lds_void_t;
__device__ __forceinline__ void copy16_to_lds(const void* base, uint32_t off, uint32_t dst) {
  const uint32_t to = __builtin_amdgcn_readfirstlane(dst);
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" : : "v"(off), "s"(base), "s"(to) : "memory");
}
__device__ __forceinline__ void copy4_to_lds(const void* base, uint32_t off, uint32_t dst) {
  const uint32_t to = __builtin_amdgcn_readfirstlane(dst);
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1" : : "v"(off), "s"(base), "s"(to) : "memory");
}
// The waits for the copies count the loads and stores issued behind them, which the compiler could move or drop: at least N of
// them stand between this place and the next one marked, on every path, or the build, which looks at the generated
// assembly, fails.
template <int N>
__device__ __forceinline__ void ring_mark() {
  asm volatile("; ring: %0 loads and stores" : : "n"(N) : "memory");
}
// s_waitcnt immediate that waits for at most n outstanding vector memory operations.
constexpr int vmcnt_imm(int n) { return (n & 15) | 0x0F70 | ((n >> 4) << 14); }

typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4_t;
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

template <typename T>
__device__ __forceinline__ T load_at(const void* base, uint32_t bytes) {
  return *reinterpret_cast<const T*>(static_cast<const char*>(base) + bytes);
}

// The scan: one workgroup per sequence, value head and slice of 16 NC state columns; eight wavefronts that walk along
// the sequence together, three barriers a block.
//   Solving half (4 wavefronts): wavefront w keeps rows 32 w .. 32 w + 31 of the state in registers, as the second operand
//   of K S just as the last update left them.  K S over its channels for all tokens; barrier; the sum over the
//   wavefronts for tokens 16 w .. 16 w + 15, R; barrier; U = T R; barrier; its rows' update.
//   Output half: Q S of 16 tokens each while the others solve, A U and the stores while they are at the next block.
// Bound by the chain through the barriers, 1.3 us or about 3000 cycles a block: 8192 tokens of 32 heads of 128 take 167 us
// with every compute unit at work and as long with one head on the machine.
template <int DK, int NC>
struct Scan {
  static constexpr int KS = DK / 32;
  static constexpr uint32_t kNone = 0x7F800000u;         // a token that writes nothing: infinity
  struct Lds {
    f32x4_t X[KS][4][NC][64];                  // K S of a wavefront's channels, 16 tokens each
    half8_t S[2][NC][KS][64];                  // the state in two parts, as an operand
    _Float16 R[2][NC][16][kTok + 8];
    _Float16 U[2][NC][16][kTok + 8];           // U times the decays to the block's end, in the state's unit, in two parts
    _Float16 O[2][2][NC][16][kTok + 8];        // U for the outputs, of two blocks, in two parts
    half4_t K[KS][2][kTok * 4];                // a wavefront's channels of K in two 16s, for their transposition
    uint16_t V[kRing][kTok][16 * NC];          // values
    float rows[kRing][4][kTok];                // row factors: beta, c, d, e
    float decay[kRing][64];                    // of the whole block, copies; NaN where it is out of the scale's premise
    float norm[KS][NC * 16];
    uint32_t top[3][NC * 16];                  // largest |beta v| of a block, as bits
    float least[3];                            // the smallest that a block's tokens write, zeros aside, or the first's rest
    float units[2][2][NC * 16];                // for the output half: ratio, and the block's unit times the scale
  };

  const DeltaArgs& a;
  const ChunkWork& ws;
  Lds& lds;
  const uint32_t lds_base;
  const int lane, w, c, g, seq, head, k_head, c0;
  SeqRows rows;
  int n, blocks, slot0;
  int slot;                                    // of the sequence's state, or -1
  bool old;                                    // it is read
  const float one = hidden_one();

  __device__ Scan(const DeltaArgs& args, const ChunkWork& work, Lds& shared, uint32_t base, int seq_, int head_, int k_head_, int c0_)
      : a(args), ws(work), lds(shared), lds_base(base), lane(threadIdx.x & 63), w(__builtin_amdgcn_readfirstlane(threadIdx.x >> 6)),
        c(lane & 15), g(lane >> 4), seq(seq_), head(head_), k_head(k_head_), c0(c0_) {}

  __device__ __forceinline__ uint32_t lds_address(const void* p) const {
    return lds_base + (uint32_t)(static_cast<const char*>(p) - reinterpret_cast<const char*>(&lds));
  }

  // A pointer that walks along the blocks, kept in scalar registers; it stays at the last one.
  struct Walk {
    const char* p;
    int64_t step;
    __device__ __forceinline__ void next(bool more) { p += more ? step : 0; }
  };
  __device__ __forceinline__ Walk walk(const void* base, int heads, int h, int bytes) const {
    return Walk{static_cast<const char*>(base) + ((int64_t)slot0 * heads + h) * bytes, (int64_t)heads * bytes};
  }

  // Where 4 channels (one of four) of a token lie: every second eight tokens with their halves of 32 words and of 4
  // exchanged, so that neither the writes (16 tokens, 2 parts at a time) nor the transposing reads (4 tokens each of two
  // eights, all parts) meet in a bank.
  __device__ __forceinline__ static int place(int token, int part) {
    const int odd = token >> 3 & 1;
    return (token * 4 + part) ^ (odd * 18);
  }

  // Four values of two results' rows as one operand, in two parts.
  __device__ __forceinline__ void operand(const f32x4_t& x, const f32x4_t& y, half8_t& hi, half8_t& lo) const {
    half4_t a0, b0, a1, b1;
    split4(x, a0, b0, one);
    split4(y, a1, b1, one);
    hi = half8_t{a0[0], a0[1], a0[2], a0[3], a1[0], a1[1], a1[2], a1[3]};
    lo = half8_t{b0[0], b0[1], b0[2], b0[3], b1[0], b1[1], b1[2], b1[3]};
  }

  // The power of two that takes x < 2^100 below 2^13, and its inverse: 2^-107 at least, so that it is a normal number times the
  // outputs' scale and 1 / kTri, too, and no output's error is above 2^-140 for that.
  __device__ __forceinline__ static void unit(float x, float& up, float& down) {
    const uint32_t e = max(min(__float_as_uint(x) >> 23, 226u), 32u);
    up = __uint_as_float((266u - e) << 23);
    down = __uint_as_float((e - 12u) << 23);
  }

  // ---- the solving half

  f32x4_t S[2][NC];                            // rows 32 w + 16 i + 4 g + r of column c
  // Of a column: its norm's bound and the unit of S behind the block; the block's unit, inverse; the ratios from the
  // unit of S before the block to the block's and to that behind it, and from the block's to that.
  float bound[NC], state_unit[NC], up[NC], ratio[NC], carry[NC], to_state[NC];
  float last_unit[NC];                         // of S as it is between blocks
  Walk k_at, t_at;
  bool bad = false;

  __device__ __forceinline__ bool owner() const { return KS == 4 || w < KS; }

  // Loads are straight-line and the same every time (past the end: the last block again), so that the waits in the
  // loop count on exactly what was issued since.
  // k_at and t_at: the block to load next.
  __device__ __forceinline__ void load_k(SolveStage& s, bool more) {
#pragma unroll
    for (int j = 0; j < 4; ++j) s.k[j] = load_at<half8_t>(k_at.p, ((j * KS + w % KS) * 64 + lane) * 16);
    k_at.next(more);
  }
  __device__ __forceinline__ void load_t(SolveStage& s, bool more) {
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      const uint32_t frag = tri_frag(w, min(ks, w >> 1)) * 2048 + lane * 16;
      s.t_hi[ks] = load_at<half8_t>(t_at.p, frag);
      s.t_lo[ks] = load_at<half8_t>(t_at.p, frag + 1024);
    }
    t_at.next(more);
  }

  // Units of a block, by column, from the bound before it (one more block is opened behind the last, which sees what
  // that one's decay says): everything in the block is below bound + 64 max|beta v|,
  // updates below three times that.  Between blocks S has a unit by its bound alone, which follows strong decays: to 2^-100 of
  // the block's, so that the ratios stay in range whatever the decay.  The updates go into S in that unit.
  __device__ __forceinline__ void open_block(int b) {
    const float decay = lds.decay[b % kRing][lane];
    const float least = lds.least[b % 3];
#pragma unroll
    for (int nc = 0; nc < NC; ++nc) {
      const float more = 64.0f * __uint_as_float(lds.top[b % 3][nc * 16 + c]);
      const float most = bound[nc] + more, was = state_unit[nc];
      bad |= !(most < 0x1p100f) || __builtin_fmaxf(least, decay * bound[nc]) < kRange * most;
      float now, state_up;
      unit(most, up[nc], now);
      ratio[nc] = was * up[nc];
      if (w == 3 && g == 0) {
        lds.units[b & 1][0][nc * 16 + c] = kTri * ratio[nc];
        lds.units[b & 1][1][nc * 16 + c] = now * (a.scale / kTri);
      }
      bound[nc] = __builtin_fmaf(decay, bound[nc], more) * 1.00001f;
      unit(__builtin_fmaxf(bound[nc], 0x1p-100f * most), state_up, state_unit[nc]);
      to_state[nc] = now * state_up;
      carry[nc] = was * state_up;
    }
  }

  // The compiler moves nothing across: memory instructions go out where the wavefront waits for LDS anyway, not in a
  // row that would hold up the next step.
  __device__ __forceinline__ static void here() { __builtin_amdgcn_sched_barrier(0); }

  __device__ __forceinline__ void solve_block(SolveStage& s, int b) {
    const int slot = b % kRing, row = 16 * w + 4 * g;
    const float4 be = *reinterpret_cast<const float4*>(&lds.rows[slot][0][row]), cc = *reinterpret_cast<const float4*>(&lds.rows[slot][1][row]);
    const float4 d4 = *reinterpret_cast<const float4*>(&lds.rows[slot][2][row]);
    const float decay = lds.decay[slot][lane];
    uint32_t v[NC][4];
#pragma unroll
    for (int nc = 0; nc < NC; ++nc)
#pragma unroll
      for (int r = 0; r < 4; ++r) v[nc][r] = lds.V[slot][row + r][nc * 16 + c];
    // this wavefront's channels of K S
    if (owner()) {
#pragma unroll
      for (int nc = 0; nc < NC; ++nc) {
        f32x4_t x[4];
        half8_t hi, lo;
        operand(S[0][nc], S[1][nc], hi, lo);
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = mfma(s.k[j], hi, f32x4_t{0.0f, 0.0f, 0.0f, 0.0f});
        // K / kPart is as good as K beside the second part: its elements are off by 2^-14 of a row's largest at most
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = mfma(s.k[j] * (_Float16)(1.0f / kPart), lo, x[j]);
        lds.S[0][nc][w][lane] = hi;
        lds.S[1][nc][w][lane] = lo;
#pragma unroll
        for (int j = 0; j < 4; ++j) lds.X[w][j][nc][lane] = x[j];
      }
    }
    lds_barrier();
    f32x4_t part[KS][NC];
#pragma unroll
    for (int nc = 0; nc < NC; ++nc)
#pragma unroll
      for (int i = 0; i < KS; ++i) part[i][nc] = lds.X[i][w][nc][lane];
    here();
    if (owner()) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const half8_t k = s.k[j];
        lds.K[w][0][place(16 * j + c, g)] = half4_t{k[0], k[1], k[2], k[3]};
        lds.K[w][1][place(16 * j + c, g)] = half4_t{k[4], k[5], k[6], k[7]};
      }
    }
    load_k(s, b + 3 < blocks);
    here();
    const float beta[4] = {be.x, be.y, be.z, be.w}, c4[4] = {cc.x, cc.y, cc.z, cc.w};
#pragma unroll
    for (int nc = 0; nc < NC; ++nc) {
      f32x4_t r4;
#pragma unroll
      for (int i = 1; i < KS; i += 2) part[i - 1][nc] += part[i][nc];
      if (KS == 4) part[0][nc] += part[2][nc];
#pragma unroll
      for (int r = 0; r < 4; ++r)
        r4[r] = __builtin_fmaf(beta[r] * __uint_as_float(v[nc][r] << 16), up[nc], -(c4[r] * ratio[nc]) * part[0][nc][r]);
      half4_t rh, rl;
      split4(r4, rh, rl, one);
      *reinterpret_cast<half4_t*>(&lds.R[0][nc][c][16 * w + 4 * g]) = rh;
      *reinterpret_cast<half4_t*>(&lds.R[1][nc][c][16 * w + 4 * g]) = rl;
    }
    lds_barrier();
    half8_t rh[2][NC], rl[2][NC];
#pragma unroll
    for (int nc = 0; nc < NC; ++nc)
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        if (ks > (w >> 1)) continue;
        rh[ks][nc] = *reinterpret_cast<const half8_t*>(&lds.R[0][nc][c][ks * 32 + g * 8]);
        rl[ks][nc] = *reinterpret_cast<const half8_t*>(&lds.R[1][nc][c][ks * 32 + g * 8]);
      }
    here();
#pragma unroll
    for (int nc = 0; nc < NC; ++nc) {
      const f32x4_t zero = {0.0f, 0.0f, 0.0f, 0.0f};
      f32x4_t u = mfma(s.t_hi[0], rh[0][nc], zero), ul = mfma(s.t_lo[0], rh[0][nc], zero);
      ul = mfma(s.t_hi[0], rl[0][nc], ul);
      if (w >= 2) {
        u = mfma(s.t_hi[1], rh[1][nc], u);
        ul = mfma(s.t_lo[1], rh[1][nc], ul);
        ul = mfma(s.t_hi[1], rl[1][nc], ul);
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) u[r] = __builtin_fmaf(ul[r], 1.0f / kPart, u[r]) * (1.0f / kTri);
      const float d[4] = {d4.x, d4.y, d4.z, d4.w};
      half4_t uh, uw, oh, ow;
      const float to = to_state[nc];
      split4(f32x4_t{u[0] * (d[0] * to), u[1] * (d[1] * to), u[2] * (d[2] * to), u[3] * (d[3] * to)}, uh, uw, one);
      *reinterpret_cast<half4_t*>(&lds.U[0][nc][c][16 * w + 4 * g]) = uh;
      *reinterpret_cast<half4_t*>(&lds.U[1][nc][c][16 * w + 4 * g]) = uw;
      split4(u, oh, ow, one);
      *reinterpret_cast<half4_t*>(&lds.O[b & 1][0][nc][c][16 * w + 4 * g]) = oh;
      *reinterpret_cast<half4_t*>(&lds.O[b & 1][1][nc][c][16 * w + 4 * g]) = ow;
    }
    half8_t kt[2][2];
    if (owner()) {
      // Transposed K: lane i of 16 addresses 4 channels of token i / 4 and gets channel i of 4 tokens.
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          half4_t p[2];
#pragma unroll
          for (int h = 0; h < 2; ++h)
            p[h] = __builtin_bit_cast(half4_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (lds_s16x4_t*)&lds.K[w][i][place(ks * 32 + g * 8 + h * 4 + (c >> 2), c & 3)]));
          kt[ks][i] = half8_t{p[0][0], p[0][1], p[0][2], p[0][3], p[1][0], p[1][1], p[1][2], p[1][3]};
        }
    }
#pragma unroll
    for (int nc = 0; nc < NC; ++nc) {
      last_unit[nc] = state_unit[nc];
#pragma unroll
      for (int i = 0; i < 2; ++i) S[i][nc] *= decay * carry[nc];
    }
    lds_barrier();
    // S <- decay S + K^T U
    half8_t uh[2][NC], ul[2][NC];
    if (owner()) {
#pragma unroll
      for (int nc = 0; nc < NC; ++nc)
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
          uh[ks][nc] = *reinterpret_cast<const half8_t*>(&lds.U[0][nc][c][ks * 32 + g * 8]);
          ul[ks][nc] = *reinterpret_cast<const half8_t*>(&lds.U[1][nc][c][ks * 32 + g * 8]);
        }
    }
    here();
    load_t(s, b + 3 < blocks);
    open_block(b + 1);
    here();
    if (owner()) {
#pragma unroll
      for (int nc = 0; nc < NC; ++nc) {
        f32x4_t low[2] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
#pragma unroll
          for (int i = 0; i < 2; ++i) low[i] = mfma(kt[ks][i], ul[ks][nc], low[i]);
#pragma unroll
          for (int i = 0; i < 2; ++i) S[i][nc] = mfma(kt[ks][i], uh[ks][nc], S[i][nc]);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) S[i][nc][r] = __builtin_fmaf(low[i][r], 1.0f / kPart, S[i][nc][r]);
      }
    }
  }

  __device__ __forceinline__ void solve() {
    SolveStage even, odd;
    k_at = walk(ws.k, a.k_heads, k_head, 4 * KS * 1024);
    t_at = walk(ws.t, a.v_heads, head, kTriFrags * 2048);
    float* state = static_cast<float*>(a.s.state) + (slot >= 0 ? slot : 0) * a.s.slot +
                   ((int64_t)head * DK + (w % KS) * 32 + 4 * g) * a.v_dim + c0 + c;
    // all CUs begin at once: what the first block needs is asked for first
#pragma unroll
    for (int nc = 0; nc < NC; ++nc)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) S[i][nc][r] = old ? state[(int64_t)(16 * i + r) * a.v_dim + nc * 16] : 0.0f;
    load_k(even, blocks > 1);
    load_t(even, blocks > 1);
    if (w == 0 && lane < 3 * 16) {
#pragma unroll
      for (int nc = 0; nc < NC; ++nc) (&lds.top[0][0])[nc * 48 + lane] = 0;
    }
#pragma unroll
    for (int nc = 0; nc < NC; ++nc) {
      float m = 0.0f;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) m += __builtin_fabsf(S[i][nc][r]);
      m = quad_sum(m);
      if (g == 0 && owner()) lds.norm[w][nc * 16 + c] = m;
    }
    lds_barrier();
#pragma unroll
    for (int nc = 0; nc < NC; ++nc) {
      bound[nc] = 0.0f;
#pragma unroll
      for (int i = 0; i < KS; ++i) bound[nc] += lds.norm[i][nc * 16 + c];
      float state_up;
      unit(bound[nc], state_up, state_unit[nc]);
#pragma unroll
      for (int i = 0; i < 2; ++i) S[i][nc] *= state_up;
    }
    load_k(odd, blocks > 2);
    load_t(odd, blocks > 2);
    lds_barrier();
    open_block(0);
    int b = 0;
    for (; b + 1 < blocks; b += 2) {
      solve_block(even, b);
      solve_block(odd, b + 1);
    }
    if (b < blocks) solve_block(even, b);
    // where a block broke the scale's premise, the slice is left as it was to the kernel behind this one
    const bool left = __builtin_amdgcn_ballot_w64(bad) != 0;
    uint8_t* flag = ws.flags + ((int64_t)seq * a.v_heads + head) * (a.v_dim / 16) + c0 / 16;
    if (threadIdx.x < NC) flag[threadIdx.x] = left;
    if (slot < 0 || left || !owner()) return;
#pragma unroll
    for (int nc = 0; nc < NC; ++nc)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) state[(int64_t)(16 * i + r) * a.v_dim + nc * 16] = S[i][nc][r] * last_unit[nc];
  }

  // ---- the output half: results transposed, a lane holds 4 neighbouring columns of token c

  static constexpr int kLoads = KS + 4;        // of a block: Q's and A's fragments

  Walk q_at, a_at, f_at, v_at, o_at;           // the block to load or copy next, and the one to write

  __device__ __forceinline__ void load_q(OutStage<KS>& s, bool more) {
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) s.q[ks] = load_at<half8_t>(q_at.p, (((w - 4) * KS + ks) * 64 + lane) * 16);
    q_at.next(more);
  }
  __device__ __forceinline__ void load_a(OutStage<KS>& s, bool more) {
    const int o = w - 4;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      const uint32_t frag = tri_frag(o, min(ks, o >> 1)) * 2048 + lane * 16;
      s.a_hi[ks] = load_at<half8_t>(a_at.p, frag);
      s.a_lo[ks] = load_at<half8_t>(a_at.p, frag + 1024);
    }
    a_at.next(more);
  }

  // Starts the copies of a block's values and row factors: one or two of a wavefront.
  __device__ __forceinline__ void copy_rows(int block) {
    const int slot = block % kRing, last = n - 1 - min(block, blocks - 1) * kTok;
    const bool more = block + 1 < blocks;
#pragma unroll
    for (int i = 0; i < 2 * NC + 2; ++i) {
      if (i % 4 != w - 4) continue;
      if (i < 2 * NC) {
        // rows behind the end repeat the last one; their beta is 0
        const int l = i * 64 + lane, row = min(l / (2 * NC), last);
        copy16_to_lds(v_at.p, (uint32_t)row * (uint32_t)a.v_tok * 2 + l % (2 * NC) * 16, lds_address(&lds.V[slot]) + i * 1024);
      } else if (i == 2 * NC) {
        copy16_to_lds(f_at.p, lane * 16, lds_address(&lds.rows[slot]));
      } else {
        copy4_to_lds(f_at.p, 4 * kTok * 4 + 4 * c, lds_address(&lds.decay[slot]));
      }
    }
    v_at.next(more);
    f_at.next(more);
  }

  // The largest |beta v| of 16 tokens, by column, for the block's units: read, then written.
  struct TopRows {
    float4 beta;
    uint32_t v[NC][4];
  };
  __device__ __forceinline__ void read_top(TopRows& t, int block) {
    const int slot = block % kRing, row = 16 * (w - 4) + 4 * g;
    t.beta = *reinterpret_cast<const float4*>(&lds.rows[slot][0][row]);
#pragma unroll
    for (int nc = 0; nc < NC; ++nc)
#pragma unroll
      for (int r = 0; r < 4; ++r) t.v[nc][r] = lds.V[slot][row + r][nc * 16 + c];
  }
  __device__ __forceinline__ void write_top(const TopRows& t, int block) {
    const float b[4] = {t.beta.x, t.beta.y, t.beta.z, t.beta.w};
#pragma unroll
    for (int nc = 0; nc < NC; ++nc) {
      uint32_t m = 0;                          // as bits, so that a NaN is the largest
#pragma unroll
      for (int r = 0; r < 4; ++r) m = max(m, __float_as_uint(b[r] * __uint_as_float(t.v[nc][r] << 16)) & 0x7FFFFFFFu);
      atomicMax(&lds.top[block % 3][nc * 16 + c], m);
    }
  }

  // For the check of a block's range, by one wavefront (by all four, a row to four lanes, the scan took 5 % longer): the least that
  // its tokens write, zeros aside, or what is left of the first one's at the end, if that is more.  A lane has a token and takes
  // the largest of four columns, which is hardly ever far below the whole row's; where it is 0 the row decides.
  __device__ __forceinline__ void write_least(int block) {
    typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
    const int slot = block % kRing;
    const float beta = lds.rows[slot][0][lane], decay = lds.decay[slot][lane];
    auto largest = [&](int part) {             // of four columns, as bits
      const uint2 v = *reinterpret_cast<const uint2*>(&lds.V[slot][lane][4 * part]);
      const u16x2_t two = __builtin_elementwise_max(__builtin_bit_cast(u16x2_t, v.x & 0x7FFF7FFFu),
                                                    __builtin_bit_cast(u16x2_t, v.y & 0x7FFF7FFFu));
      return (uint32_t)max(two[0], two[1]);
    };
    uint32_t most = largest(0);
    if (__builtin_amdgcn_ballot_w64(most == 0 && beta > 0.0f) != 0) {
#pragma unroll
      for (int part = 1; part < 4 * NC; ++part) most = max(most, largest(part));
    }
    const float m = beta * __uint_as_float(most << 16);
    const uint32_t least = wave_min(m > 0.0f ? __float_as_uint(m) : kNone);
    const float first = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(m)));
    if (lane == 63) lds.least[block % 3] = __builtin_fmaxf(__uint_as_float(least), decay * first);
  }

  // A U and the stores of a block, its Q S in y.
  __device__ __forceinline__ void store_out(const OutStage<KS>& s, f32x4_t (&y)[NC], const float4 (&scale)[NC], int b,
                                            uint32_t lane_at) {
    const int o = w - 4, rows_here = min(n - b * kTok, kTok);
    // a block's rows as a buffer: writes past the sequence's end go nowhere
    const __amdgpu_buffer_rsrc_t out = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<char*>(o_at.p), 0, ((uint32_t)(rows_here - 1) * (uint32_t)a.o_tok + 16 * NC) * 2, 0x00027000);
#pragma unroll
    for (int nc = 0; nc < NC; ++nc) {
      f32x4_t low = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        if (ks > (o >> 1)) continue;
        const half8_t hi = *reinterpret_cast<const half8_t*>(&lds.O[b & 1][0][nc][c][ks * 32 + g * 8]);
        const half8_t lo = *reinterpret_cast<const half8_t*>(&lds.O[b & 1][1][nc][c][ks * 32 + g * 8]);
        y[nc] = mfma(hi, s.a_hi[ks], y[nc]);
        low = mfma(hi, s.a_lo[ks], low);
        low = mfma(lo, s.a_hi[ks], low);
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) y[nc][r] = __builtin_fmaf(low[r], 1.0f / kPart, y[nc][r]);
      const u32x2_t two = {bf16_pair(y[nc][0] * scale[nc].x, y[nc][1] * scale[nc].y),
                           bf16_pair(y[nc][2] * scale[nc].z, y[nc][3] * scale[nc].w)};
      __builtin_amdgcn_raw_buffer_store_b64(two, out, lane_at, nc * 32, 0);
    }
    o_at.p += o_at.step;
  }

  // LAST: behind the loop over pairs of blocks.  No wait follows, and its loads, which nobody needs, may be dropped.
  template <bool LAST = false>
  __device__ __forceinline__ void out_block(OutStage<KS>& s, int b, uint32_t lane_at) {
    // The copies begin with two blocks (all workgroups begin at once, and wait for the first) and go on by two a block,
    // 2 b + 2 and 2 b + 3, up to a lead of kAhead = 6.  Then this wavefront waits until its part of the next block's are
    // in, by what it has issued since at least; a block issues its copies, kLoads loads and a store.  For block 1 that is
    // kLoads loads and two copies, for 2 more; for 3 two blocks and four copies, for 4 to 8 more; from 9 on kAhead - 1
    // blocks and copies.
    ring_mark<LAST ? 0 : kLoads + 1>();
    int turn = b;
    asm("" : "+s"(turn));                      // one loop for all of them
    if (turn < 4) {
      copy_rows(2 * b + 2);
      copy_rows(2 * b + 3);
    } else {
      copy_rows(b + kAhead);
    }
    if (turn < 2)
      __builtin_amdgcn_s_waitcnt(vmcnt_imm(kLoads + 2));
    else if (turn < 8)
      __builtin_amdgcn_s_waitcnt(vmcnt_imm(2 * (kLoads + 1) + 4));
    else
      __builtin_amdgcn_s_waitcnt(vmcnt_imm((kAhead - 1) * (kLoads + 1)));
    lds_barrier();
    f32x4_t y[NC];
    float4 scale[NC];
    half8_t state[2][NC][KS];
#pragma unroll
    for (int part = 0; part < 2; ++part)
#pragma unroll
      for (int nc = 0; nc < NC; ++nc)
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) state[part][nc][ks] = lds.S[part][nc][ks][lane];
    const float e = lds.rows[b % kRing][3][16 * (w - 4) + c];
    here();
    TopRows top;                               // used behind the next barrier
    read_top(top, b + 1);
    here();
#pragma unroll
    for (int nc = 0; nc < NC; ++nc) {
      f32x4_t low = {0.0f, 0.0f, 0.0f, 0.0f};
      y[nc] = low;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        y[nc] = mfma(state[0][nc][ks], s.q[ks], y[nc]);
        low = mfma(state[1][nc][ks], s.q[ks], low);
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) y[nc][r] = __builtin_fmaf(low[r], 1.0f / kPart, y[nc][r]);
      const float4 ratio = *reinterpret_cast<const float4*>(&lds.units[b & 1][0][nc * 16 + 4 * g]);
      scale[nc] = *reinterpret_cast<const float4*>(&lds.units[b & 1][1][nc * 16 + 4 * g]);
      y[nc][0] *= e * ratio.x;
      y[nc][1] *= e * ratio.y;
      y[nc][2] *= e * ratio.z;
      y[nc][3] *= e * ratio.w;
    }
    lds_barrier();
    write_top(top, b + 1);
    if (w == 4) write_least(b + 1);
    load_q(s, b + 3 < blocks);
    if (w == 7 && lane < NC * 16) lds.top[(b + 2) % 3][lane] = 0;
    lds_barrier();
    store_out(s, y, scale, b, lane_at);
    load_a(s, b + 3 < blocks);
  }

  __device__ __forceinline__ void output() {
    const uint32_t lane_at = (uint32_t)((16 * (w - 4) + c) * (uint32_t)a.o_tok + 4 * g) * 2;
    OutStage<KS> even, odd;
    q_at = walk(ws.q, a.k_heads, k_head, 4 * KS * 1024);
    a_at = walk(ws.a, a.v_heads, head, kTriFrags * 2048);
    f_at = walk(ws.factors, a.v_heads, head, kFactors * 4);
    v_at = Walk{reinterpret_cast<const char*>(a.v + rows.first * a.v_tok + head * a.v_head + c0), kTok * 2 * a.v_tok};
    o_at = Walk{reinterpret_cast<const char*>(a.out + rows.first * a.o_tok + head * a.o_head + c0), kTok * 2 * a.o_tok};
    copy_rows(0);
    ring_mark<kLoads>();
    load_q(even, blocks > 1);
    load_a(even, blocks > 1);
    ring_mark<0>();
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(kLoads));       // the first block's copies are in
    lds_barrier();
    TopRows top;
    read_top(top, 0);
    write_top(top, 0);
    if (w == 4) write_least(0);
    copy_rows(1);
    ring_mark<kLoads>();
    load_q(odd, blocks > 2);
    load_a(odd, blocks > 2);
    lds_barrier();
    int b = 0;
    for (; b + 1 < blocks; b += 2) {
      out_block(even, b, lane_at);
      out_block(odd, b + 1, lane_at);
    }
    if (b < blocks) out_block<true>(even, b, lane_at);
    ring_mark<0>();
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));   // no copy outlives the workgroup's LDS
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
  Scan<DK, NC> scan(a, ws, lds, (uint32_t)(uintptr_t)(lds_void_t*)&lds, seq, k_head * group + part / slices, k_head, part % slices * 16 * NC);
  scan.rows = seq_rows(a.s, seq);
  scan.n = scan.rows.end - scan.rows.first;
  scan.slot = seq_slot(a.s, seq);
  scan.old = scan.slot >= 0 && scalar_load(a.s.kv_len + seq) > scan.n;
  if (scan.n <= ws.short_len) return;
  scan.blocks = (scan.n + kTok - 1) / kTok;
  scan.slot0 = scan.rows.first / kTok + seq;
  if (scan.w < 4)
    scan.solve();
  else
    scan.output();
}

template <int DK, int NC>
int launch_scan(const DeltaArgs& a, const ChunkWork& ws, hipStream_t stream) {
  const int64_t pairs = (int64_t)a.s.num_seqs * a.k_heads;
  const int64_t grid = (pairs + 7) / 8 * 8 * (a.v_heads / a.k_heads) * (a.v_dim / (16 * NC));
  if (grid * kScanThreads > (int64_t)UINT32_MAX) return NVFP4_ERR_UNSUPPORTED;           // threads of a launch
  chunk_scan_kernel<DK, NC><<<(unsigned)grid, kScanThreads, 0, stream>>>(a, ws);
  return hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP;
}

template <int DK>
int launch_dk(const DeltaArgs& a, const ChunkWork& ws, int64_t max_q, hipStream_t stream) {
  DeviceInfo dev;
  const int st = device_info(stream, dev);
  if (st != NVFP4_OK) return st;
  const int64_t prepare = ws.blocks * a.k_heads * ((a.v_heads / a.k_heads + 1) / 2);
  if (prepare * kPrepareThreads > (int64_t)UINT32_MAX) return NVFP4_ERR_UNSUPPORTED;
  chunk_prepare_kernel<DK><<<(unsigned)prepare, kPrepareThreads, 0, stream>>>(a, ws);
  if (hipGetLastError() != hipSuccess) return NVFP4_ERR_HIP;
  // Slices of 16 columns while one round of workgroups holds them all, else of 32: a block of the scan takes 1.3 us
  // with 16 columns and 2.1 us with 32 (whole calls, one sequence of 8192 tokens, 256 slices of 16: 228 against 324 us; eight
  // of 1023, 2048 slices: 252 against 212).  As many sequences as the tokens give of the longest.
  const int64_t longest = max_q > a.s.tokens ? a.s.tokens : max_q > kTok ? max_q : kTok;
  const int64_t seqs = (a.s.tokens + longest - 1) / longest;
  const int64_t slices = (seqs < a.s.num_seqs ? seqs : a.s.num_seqs) * a.v_heads * (a.v_dim / 16);
  return slices <= dev.cus ? launch_scan<DK, 1>(a, ws, stream) : launch_scan<DK, 2>(a, ws, stream);
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
  ws.a = reinterpret_cast<_Float16*>(take(ws.blocks * v_heads * kTriFrags * 2 * 1024));
  ws.factors = reinterpret_cast<float*>(take(ws.blocks * v_heads * kFactors * 4));
  ws.flags = reinterpret_cast<uint8_t*>(take(num_seqs * v_heads * (v_dim / 16)));
  return (size_t)(p - static_cast<char*>(base));
}

int launch_chunks(const DeltaArgs& a, const ChunkWork& ws, int64_t max_q, int k_dim, hipStream_t stream) {
  return k_dim == 128 ? launch_dk<128>(a, ws, max_q, stream) : launch_dk<64>(a, ws, max_q, stream);
}

}  // namespace nvfp4
