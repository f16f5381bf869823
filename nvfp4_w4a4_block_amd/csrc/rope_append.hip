// Per-head norms of queries and keys with the position rotation (qk_norm_rope), and appending keys
// and values to the paged cache with both on the way (kv_append), for gfx950.
//
// What is computed, per head vector x of D channels, in fp32 and rounded once when stored:
//   x <- x * w / sqrt(sum(x^2) / D + eps)
//   (x_a, x_b) <- (x_a cos_i - x_b sin_i, x_b cos_i + x_a sin_i) over the channel pairs i of the first
//   R channels; cos and sin from the position's table row
// and for the cache the codec's E4M3 byte of the fp32 value under the head's scale, or bf16.
//
// HBM-bound: every element is read once and written once.  A lane holds 8 consecutive channels (16 B
// of bf16 in, 16 B of bf16 or 8 B of E4M3 out), a head vector is spread over D / 8 lanes (rounded up
// to a power of two).  A wavefront takes ONE token and up to U groups of 64 / lanes head vectors, each group of
// queries, keys or values only: sequence, position, page, kind and their addresses are wave-uniform and
// looked up once, all loads go out first, and a lane's angles serve every group (its channels are the same in
// all).  The partner channel of the half-split rotation is R / 16 lanes away (one cross-lane read per
// channel); interleaved pairs lie in the lane.  The sum of squares is a butterfly over the vector's lanes.
// Measured: norms and rotation of 8192 tokens of 48 heads of 128 in 44 us (4.7 TB/s; a copy reaches 5.0), with values
// and an E4M3 cache in 56 to 59 us (3.8 to 4.0 TB/s, limited by the wavefronts in flight: their lookups come before their
// compute).  Two groups a wavefront; four cost occupancy (60 to 63 us), one repeats the lookups (24 against 22 us for
// 4096 tokens).
#include "fp8_device.h"
#include "paged_device.h"

namespace nvfp4 {

namespace {

constexpr int kThreads = 256;
// Groups of a wavefront where there are many: an fp32 lane has twice the bytes in flight already (4096 tokens of 48
// heads of 128: 45.3 us with two groups, 43.9 with one).
template <typename XT>
constexpr int kGroups = sizeof(XT) == 2 ? 2 : 1;

__device__ __forceinline__ void load8(const float* x, float (&e)[8]) {
  const float4 a = reinterpret_cast<const float4*>(x)[0], b = reinterpret_cast<const float4*>(x)[1];
  e[0] = a.x; e[1] = a.y; e[2] = a.z; e[3] = a.w;
  e[4] = b.x; e[5] = b.y; e[6] = b.z; e[7] = b.w;
}

// 8 channels as they lie in memory, widened only when their group's turn comes: half the registers for bf16.
template <typename XT>
struct Raw {
  uint4 w[sizeof(XT) / 2];
};

template <typename XT>
__device__ __forceinline__ void load_raw(const XT* x, Raw<XT>& r) {
#pragma unroll
  for (int i = 0; i < (int)sizeof(XT) / 2; ++i) r.w[i] = reinterpret_cast<const uint4*>(x)[i];
}

template <typename XT>
__device__ __forceinline__ void widen_raw(const Raw<XT>& r, float (&e)[8]) {
  constexpr int N = sizeof(XT) / 2;
#pragma unroll
  for (int i = 0; i < N; ++i) widen(r.w[i], e + i * (8 / N), static_cast<const XT*>(nullptr));
}

__device__ __forceinline__ uint4 pack_bf16(const float (&e)[8]) {
  return make_uint4(bf16_pair(e[0], e[1]), bf16_pair(e[2], e[3]), bf16_pair(e[4], e[5]), bf16_pair(e[6], e[7]));
}

__device__ __forceinline__ uint2 pack_fp8(const float (&e)[8], const FastQuotient& f) {
  bool nan = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) nan |= e[i] != e[i];
  if (fast_scale(f.s) && !nan) return make_uint2(fp8x4_fast(e, f), fp8x4_fast(e + 4, f));
  return make_uint2(fp8x4_exact(e, f.s), fp8x4_exact(e + 4, f.s));
}

// The operand of a kind, field by field: a reference into the kernel's arguments would put them in memory.
__device__ __forceinline__ HeadsView pick(int kind, const HeadsView& q, const HeadsView& k, const HeadsView& v) {
  return HeadsView{kind == 0 ? q.data : (kind == 1 ? k.data : v.data), kind == 0 ? q.tok : (kind == 1 ? k.tok : v.tok),
                   kind == 0 ? q.head : (kind == 1 ? k.head : v.head), kind == 0 ? q.heads : (kind == 1 ? k.heads : v.heads)};
}

// 1 / sqrt(v) as hi + lo: one Newton step from the hardware's reciprocal root, its residual 1 - v r^2 in twice the
// precision, kept in two parts, so that x hi + x lo is rounded once.  (Root and quotient each rounded were less exact
// than the formula step by step: 5.8e-8 against 5.4e-8 of fp32 norms and rotations, this 4.7e-8.)  v outside the range
// where nothing in the step overflows or loses bits (0 and infinite among it) takes the root and quotient themselves.
__device__ __forceinline__ void reciprocal_root(float v, float& hi, float& lo) {
  if (v >= 0x1p-90f && v <= 0x1p90f) {
    const float r = __builtin_amdgcn_rsqf(v), t = v * r;
    const float e = __builtin_fmaf(-__builtin_fmaf(v, r, -t), r, __builtin_fmaf(-t, r, 1.0f));
    const float d = 0.5f * r * e;
    hi = r + d;
    lo = d - (hi - r);
  } else {
    hi = 1.0f / __builtin_sqrtf(v);
    lo = 0.0f;
  }
}

__device__ __forceinline__ FastQuotient quotient_of(float s) { return FastQuotient{s, 1.0f / s, 440.0f * s}; }

// LPR lanes per head vector (power of two), U groups per wavefront, XT the input type, APPEND: keys and values go
// to the cache.
template <typename XT, int LPR, int U, bool APPEND>
__global__ __launch_bounds__(kThreads) void rope_append_kernel(RopeAppendArgs a) {
  constexpr int RPW = 64 / LPR;                 // head vectors per group
  const int lane = threadIdx.x & 63;
  const int job = __builtin_amdgcn_readfirstlane(blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6));
  const int token = job / a.jobs, group0 = (job - token * a.jobs) * U;
  if (token >= a.tokens) return;
  const int li = lane & (LPR - 1), d0 = li * 8; // lane in its head vector, its first channel
  const int gq = (a.q.heads + RPW - 1) / RPW, gk = (a.k.heads + RPW - 1) / RPW;

  // The sequence's search goes out ahead of the vectors' loads, which it would otherwise wait for (vector loads
  // return in order); up to 63 sequences are one probe per lane.
  const int32_t* cu = a.cu_q;
  const bool one_probe = APPEND && a.num_seqs < 64;
  int probe = 0;
  if (one_probe) probe = cu[lane < a.num_seqs ? lane : a.num_seqs];
  __builtin_amdgcn_sched_barrier(0);
  Raw<XT> raw[U];
  int kind[U], head[U];                         // 0: query, 1: key, 2: value
  bool live[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int g = group0 + u;
    kind[u] = g < gq ? 0 : (g < gq + gk ? 1 : 2);
    const HeadsView x = pick(kind[u], a.q, a.k, a.v);
    head[u] = (kind[u] == 0 ? g : (kind[u] == 1 ? g - gq : g - gq - gk)) * RPW + lane / LPR;
    live[u] = g < a.groups && head[u] < x.heads && d0 < a.dim;
    raw[u] = Raw<XT>{};
    if (live[u]) load_raw(static_cast<const XT*>(x.data) + token * x.tok + head[u] * x.head + d0, raw[u]);
  }

  int64_t place = 0;                            // the token's place in its sequence
  int64_t page_row = 0;                         // its row in a page
  uint8_t *k_page = nullptr, *v_page = nullptr;
  if (APPEND) {
    const int seq = one_probe
        ? __builtin_popcountll(__builtin_amdgcn_ballot_w64(lane <= a.num_seqs && probe <= token)) - 1
        : wave_search(a.num_seqs + 1, [=](int j) { return cu[j] <= token; });
    if (seq < 0 || seq >= a.num_seqs) return;   // the token belongs to nobody
    place = (int64_t)scalar_load(a.kv_len + seq) - ((int64_t)scalar_load(a.cu_q + seq + 1) - token);
    const int64_t block = place >> a.page_shift;
    if (place >= 0 && block < a.table_width) {
      const int page = scalar_load(a.page_table + seq * a.table_stride + block);
      if (page >= 0 && page < a.num_pages) {
        k_page = a.k_cache + page * a.k_page;
        v_page = a.v_cache + page * a.v_page;
        page_row = place & ((1 << a.page_shift) - 1);
      }
    }
  }

  const int half = a.rot / 2;
  const int64_t pos = a.table && a.positions ? scalar_load(a.positions + token) : place;
  const bool known = pos >= 0 && pos < a.table_rows;
  const bool turns = a.table && d0 < a.rot, first = d0 < half;
  float c[8], n[8];                             // interleaved: the first four
  if (turns && known && kind[0] != 2) {         // groups are in the order of their kinds
    const float* t = a.table + pos * a.rot;
    if (a.interleaved) {
      const float4 x = *reinterpret_cast<const float4*>(t + d0 / 2), y = *reinterpret_cast<const float4*>(t + half + d0 / 2);
      c[0] = x.x; c[1] = x.y; c[2] = x.z; c[3] = x.w;
      n[0] = y.x; n[1] = y.y; n[2] = y.z; n[3] = y.w;
    } else {
      const int i0 = first ? d0 : d0 - half;
      load8(t + i0, c);
      load8(t + half + i0, n);
      // the sine with the sign it takes in this half: x c + partner n
#pragma unroll
      for (int i = 0; i < 8; ++i) n[i] = first ? -n[i] : n[i];
    }
  }
  float g[8];                                   // the weight of the current kind
  int g_kind = -1;
  FastQuotient f{0.0f, 0.0f, 0.0f};
  int f_kind = -1;

#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (group0 + u >= a.groups) break;
    float v[8];
    widen_raw(raw[u], v);
    if (kind[u] != 2) {
      const float* w = kind[u] == 0 ? a.q_weight : a.k_weight;
      if (w) {
        if (g_kind != kind[u] && d0 < a.dim) load8(w + d0, g);
        g_kind = kind[u];
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = __builtin_fmaf(v[i], v[i], sum);
#pragma unroll
        for (int m = 1; m < LPR; m *= 2) sum += __shfl_xor(sum, m, 64);
        if (live[u]) {
          float r, r_lo;
          reciprocal_root(sum / (float)a.dim + a.eps, r, r_lo);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = __builtin_fmaf(v[i], r, v[i] * r_lo) * g[i];
        }
      }
      if (a.table) {
        if (a.interleaved) {
          if (turns && known) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float x = v[2 * i], y = v[2 * i + 1];
              v[2 * i] = __builtin_fmaf(x, c[i], -(y * n[i]));
              v[2 * i + 1] = __builtin_fmaf(y, c[i], x * n[i]);
            }
          }
        } else {
          const int partner = lane + (first ? half / 8 : -(half / 8));
          float o[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = __shfl(v[i], partner & 63, 64);     // every lane takes part
          if (turns && known) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = __builtin_fmaf(v[i], c[i], o[i] * n[i]);
          }
        }
        if (turns && !known) {
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = __builtin_nanf("");
        }
      }
    }
    if (kind[u] == 0 || !APPEND) {
      if (!live[u]) continue;
      const HeadsView o = pick(kind[u], a.q_out, a.k_out, a.k_out);
      const int64_t at = token * o.tok + head[u] * o.head + d0;
      if (a.out_bf16) {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(o.data) + at) = pack_bf16(v);
      } else {
        float4* p = reinterpret_cast<float4*>(static_cast<float*>(o.data) + at);
        p[0] = make_float4(v[0], v[1], v[2], v[3]);
        p[1] = make_float4(v[4], v[5], v[6], v[7]);
      }
    } else {
      if (!k_page) return;                      // no page: keys and values are dropped
      uint8_t* base = kind[u] == 1 ? k_page : v_page;
      const int64_t at = (((int64_t)head[u] << a.page_shift) + page_row) * a.dim + d0;
      if (a.fp8) {
        // one scale per cache: its reciprocal serves every group of the kind
        if (a.scale_stride != 0) {
          if (live[u]) f = quotient_of((kind[u] == 1 ? a.k_scale : a.v_scale)[head[u]]);
        } else if (f_kind != kind[u]) {
          f = quotient_of(scalar_load(kind[u] == 1 ? a.k_scale : a.v_scale));
          f_kind = kind[u];
        }
        if (live[u]) *reinterpret_cast<uint2*>(base + at) = pack_fp8(v, f);
      } else if (live[u]) {
        *reinterpret_cast<uint4*>(base + 2 * at) = pack_bf16(v);
      }
    }
  }
}

template <typename XT, int LPR, bool APPEND>
int launch_groups(RopeAppendArgs a, hipStream_t stream) {
  constexpr int RPW = 64 / LPR;
  auto groups = [](const HeadsView& x) { return (x.heads + RPW - 1) / RPW; };
  a.groups = groups(a.q) + groups(a.k) + (APPEND ? groups(a.v) : 0);
  // Enough wavefronts to fill the GPU: several groups each, else one for the shortest path (12 groups of 128 channels
  // a token: 2048 tokens 13.3 us with two groups and 13.8 with one, 512 tokens 5.9 and 5.6).
  const bool many = (int64_t)a.tokens * a.groups >= 2 * 8192;
  const int u = many ? kGroups<XT> : 1;
  a.jobs = (a.groups + u - 1) / u;
  const int64_t jobs = (int64_t)a.tokens * a.jobs;
  if (jobs * 64 + kThreads > (int64_t)UINT32_MAX) return NVFP4_ERR_UNSUPPORTED;      // threads of a launch
  const unsigned grid = (unsigned)((jobs + kThreads / 64 - 1) / (kThreads / 64));
  if (many)
    rope_append_kernel<XT, LPR, kGroups<XT>, APPEND><<<grid, kThreads, 0, stream>>>(a);
  else
    rope_append_kernel<XT, LPR, 1, APPEND><<<grid, kThreads, 0, stream>>>(a);
  return hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP;
}

template <typename XT, bool APPEND>
int launch_lanes(const RopeAppendArgs& a, hipStream_t stream) {
  if (a.dim <= 16) return launch_groups<XT, 2, APPEND>(a, stream);
  if (a.dim <= 32) return launch_groups<XT, 4, APPEND>(a, stream);
  if (a.dim <= 64) return launch_groups<XT, 8, APPEND>(a, stream);
  if (a.dim <= 128) return launch_groups<XT, 16, APPEND>(a, stream);
  if (a.dim <= 256) return launch_groups<XT, 32, APPEND>(a, stream);
  return launch_groups<XT, 64, APPEND>(a, stream);
}

}  // namespace

int launch_rope_append(const RopeAppendArgs& a, int x_dtype, bool append, hipStream_t stream) {
  if (x_dtype == NVFP4_BF16)
    return append ? launch_lanes<uint16_t, true>(a, stream) : launch_lanes<uint16_t, false>(a, stream);
  return append ? launch_lanes<float, true>(a, stream) : launch_lanes<float, false>(a, stream);
}

}  // namespace nvfp4
