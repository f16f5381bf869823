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
// to a power of two), so a wavefront takes 64 / lanes vectors of ONE token at a time: the token's
// sequence, position, page and table row are wave-uniform and looked up once.  The partner channel of
// the half-split rotation is R / 16 lanes away (one cross-lane read per channel); interleaved pairs
// lie in the lane.  The sum of squares is a butterfly over the vector's lanes.
#include "fp8_device.h"
#include "paged_device.h"

namespace nvfp4 {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ void load8(const uint16_t* x, float (&e)[8]) {
  widen(*reinterpret_cast<const uint4*>(x), e, x);
}
__device__ __forceinline__ void load8(const float* x, float (&e)[8]) {
  const float4 a = reinterpret_cast<const float4*>(x)[0], b = reinterpret_cast<const float4*>(x)[1];
  e[0] = a.x; e[1] = a.y; e[2] = a.z; e[3] = a.w;
  e[4] = b.x; e[5] = b.y; e[6] = b.z; e[7] = b.w;
}

__device__ __forceinline__ uint4 pack_bf16(const float (&e)[8]) {
  return make_uint4(bf16_pair(e[0], e[1]), bf16_pair(e[2], e[3]), bf16_pair(e[4], e[5]), bf16_pair(e[6], e[7]));
}

__device__ __forceinline__ uint2 pack_fp8(const float (&e)[8], float s) {
  bool nan = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) nan |= e[i] != e[i];
  if (fast_scale(s) && !nan) {
    const FastQuotient f{s, 1.0f / s, 440.0f * s};
    return make_uint2(fp8x4_fast(e, f), fp8x4_fast(e + 4, f));
  }
  return make_uint2(fp8x4_exact(e, s), fp8x4_exact(e + 4, s));
}


// LPR lanes per head vector (power of two), XT the input type, APPEND: keys and values go to the cache.
template <typename XT, int LPR, bool APPEND>
__global__ __launch_bounds__(kThreads) void rope_append_kernel(RopeAppendArgs a) {
  constexpr int RPW = 64 / LPR;                 // head vectors per wavefront
  const int lane = threadIdx.x & 63;
  const int job = __builtin_amdgcn_readfirstlane(blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6));
  const int token = job / a.groups, group = job - token * a.groups;
  if (token >= a.tokens) return;
  const int li = lane & (LPR - 1);              // lane in its head vector
  const int row = group * RPW + lane / LPR;     // q heads, then k heads, then v heads
  const int d0 = li * 8;
  const int kind = row < a.q.heads ? 0 : (row < a.q.heads + a.k.heads ? 1 : 2);
  const int h = kind == 0 ? row : (kind == 1 ? row - a.q.heads : row - a.q.heads - a.k.heads);
  const bool live = row < a.q.heads + a.k.heads + (APPEND ? a.v.heads : 0) && d0 < a.dim;

  // the vector's load goes out before the lookups below
  float e[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) e[i] = 0.0f;
  if (live) {
    const HeadsView& x = kind == 0 ? a.q : (kind == 1 ? a.k : a.v);
    load8(static_cast<const XT*>(x.data) + token * x.tok + h * x.head + d0, e);
  }

  int64_t place = 0;                            // the token's place in its sequence
  int seq = 0;
  if (APPEND) {
    seq = wave_search(a.num_seqs + 1, [&](int j) { return a.cu_q[j] <= token; });
    if (seq < 0 || seq >= a.num_seqs) return;   // the token belongs to nobody
    place = (int64_t)a.kv_len[seq] - ((int64_t)a.cu_q[seq + 1] - token);
  }

  if (kind != 2) {
    const float* w = kind == 0 ? a.q_weight : a.k_weight;
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += e[i] * e[i];
#pragma unroll
    for (int m = 1; m < LPR; m *= 2) sum += __shfl_xor(sum, m, 64);
    if (w && live) {
      const float r = 1.0f / __builtin_sqrtf(sum / (float)a.dim + a.eps);
      float g[8];
      load8(w + d0, g);
#pragma unroll
      for (int i = 0; i < 8; ++i) e[i] = e[i] * r * g[i];
    }
  }
  if (a.table) {
    const int64_t pos = a.positions ? a.positions[token] : place;
    const bool known = pos >= 0 && pos < a.table_rows;
    const float* t = a.table + (known ? pos : 0) * a.rot;
    const int half = a.rot / 2;
    const bool turns = d0 < a.rot && kind != 2;
    const float nan = __builtin_nanf("");
    if (a.interleaved) {
      if (turns && known) {
        const float4 c = *reinterpret_cast<const float4*>(t + d0 / 2);
        const float4 n = *reinterpret_cast<const float4*>(t + half + d0 / 2);
        const float cc[4] = {c.x, c.y, c.z, c.w}, nn[4] = {n.x, n.y, n.z, n.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float x = e[2 * i], y = e[2 * i + 1];
          e[2 * i] = x * cc[i] - y * nn[i];
          e[2 * i + 1] = y * cc[i] + x * nn[i];
        }
      }
    } else {
      // every lane takes part in the cross-lane reads
      const int step = half / 8;
      const bool first = d0 < half;
      const int partner = lane + (first ? step : -step);
      float o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = __shfl(e[i], partner & 63, 64);
      if (turns && known) {
        const int i0 = first ? d0 : d0 - half;
        float c[8], n[8];
        load8(t + i0, c);
        load8(t + half + i0, n);
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = first ? e[i] * c[i] - o[i] * n[i] : e[i] * c[i] + o[i] * n[i];
      }
    }
    if (turns && !known)
#pragma unroll
      for (int i = 0; i < 8; ++i) e[i] = nan;
  }
  if (!live) return;

  if (kind == 0 || !APPEND) {
    const HeadsView& o = kind == 0 ? a.q_out : a.k_out;
    const int64_t at = token * o.tok + h * o.head + d0;
    if (a.out_bf16) {
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(o.data) + at) = pack_bf16(e);
    } else {
      float4* p = reinterpret_cast<float4*>(static_cast<float*>(o.data) + at);
      p[0] = make_float4(e[0], e[1], e[2], e[3]);
      p[1] = make_float4(e[4], e[5], e[6], e[7]);
    }
    return;
  }
  const int64_t block = place >> a.page_shift;
  if (place < 0 || block >= a.table_width) return;
  const int page = a.page_table[seq * a.table_stride + block];
  if (page < 0 || page >= a.num_pages) return;
  const int64_t in_page =
      (((int64_t)h << a.page_shift) + (place & ((1 << a.page_shift) - 1))) * a.dim + d0;
  uint8_t* base = kind == 1 ? a.k_cache + page * a.k_page : a.v_cache + page * a.v_page;
  if (a.fp8) {
    const float s = (kind == 1 ? a.k_scale : a.v_scale)[h * a.scale_stride];
    *reinterpret_cast<uint2*>(base + in_page) = pack_fp8(e, s);
  } else {
    *reinterpret_cast<uint4*>(base + 2 * in_page) = pack_bf16(e);
  }
}

template <typename XT, bool APPEND>
int launch_lanes(RopeAppendArgs a, hipStream_t stream) {
  int lanes = 2;
  while (lanes * 8 < a.dim) lanes *= 2;
  const int rows = a.q.heads + a.k.heads + (APPEND ? a.v.heads : 0);
  a.groups = (rows + 64 / lanes - 1) / (64 / lanes);
  const int64_t jobs = (int64_t)a.tokens * a.groups;
  if (jobs > INT32_MAX - 8) return NVFP4_ERR_UNSUPPORTED;
  const unsigned grid = (unsigned)((jobs + kThreads / 64 - 1) / (kThreads / 64));
  switch (lanes) {
    case 2: rope_append_kernel<XT, 2, APPEND><<<grid, kThreads, 0, stream>>>(a); break;
    case 4: rope_append_kernel<XT, 4, APPEND><<<grid, kThreads, 0, stream>>>(a); break;
    case 8: rope_append_kernel<XT, 8, APPEND><<<grid, kThreads, 0, stream>>>(a); break;
    case 16: rope_append_kernel<XT, 16, APPEND><<<grid, kThreads, 0, stream>>>(a); break;
    case 32: rope_append_kernel<XT, 32, APPEND><<<grid, kThreads, 0, stream>>>(a); break;
    default: rope_append_kernel<XT, 64, APPEND><<<grid, kThreads, 0, stream>>>(a); break;
  }
  return hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP;
}

}  // namespace

int launch_rope_append(const RopeAppendArgs& a, int x_dtype, bool append, hipStream_t stream) {
  if (x_dtype == NVFP4_BF16)
    return append ? launch_lanes<uint16_t, true>(a, stream) : launch_lanes<uint16_t, false>(a, stream);
  return append ? launch_lanes<float, true>(a, stream) : launch_lanes<float, false>(a, stream);
}

}  // namespace nvfp4
