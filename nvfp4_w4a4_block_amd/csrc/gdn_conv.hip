// The short causal convolution in front of the gated delta rule, with its state and SiLU (gfx950):
//   y[t, c] = silu(bias[c] + sum_j w[c, j] x[t - (W - 1) + j, c]),  W = 2, 3 or 4
// over the tokens of each sequence; inputs before its first new token come from its state (the last W - 1 inputs),
// which is replaced by the last W - 1 inputs of all.
//
// HBM-bound: every input is read once and written once (8192 tokens of 8192 bf16 channels, 268 MB: 56-62 us, 4.3-4.8
// TB/s).  A lane holds 8 channels, a wavefront 512, and walks along a
// run of tokens with the last W - 1 inputs in registers; sequences that end inside the run are walked through.  The
// state is read for the first W - 1 tokens of a sequence only: the wavefront that has a sequence's first token takes
// those tokens all, even past the end of its run, and then replaces the state, so no other wavefront reads what it
// writes.
#include "seq_device.h"

namespace nvfp4 {

namespace {

constexpr int kThreads = 256;
constexpr int kTogether = 4;       // tokens loaded at once

// 8 channels as they lie in memory.
template <typename T>
struct Raw {
  uint4 w[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ void load_raw(const T* p, Raw<T>& r) {
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.w[i] = reinterpret_cast<const uint4*>(p)[i];
}
template <typename T>
__device__ __forceinline__ void widen_raw(const Raw<T>& r, float (&v)[8]) {
  constexpr int N = sizeof(T) / 2;
#pragma unroll
  for (int i = 0; i < N; ++i) widen(r.w[i], v + i * (8 / N), static_cast<const T*>(nullptr));
}
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]) {
  Raw<T> r;
  load_raw(p, r);
  widen_raw(r, v);
}

__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

template <typename XT, int W>
__global__ __launch_bounds__(kThreads) void conv_kernel(ConvArgs a) {
  const int lane = threadIdx.x & 63;
  const int job = __builtin_amdgcn_readfirstlane(blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6));
  const int tile = job / a.tiles;
  const int t0 = tile * a.run;
  const int c0 = (job - tile * a.tiles) * 512 + lane * 8;
  if (t0 >= a.s.tokens) return;
  const bool live = c0 < a.channels;
  const XT* x = static_cast<const XT*>(a.x);
  const int32_t* cu = a.s.cu_q;
  int seq = wave_search(a.s.num_seqs + 1, [=](int j) { return cu[j] <= t0; });
  if (seq >= a.s.num_seqs) return;             // behind the last sequence

  float w[W][8], bias[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) bias[i] = 0.0f;
  if (live) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < W; ++j) w[j][i] = a.weight[(int64_t)(c0 + i) * W + j];
    if (a.bias) load8(a.bias + c0, bias);
  }

  int t = t0;
  const int stop = t0 + a.run < a.s.tokens ? t0 + a.run : a.s.tokens;
  if (seq < 0) {                               // rows before the first sequence belong to nobody
    seq = 0;
    t = clamp_int(scalar_load(cu), t, stop);
  }
  for (; seq < a.s.num_seqs && t < stop; ++seq) {
    const SeqRows r = seq_rows(a.s, seq);
    if (r.first >= stop) break;
    if (r.end <= t) continue;
    t = t < r.first ? r.first : t;
    const int n = r.end - r.first;
    const bool head = t == r.first;
    if (!head && t - r.first < W - 1) {        // taken by the wavefront of the first token
      t = r.first + W - 1 < r.end ? r.first + W - 1 : r.end;
      if (t >= stop) break;
      if (t == r.end) continue;
    }
    float h[W - 1][8];                         // the last W - 1 inputs, oldest first
    const int slot = seq_slot(a.s, seq);
    const bool old = slot >= 0 && scalar_load(a.s.kv_len + seq) > n;
    XT* state = static_cast<XT*>(a.s.state) + (slot >= 0 ? slot : 0) * a.s.slot + c0;
    int end = r.end < stop ? r.end : stop;
    if (head) {
      const int most = r.first + W - 1 < r.end ? r.first + W - 1 : r.end;
      end = end > most ? end : most;
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
#pragma unroll
      for (int i = 0; i < 8; ++i) h[j][i] = 0.0f;
      if (!live) continue;
      if (head) {
        if (old) load8(state + j * (int64_t)a.channels, h[j]);
      } else {
        load8(x + (t - (W - 1) + j) * a.x_row + c0, h[j]);
      }
    }
    if (head && slot >= 0 && live) {           // the last W - 1 inputs of all
      float kept[W - 1][8];
#pragma unroll
      for (int j = 0; j < W - 1; ++j) {
        const int i = n - (W - 1) + j;
#pragma unroll
        for (int e = 0; e < 8; ++e) kept[j][e] = 0.0f;
        if (i >= 0)
          load8(x + (r.first + i) * a.x_row + c0, kept[j]);
        else
#pragma unroll
          for (int m = 1; m < W - 1; ++m)      // the old state moved up by the n < W - 1 new tokens
            if (m == n && j + m < W - 1)
#pragma unroll
              for (int e = 0; e < 8; ++e) kept[j][e] = h[(j + m) % (W - 1)][e];
      }
#pragma unroll
      for (int j = 0; j < W - 1; ++j) store8(state + j * (int64_t)a.channels, kept[j]);
    }
    if (!live) {
      t = t < end ? end : t;
      continue;
    }
    auto token = [&](const Raw<XT>& raw, int at) {
      float v[8], y[8];
      widen_raw(raw, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float s = bias[i];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) s = __builtin_fmaf(w[j][i], h[j][i], s);
        s = __builtin_fmaf(w[W - 1][i], v[i], s);
        // the hardware's exponential and reciprocal, a unit in the last place each: the exact quotient's ten
        // instructions an element made the kernel slower than its bytes
        y[i] = s * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(s * -1.44269504088896340736f));
#pragma unroll
        for (int j = 0; j + 1 < W - 1; ++j) h[j][i] = h[j + 1][i];
        h[W - 2][i] = v[i];
      }
      if (a.out_bf16)
        store8(static_cast<uint16_t*>(a.y) + at * a.y_row + c0, y);
      else
        store8(static_cast<float*>(a.y) + at * a.y_row + c0, y);
    };
    const XT* p = x + c0;
    for (; t + kTogether <= end; t += kTogether) {
      Raw<XT> raw[kTogether];
#pragma unroll
      for (int i = 0; i < kTogether; ++i) load_raw(p + (t + i) * a.x_row, raw[i]);
#pragma unroll
      for (int i = 0; i < kTogether; ++i) token(raw[i], t + i);
    }
    for (; t < end; ++t) {
      Raw<XT> raw;
      load_raw(p + t * a.x_row, raw);
      token(raw, t);
    }
  }
}

template <typename XT>
int launch_width(const ConvArgs& a, int width, unsigned grid, hipStream_t stream) {
  if (width == 4)
    conv_kernel<XT, 4><<<grid, kThreads, 0, stream>>>(a);
  else if (width == 3)
    conv_kernel<XT, 3><<<grid, kThreads, 0, stream>>>(a);
  else
    conv_kernel<XT, 2><<<grid, kThreads, 0, stream>>>(a);
  return hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP;
}

}  // namespace

int launch_gdn_conv(const ConvArgs& args, int x_dtype, int width, hipStream_t stream) {
  ConvArgs a = args;
  a.tiles = (a.channels + 511) / 512;
  a.run = 1;
  // Runs share the loads of weights and of the inputs before them, and cost a small call its parallelism: as long as 16
  // tokens while that leaves four wavefronts a compute unit (8192 channels, runs of 1 / 4 / 16: 256 tokens 7.9 / 5.2 / 8.3
  // us, 1024 tokens 25.2 / 11.8 / 10.5 us, 4096 tokens 84.4 / 34.2 / 27.4 us; 512 channels, 1024 tokens 4.3 / 4.6 / 7.9 us).
  while (a.run < 16 && (int64_t)a.s.tokens * a.tiles / (2 * a.run) >= 1024) a.run *= 2;
  const int64_t jobs = (int64_t)((a.s.tokens + a.run - 1) / a.run) * a.tiles;
  const int64_t grid64 = (jobs + kThreads / 64 - 1) / (kThreads / 64);
  if (grid64 * kThreads > (int64_t)UINT32_MAX) return NVFP4_ERR_UNSUPPORTED;           // threads of a launch
  const unsigned grid = (unsigned)grid64;
  return x_dtype == NVFP4_BF16 ? launch_width<uint16_t>(a, width, grid, stream) : launch_width<float>(a, width, grid, stream);
}

}  // namespace nvfp4
