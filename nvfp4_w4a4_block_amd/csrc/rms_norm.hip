// Root-mean-square norms in front of and behind the 4-bit linears, with their neighbours fused and the output
// quantized on the way (gfx950):
//   add_rms_norm    r' = rnd(x + r), y = r' w / sqrt(mean(r'^2) + eps)           over a row
//   gated_rms_norm  y = x w / sqrt(mean(x^2) + eps) * z sigmoid(z)                over each head of a row
// and from y, any of: bf16 or fp32; NVFP4 as the quantizer encodes fl32(y), under a given global scale or one per row
// (max|y| / 2688); FP8 (E4M3) bytes under a given scale or one per row (max|y| / 448).
//
// HBM-bound: every element is read once and written once (calls on inputs in turn: 4096 x 5120 bf16 with residual to NVFP4,
// 138 MB, 31 us, 4.4 TB/s; gated, 8192 x 4096 to bf16, 201 MB, 37 us, 5.4 TB/s; 30 us on the same inputs every time, which
// partly stay in the 256 MB cache).  A workgroup takes one row and keeps it in registers, a thread 16 consecutive elements
// (an NVFP4 block) at a time, so that the statistics, the row's maximum and the encoding need one pass over memory.  Rows
// of at most 64 blocks share workgroups, as many to a wavefront as it holds.
//
// Arithmetic: in 64 bits from the stored r' (x and z) to y: codes of values next to a rounding border do not depend on the
// order of a sum.  The NVFP4 bytes are the quantizer's of fl32(y), the FP8 bytes the values nearest to y / scale, with one
// rounding and, per row, max|y| / 448 before its own to fp32 (quotients of fl32(y) in fp32 put one byte in about three
// million on a border's other side; 2049 x 4096 fp32: 12 us, 11 that way).  gated_rms_norm without a quantized output works
// in fp32, which hides its exponential behind the loads, but for heads that fp32 does not hold (8192 tokens of 32 heads of
// 128, inputs in turn, bf16 output: 37 us; on the same inputs 30, 58 in 64 bits; NVFP4 output, in 64 bits: 57 us, FP8
// 62 us, bound by their thousand instructions, half of them of 64 bits, for 16 elements).
#include <type_traits>

#include "fp8_device.h"
#include "gdn_internal.h"

namespace nvfp4 {

namespace {

enum Format { kNone = 0, kNvfp4 = 1, kFp8 = 2 };

template <typename T>
struct Block16 {
  uint4 w[sizeof(T)];
};

template <typename T>
__device__ __forceinline__ void load16(const T* p, float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < (int)sizeof(T); ++i)
    widen(reinterpret_cast<const uint4*>(p)[i], v + i * (16 / sizeof(T)), static_cast<const T*>(nullptr));
}

__device__ __forceinline__ float one(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }
__device__ __forceinline__ float one(const float* p) { return *p; }

__device__ __forceinline__ void store16(uint16_t* p, const float (&v)[16]) {
  uint4* o = reinterpret_cast<uint4*>(p);
  o[0] = make_uint4(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7]));
  o[1] = make_uint4(bf16_pair(v[8], v[9]), bf16_pair(v[10], v[11]), bf16_pair(v[12], v[13]), bf16_pair(v[14], v[15]));
}
__device__ __forceinline__ void store16(float* p, const float (&v)[16]) {
  float4* o = reinterpret_cast<float4*>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
}

__device__ __forceinline__ float rounded(float v, const uint16_t*) { return __uint_as_float((uint32_t)f32_to_bf16_rne(v) << 16); }
__device__ __forceinline__ float rounded(float v, const float*) { return v; }

// Sum over a row: `lanes` of a wavefront, or all the workgroup's threads; every thread of the row gets it.
__device__ __forceinline__ double group_sum(double v, double* lds, int lanes) {
  for (int m = 1; m < lanes; m *= 2) v += __shfl_xor(v, m, 64);
  if (!lds) return v;
  const int waves = blockDim.x >> 6;
  if (waves == 1) return v;
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  double s = 0.0;
  for (int i = 0; i < waves; ++i) s += lds[i];
  return s;
}

// Largest, likewise: of magnitudes' bits, NaN above infinity above the rest.
template <typename T>
__device__ __forceinline__ T group_max(T v, T* lds, int lanes) {
  for (int m = 1; m < lanes; m *= 2) v = max(v, __shfl_xor(v, m, 64));
  if (!lds) return v;
  const int waves = blockDim.x >> 6;
  if (waves == 1) return v;
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  for (int i = 0; i < waves; ++i) v = max(v, lds[i]);
  return v;
}

// E4M3 bytes of y f from 64 bits, one rounding: the product's upper 21 bits, the last one set where any below are (so that
// it lies on no border that the product does not), go through fp32 exactly.
template <bool MAY_BE_NAN>
__device__ __forceinline__ uint4 fp8_16(const double (&y)[16], double f) {
  float t[16];
  bool nan = false;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint64_t bits = __builtin_bit_cast(uint64_t, y[i] * f);
    const uint32_t hi = (uint32_t)(bits >> 32) | min((uint32_t)bits, 1u);
    t[i] = (float)__builtin_bit_cast(double, (uint64_t)hi << 32);
    if (MAY_BE_NAN) nan |= t[i] != t[i];
  }
  if (MAY_BE_NAN && nan)
    return make_uint4(fp8x4_exact(t, 1.0f), fp8x4_exact(t + 4, 1.0f), fp8x4_exact(t + 8, 1.0f), fp8x4_exact(t + 12, 1.0f));
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float c[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) c[j] = __builtin_amdgcn_fmed3f(t[4 * i + j], -448.0f, 448.0f);
    w[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c[2], c[3], __builtin_amdgcn_cvt_pk_fp8_f32(c[0], c[1], 0, false), true);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// z sigmoid(z) to about 2^-44.  e^-z = 2^n 2^f, |f| <= 1/2, n by adding 1.5 * 2^52, whose last bits are then n; 2^f by the
// polynomial of degree 9 through its values at ten Chebyshev nodes (off by 2^-46); the quotient by a Newton step from the
// hardware's estimate (2^-24 or better).  Minus infinity gives what the formula does, -inf * 0: not a number.
__device__ __forceinline__ double silu64(float gate) {
  const double z = gate == -__builtin_inff() ? __builtin_nanf("") : gate;
  const double t = (double)__builtin_amdgcn_fmed3f(gate, -700.0f, 700.0f) * -1.4426950408889634074;
  const double m = t + 0x1.8p52, f = t - (m - 0x1.8p52);
  double p = 1.0205905413765595e-07;
  p = __builtin_fma(p, f, 1.325964524488711e-06);
  p = __builtin_fma(p, f, 1.5252672924850737e-05);
  p = __builtin_fma(p, f, 0.0001540343375125101);
  p = __builtin_fma(p, f, 0.0013333558200794592);
  p = __builtin_fma(p, f, 0.009618129193934313);
  p = __builtin_fma(p, f, 0.05550410866465167);
  p = __builtin_fma(p, f, 0.2402265069564034);
  p = __builtin_fma(p, f, 0.6931471805599462);
  p = __builtin_fma(p, f, 1.0000000000000135);
  const double d = 1.0 + __builtin_ldexp(p, (int)(uint32_t)__builtin_bit_cast(uint64_t, m));
  const double r = __builtin_amdgcn_rcp(d);
  return z * __builtin_fma(__builtin_fma(-d, r, 1.0), r, r);
}

// In fp32, by the hardware's exponential and reciprocal (a unit in the last place each); the exponential's argument is
// rounded, so |z| 2^-24 relative.
__device__ __forceinline__ float silu32(float z) {
  return z * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -1.44269504088896340736f));
}

__device__ __forceinline__ double root(double v) { return __builtin_sqrt(v); }
__device__ __forceinline__ float root(float v) { return __builtin_sqrtf(v); }

constexpr int kSharedThreads = 256;

// XT: type of x; AT: type of the residual (its output has the same) or of the gates; NB: blocks of a thread, 0 for rows
// that share a workgroup, 2^row_lanes_log threads each.
template <typename XT, typename AT, int BLOCKS, bool GATED, int FORMAT>
__global__ __launch_bounds__(1024) void rms_norm_kernel(NormArgs a) {
  constexpr bool SHARED = BLOCKS == 0;
  constexpr int NB = SHARED ? 1 : BLOCKS;
  __shared__ double sums_of[16];
  typedef typename std::conditional<FORMAT == kFp8, unsigned long long, unsigned>::type Top;
  __shared__ Top tops_of[16];
  double* sums = SHARED ? nullptr : sums_of;
  Top* tops = SHARED ? nullptr : tops_of;
  const int lanes = SHARED ? 1 << a.row_lanes_log : 64;
  const int64_t row = SHARED ? (int64_t)(blockIdx.x * kSharedThreads + threadIdx.x) >> a.row_lanes_log : (int64_t)blockIdx.x;
  if (SHARED && row >= a.rows) return;
  const int tid = SHARED ? threadIdx.x & (lanes - 1) : threadIdx.x, threads = blockDim.x;
  float v[NB][16];
  double exact[FORMAT == kFp8 ? NB : 1][16];   // FP8: y is this times inv_of
  double inv_of[NB];
  bool live[NB], again[NB];
  double sum = 0.0;
#pragma unroll
  for (int n = 0; n < NB; ++n) {
    const int b = tid + n * threads;
    live[n] = b < a.blocks;
#pragma unroll
    for (int i = 0; i < 16; ++i) v[n][i] = 0.0f;
    if (GATED) {
      typedef typename std::conditional<FORMAT == kNone, float, double>::type Real;
      Real y[16], total = 0;
#pragma unroll
      for (int i = 0; i < 16; ++i) y[i] = 0;
      if (live[n]) {
        const int head = b / a.head_blocks, c = (b - head * a.head_blocks) * 16;
        float z[16], w[16];
        load16(static_cast<const XT*>(a.x) + row * a.x_row + head * a.x_head + c, v[n]);
        load16(static_cast<const AT*>(a.aux) + row * a.aux_row + head * a.aux_head + c, z);
        load16(a.weight + c, w);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const Real x = v[n][i];
          total += x * x;
          y[i] = x * (Real)w[i] * (FORMAT == kNone ? (Real)silu32(z[i]) : (Real)silu64(z[i]));
        }
      }
      // a head's blocks lie in neighbouring lanes
      for (int m = 1; m < a.head_blocks; m *= 2) total += __shfl_xor(total, m, 64);
      const Real mean = total / (Real)(a.head_blocks * 16) + (Real)a.eps, inv = (Real)1 / root(mean);
      if (FORMAT == kNone) {
        // what fp32 does not hold: squares that overflow or vanish, products with the gate that overflow ahead of the norm
        float most = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) most = __builtin_fmaxf(most, __builtin_fabsf((float)y[i]));
        again[n] = live[n] && (!(total < (Real)0x1p100) || mean < (Real)0x1p-40 || most > 0x1p100f);
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        if (FORMAT == kFp8)
          exact[n][i] = y[i];
        else
          v[n][i] = (float)(y[i] * inv);
      }
      inv_of[n] = inv;
    } else if (live[n]) {
      load16(static_cast<const XT*>(a.x) + row * a.x_row + b * 16, v[n]);
      if (a.aux) {
        float r[16];
        load16(static_cast<const AT*>(a.aux) + row * a.aux_row + b * 16, r);
#pragma unroll
        for (int i = 0; i < 16; ++i) v[n][i] = rounded(v[n][i] + r[i], static_cast<const AT*>(nullptr));
        if (a.residual_out) store16(static_cast<AT*>(a.residual_out) + row * a.residual_out_row + b * 16, v[n]);
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) sum = __builtin_fma((double)v[n][i], (double)v[n][i], sum);
    }
  }
  if (!GATED) {
    sum = group_sum(sum, sums, lanes);
    const double inv = 1.0 / __builtin_sqrt(sum / (double)(a.blocks * 16) + (double)a.eps);
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      if (!live[n]) continue;
      float w[16];
      load16(a.weight + (tid + n * threads) * 16, w);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const double y = (double)v[n][i] * (double)w[i];
        if (FORMAT == kFp8)
          exact[n][i] = y;
        else
          v[n][i] = (float)(y * inv);
      }
      inv_of[n] = inv;
    }
  }
  if (GATED && FORMAT == kNone) {
    // such heads once more, in 64 bits and from memory, so that nothing is kept ready for it
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      if (__builtin_amdgcn_ballot_w64(again[n]) == 0) continue;
      const int b = tid + n * threads, head = b / a.head_blocks, c = (b - head * a.head_blocks) * 16;
      const XT* x = static_cast<const XT*>(a.x) + row * a.x_row + head * a.x_head + c;
      const AT* z = static_cast<const AT*>(a.aux) + row * a.aux_row + head * a.aux_head + c;
      double squares = 0.0;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const double v = live[n] ? one(x + i) : 0.0f;
        squares = __builtin_fma(v, v, squares);
      }
      for (int m = 1; m < a.head_blocks; m *= 2) {
        squares += __shfl_xor(squares, m, 64);
        again[n] |= __shfl_xor((int)again[n], m, 64) != 0;
      }
      if (!again[n] || !live[n]) continue;
      const double inv = 1.0 / __builtin_sqrt(squares / (double)(a.head_blocks * 16) + (double)a.eps);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        v[n][i] = (float)((double)one(x + i) * (double)a.weight[c + i] * silu64(one(z + i)) * inv);
        __builtin_amdgcn_sched_barrier(0);               // one after the other: few registers
      }
    }
  }
  if (a.y) {
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      if (!live[n]) continue;
      const int64_t at = row * a.y_row + (tid + n * threads) * 16;
      if (FORMAT == kFp8) {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[n][i] = (float)(exact[n][i] * inv_of[n]);
      }
      if (a.y_bf16)
        store16(static_cast<uint16_t*>(a.y) + at, v[n]);
      else
        store16(static_cast<float*>(a.y) + at, v[n]);
    }
  }
  if (FORMAT == kNvfp4) {
    float s;
    if (a.given) {
      s = a.global[0];
    } else {
      unsigned top = 0;
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int i = 0; i < 16; ++i) top = !live[n] ? top : max(top, __float_as_uint(v[n][i]) & 0x7FFFFFFFu);
      top = group_max(top, reinterpret_cast<unsigned*>(tops), lanes);
      s = __uint_as_float(top) / kGlobalDivisor;
      if (tid == 0) a.global[row] = s;
    }
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      if (!live[n]) continue;
      const int64_t b = row * a.blocks + tid + n * threads;
      uint32_t scale, lo, hi;
      encode_block(v[n], s, scale, lo, hi);
      a.scales[b] = (uint8_t)scale;
      reinterpret_cast<uint2*>(a.codes)[b] = make_uint2(lo, hi);
    }
  }
  if (FORMAT == kFp8) {
    double r;                                  // 1 / scale
    bool finite = false;                       // known of the whole row
    if (a.given) {
      r = 1.0 / (double)a.global[0];
    } else {
      double most = 0.0;
      bool nan = false;
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        if (!live[n]) continue;
        double m = 0.0;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          nan |= exact[n][i] != exact[n][i];
          m = __builtin_fmax(m, __builtin_fabs(exact[n][i]));
        }
        m *= inv_of[n];
        nan |= m != m;
        most = __builtin_fmax(most, m);
      }
      unsigned long long top = nan ? 0x7FF8000000000000ull : __builtin_bit_cast(unsigned long long, most);
      top = group_max(top, reinterpret_cast<unsigned long long*>(tops), lanes);
      const double s = __builtin_bit_cast(double, top) / 448.0;
      if (tid == 0) a.global[row] = (float)s;
      finite = top < 0x7FF0000000000000ull;
      r = s == 0.0 ? 0.0 : 1.0 / s;            // a row of zeros has scale 0: signed zeros
    }
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      if (!live[n]) continue;
      const int64_t b = row * a.blocks + tid + n * threads;
      const double f = inv_of[n] * r;
      reinterpret_cast<uint4*>(a.codes)[b] = finite ? fp8_16<false>(exact[n], f) : fp8_16<true>(exact[n], f);
    }
  }
}

template <typename XT, typename AT, bool GATED, int FORMAT>
int launch_format(const NormArgs& a, hipStream_t stream) {
  const int waves = (a.blocks + 63) / 64;
  if (waves == 1) {
    // 20863 rows of 8 blocks, gated, FP8: 34.9 us with a wavefront each
    NormArgs s = a;
    while ((1 << s.row_lanes_log) < a.blocks) ++s.row_lanes_log;
    const int64_t threads = (int64_t)a.rows << s.row_lanes_log;
    rms_norm_kernel<XT, AT, 0, GATED, FORMAT><<<(unsigned)((threads + kSharedThreads - 1) / kSharedThreads), kSharedThreads, 0, stream>>>(s);
  } else if (waves <= 16)
    rms_norm_kernel<XT, AT, 1, GATED, FORMAT><<<a.rows, waves * 64, 0, stream>>>(a);
  else
    rms_norm_kernel<XT, AT, 2, GATED, FORMAT><<<a.rows, (waves + 1) / 2 * 64, 0, stream>>>(a);
  return hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP;
}

template <typename XT, typename AT, bool GATED>
int launch_types(const NormArgs& a, int format, hipStream_t stream) {
  if (format == kNvfp4) return launch_format<XT, AT, GATED, kNvfp4>(a, stream);
  if (format == kFp8) return launch_format<XT, AT, GATED, kFp8>(a, stream);
  return launch_format<XT, AT, GATED, kNone>(a, stream);
}

}  // namespace

int launch_rms_norm(const NormArgs& a, bool gated, int x_dtype, int aux_dtype, int format, hipStream_t stream) {
  const bool xb = x_dtype == NVFP4_BF16, ab = aux_dtype == NVFP4_BF16;
  if (gated)
    return xb ? (ab ? launch_types<uint16_t, uint16_t, true>(a, format, stream) : launch_types<uint16_t, float, true>(a, format, stream))
              : (ab ? launch_types<float, uint16_t, true>(a, format, stream) : launch_types<float, float, true>(a, format, stream));
  return xb ? (ab ? launch_types<uint16_t, uint16_t, false>(a, format, stream) : launch_types<uint16_t, float, false>(a, format, stream))
            : (ab ? launch_types<float, uint16_t, false>(a, format, stream) : launch_types<float, float, false>(a, format, stream));
}

}  // namespace nvfp4
