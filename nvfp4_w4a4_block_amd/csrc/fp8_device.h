// FP8 (E4M3FN) encode and decode of fp32 values under a scale, shared by the KV-cache codec and
// the paged-cache kernels:
//   encode: byte = sign | E4M3_RNE_SAT(fl32(|x| / s)); +-inf -> +-448; NaN -> 0x7F
//   decode: fl32(E4M3(byte) * s); 0x7F / 0xFF -> NaN
// The fast path (scales in [2^-64, 2^64], non-NaN inputs) gives the bytes of the exact one; the
// codec's file states why.
#pragma once

#include "nvfp4_device.h"

namespace nvfp4 {

__device__ __forceinline__ uint32_t fp8_encode(float x, float s) {
  const float t = x / s;                                    // IEEE binary32 division
  const float a = __builtin_fabsf(t);
  if (a != a) return 0x7Fu;
  return e4m3_encode_rne_sat(a) | ((__float_as_uint(t) >> 24) & 0x80u);
}

// Operands of the fast quantize path: s, r = fl32(1 / s) and the clamp fl32(440 s).
struct FastQuotient {
  float s, r, lim;
};

__device__ __forceinline__ bool fast_scale(float s) { return s >= 0x1p-64f && s <= 0x1p64f; }

__device__ __forceinline__ float fast_quotient(float x, const FastQuotient& f) {
  return div_rn(__builtin_amdgcn_fmed3f(x, -f.lim, f.lim), f.s, f.r);
}

// Bytes of e[0..3] in one dword (element 0 in the low byte), fast path, non-NaN inputs.
__device__ __forceinline__ uint32_t fp8x4_fast(const float* e, const FastQuotient& f) {
  uint32_t w = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(fast_quotient(e[0], f), fast_quotient(e[1], f), 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(fast_quotient(e[2], f), fast_quotient(e[3], f), (int)w, true);
}

__device__ __forceinline__ uint32_t fp8x4_exact(const float* e, float s) {
  return fp8_encode(e[0], s) | fp8_encode(e[1], s) << 8 | fp8_encode(e[2], s) << 16 | fp8_encode(e[3], s) << 24;
}

// fl32(E4M3(byte) * s) of the four bytes of w (byte 0 first): the hardware decode is exact
// and gives NaN for 0x7F / 0xFF, which the multiply keeps.
__device__ __forceinline__ void fp8x4_decode(int w, float s, float* e) {
  const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(w, false);
  const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8(w, true);
  e[0] = lo[0] * s;
  e[1] = lo[1] * s;
  e[2] = hi[0] * s;
  e[3] = hi[1] * s;
}

}  // namespace nvfp4
