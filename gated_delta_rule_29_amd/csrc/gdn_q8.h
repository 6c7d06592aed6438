// gdn_q8.h -- eight values to and from e4m3 (OCP: no infinity, largest 448) on a scale.
#pragma once

#include "gdn_layer_device.h"

namespace gdn {

// The scale of values whose largest magnitude has these bits; a NaN stays one (fmaxf would drop it).
__device__ __forceinline__ float q8_scale(unsigned amax) {
  const float a = __uint_as_float(amax);
  return (a == a ? fmaxf(a, 1e-12f) : a) / 448.f;
}

__device__ __forceinline__ u32x2v q8_convert(const float (&v)[8]) {
  u32x2v r;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h], v[4 * h + 1], 0, false);
    r[h] = (unsigned)__builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h + 2], v[4 * h + 3], w, true);
  }
  return r;
}

// e4m3 bytes of the quotients x / scale, to nearest even.  A product with the scale's reciprocal is off from the
// quotient by less than 2^-21 of it, and may lie on the other side of a value half way between two e4m3 values: where
// the products 2^-21 below and above it do not become the same bytes, in any of the wave's lanes, and for scales that
// are not finite, the quotients are formed.  (8 divisions are 80 instructions, this is 40: 33 -> 22 us for 8192 tokens
// of 8 heads of 128 columns.)  A product above 448 is so by less than 2^-20 of it, and becomes 448.
__device__ __forceinline__ u32x2v q8_pack(const float (&x)[8], float scale) {
  const float inv = __builtin_amdgcn_rcpf(scale);
  float lo[8], hi[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float y = x[i] * inv;
    lo[i] = y * (1.f - 0x1p-21f);
    hi[i] = y * (1.f + 0x1p-21f);
  }
  const u32x2v q = q8_convert(lo), t = q8_convert(hi);
  if (__ballot(!(scale < __builtin_inff()) || q[0] != t[0] || q[1] != t[1]) == 0) return q;
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = x[i] / scale;
    v[i] = v[i] > 448.f ? 448.f : (v[i] < -448.f ? -448.f : v[i]);  // NaN passes
  }
  return q8_convert(v);
}

__device__ __forceinline__ void q8_unpack(u32x2v w, float (&x)[8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const auto a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[h], false);
    const auto b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[h], true);
    x[4 * h] = a[0];
    x[4 * h + 1] = a[1];
    x[4 * h + 2] = b[0];
    x[4 * h + 3] = b[1];
  }
}

// The same as bf16, which holds every e4m3 value.
__device__ __forceinline__ bf16x8 q8_bf16(u32x2v w) {
  typedef bf16 bf16x2 __attribute__((ext_vector_type(2)));
  bf16x8 r;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[h], 1.f, false);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[h], 1.f, true);
    r[4 * h] = a[0];
    r[4 * h + 1] = a[1];
    r[4 * h + 2] = b[0];
    r[4 * h + 3] = b[1];
  }
  return r;
}

}  // namespace gdn
