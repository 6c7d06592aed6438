// gdn_q8.h -- eight values to and from e4m3 (OCP: no infinity, largest 448) on a scale.
#pragma once

#include "gdn_layer_device.h"

namespace gdn {

// The scale of values whose largest magnitude has these bits; a NaN stays one (fmaxf would drop it).
__device__ __forceinline__ float q8_scale(unsigned amax) {
  const float a = __uint_as_float(amax);
  return (a == a ? fmaxf(a, 1e-12f) : a) / 448.f;
}

// e4m3 bytes of x / scale, to nearest even.  Divided for: a product with the reciprocal may lie on the other
// side of a value half way between two e4m3 values.
__device__ __forceinline__ u32x2v q8_pack(const float (&x)[8], float scale) {
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = x[i] / scale;
    v[i] = v[i] > 448.f ? 448.f : (v[i] < -448.f ? -448.f : v[i]);  // NaN passes
  }
  u32x2v r;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h], v[4 * h + 1], 0, false);
    r[h] = (unsigned)__builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h + 2], v[4 * h + 3], w, true);
  }
  return r;
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
