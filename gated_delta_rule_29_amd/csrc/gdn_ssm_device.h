// gdn_ssm_device.h -- device-side pieces of the selective scan that its forward and backward share.
#pragma once

#include "../../include/gdn.h"
#include "gdn_layer_device.h"

namespace gdn {

// A lane's NPL states of channel c: st[c][j * NPL ..], zero behind the N-th and where st is null.
// One vector access where the lanes' shares are whole (N = LN * NPL); states are 16-byte aligned.
template <int NPL>
__device__ __forceinline__ void load_state(const float* st, int c, int j, int N, float (&h)[NPL]) {
  if (!st) {
#pragma unroll
    for (int i = 0; i < NPL; ++i) h[i] = 0.f;
    return;
  }
  const float* q = st + (int64_t)c * N + j * NPL;
  if (NPL == 4 && N % 4 == 0) {
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    if (j * NPL < N) v = *reinterpret_cast<const f32x4*>(q);
#pragma unroll
    for (int i = 0; i < NPL; ++i) h[i] = v[i % 4];
  } else {
#pragma unroll
    for (int i = 0; i < NPL; ++i) h[i] = j * NPL + i < N ? q[i] : 0.f;
  }
}
template <int NPL>
__device__ __forceinline__ void store_state(float* st, int c, int j, int N, const float (&h)[NPL]) {
  float* q = st + (int64_t)c * N + j * NPL;
  if (NPL == 4 && N % 4 == 0) {
    f32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = h[i % NPL];
    if (j * NPL < N) *reinterpret_cast<f32x4*>(q) = v;
  } else {
#pragma unroll
    for (int i = 0; i < NPL; ++i)
      if (j * NPL + i < N) q[i] = h[i];
  }
}

// B and C of the 32 tokens from tb on as fp32 pairs bc[token][n][B, C]; zero for n >= N and for tokens
// behind t1.
template <typename T, int NP>
__device__ __forceinline__ void stage_bc(const SsmParams& p, int tb, int t1, float* bc) {
  for (int e = threadIdx.x; e < kSsmChunk * NP; e += blockDim.x) {
    const int tk = e / NP, n = e % NP, t = tb + tk;
    const bool v = n < p.N && t < t1;
    bc[2 * e] = v ? to_f(static_cast<const T*>(p.Bm)[t * p.b_pitch + n]) : 0.f;
    bc[2 * e + 1] = v ? to_f(static_cast<const T*>(p.Cm)[t * p.c_pitch + n]) : 0.f;
  }
}

template <int NPL>
__device__ __forceinline__ void read_bc(const float* q, float (&b)[NPL], float (&c)[NPL]) {
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    b[i] = q[2 * i];
    c[i] = q[2 * i + 1];
  }
}

// Sum over a channel's LN lanes, in each of them.
template <int LN>
__device__ __forceinline__ float group_sum(float x) {
  x += dpp<kDppXor1>(x);
  x += dpp<kDppXor2>(x);
  if constexpr (LN == 16) {
    x += dpp<kDppHalfMirror>(x);
    x += dpp<kDppMirror>(x);
  }
  return x;
}

// Pieces of `len` tokens before sequence pc.seq.
__device__ __forceinline__ int64_t find_piece_before(const Seqs& s, const Piece& pc, int len, int lane) {
  if (!s.cu) return (int64_t)pc.seq * ((s.T + len - 1) / len);
  int sum = 0;
  for (int i = lane; i < pc.seq; i += 64) sum += (max(seq_begin(s, i + 1) - seq_begin(s, i), 0) + len - 1) / len;
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) sum += __shfl_xor(sum, m, 64);
  return sum;
}

struct SeqPieces {
  int first, count;  // a sequence's pieces
};
__device__ __forceinline__ SeqPieces pieces_of(const Seqs& s, int seq, int len, int lane) {
  Piece pc;
  pc.seq = seq;
  SeqPieces r;
  r.first = (int)find_piece_before(s, pc, len, lane);
  r.count = (max(seq_begin(s, seq + 1) - seq_begin(s, seq), 0) + len - 1) / len;
  return r;
}

// f(T{}, LN, NPL) for these types and states: four lanes a channel up to 16 states, 16 beyond.
template <typename F>
hipError_t ssm_dispatch(int dtype, int N, F&& f) {
  using std::integral_constant;
  auto states = [&](auto t) {
    if (N <= 16) return f(t, integral_constant<int, 4>{}, integral_constant<int, 4>{});
    if (N <= 32) return f(t, integral_constant<int, 16>{}, integral_constant<int, 2>{});
    return f(t, integral_constant<int, 16>{}, integral_constant<int, 4>{});
  };
  return dtype == GDN_DTYPE_BF16 ? states(bf16{}) : states(float{});
}

}  // namespace gdn
