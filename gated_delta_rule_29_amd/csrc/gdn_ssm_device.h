// gdn_ssm_device.h -- device-side pieces of the selective scan that its forward and backward share.
#pragma once

#include "../../include/gdn.h"
#include "gdn_layer_device.h"

namespace gdn {

// A lane's NPL states of channel c: st[c][j * NPL ..], zero behind the N-th and where st is null.
// One vector access where N is a multiple of a lane's four; states are 16-byte aligned then.
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

constexpr unsigned kNowhere = 0x80000000u;  // an offset behind the end of every buffer here

// A buffer over `rows` rows of `width` elements from row `row` on: loads behind the last one give 0, so
// that no load needs a branch (a branch around each load would have each waited for by itself).
// row, rows and the pitch are the same in all lanes.
template <typename T>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t window(const void* base, int64_t pitch, int row, int rows, int width) {
  const T* p = static_cast<const T*>(base) + row * pitch;
  const int bytes = rows > 0 ? (int)(((rows - 1) * pitch + width) * (int64_t)sizeof(T)) : 0;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<T*>(p), 0, bytes, 0x00020000);
}
// The element at byte offset off, as its bits.  (All of the offset is in the lane's part: the scalar
// part of a buffer offset is not compared with the buffer's end.)
template <typename T>
__device__ __forceinline__ unsigned load_bits(__amdgpu_buffer_rsrc_t r, unsigned off) {
  if constexpr (sizeof(T) == 2) return (unsigned short)__builtin_amdgcn_raw_buffer_load_b16(r, off, 0, 0);
  else return __builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0);
}
// A store there; dropped behind the buffer's end.
template <typename T>
__device__ __forceinline__ void store_bits(__amdgpu_buffer_rsrc_t r, T v, unsigned off) {
  if constexpr (sizeof(T) == 2) __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(short, v), r, off, 0, 0);
  else __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(int, v), r, off, 0, 0);
}
template <typename T>
__device__ __forceinline__ float of_bits(unsigned b) {
  return __uint_as_float(sizeof(T) == 2 ? b << 16 : b);
}

// B and C of TOK tokens on their way to LDS: load() asks for them, store() writes them as fp32 pairs
// bc[token][n][B, C], zero for n >= N and for tokens behind the end.
template <typename T, int NP, int TOK, int THREADS>
struct StageBC {
  static constexpr int PER = (TOK * NP + THREADS - 1) / THREADS;
  unsigned b[PER], c[PER];
  __device__ __forceinline__ void load(const SsmParams& p, int tb, int rows) {
    const auto rb = window<T>(p.Bm, p.b_pitch, tb, rows, p.N), rc = window<T>(p.Cm, p.c_pitch, tb, rows, p.N);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = i * THREADS + threadIdx.x, tk = e / NP, n = e % NP;
      const bool v = n < p.N && tk < TOK;
      b[i] = load_bits<T>(rb, v ? (unsigned)(tk * (int)p.b_pitch + n) * sizeof(T) : kNowhere);
      c[i] = load_bits<T>(rc, v ? (unsigned)(tk * (int)p.c_pitch + n) * sizeof(T) : kNowhere);
    }
  }
  __device__ __forceinline__ void store(float* bc) const {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = i * THREADS + threadIdx.x;
      if (PER * THREADS == TOK * NP || e < TOK * NP)
        *reinterpret_cast<float2*>(bc + 2 * e) = make_float2(of_bits<T>(b[i]), of_bits<T>(c[i]));
    }
  }
};

template <int NPL>
__device__ __forceinline__ void read_bc(const float* q, float (&b)[NPL], float (&c)[NPL]) {
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    b[i] = q[2 * i];
    c[i] = q[2 * i + 1];
  }
}

// One token's decay e^{de A}, A2 = A log2(e).  The hardware exponential is within an ulp, but a little low on
// average just below 1 (by 0.115 of 2^-24 for decays of 1e-5 to 1e-3 a token, measured over 2^20
// arguments an octave): a state that lasts 10^4 tokens would lose 7e-5 of itself.  An argument higher by
// 0.115 * 2^-24 / ln 2 = 9.9e-9 takes that mean away and costs nothing; a decay of 1 (de = 0) stays 1.
__device__ __forceinline__ float decay(float de, float A2) {
  return __builtin_amdgcn_exp2f(__builtin_fmaf(de, A2, 9.9e-9f));
}

// A channel's decay factors A log2(e) of a lane's states, zero behind the N-th.
template <int NPL>
__device__ __forceinline__ void load_decay(const SsmParams& p, int cc, int j, float (&A2)[NPL]) {
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const int n = j * NPL + i;
    A2[i] = n < p.N ? p.A[(int64_t)cc * p.N + n] * kLog2e : 0.f;
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

// The piece with its fields known to be the same in all lanes.
__device__ __forceinline__ Piece uniform(Piece p) {
  p.seq = __builtin_amdgcn_readfirstlane(p.seq);
  p.k = __builtin_amdgcn_readfirstlane(p.k);
  p.before = __builtin_amdgcn_readfirstlane(p.before);
  p.begin = __builtin_amdgcn_readfirstlane(p.begin);
  p.end = __builtin_amdgcn_readfirstlane(p.end);
  return p;
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

// Offsets on the device that are not those of the host (against the contract) must not lead out of
// what the host sized: numbers of pieces and chunks are held to its totals.
struct SeqPieces {
  int first, count;  // a sequence's pieces
};
__device__ __forceinline__ SeqPieces pieces_of(const Seqs& s, int seq, int len, int total, int lane) {
  Piece pc;
  pc.seq = seq;
  SeqPieces r;
  r.first = min((int)find_piece_before(s, pc, len, lane), total);
  r.count = min((max(seq_begin(s, seq + 1) - seq_begin(s, seq), 0) + len - 1) / len, total - r.first);
  return r;
}

// What a workgroup of four waves does: a segment of len tokens, 4 * 64 / LN channels of it, and this lane's part.
template <int LN>
struct Place {
  static constexpr int CH = 64 / LN;
  int lane, wv, j, seg, grp, c, cc, t0, t1;
  bool cv;  // the lane has a channel (loads of a lane without one read the last channel's)
  Piece pc;
  // total: the pieces of len tokens in all (as many as sequences where none is cut)
  __device__ __forceinline__ Place(const SsmParams& p, int groups, int len, int total) {
    // Four lanes a channel: a workgroup's 64 channels are whole cache lines, and the segments that a
    // summary leaves out are spread over the XCDs (in contiguous stretches they left half of
    // them idle).  16 lanes: neighbours share lines and belong on one XCD.
    const int bid = LN == 4 ? blockIdx.x : xcd_contiguous(blockIdx.x, gridDim.x);
    lane = threadIdx.x & 63;
    wv = threadIdx.x >> 6;
    j = lane % LN;
    seg = bid / groups;
    grp = bid - seg * groups;
    c = (grp * 4 + wv) * CH + lane / LN;
    cv = c < p.D;
    cc = cv ? c : p.D - 1;
    pc = uniform(total == p.s.n ? whole_sequence(p.s, seg) : find_piece(p.s, seg, len, lane));
    t0 = pc.begin + pc.k * len;
    t1 = min(t0 + len, pc.end);
  }
};

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
