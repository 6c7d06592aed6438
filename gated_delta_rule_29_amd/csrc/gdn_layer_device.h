// gdn_layer_device.h -- device-side pieces shared by the layer operators (convolution, selective
// scan, norm): vectors of inputs as fp32, the activations, lane exchanges, sequence lookup.
#pragma once

#include <utility>

#include "gdn_device.h"
#include "gdn_layer.h"

namespace gdn {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

typedef unsigned u32x2v __attribute__((ext_vector_type(2)));
typedef unsigned u32x4v __attribute__((ext_vector_type(4)));

// Calls f(std::integral_constant<int, 0>) .. f(std::integral_constant<int, N - 1>): an unrolled
// loop whose index is a constant expression (the lane-exchange builtins need one).
template <typename F, int... I>
__device__ __forceinline__ void static_for_impl(F&& f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void static_for(F&& f) {
  static_for_impl(static_cast<F&&>(f), std::make_integer_sequence<int, N>{});
}

// V consecutive values as fp32 and back: one access of 8 or 16 bytes, aligned to its size, or V is 1.
template <typename T, int V>
__device__ __forceinline__ void loadv(const T* p, float (&x)[V]) {
  if constexpr (V == 1) {
    x[0] = to_f(*p);
  } else {
    constexpr int WORDS = V * sizeof(T) / 4;
    typedef unsigned Words __attribute__((ext_vector_type(WORDS)));
    const Words r = *reinterpret_cast<const Words*>(p);
#pragma unroll
    for (int i = 0; i < WORDS; ++i) {
      if constexpr (sizeof(T) == 4) {
        x[i] = __uint_as_float(r[i]);
      } else {
        x[2 * i] = __uint_as_float(r[i] << 16);
        x[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
      }
    }
  }
}

template <typename T, int V>
__device__ __forceinline__ void storev(T* p, const float (&x)[V]) {
  if constexpr (V == 1) {
    *p = to_t<T>(x[0]);
  } else {
    typedef T Vt __attribute__((ext_vector_type(V)));
    Vt r;
#pragma unroll
    for (int i = 0; i < V; ++i) r[i] = to_t<T>(x[i]);
    *reinterpret_cast<Vt*>(p) = r;
  }
}

// 1 / (1 + e^-x): the hardware exponential and reciprocal, each within one ulp.
__device__ __forceinline__ float sigmoid_f(float x) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-kLog2e * x));
}

// log(1 + e^x) = max(x, 0) + log1p(e^-|x|), with log1p(e) = 2 atanh(s), s = e / (2 + e) <= 1/3.
// atanh(s) / s is a polynomial of degree 4 in s^2, fitted on [0, 1/9] to 7.8e-9 relative (an eighth
// of fp32's half step).  log(1 + e) itself would lose e's low bits for the small step sizes that
// matter most.  `sig`: the derivative, 1 / (1 + e^-x).
__device__ __forceinline__ float softplus_f(float x, float* sig) {
  const float e = __builtin_amdgcn_exp2f(-kLog2e * __builtin_fabsf(x));
  const float s = e * __builtin_amdgcn_rcpf(2.f + e), q = s * s;
  float t = 0x1.208bdp-3f;
  t = __builtin_fmaf(t, q, 0x1.1e510ap-3f);
  t = __builtin_fmaf(t, q, 0x1.99dae6p-3f);
  t = __builtin_fmaf(t, q, 0x1.5554ep-2f);
  t = __builtin_fmaf(t, q, 1.f);
  if (sig) {
    const float r = __builtin_amdgcn_rcpf(1.f + e);
    *sig = x >= 0.f ? r : e * r;
  }
  return __builtin_fmaf(2.f * s, t, fmaxf(x, 0.f));  // a NaN in x is in s too
}

template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
  return __uint_as_float(__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(x), CTRL, 0xf, 0xf, true));
}
// Lane-exchange controls: within four lanes the value of lane k, or of lane ^ 1 / ^ 2; within 16
// lanes that of lane k, of lane ^ 15 (mirror) or of lane ^ 7 (mirrored halves).
constexpr int dpp_quad(int k) { return k * 0x55; }
constexpr int kDppXor1 = 0xB1, kDppXor2 = 0x4E, kDppMirror = 0x140, kDppHalfMirror = 0x141;
constexpr int dpp_row(int k) { return 0x150 + k; }

// Value of lane k of this lane's group of LN lanes.
template <int LN, int K>
__device__ __forceinline__ float lane_of(float x) {
  if constexpr (LN == 4) return dpp<dpp_quad(K)>(x);
  else return dpp<dpp_row(K)>(x);
}

// The same as a move of its own, for a value that several products take: a product with a lane
// exchange in it issues at the full 4 cycles, a plain one beside another wave's in about 2.5.
template <int LN, int K>
__device__ __forceinline__ float shared_lane(float x) {
  float r = lane_of<LN, K>(x);
  asm("" : "+v"(r));  // no instruction; keeps the move from being folded into the products
  return r;
}

// v[k] of LN lanes each: lane j of the group gets sum over the group's lanes of v[j].  Every step
// halves the number of values: a lane keeps one half and hands the other to a partner that
// keeps that.
template <int LN>
__device__ __forceinline__ float reduce_scatter(const float (&v)[LN], int j) {
  if constexpr (LN == 4) {
    const bool b1 = j & 2, b0 = j & 1;
    const float p = (b1 ? v[2] : v[0]) + dpp<kDppXor2>(b1 ? v[0] : v[2]);
    const float q = (b1 ? v[3] : v[1]) + dpp<kDppXor2>(b1 ? v[1] : v[3]);
    return (b0 ? q : p) + dpp<kDppXor1>(b0 ? p : q);
  } else {
    static_assert(LN == 16, "4 or 16 lanes");
    const bool b3 = j & 8, b2 = j & 4, b1 = j & 2, b0 = j & 1;
    float p[8], q[4], r[2];
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = (b3 ? v[i + 8] : v[i]) + dpp<kDppMirror>(b3 ? v[i] : v[i + 8]);
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = (b2 ? p[i + 4] : p[i]) + dpp<kDppHalfMirror>(b2 ? p[i] : p[i + 4]);
#pragma unroll
    for (int i = 0; i < 2; ++i) r[i] = (b1 ? q[i + 2] : q[i]) + dpp<kDppXor2>(b1 ? q[i] : q[i + 2]);
    return (b0 ? r[1] : r[0]) + dpp<kDppXor1>(b0 ? r[0] : r[1]);
  }
}

// The value of the row of 16 lanes beside this one (0 <-> 1, 2 <-> 3), and of the other half wave:
// swapping a register with its own copy leaves the two halves side by side.
__device__ __forceinline__ float add_rows16(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float add_halves(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Sum over the wave, in every lane.
__device__ __forceinline__ float wave_sum(float x) {
  x += dpp<kDppXor1>(x);
  x += dpp<kDppXor2>(x);
  x += dpp<kDppHalfMirror>(x);
  x += dpp<kDppMirror>(x);
  return add_halves(add_rows16(x));
}

// out(c, sum over r < rows of part[r][c]) for every column c < cols: 64 columns a workgroup, 16
// waves that each take every 16th row, joined in a fixed order.  Added in 64 bits: a long call has
// many thousands of rows, and a running fp32 sum of n terms of one sign loses up to n / 2 units of
// 2^-24.
template <typename Out>
__global__ __launch_bounds__(1024) void column_sum_kernel(const float* __restrict__ part, int rows, int64_t cols,
                                                          int64_t first, Out out) {
  __shared__ double acc[16][64];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int64_t c = first + (int64_t)blockIdx.x * 64 + lane;
  double s = 0.0;
  if (c < cols) {
#pragma unroll 4
    for (int r = wv; r < rows; r += 16) s += part[(int64_t)r * cols + c];
  }
  acc[wv][lane] = s;
  __syncthreads();
  if (wv == 0 && c < cols) {
    double t = acc[0][lane];
#pragma unroll
    for (int i = 1; i < 16; ++i) t += acc[i][lane];
    out(c, (float)t);
  }
}
template <typename Out>
hipError_t column_sum(const float* part, int rows, int64_t cols, Out out, hipStream_t st) {
  // (a launch takes fewer than 2^32 threads, 16 a column)
  constexpr int64_t most = int64_t{1} << 27;
  for (int64_t first = 0; first < cols; first += most) {
    const int64_t n = cols - first < most ? cols - first : most;
    column_sum_kernel<<<dim3((unsigned)((n + 63) / 64)), 1024, 0, st>>>(part, rows, cols, first, out);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// Whether a row before row b uses the same slot: the first row of a slot is the one that counts.
// Called by all threads of the workgroup.
__device__ __forceinline__ bool slot_taken(const int* slots, int b, int slot) {
  int hit = 0;
  for (int i = threadIdx.x; i < b; i += blockDim.x) hit |= slots[i] == slot;
  return __syncthreads_or(hit);
}

// Workgroups are dealt to the eight XCDs in turn; this numbering gives each XCD (and its L2) a
// contiguous stretch of them, for any number of workgroups.
__device__ __forceinline__ int xcd_contiguous(int bid, int n) {
  const int x = bid & 7, q = n >> 3, r = n & 7;
  return x * q + min(x, r) + (bid >> 3);
}

// Offsets of a packed batch are the caller's; a value outside the rows is read as the nearest
// one inside, so that no offset leads out of a tensor.
__device__ __forceinline__ int seq_begin(const Seqs& s, int i) {
  return s.cu ? min(max(s.cu[i], 0), s.rows) : i * s.T;
}

// The sequence that holds row t (the last one that starts at or before it).
__device__ __forceinline__ int seq_of_row(const Seqs& s, int t) {
  if (!s.cu) return t / s.T;
  int lo = 0, hi = s.n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (s.cu[mid] <= t) lo = mid; else hi = mid;
  }
  return lo;
}

// Piece `id` of the sequences cut into pieces of `len` tokens each: its sequence, its number in
// it, and the number of pieces before the sequence.  One wave looks at 64 sequences at a time.
struct Piece {
  int seq, k, before, begin, end;  // begin, end: the sequence's rows
};
// A sequence as its one piece (seq < 0: it has no tokens).
__device__ __forceinline__ Piece whole_sequence(const Seqs& s, int i) {
  Piece r;
  r.k = 0;
  r.before = i;
  r.begin = seq_begin(s, i);
  r.end = seq_begin(s, i + 1);
  r.seq = r.end > r.begin ? i : -1;
  return r;
}
__device__ __forceinline__ Piece find_piece(const Seqs& s, int id, int len, int lane) {
  Piece r;
  if (!s.cu) {
    const int per = (s.T + len - 1) / len;
    r.seq = id / per;
    r.k = id - r.seq * per;
    r.before = r.seq * per;
    r.begin = r.seq * s.T;
    r.end = r.begin + s.T;
    return r;
  }
  int before = 0;
  for (int base = 0; base < s.n; base += 64) {
    const int i = base + lane;
    const int b = i < s.n ? seq_begin(s, i) : 0, e = i < s.n ? seq_begin(s, i + 1) : 0;
    const int c = e > b ? (e - b + len - 1) / len : 0;
    int inc = c;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int o = __shfl_up(inc, off, 64);
      if (lane >= off) inc += o;
    }
    const unsigned long long m = __ballot(id < before + inc && id >= before + inc - c);
    if (m) {
      const int l = __builtin_ctzll(m);
      r.seq = base + l;
      r.before = before + __shfl(inc - c, l, 64);
      r.k = id - r.before;
      r.begin = __shfl(b, l, 64);
      r.end = __shfl(e, l, 64);
      return r;
    }
    before += __shfl(inc, 63, 64);
  }
  r.seq = -1;
  r.k = r.before = r.begin = r.end = 0;
  return r;
}

}  // namespace gdn
