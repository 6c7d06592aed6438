// gdn_norm.hip -- root-mean-square norm with the residual's addition, with an output in the inputs'
// type or in 8 bits (e4m3) with scales, and its gradient.
//
//   s = x + residual, stored in the residual's type;  r = 1 / sqrt(mean_c s_c^2 + eps) of the stored s
//   y_c = s_c r w_c
//   8 bits: scale = max(max |y|, 1e-12) / 448 over a row or over 128 columns, q = e4m3(y / scale)
//   ds = r (dy w - s r^2 mean(dy w s)) + dsum,   dw_c = sum over rows of dy_c s_c r
//
// One row's values stay in the registers of TPR threads: every input is read once, and the kernels run at
// the rate of a large copy (5.2 TB/s) or above it: 16384 rows of 4096 bf16 with a bf16 residual 90 us (537 MB:
// 6.0 TB/s, part of which the 256 MB cache takes) and their gradient 112 us (537 MB and 17 MB of
// weight-gradient shares: 4.9 TB/s); 8192 rows of 4096 with an fp32 residual to 8 bits in 128-column blocks
// 72 us (370 MB: 5.2 TB/s).  A single row takes 2.6 us.
#include "../../include/gdn.h"
#include "gdn_layer_device.h"

namespace gdn {

namespace {

constexpr int kBlock = 128;        // columns of a scale block
constexpr float kE4m3Max = 448.f;  // largest e4m3 value

// V consecutive values (8, in 16-byte accesses, or 1).
template <typename T, int V>
__device__ __forceinline__ void load_vec(const T* p, float (&x)[V]) {
  if constexpr (V == 8 && sizeof(T) == 4) {
    float a[4], b[4];
    loadv<T, 4>(p, a);
    loadv<T, 4>(p + 4, b);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = a[i];
      x[4 + i] = b[i];
    }
  } else {
    loadv<T, V>(p, x);
  }
}
template <typename T, int V>
__device__ __forceinline__ void store_vec(T* p, const float (&x)[V]) {
  if constexpr (V == 8 && sizeof(T) == 4) {
    const float a[4] = {x[0], x[1], x[2], x[3]}, b[4] = {x[4], x[5], x[6], x[7]};
    storev<T, 4>(p, a);
    storev<T, 4>(p + 4, b);
  } else {
    storev<T, V>(p, x);
  }
}

// Sum over the TPR threads of a row, in each of them; red: TPR / 64 floats of the row's own.
template <int TPR>
__device__ __forceinline__ float row_sum(float x, float* red) {
  x = wave_sum(x);
  if constexpr (TPR > 64) {
    const int wv = (threadIdx.x % TPR) >> 6;
    __syncthreads();  // red's last readers are done
    if ((threadIdx.x & 63) == 0) red[wv] = x;
    __syncthreads();
    x = red[0];
#pragma unroll
    for (int i = 1; i < TPR / 64; ++i) x += red[i];
  }
  return x;
}

// Largest of unsigned values (the bits of non-negative floats, where a NaN is above all) over
// 16 lanes, a wave, or a row's threads.
__device__ __forceinline__ unsigned max16(unsigned x) {
  x = max(x, __float_as_uint(dpp<kDppXor1>(__uint_as_float(x))));
  x = max(x, __float_as_uint(dpp<kDppXor2>(__uint_as_float(x))));
  x = max(x, __float_as_uint(dpp<kDppHalfMirror>(__uint_as_float(x))));
  return max(x, __float_as_uint(dpp<kDppMirror>(__uint_as_float(x))));
}
__device__ __forceinline__ unsigned wave_max(unsigned x) {
  x = max16(x);
  const auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
  x = max(r[0], r[1]);
  const auto q = __builtin_amdgcn_permlane32_swap(x, x, false, false);
  return max(q[0], q[1]);
}
template <int TPR>
__device__ __forceinline__ unsigned row_max(unsigned x, float* red) {
  x = wave_max(x);
  if constexpr (TPR > 64) {
    const int wv = (threadIdx.x % TPR) >> 6;
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[wv] = __uint_as_float(x);
    __syncthreads();
    x = __float_as_uint(red[0]);
#pragma unroll
    for (int i = 1; i < TPR / 64; ++i) x = max(x, __float_as_uint(red[i]));
  }
  return x;
}

__device__ __forceinline__ float scale_of(unsigned amax) {
  // a NaN stays one: fmaxf would drop it
  const float a = __uint_as_float(amax);
  return (a == a ? fmaxf(a, 1e-12f) : a) / kE4m3Max;
}

// e4m3 bytes of y / scale (to nearest even).  The quotient is at most 448 but for its last bit.  It is
// divided for: a product with the scale's reciprocal may be a unit or two away from it, on the other side
// of a value half way between two e4m3 values.
template <int V>
__device__ __forceinline__ void store_q8(uint8_t* q, const float (&y)[V], float scale) {
  float v[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    v[i] = y[i] / scale;
    v[i] = v[i] > kE4m3Max ? kE4m3Max : (v[i] < -kE4m3Max ? -kE4m3Max : v[i]);  // NaN passes
  }
  if constexpr (V == 8) {
    u32x2v r;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h], v[4 * h + 1], 0, false);
      r[h] = (unsigned)__builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h + 2], v[4 * h + 3], w, true);
    }
    *reinterpret_cast<u32x2v*>(q) = r;
  } else {
    *q = (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[0], 0, false);
  }
}

// Q8: 0 the inputs' type, 1 e4m3 with one scale a row, 2 with one for 128 columns.
template <typename T, typename RT, int V, int TPR, int NV, int Q8>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void norm_fwd_kernel(NormParams p) {
  constexpr int RPW = TPR < 256 ? 256 / TPR : 1;
  __shared__ float red[RPW * (TPR / 64)];
  __shared__ unsigned half[Q8 == 2 && V == 1 && TPR > 64 ? kNormMaxD / 64 + 1 : 1];  // maxima of 64 columns
  const int sub = threadIdx.x / TPR, tid = threadIdx.x % TPR;
  const int row = blockIdx.x * RPW + sub;
  if (TPR == 64 && row >= p.M) return;  // (one row a workgroup otherwise)
  float* rd = red + sub * (TPR / 64);
  const T* x = static_cast<const T*>(p.x) + row * p.x_pitch;
  const RT* res = p.residual ? static_cast<const RT*>(p.residual) + row * p.r_pitch : nullptr;
  float v[NV][V];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * TPR + tid) * V;
    if (c < p.D) {
      load_vec<T, V>(x + c, v[i]);
      if (res) {
        float r[V];
        load_vec<RT, V>(res + c, r);
#pragma unroll
        for (int k = 0; k < V; ++k) v[i][k] = to_f(to_t<RT>(v[i][k] + r[k]));  // the stored sum is the one that is normalised
        if (p.sum) store_vec<RT, V>(static_cast<RT*>(p.sum) + (int64_t)row * p.D + c, v[i]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < V; ++k) v[i][k] = 0.f;
    }
#pragma unroll
    for (int k = 0; k < V; ++k) ss = __builtin_fmaf(v[i][k], v[i][k], ss);
  }
  ss = row_sum<TPR>(ss, rd);
  const float r = 1.f / sqrtf(ss / (float)p.D + p.eps);
  if (p.rstd && tid == 0) p.rstd[row] = r;
  unsigned amax = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * TPR + tid) * V;
    if (c < p.D) {
      float w[V];
      load_vec<float, V>(p.w + c, w);
#pragma unroll
      for (int k = 0; k < V; ++k) v[i][k] = v[i][k] * r * w[k];
      if constexpr (Q8 == 0) store_vec<T, V>(static_cast<T*>(p.y) + (int64_t)row * p.D + c, v[i]);
    }
    if constexpr (Q8 == 1) {
#pragma unroll
      for (int k = 0; k < V; ++k) amax = max(amax, __float_as_uint(v[i][k]) & 0x7fffffffu);
    }
    if constexpr (Q8 == 2) {
      unsigned m = 0;
#pragma unroll
      for (int k = 0; k < V; ++k) m = max(m, __float_as_uint(v[i][k]) & 0x7fffffffu);
      if constexpr (V == 8) {
        // 16 lanes hold one block
        const float s = scale_of(max16(m));
        if (c < p.D) {
          if (tid % 16 == 0) p.scale[(int64_t)row * ((p.D + kBlock - 1) / kBlock) + c / kBlock] = s;
          store_q8<V>(static_cast<uint8_t*>(p.y) + (int64_t)row * p.D + c, v[i], s);
        }
      } else if constexpr (TPR > 64) {
        m = wave_max(m);  // a wave holds half a block
        if ((tid & 63) == 0 && c < p.D) half[c / 64] = m;
      }
    }
  }
  if constexpr (Q8 == 1) {
    const float s = scale_of(row_max<TPR>(amax, rd));
    if (tid == 0) p.scale[row] = s;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + tid) * V;
      if (c < p.D) store_q8<V>(static_cast<uint8_t*>(p.y) + (int64_t)row * p.D + c, v[i], s);
    }
  }
  if constexpr (Q8 == 2 && V == 1 && TPR == 64) {
    // two vectors of the row's one wave hold a block
    const int nb = (p.D + kBlock - 1) / kBlock;
#pragma unroll
    for (int b = 0; b < NV / 2; ++b) {
      const unsigned m = wave_max(max(__float_as_uint(v[2 * b][0]) & 0x7fffffffu, __float_as_uint(v[2 * b + 1][0]) & 0x7fffffffu));
      const float s = scale_of(m);
      if (tid == 0 && b < nb) p.scale[(int64_t)row * nb + b] = s;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int c = (2 * b + h) * TPR + tid;
        if (c < p.D) store_q8<V>(static_cast<uint8_t*>(p.y) + (int64_t)row * p.D + c, v[2 * b + h], s);
      }
    }
  }
  if constexpr (Q8 == 2 && V == 1 && TPR > 64) {
    const int nb = (p.D + kBlock - 1) / kBlock, last = (p.D - 1) / 64;
    __syncthreads();
    auto scale = [&](int b) { return scale_of(max(half[2 * b], half[min(2 * b + 1, last)])); };
    for (int i = tid; i < nb; i += TPR) p.scale[(int64_t)row * nb + i] = scale(i);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = i * TPR + tid;
      if (c < p.D) store_q8<V>(static_cast<uint8_t*>(p.y) + (int64_t)row * p.D + c, v[i], scale(c / kBlock));
    }
  }
}

// The rows of a gradient call are dealt to `groups` row workers (a workgroup, or one of its waves
// where rows are short); each keeps its share of dw in registers.  A worker of a long call has thousands of
// rows, and a running fp32 sum of n terms of one sign loses up to n / 2 units of 2^-24: every kFold
// rows the registers are added to the share in the workspace.
constexpr int kFold = 64;
template <typename T, typename RT, int V, int TPR, int NV>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void norm_bwd_kernel(NormBwdParams p, int groups) {
  constexpr int RPW = TPR < 256 ? 256 / TPR : 1;
  __shared__ float red[RPW * (TPR / 64)];
  const int sub = threadIdx.x / TPR, tid = threadIdx.x % TPR;
  const int worker = blockIdx.x * RPW + sub;
  if (TPR == 64 && worker >= groups) return;
  float* rd = red + sub * (TPR / 64);
  float dw[NV][V] = {};
  const float inv_d = 1.f / (float)p.D;
  // dw to the workspace: as its first rows' sums, or added to those that are there
  auto fold = [&](bool first) {
    int at = tid;
    asm volatile("" : "+v"(at));  // no instruction; keeps the addresses from holding registers between
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + at) * V;
      if (c < p.D) {
        float* q = p.part + (int64_t)worker * p.D + c;
        if (!first) {
          float old[V];
          load_vec<float, V>(q, old);
#pragma unroll
          for (int k = 0; k < V; ++k) dw[i][k] += old[k];
        }
        store_vec<float, V>(q, dw[i]);
#pragma unroll
        for (int k = 0; k < V; ++k) dw[i][k] = 0.f;
      }
    }
  };
  for (int first = worker; first < p.M; first += kFold * groups) {
    const int end = min(p.M, first + kFold * groups);
    for (int row = first; row < end; row += groups) {
      const T* dy = static_cast<const T*>(p.dy) + row * p.dy_pitch;
      const RT* s = static_cast<const RT*>(p.s) + row * p.s_pitch;
      const float r = p.rstd[row];
      float g[NV][V], v[NV][V], dot = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + tid) * V;
        if (c < p.D) {
          float w[V];
          load_vec<T, V>(dy + c, g[i]);
          load_vec<RT, V>(s + c, v[i]);
          load_vec<float, V>(p.w + c, w);
#pragma unroll
          for (int k = 0; k < V; ++k) {
            v[i][k] *= r;
            dw[i][k] = __builtin_fmaf(g[i][k], v[i][k], dw[i][k]);
            g[i][k] *= w[k];
            dot = __builtin_fmaf(g[i][k], v[i][k], dot);
          }
        }
      }
      dot = row_sum<TPR>(dot, rd) * inv_d;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + tid) * V;
        if (c < p.D) {
          float o[V];
#pragma unroll
          for (int k = 0; k < V; ++k) o[k] = r * (g[i][k] - v[i][k] * dot);
          if (p.dsum) {
            float d[V];
            load_vec<RT, V>(static_cast<const RT*>(p.dsum) + row * p.dsum_pitch + c, d);
#pragma unroll
            for (int k = 0; k < V; ++k) o[k] += d[k];
          }
          store_vec<RT, V>(static_cast<RT*>(p.dres) + (int64_t)row * p.D + c, o);
          if (p.dx) store_vec<T, V>(static_cast<T*>(p.dx) + (int64_t)row * p.D + c, o);
        }
      }
    }
    fold(first == worker);
  }
}

struct NormWeightOut {
  float* dw;
  __device__ void operator()(int64_t c, float s) const { dw[c] = s; }
};

bool al16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// Threads of a row and vectors of a thread: 64 threads for short rows, 256 for up to 8192 columns
// in 16-byte vectors, 1024 beyond that and for single columns.  (The gradient's registers do not hold its
// widest instances: beyond 16384 columns 7 to 12 are spilled, of more than 4096 single columns 54 to 56:
// 4096 rows of 4097 bf16 take 104 us, 1 TB/s.)
template <typename F>
hipError_t by_width(int D, bool vec, F&& f) {
  using std::integral_constant;
  if (vec) {
    using V = integral_constant<int, 8>;
    if (D <= 512) return f(V{}, integral_constant<int, 64>{}, integral_constant<int, 1>{});
    if (D <= 2048) return f(V{}, integral_constant<int, 256>{}, integral_constant<int, 1>{});
    if (D <= 4096) return f(V{}, integral_constant<int, 256>{}, integral_constant<int, 2>{});
    if (D <= 8192) return f(V{}, integral_constant<int, 256>{}, integral_constant<int, 4>{});
    if (D <= 16384) return f(V{}, integral_constant<int, 1024>{}, integral_constant<int, 2>{});
    return f(V{}, integral_constant<int, 1024>{}, integral_constant<int, 4>{});
  }
  using V = integral_constant<int, 1>;
  if (D <= 512) return f(V{}, integral_constant<int, 64>{}, integral_constant<int, 8>{});
  if (D <= 4096) return f(V{}, integral_constant<int, 1024>{}, integral_constant<int, 4>{});
  return f(V{}, integral_constant<int, 1024>{}, integral_constant<int, 32>{});
}

template <typename F>
hipError_t by_type(int dtype, int rdtype, F&& f) {
  if (dtype == GDN_DTYPE_F32) return f(float{}, float{});
  return rdtype == GDN_DTYPE_BF16 ? f(bf16{}, bf16{}) : f(bf16{}, float{});
}

// The call for M of the rows, from row m0 on.
template <typename T, typename RT>
NormParams rows_from(NormParams p, int m0, int M) {
  const int64_t out = (int64_t)m0 * p.D;
  p.x = static_cast<const T*>(p.x) + m0 * p.x_pitch;
  if (p.residual) p.residual = static_cast<const RT*>(p.residual) + m0 * p.r_pitch;
  if (p.sum) p.sum = static_cast<RT*>(p.sum) + out;
  if (p.rstd) p.rstd += m0;
  if (p.scale) {
    p.y = static_cast<uint8_t*>(p.y) + out;
    p.scale += m0 * (int64_t)(p.block ? (p.D + kBlock - 1) / kBlock : 1);
  } else {
    p.y = static_cast<T*>(p.y) + out;
  }
  p.M = M;
  return p;
}

// Row workers of a gradient call: four workgroups a CU at most.
int bwd_groups(int M, int D) {
  const int most = D <= 512 ? 4096 : 1024;
  return M < most ? M : most;
}

}  // namespace

size_t norm_bwd_ws_bytes(int M, int D) { return (size_t)bwd_groups(M, D) * D * 4; }

hipError_t launch_norm_fwd(const NormParams& p, int dtype, int rdtype, hipStream_t st) {
  const bool q8 = p.scale != nullptr;
  const bool vec = p.D % 8 == 0 && p.x_pitch % 8 == 0 && (!p.residual || p.r_pitch % 8 == 0) && al16(p.x) &&
                   al16(p.residual) && al16(p.sum) && al16(p.w) && (reinterpret_cast<uintptr_t>(p.y) % (q8 ? 8 : 16)) == 0;
  return by_type(dtype, rdtype, [&](auto t, auto rt) {
    return by_width(p.D, vec, [&](auto v, auto tpr, auto nv) {
      constexpr int TPR = decltype(tpr)::value, wg = TPR < 256 ? 256 : TPR, rpw = wg / TPR;
      using T = decltype(t);
      using RT = decltype(rt);
      // A launch takes fewer than 2^32 threads, which a few million rows reach: more rows, more launches.
      constexpr int most = (1 << 30) / wg * rpw;
      for (int m0 = 0; m0 < p.M; m0 += most) {
        const NormParams q = rows_from<T, RT>(p, m0, min(p.M - m0, most));
        const dim3 grid((q.M + rpw - 1) / rpw);
        if (!q8) norm_fwd_kernel<T, RT, v(), TPR, nv(), 0><<<grid, wg, 0, st>>>(q);
        else if (p.block == 0) norm_fwd_kernel<T, RT, v(), TPR, nv(), 1><<<grid, wg, 0, st>>>(q);
        else norm_fwd_kernel<T, RT, v(), TPR, nv(), 2><<<grid, wg, 0, st>>>(q);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
      }
      return hipSuccess;
    });
  });
}

hipError_t launch_norm_bwd(const NormBwdParams& p, int dtype, int sdtype, hipStream_t st) {
  const bool vec = p.D % 8 == 0 && p.dy_pitch % 8 == 0 && p.s_pitch % 8 == 0 && (!p.dsum || p.dsum_pitch % 8 == 0) &&
                   al16(p.dy) && al16(p.s) && al16(p.dsum) && al16(p.w) && al16(p.dres) && al16(p.dx);
  const int groups = bwd_groups(p.M, p.D);
  return by_type(dtype, sdtype, [&](auto t, auto rt) {
    return by_width(p.D, vec, [&](auto v, auto tpr, auto nv) {
      constexpr int TPR = decltype(tpr)::value, wg = TPR < 256 ? 256 : TPR, rpw = wg / TPR;
      norm_bwd_kernel<decltype(t), decltype(rt), v(), TPR, nv()><<<dim3((groups + rpw - 1) / rpw), wg, 0, st>>>(p, groups);
      hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
      return column_sum(p.part, groups, p.D, NormWeightOut{p.dw}, st);
    });
  });
}

}  // namespace gdn
