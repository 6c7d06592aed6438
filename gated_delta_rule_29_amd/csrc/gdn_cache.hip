// gdn_cache.hip -- the paged cache of keys and values: written, in the inputs' type or in 8 bits (e4m3) with
// a scale for each token and head, and read back.
//
//   8 bits: scale = max(max |x|, 1e-12) / 448 over a head's D columns, q = e4m3(x / scale)
//
// A row (one token and head) is held by 8 to 64 lanes, 8 columns each, so that the scale's maximum is a
// lane exchange and every input is read once.  Bound by memory.
#include "../../include/gdn.h"
#include "gdn_attn.h"
#include "gdn_layer_device.h"
#include "gdn_q8.h"

namespace gdn {

namespace {

constexpr int kThreads = 256;

// 8 columns c .. c + 7 of a row of D as fp32, 0 beyond it.
template <typename T, bool VEC>
__device__ __forceinline__ void load_row8(const T* p, int c, int D, float (&x)[8]) {
  if constexpr (VEC) {
    if (c < D) {
      load8f(p + c, x);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = 0.f;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = c + i < D ? to_f(p[c + i]) : 0.f;
  }
}
template <typename T, bool VEC>
__device__ __forceinline__ void store_row8(T* p, int c, int D, const float (&x)[8]) {
  if constexpr (VEC) {
    if (c < D) {
      if constexpr (sizeof(T) == 4) {
        const float a[4] = {x[0], x[1], x[2], x[3]}, b[4] = {x[4], x[5], x[6], x[7]};
        storev<T, 4>(p + c, a);
        storev<T, 4>(p + c + 4, b);
      } else {
        storev<T, 8>(p + c, x);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < D) p[c + i] = to_t<T>(x[i]);
  }
}

// Largest of unsigned values over LPR lanes (8, 16, 32 or 64).
template <int LPR>
__device__ __forceinline__ unsigned lanes_max(unsigned x) {
  x = max(x, __float_as_uint(dpp<kDppXor1>(__uint_as_float(x))));
  x = max(x, __float_as_uint(dpp<kDppXor2>(__uint_as_float(x))));
  x = max(x, __float_as_uint(dpp<kDppHalfMirror>(__uint_as_float(x))));
  if constexpr (LPR >= 16) x = max(x, __float_as_uint(dpp<kDppMirror>(__uint_as_float(x))));
  if constexpr (LPR >= 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    x = max(r[0], r[1]);
  }
  if constexpr (LPR >= 64) {
    const auto r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    x = max(r[0], r[1]);
  }
  return x;
}

// Which of a workgroup's tokens [t0, t0 + n) count: the first one of a slot does, so that no place is
// written twice.  Slots of earlier tokens are looked up in a bitmap of the workgroup's own (a hash of 32768
// places: 64 entries give a stray hit in 500 slots), and compared where it says so.  The bitmap is built by
// LDS atomics, whose order does not change it.
constexpr int kMapWords = 1024;
constexpr int kMaxTokens = 64;
__device__ __forceinline__ void find_live(const int* slots, int t0, int n, int limit, int* own, int* dead,
                                          unsigned* map) {
  for (int i = threadIdx.x; i < kMapWords; i += kThreads) map[i] = 0;
  __syncthreads();
  if ((int)threadIdx.x < n) {
    const int s = slots[t0 + threadIdx.x];
    own[threadIdx.x] = s;
    dead[threadIdx.x] = s < 0 || s >= limit;
    atomicOr(&map[(s >> 5) & (kMapWords - 1)], 1u << (s & 31));
  }
  __syncthreads();
  const int end = t0 + n;
  for (int b = threadIdx.x * 4; b < end; b += kThreads * 4) {
    int s[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) s[e] = b + e < end ? slots[b + e] : -1;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (map[(s[e] >> 5) & (kMapWords - 1)] >> (s[e] & 31) & 1)
        for (int j = max(b + e + 1 - t0, 0); j < n; ++j)
          if (own[j] == s[e]) dead[j] = 1;
  }
  __syncthreads();
}

// The rows of a workgroup, (token, k or v, head): its lanes take kThreads / LPR at a time, and ask for
// kBatch of them before they use the first.
constexpr int kBatch = 4;
struct Row {
  int t, h;
  bool val, live;
  int64_t at;  // in the cache
};
__device__ __forceinline__ Row row_of(const CacheRowsParams& p, int r, int rows, int nh, int h0, const int* slot,
                                      const int* dead) {
  Row w;
  w.t = r / (2 * nh);
  const int hv = r - w.t * 2 * nh;
  w.val = hv >= nh;
  w.h = h0 + (w.val ? hv - nh : hv);
  w.live = r < rows;
  const int s = w.live ? slot[w.t] : 0;
  w.live = w.live && !(dead ? dead[w.t] : s < 0 || s >= p.c.pages * p.c.P);
  const int page = w.live ? s / p.c.P : 0, place = w.live ? s - page * p.c.P : 0;
  w.at = ((int64_t)page * p.c.H + w.h) * p.c.P + place;
  return w;
}

template <typename T, bool Q8, bool VEC, int LPR>
__global__ __launch_bounds__(kThreads) void cache_write_kernel(CacheRowsParams p, int tokens, int heads, int groups) {
  __shared__ int own[kMaxTokens], dead[kMaxTokens];
  __shared__ unsigned map[kMapWords];
  const int t0 = (blockIdx.x / groups) * tokens, h0 = (blockIdx.x % groups) * heads;
  const int nt = min(tokens, p.T - t0), nh = min(heads, p.c.H - h0);
  find_live(p.slots, t0, nt, p.c.pages * p.c.P, own, dead, map);
  const int c = (threadIdx.x % LPR) * 8;
  const int rows = nt * nh * 2;
  constexpr int STEP = kThreads / LPR;
  for (int r0 = threadIdx.x / LPR; r0 < rows; r0 += kBatch * STEP) {
    float x[kBatch][8];
    Row w[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      w[b] = row_of(p, r0 + b * STEP, rows, nh, h0, own, dead);
      const Heads& in = w[b].val ? p.v : p.k;
      if (w[b].live)
        load_row8<T, VEC>(static_cast<const T*>(in.p) + (t0 + w[b].t) * in.pitch + w[b].h * in.head, c, p.c.D, x[b]);
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      if (!w[b].live) continue;
      void* to = w[b].val ? p.c.v : p.c.k;
      if constexpr (Q8) {
        unsigned m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[b][i]) & 0x7fffffffu);  // a NaN is above all
        const float scale = q8_scale(lanes_max<LPR>(m));
        uint8_t* q = static_cast<uint8_t*>(to) + w[b].at * p.c.D;
        const u32x2v v = q8_pack(x[b], scale);
        if constexpr (VEC) {
          if (c < p.c.D) *reinterpret_cast<u32x2v*>(q + c) = v;
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (c + i < p.c.D) q[c + i] = (uint8_t)(v[i / 4] >> (8 * (i % 4)));
        }
        if (c == 0) (w[b].val ? p.c.vs : p.c.ks)[w[b].at] = scale;
      } else {
        store_row8<T, VEC>(static_cast<T*>(to) + w[b].at * p.c.D, c, p.c.D, x[b]);
      }
    }
  }
}

template <typename T, bool Q8, bool VEC, int LPR>
__global__ __launch_bounds__(kThreads) void cache_read_kernel(CacheRowsParams p, int tokens, int heads, int groups) {
  const int t0 = (blockIdx.x / groups) * tokens, h0 = (blockIdx.x % groups) * heads;
  const int nt = min(tokens, p.T - t0), nh = min(heads, p.c.H - h0);
  const int c = (threadIdx.x % LPR) * 8;
  const int rows = nt * nh * 2;
  constexpr int STEP = kThreads / LPR;
  for (int r0 = threadIdx.x / LPR; r0 < rows; r0 += kBatch * STEP) {
    float x[kBatch][8], scale[kBatch];
    u32x2v q[kBatch];
    Row w[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      w[b] = row_of(p, r0 + b * STEP, rows, nh, h0, p.slots + t0, nullptr);
      const void* from = w[b].val ? p.c.v : p.c.k;
      q[b] = u32x2v{0u, 0u};
      scale[b] = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) x[b][i] = 0.f;
      if (!w[b].live) continue;
      if constexpr (Q8) {
        const uint8_t* row = static_cast<const uint8_t*>(from) + w[b].at * p.c.D;
        scale[b] = (w[b].val ? p.c.vs : p.c.ks)[w[b].at];
        if constexpr (VEC) {
          if (c < p.c.D) q[b] = *reinterpret_cast<const u32x2v*>(row + c);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (c + i < p.c.D) q[b][i / 4] |= (unsigned)row[c + i] << (8 * (i % 4));
        }
      } else {
        load_row8<T, VEC>(static_cast<const T*>(from) + w[b].at * p.c.D, c, p.c.D, x[b]);
      }
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      if (r0 + b * STEP >= rows) continue;
      if constexpr (Q8) {
        q8_unpack(q[b], x[b]);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[b][i] *= scale[b];
      }
      T* to = static_cast<T*>(w[b].val ? p.vo : p.ko) + ((int64_t)(t0 + w[b].t) * p.c.H + w[b].h) * p.c.D;
      store_row8<T, VEC>(to, c, p.c.D, x[b]);
    }
  }
}

template <typename T, bool Q8, bool VEC, bool WRITE, int LPR>
hipError_t launch(const CacheRowsParams& p, hipStream_t st) {
  // Tokens of a workgroup: enough rows for four rounds of its lanes where that still fills the chip; for
  // writing, more in very long calls, where each workgroup looks through all earlier slots.
  const int per = kThreads / LPR;  // rows at a time
  int tokens = 1;
  while (tokens < 16 && tokens * 2 * p.c.H < 4 * per && p.T / (2 * tokens) >= 512) tokens *= 2;
  if (WRITE) {
    if (p.T > 2048 && tokens < 16) tokens = 16;
    if (p.T > 16384) tokens = kMaxTokens;
  }
  int heads = p.c.H;
  const int64_t tiles = (p.T + tokens - 1) / tokens;
  // one token's heads in several workgroups where there are few tokens
  while (heads > 1 && tiles * ((p.c.H + heads - 1) / heads) < 256 && tokens * 2 * heads > per) heads = (heads + 1) / 2;
  const int groups = (p.c.H + heads - 1) / heads;
  if (tiles * groups > kMaxGroups) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)(tiles * groups));
  if constexpr (WRITE) cache_write_kernel<T, Q8, VEC, LPR><<<grid, kThreads, 0, st>>>(p, tokens, heads, groups);
  else cache_read_kernel<T, Q8, VEC, LPR><<<grid, kThreads, 0, st>>>(p, tokens, heads, groups);
  return hipGetLastError();
}

template <typename T, bool Q8, bool VEC, bool WRITE>
hipError_t by_width(const CacheRowsParams& p, hipStream_t st) {
  if (p.c.D <= 64) return launch<T, Q8, VEC, WRITE, 8>(p, st);
  if (p.c.D <= 128) return launch<T, Q8, VEC, WRITE, 16>(p, st);
  if (p.c.D <= 256) return launch<T, Q8, VEC, WRITE, 32>(p, st);
  return launch<T, Q8, VEC, WRITE, 64>(p, st);
}

template <typename T, bool WRITE>
hipError_t by_type(const CacheRowsParams& p, bool q8, hipStream_t st) {
  constexpr int E = sizeof(T);
  const auto odd = [](const void* q, int64_t a, int64_t b, int64_t to) {
    return ((uint64_t)(uintptr_t)q | (uint64_t)a | (uint64_t)b) % to != 0;
  };
  // rows of 8 columns at a time: D a multiple of 8, every row aligned to its vectors
  const int64_t c = q8 ? 8 : 16, row = (int64_t)p.c.D * (q8 ? 1 : E);
  bool vec = p.c.D % 8 == 0 && !odd(p.c.k, row, 0, c) && !odd(p.c.v, row, 0, c);
  if (WRITE) {
    vec = vec && !odd(p.k.p, p.k.pitch * E, p.k.head * E, 16) && !odd(p.v.p, p.v.pitch * E, p.v.head * E, 16);
  } else {
    vec = vec && !odd(p.ko, (int64_t)p.c.D * E, 0, 16) && !odd(p.vo, 0, 0, 16);
  }
  if (q8) return vec ? by_width<T, true, true, WRITE>(p, st) : by_width<T, true, false, WRITE>(p, st);
  return vec ? by_width<T, false, true, WRITE>(p, st) : by_width<T, false, false, WRITE>(p, st);
}

}  // namespace

hipError_t launch_cache_write(const CacheRowsParams& p, int dtype, bool q8, hipStream_t st) {
  return dtype == GDN_DTYPE_BF16 ? by_type<bf16, true>(p, q8, st) : by_type<float, true>(p, q8, st);
}
hipError_t launch_cache_read(const CacheRowsParams& p, int dtype, bool q8, hipStream_t st) {
  return dtype == GDN_DTYPE_BF16 ? by_type<bf16, false>(p, q8, st) : by_type<float, false>(p, q8, st);
}

}  // namespace gdn
