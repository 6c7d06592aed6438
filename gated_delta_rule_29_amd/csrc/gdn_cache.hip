// gdn_cache.hip -- the paged cache of keys and values: written, in the inputs' type or in 8 bits (e4m3) with
// a scale for each token and head, and read back.
//
//   8 bits: scale = max(max |x|, 1e-12) / 448 over a head's D columns, q = e4m3(x / scale)
//
// A row (one token and head) is held by 8 to 64 lanes, 8 columns each, so that the scale's maximum is a
// lane exchange and every input is read once.  Reading is bound by memory (16384 tokens of 8 heads of 128 columns out
// of pages of 16: 17.5 us, 5.8 TB/s of what it reads and writes, part of it out of the last caches).  Writing 8 bits
// is bound by its instructions, some 1240 a wave of 16 rows (vector units busy 64%): addresses in 64 bits, the
// maximum, conversions, and the look through earlier slots (8192 tokens of 8 heads of 128 columns: 21 us, 2.5 TB/s).  16 columns a lane, and
// neighbouring tokens on one die, were no faster.  In the inputs' type they are written in 15.4 us (67 MB, 4.4 TB/s).
// Single tokens (64 of them: 4.4 us) are one chain of loads.
#include "../../include/gdn.h"
#include "gdn_attn.h"
#include "gdn_layer_device.h"
#include "gdn_q8.h"

namespace gdn {

namespace {

constexpr int kThreads = 256;

// Columns c .. c + 7 of a row of D, 0 beyond it: as they are in memory while they are on their way (a
// conversion would wait for them), and as fp32.  VEC: in 16-byte accesses.
template <typename T, bool VEC>
struct Row8 {
  u32x4v v[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p, int c, int D) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i)
      if (c + i * 16 / (int)sizeof(T) < D) v[i] = reinterpret_cast<const u32x4v*>(p + c)[i];
  }
  __device__ __forceinline__ void values(float (&x)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (sizeof(T) == 4) x[i] = __uint_as_float(v[i / 4][i % 4]);
      else x[i] = __uint_as_float(i & 1 ? v[i / 8][i % 8 / 2] & 0xffff0000u : v[i / 8][i % 8 / 2] << 16);
    }
  }
};
template <typename T>
struct Row8<T, false> {
  T v[8];
  __device__ __forceinline__ void load(const T* p, int c, int D) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < D) v[i] = p[c + i];
  }
  __device__ __forceinline__ void values(float (&x)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = to_f(v[i]);
  }
};
template <typename T, bool VEC>
__device__ __forceinline__ void store_row8(T* p, int c, int D, const float (&x)[8]) {
  if constexpr (VEC) {
    constexpr int W = 16 / sizeof(T);
#pragma unroll
    for (int i = 0; i < 8; i += W)
      if (c + i < D) {
        float w[W];
#pragma unroll
        for (int j = 0; j < W; ++j) w[j] = x[i + j];
        storev<T, W>(p + c + i, w);
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
constexpr int kLook = 8;  // earlier slots that a thread asks for together
struct Slots {
  int mine, s[kLook];
};
__device__ __forceinline__ Slots ask_slots(const int* slots, int t0, int n) {
  Slots r;
  r.mine = (int)threadIdx.x < n ? slots[t0 + threadIdx.x] : -1;
#pragma unroll
  for (int e = 0; e < kLook; ++e) {
    const int i = (int)threadIdx.x + e * kThreads;
    r.s[e] = i < t0 + n ? slots[i] : -1;
  }
  return r;
}
__device__ __forceinline__ void find_live(const int* slots, Slots r, int t0, int n, int limit, int* own, int* dead,
                                          unsigned* map) {
  for (int i = threadIdx.x; i < kMapWords; i += kThreads) map[i] = 0;
  int(&s)[kLook] = r.s;
  const int mine = r.mine;
  __syncthreads();
  if ((int)threadIdx.x < n) {
    own[threadIdx.x] = mine;
    dead[threadIdx.x] = mine < 0 || mine >= limit;
    atomicOr(&map[(mine >> 5) & (kMapWords - 1)], 1u << (mine & 31));
  }
  __syncthreads();
  for (int b = threadIdx.x;; b += kLook * kThreads) {
    unsigned hits = 0;  // (a slot of -1, behind the end, may hit too)
#pragma unroll
    for (int e = 0; e < kLook; ++e) hits |= (map[(s[e] >> 5) & (kMapWords - 1)] >> (s[e] & 31) & 1) << e;
    for (; hits; hits &= hits - 1) {
      const int i = b + __builtin_ctz(hits) * kThreads;
      if (i >= t0 + n) break;
      const int slot = slots[i];
      for (int j = max(i + 1 - t0, 0); j < n; ++j)
        if (own[j] == slot) dead[j] = 1;
    }
    if (b + kLook * kThreads >= t0 + n) break;
#pragma unroll
    for (int e = 0; e < kLook; ++e) {
      const int i = b + (kLook + e) * kThreads;
      s[e] = i < t0 + n ? slots[i] : -1;
    }
  }
  __syncthreads();
}

// The rows of a workgroup, (token, k or v, head): its lanes take kThreads / LPR at a time, and ask for
// kBatch of them before they use the first.
constexpr int kBatch = 4;
struct Row {
  int t, h;
  bool val, there;
};
struct RowGrid {
  int tokens, heads;     // of a workgroup
  Divisor groups, pair;  // workgroups for the heads of a token; 2 * heads
  int pshift;            // a page has 2^pshift places
};
__device__ __forceinline__ int quotient(int n, const Divisor& d) { return (int)(((uint64_t)(uint32_t)n * d.mul) >> d.shift); }
__device__ __forceinline__ Row row_of(const CacheRowsParams& p, const RowGrid& g, int r, int rows, int h0) {
  Row w;
  w.t = quotient(r, g.pair);
  const int hv = r - w.t * (int)g.pair.by;
  w.val = hv >= g.heads;
  w.h = h0 + (w.val ? hv - g.heads : hv);
  w.there = r < rows && w.h < p.c.H;
  return w;
}
__device__ __forceinline__ int64_t cache_row(const Cache& c, int pshift, int slot, int h) {
  const int page = slot >> pshift;
  return ((int64_t)page * c.H + h) * c.P + (slot - (page << pshift));
}

template <typename T, bool Q8, bool VEC, int LPR>
__global__ __launch_bounds__(kThreads) void cache_write_kernel(CacheRowsParams p, RowGrid g) {
  __shared__ int own[kMaxTokens], dead[kMaxTokens];
  __shared__ unsigned map[kMapWords];
  const int tile = quotient(blockIdx.x, g.groups), t0 = tile * g.tokens;
  const int h0 = (blockIdx.x - tile * (int)g.groups.by) * g.heads, nt = min(g.tokens, p.T - t0);
  const int c = (threadIdx.x % LPR) * 8;
  const int rows = nt * g.heads * 2;
  constexpr int STEP = kThreads / LPR;
  Row8<T, VEC> in[kBatch];
  Row w[kBatch];
  auto ask = [&](int r0) {
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      w[b] = row_of(p, g, r0 + b * STEP, rows, h0);
      const Heads& from = w[b].val ? p.v : p.k;
      in[b] = {};
      if (w[b].there)
        in[b].load(static_cast<const T*>(from.p) + (t0 + w[b].t) * from.pitch + w[b].h * from.head, c, p.c.D);
    }
  };
  int r0 = threadIdx.x / LPR;
  const Slots slots = ask_slots(p.slots, t0, nt);
  ask(r0);  // (under way while the slots are looked through)
  find_live(p.slots, slots, t0, nt, p.c.pages * p.c.P, own, dead, map);
  while (r0 < rows) {
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      if (!w[b].there || dead[w[b].t]) continue;
      const int64_t at = cache_row(p.c, g.pshift, own[w[b].t], w[b].h);
      void* to = w[b].val ? p.c.v : p.c.k;
      float x[8];
      in[b].values(x);
      if constexpr (Q8) {
        unsigned m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[i]) & 0x7fffffffu);  // a NaN is above all
        const float scale = q8_scale(lanes_max<LPR>(m));
        uint8_t* q = static_cast<uint8_t*>(to) + at * p.c.D;
        const u32x2v v = q8_pack(x, scale);
        if constexpr (VEC) {
          if (c < p.c.D) *reinterpret_cast<u32x2v*>(q + c) = v;
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (c + i < p.c.D) q[c + i] = (uint8_t)(v[i / 4] >> (8 * (i % 4)));
        }
        if (c == 0) (w[b].val ? p.c.vs : p.c.ks)[at] = scale;
      } else {
        store_row8<T, VEC>(static_cast<T*>(to) + at * p.c.D, c, p.c.D, x);
      }
    }
    r0 += kBatch * STEP;
    if (r0 < rows) ask(r0);
  }
}

template <typename T, bool Q8, bool VEC, int LPR>
__global__ __launch_bounds__(kThreads) void cache_read_kernel(CacheRowsParams p, RowGrid g) {
  const int tile = quotient(blockIdx.x, g.groups), t0 = tile * g.tokens;
  const int h0 = (blockIdx.x - tile * (int)g.groups.by) * g.heads, nt = min(g.tokens, p.T - t0);
  const int c = (threadIdx.x % LPR) * 8;
  const int rows = nt * g.heads * 2;
  constexpr int STEP = kThreads / LPR;
  for (int r0 = threadIdx.x / LPR; r0 < rows; r0 += kBatch * STEP) {
    float scale[kBatch];
    u32x2v q[kBatch];
    Row8<T, VEC> in[kBatch];
    Row w[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      w[b] = row_of(p, g, r0 + b * STEP, rows, h0);
      const void* from = w[b].val ? p.c.v : p.c.k;
      q[b] = u32x2v{0u, 0u};
      scale[b] = 0.f;
      in[b] = {};
      const int slot = w[b].there ? p.slots[t0 + w[b].t] : -1;
      if (slot < 0 || slot >= p.c.pages * p.c.P) continue;
      const int64_t at = cache_row(p.c, g.pshift, slot, w[b].h);
      if constexpr (Q8) {
        const uint8_t* row = static_cast<const uint8_t*>(from) + at * p.c.D;
        scale[b] = (w[b].val ? p.c.vs : p.c.ks)[at];
        if constexpr (VEC) {
          if (c < p.c.D) q[b] = *reinterpret_cast<const u32x2v*>(row + c);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (c + i < p.c.D) q[b][i / 4] |= (unsigned)row[c + i] << (8 * (i % 4));
        }
      } else {
        in[b].load(static_cast<const T*>(from) + at * p.c.D, c, p.c.D);
      }
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      if (!w[b].there) continue;
      float x[8];
      if constexpr (Q8) {
        q8_unpack(q[b], x);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= scale[b];
      } else {
        in[b].values(x);
      }
      T* to = static_cast<T*>(w[b].val ? p.vo : p.ko) + ((int64_t)(t0 + w[b].t) * p.c.H + w[b].h) * p.c.D;
      store_row8<T, VEC>(to, c, p.c.D, x);
    }
  }
}

template <typename T, bool Q8, bool VEC, bool WRITE, int LPR>
hipError_t launch(const CacheRowsParams& p, hipStream_t st) {
  // Tokens of a workgroup: as many rows as its lanes ask for together, where that still fills the chip.  Writing looks
  // through all earlier slots in every workgroup: more tokens in very long calls.
  const int per = kThreads / LPR;  // rows at a time
  int tokens = 1;
  while (tokens < 16 && tokens * 4 * p.c.H <= kBatch * per && p.T / (2 * tokens) >= 512) tokens *= 2;
  if (WRITE && p.T > 16384) tokens = p.T > 65536 ? kMaxTokens : 16;
  int heads = p.c.H;
  const int64_t tiles = (p.T + tokens - 1) / tokens;
  // one token's heads in several workgroups where there are few tokens
  while (heads > 1 && tiles * ((p.c.H + heads - 1) / heads) < 256 && tokens * 2 * heads > per) heads = (heads + 1) / 2;
  const int groups = (p.c.H + heads - 1) / heads;
  if (tiles * groups > kMaxGroups) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)(tiles * groups));
  const RowGrid g{tokens, heads, divisor((uint32_t)groups), divisor(2u * heads), __builtin_ctz((unsigned)p.c.P)};
  if constexpr (WRITE) cache_write_kernel<T, Q8, VEC, LPR><<<grid, kThreads, 0, st>>>(p, g);
  else cache_read_kernel<T, Q8, VEC, LPR><<<grid, kThreads, 0, st>>>(p, g);
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
