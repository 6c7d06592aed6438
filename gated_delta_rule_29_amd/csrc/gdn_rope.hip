// gdn_rope.hip -- rotary positions and their gradient.
//
//   Pair i of a head's first R columns, (u, w), is turned by a_i = 2 pi pos f_i and scaled by m:
//   (m (u cos a - w sin a), m (u sin a + w cos a)); the other columns pass.  The gradient turns backwards.
//
// Angles.  f_i is a 64-bit fraction of a turn, so pos * f_i mod 2^64 is the angle's fraction of a turn for
// any 32-bit position, exact up to f_i's own 2^-65: whole turns drop out of the integer product, where a
// product of fp32 numbers would be off by pos * 2^-25 radians.  Its upper 32 bits are taken to the nearest
// quarter turn and a remainder of an eighth of a turn at most.
//
// A workgroup takes a few tokens: it forms their cosines and sines once, in LDS, and streams the heads
// through them in 16-byte vectors.  Bound by memory: 8192 tokens of 40 heads of 128 columns, bf16, 64 columns
// turned: 27 us, 6.2 TB/s of what it reads and writes (partly in the last caches; 35 us call after call);
// 16384 tokens of 18 heads of 256: 62 us, 4.9 TB/s, the rate of a large copy.  A token of 40 heads: 2.4 us, a chain
// of three loads.
#include "../../include/gdn.h"
#include "gdn_attn.h"
#include "gdn_layer_device.h"

namespace gdn {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxAngles = 4096;  // of a workgroup: cosines and sines in 32 KB of LDS

// Cosine and sine of `turn` * 2^-32 turns.  The remainder's angle is at most pi / 4, where the Taylor
// polynomials below end at 2e-9 (sine: the term in x^11) and 1e-10 (cosine: x^12), under 2^-24 / 16.
__device__ __forceinline__ void cos_sin(uint32_t turn, float* c, float* s) {
  const uint32_t q = (turn + (1u << 29)) >> 30;
  const float x = (float)(int32_t)(turn - (q << 30)) * 0x1.921fb6p-30f;  // 2 pi / 2^32
  const float t = x * x;
  float a = 2.7557319e-6f, b = -2.7557319e-7f;
  a = __builtin_fmaf(a, t, -1.9841270e-4f);
  a = __builtin_fmaf(a, t, 8.3333333e-3f);
  a = __builtin_fmaf(a, t, -1.6666667e-1f);
  const float sn = __builtin_fmaf(a * t, x, x);
  b = __builtin_fmaf(b, t, 2.4801587e-5f);
  b = __builtin_fmaf(b, t, -1.3888889e-3f);
  b = __builtin_fmaf(b, t, 4.1666667e-2f);
  b = __builtin_fmaf(b, t, -0.5f);
  const float cs = __builtin_fmaf(b, t, 1.f);
  const float cc = q & 1 ? sn : cs, ss = q & 1 ? cs : sn;  // up to signs
  *c = (q + 1) & 2 ? -cc : cc;
  *s = q & 2 ? -ss : ss;
}

struct RopeGrid {
  int tokens, heads;  // of a workgroup
  unsigned groups;    // workgroups for the heads of a token
};

template <typename T, int V, bool INTER>
__global__ __launch_bounds__(kThreads) void rope_kernel(RopeParams p, RopeGrid g) {
  extern __shared__ float2 cs[];
  const unsigned half = p.R / 2;
  const int t0 = (blockIdx.x / g.groups) * g.tokens, h0 = (blockIdx.x % g.groups) * g.heads;
  const unsigned tokens = min(g.tokens, p.T - t0), heads = min(g.heads, p.H - h0);
  for (unsigned i = threadIdx.x; i < tokens * half; i += kThreads) {
    const unsigned t = i / half, f = i - t * half;
    const uint64_t a = (uint64_t)(int64_t)p.pos[t0 + t] * p.table[f];
    float c, s;
    cos_sin((uint32_t)((a + 0x80000000u) >> 32), &c, &s);
    cs[i] = make_float2(c * p.magnitude, (p.back ? -s : s) * p.magnitude);
  }
  __syncthreads();
  // Items of a head: INTER: one vector, turned or not; halves: two vectors that are turned into one
  // another, then the vectors that pass.
  constexpr int PV = INTER && V == 2 ? 1 : V;  // columns that pass: one at a time where nothing is aligned
  const unsigned turned = INTER ? p.R / V : half / V;
  const unsigned per = turned + (p.D - p.R) / PV, n = tokens * heads * per;
  const T* x = static_cast<const T*>(p.x.p);
  T* y = static_cast<T*>(p.y);
#pragma unroll 2
  for (unsigned i = threadIdx.x; i < n; i += kThreads) {
    const unsigned th = i / per, j = i - th * per, t = th / heads, h = th - t * heads;
    const T* px = x + (t0 + t) * p.x.pitch + (h0 + h) * p.x.head;
    T* py = y + ((int64_t)(t0 + t) * p.H + h0 + h) * p.D;
    if (j >= turned) {
      const unsigned c = p.R + (j - turned) * PV;
      float v[PV];
      loadv<T, PV>(px + c, v);
      storev<T, PV>(py + c, v);
    } else if constexpr (INTER) {
      const float2* a = cs + t * half + j * (V / 2);
      float v[V], r[V];
      if constexpr (V == 2) {
        v[0] = to_f(px[2 * j]);
        v[1] = to_f(px[2 * j + 1]);
      } else {
        loadv<T, V>(px + j * V, v);
      }
#pragma unroll
      for (int e = 0; e < V; e += 2) {
        const float2 w = a[e / 2];
        r[e] = v[e] * w.x - v[e + 1] * w.y;
        r[e + 1] = v[e] * w.y + v[e + 1] * w.x;
      }
      if constexpr (V == 2) {
        py[2 * j] = to_t<T>(r[0]);
        py[2 * j + 1] = to_t<T>(r[1]);
      } else {
        storev<T, V>(py + j * V, r);
      }
    } else {
      const float2* a = cs + t * half + j * V;
      float u[V], v[V], r[V], q[V];
      loadv<T, V>(px + j * V, u);
      loadv<T, V>(px + half + j * V, v);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float2 w = a[e];
        r[e] = u[e] * w.x - v[e] * w.y;
        q[e] = u[e] * w.y + v[e] * w.x;
      }
      storev<T, V>(py + j * V, r);
      storev<T, V>(py + half + j * V, q);
    }
  }
}

template <typename T, int V, bool INTER>
hipError_t launch(const RopeParams& p, hipStream_t st) {
  constexpr int PV = INTER && V == 2 ? 1 : V;
  const int64_t half = p.R / 2, per = (INTER ? p.R / V : half / V) + (p.D - p.R) / PV, row = per * p.H;
  // about 1024 items a workgroup (4 a thread), fewer where that leaves compute units idle
  int64_t want = 1024;
  while (want > kThreads && row * p.T < want * 512) want /= 2;
  RopeGrid g;
  g.tokens = (int)(want > row ? want / row : 1);
  const int64_t fit = half ? kMaxAngles / half : p.T;
  if (g.tokens > fit) g.tokens = fit > 1 ? (int)fit : 1;
  if (g.tokens > p.T) g.tokens = p.T;
  const int64_t heads = g.tokens > 1 || row <= 2 * want ? p.H : (want + per - 1) / per;
  g.heads = (int)(heads < p.H ? heads : p.H);
  g.groups = (p.H + g.heads - 1) / g.heads;
  const int64_t blocks = (int64_t)((p.T + g.tokens - 1) / g.tokens) * g.groups;
  if (blocks > kMaxGroups) return hipErrorInvalidConfiguration;
  rope_kernel<T, V, INTER><<<dim3((unsigned)blocks), kThreads, (size_t)g.tokens * half * sizeof(float2), st>>>(p, g);
  return hipGetLastError();
}

bool aligned(const void* p, int64_t a, int64_t b, int64_t c, int e) {
  const uint64_t m = (uint64_t)(uintptr_t)p | (uint64_t)a * e | (uint64_t)b * e | (uint64_t)c * e;
  return m % 16 == 0;
}

template <typename T>
hipError_t rope_any(const RopeParams& p, hipStream_t st) {
  constexpr int V = 16 / sizeof(T), E = sizeof(T);
  // vectors start at multiples of 16 bytes of a head, the second half's among them
  const bool vec = aligned(p.x.p, p.T > 1 ? p.x.pitch : 0, p.H > 1 ? p.x.head : 0, p.D, E) &&
                   aligned(p.y, p.R, p.inter ? 0 : p.R / 2, 0, E);
  if (p.inter) return vec ? launch<T, V, true>(p, st) : launch<T, 2, true>(p, st);
  return vec ? launch<T, V, false>(p, st) : launch<T, 1, false>(p, st);
}

}  // namespace

hipError_t launch_rope(const RopeParams& p, int dtype, hipStream_t st) {
  return dtype == GDN_DTYPE_BF16 ? rope_any<bf16>(p, st) : rope_any<float>(p, st);
}

}  // namespace gdn
