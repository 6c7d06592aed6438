// gdn_attn_f32.hip -- attention over a paged cache with fp32 activations, for few rows and many.
//
//   z_j = scale q . k_j over the keys that the row sees,  o = sum_j e^{z_j - m} v_j / sum_j e^{z_j - m}
//
// All of it in fp32, on the fp32 16x16x4 matrix instructions (157 TFLOP/s at best, a sixteenth of bf16's, so
// operands come straight from memory and the caches: keys as rows, values as columns).  A workgroup has a tile
// of 16 or 32 rows, its four waves every fourth 16 keys each, as in the few-row kernel for bf16.  Bound by the
// latency of its loads: cross attention of 777, 5 and 130 tokens to 300, 1 and 77 states, 12 heads of 64 columns:
// 26 us.  One token after 131071 keys of 8 heads of 128 columns: 194 us (1074 MB, 5.5 TB/s), over 8 bits 111 (277 MB,
// 2.5 TB/s); 512 after 4000, 32 query heads: 386 us, 63% of the matrix rate.
#include "../../include/gdn.h"
#include "gdn_attn_device.h"
#include "gdn_q8.h"

namespace gdn {

namespace {

constexpr int kWaves = 4;
constexpr int kTile = 16;

__device__ __forceinline__ bool odd_f(float x) { return (__float_as_uint(x) & 0x7f800000u) == 0x7f800000u; }
template <bool Q8, int D, int MT>
__global__ __launch_bounds__(256) void attn_f32_kernel(AttnParams p) {
  constexpr int ROWS = 16 * MT, KS = D / 32, DB = D / 16, CB = Q8 ? D : 4 * D;
  __shared__ __attribute__((aligned(1024))) char lds[kWaves * ROWS * (D + 6) * 4];
  const int lane = threadIdx.x & 63, wv = uni(threadIdx.x >> 6), li = lane & 15, lq = lane >> 4;
  const int id = quotient(blockIdx.x, p.by_heads), h = blockIdx.x - id * p.Hk;
  Unit u;
  if (!find_unit<true>(p, id, lane, &u)) return;

  f32x8 q[MT][KS];
  int last[MT], first[MT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    const int row = u.row0 + 16 * mt + li;
    last[mt] = last_key(p, u, row);
    first[mt] = first_key(p, last[mt]);
    const int t = quotient(row, p.by_group);
    const float* from = static_cast<const float*>(p.q.p) + (int64_t)(u.begin + t) * p.q.pitch +
                        (h * p.G + row - t * p.G) * p.q.head + 8 * lq;
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int j = 0; j < 8; ++j) q[mt][s][j] = 16 * mt + li < u.nrows ? from[32 * s + j] : 0.f;
  }
  const int all_last = last_key(p, u, u.row0), all_first = first_key(p, last_key(p, u, u.row0 + u.nrows - 1));

  f32x4 o[MT][DB];
  float m[MT], l[MT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    m[mt] = -__builtin_inff();
    l[mt] = 0.f;
#pragma unroll
    for (int b = 0; b < DB; ++b) o[mt][b] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  for (int key = u.lo + kTile * wv; key < u.hi; key += kTile * kWaves) {
    const int page = p.table[u.seq * p.table_pitch + (key >> p.pshift)];
    const Window w = page_rows(p, page, h, key, kTile, u.hi, CB);
    const __amdgpu_buffer_rsrc_t rk = dma::store_rsrc(const_cast<char*>(static_cast<const char*>(p.k)) + w.at, w.bytes);
    const __amdgpu_buffer_rsrc_t rv = dma::store_rsrc(const_cast<char*>(static_cast<const char*>(p.v)) + w.at, w.bytes);
    f32x8 k[KS];
    float v[DB][4];  // value of key 4 lq + j, column 16 b + li
    f32x4 ks, vs;
    if constexpr (Q8) {
      const int64_t at = w.at / CB;
      const int rows = w.bytes / CB;
      const __amdgpu_buffer_rsrc_t r1 = dma::store_rsrc(const_cast<float*>(p.ks) + at, rows * 4);
      const __amdgpu_buffer_rsrc_t r2 = dma::store_rsrc(const_cast<float*>(p.vs) + at, rows * 4);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        ks[r] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r1, 16 * lq + 4 * r, 0, 0));
        vs[r] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r2, 16 * lq + 4 * r, 0, 0));
      }
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        float x[8];
        q8_unpack(__builtin_bit_cast(u32x2v, __builtin_amdgcn_raw_buffer_load_b64(rk, li * CB + 32 * s + 8 * lq, 0, 0)), x);
#pragma unroll
        for (int j = 0; j < 8; ++j) k[s][j] = x[j];
      }
#pragma unroll
      for (int b = 0; b < DB; ++b)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          v[b][j] = __builtin_amdgcn_cvt_f32_fp8(
              (int)__builtin_amdgcn_raw_buffer_load_b8(rv, (4 * lq + j) * CB + 16 * b + li, 0, 0), 0);
    } else {
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const u32x4v x = __builtin_bit_cast(
              u32x4v, __builtin_amdgcn_raw_buffer_load_b128(rk, li * CB + 128 * s + 32 * lq + 16 * e, 0, 0));
#pragma unroll
          for (int j = 0; j < 4; ++j) k[s][4 * e + j] = __uint_as_float(x[j]);
        }
#pragma unroll
      for (int b = 0; b < DB; ++b)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          v[b][j] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rv, (4 * lq + j) * CB + 64 * b + 4 * li, 0, 0));
    }
    const bool part = key + kTile - 1 > all_last || key < all_first;  // not all rows see all keys
    const bool edge = part || key + kTile > u.hi;
    bool odd = false;  // infinities or NaN among values that some rows do not see
    if (part) {
#pragma unroll
      for (int b = 0; b < DB; ++b)
#pragma unroll
        for (int j = 0; j < 4; ++j) odd |= odd_f(v[b][j]);
      odd = __ballot(odd) != 0;
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      f32x4 z{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < KS; ++s) z = mma16(k[s], q[mt][s], z);
      float top = -__builtin_inff();
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        float x = z[r] * p.scale;
        if constexpr (Q8) x *= ks[r];
        if (edge) {
          const int kk = key + 4 * lq + r;
          x = kk < u.hi && kk <= last[mt] && kk >= first[mt] ? x : -__builtin_inff();
        }
        z[r] = x;
        top = fmaxf(top, x);
      }
      top = max_rows16(top);
      if (__ballot(top > m[mt])) {
        const float now = fmaxf(m[mt], top), a = part_weight(m[mt], now);
        m[mt] = now;
        l[mt] *= a;
#pragma unroll
        for (int b = 0; b < DB; ++b) o[mt][b] *= a;
      }
      const float base = m[mt] == -__builtin_inff() ? 0.f : m[mt];
      float e[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        e[r] = __builtin_amdgcn_exp2f(z[r] - base);
        l[mt] += e[r];
        // (a hidden key's scale may be anything)
        if constexpr (Q8) e[r] = edge && z[r] == -__builtin_inff() ? 0.f : e[r] * vs[r];
      }
      if (!odd) {
#pragma unroll
        for (int b = 0; b < DB; ++b)
#pragma unroll
          for (int j = 0; j < 4; ++j) o[mt][b] = mma4(v[b][j], e[j], o[mt][b]);
      } else {
        // a product with a weight of 0 would not be 0: such values are added where they are seen, and taken out
#pragma unroll 1
        for (int j = 0; j < kTile; ++j) {
          const bool seen = key + j < u.hi && key + j <= last[mt] && key + j >= first[mt];
#pragma unroll
          for (int b = 0; b < DB; ++b) {
            float x[4];  // columns 16 b + 4 lq + r, as the outputs
            if constexpr (Q8) {
              const int w = (int)__builtin_amdgcn_raw_buffer_load_b32(rv, j * CB + 16 * b + 4 * lq, 0, 0);
              const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(w, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(w, true);
              x[0] = lo[0], x[1] = lo[1], x[2] = hi[0], x[3] = hi[1];
            } else {
              const u32x4v w = __builtin_bit_cast(
                  u32x4v, __builtin_amdgcn_raw_buffer_load_b128(rv, j * CB + 64 * b + 16 * lq, 0, 0));
#pragma unroll
              for (int r = 0; r < 4; ++r) x[r] = __uint_as_float(w[r]);
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) o[mt][b][r] += seen && odd_f(x[r]) ? x[r] : 0.f;
            __builtin_amdgcn_sched_barrier(0);  // (rare: few registers before speed)
          }
        }
#pragma unroll
        for (int b = 0; b < DB; ++b)
#pragma unroll
          for (int j = 0; j < 4; ++j) o[mt][b] = mma4(odd_f(v[b][j]) ? 0.f : v[b][j], e[j], o[mt][b]);
      }
    }
  }

  float* ol = reinterpret_cast<float*>(lds);
  float* ml = ol + kWaves * ROWS * (D + 4);
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    const float sum = add_halves(add_rows16(l[mt]));
    const int col = wv * ROWS + 16 * mt + li;
    if (lq == 0) {
      ml[2 * col] = m[mt];
      ml[2 * col + 1] = sum;
    }
#pragma unroll
    for (int b = 0; b < DB; ++b) *reinterpret_cast<f32x4*>(ol + col * (D + 4) + 16 * b + 4 * lq) = o[mt][b];
  }
  __syncthreads();
  join_waves<float, D, ROWS, kWaves>(p, u, h, ol, ml);
}

template <bool Q8, int D, int MT>
hipError_t launch(const AttnParams& p, hipStream_t st) {
  const int64_t groups = ((int64_t)p.plan.units + p.plan.spare) * p.Hk;
  attn_f32_kernel<Q8, D, MT><<<dim3((unsigned)groups), 256, 0, st>>>(p);
  return hipGetLastError();
}
template <bool Q8, int D>
hipError_t by_rows(const AttnParams& p, hipStream_t st) {
  if constexpr (D == 256) return launch<Q8, D, 1>(p, st);  // (the plan has tiles of 16 rows)
  else return p.plan.rows == 16 ? launch<Q8, D, 1>(p, st) : launch<Q8, D, 2>(p, st);
}
template <bool Q8>
hipError_t by_width(const AttnParams& p, hipStream_t st) {
  return p.D == 64 ? by_rows<Q8, 64>(p, st) : (p.D == 128 ? by_rows<Q8, 128>(p, st) : by_rows<Q8, 256>(p, st));
}

}  // namespace

hipError_t launch_attn_f32(const AttnParams& p, bool q8, hipStream_t st) {
  return q8 ? by_width<true>(p, st) : by_width<false>(p, st);
}

}  // namespace gdn
