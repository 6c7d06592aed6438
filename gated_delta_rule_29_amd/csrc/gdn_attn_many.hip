// gdn_attn_many.hip -- attention of many rows (chunks of a prompt, cross attention) over a paged cache.
//
//   z_j = scale q . k_j over the keys that the row sees,  o = sum_j e^{z_j - m} v_j / sum_j e^{z_j - m}
//
// in one pass with a running maximum m and sum.  A workgroup's waves each keep 32 rows (new tokens times the
// query heads of a kv head) in registers, queries and outputs; tiles of 64 keys and values go through LDS,
// the next one under way while this one is worked on.  Both products run on 32x32x16 matrix instructions,
// transposed: scores^T = K Q^T leaves each row's scores in one lane column, so that its maximum and sum need
// one lane exchange, and its accumulators are the second product's operand (outputs^T = V^T P^T) as they are:
// half h of the wave has keys 8 i + 4 h + r of each 16.
#include "../../include/gdn.h"
#include "gdn_attn_device.h"
#include "gdn_q8.h"

namespace gdn {

namespace {

constexpr int kTile = 64;  // keys of a tile
// kinds of instructions for the scheduler
constexpr int kValu = 0x2, kMfma = 0x8, kDsRead = 0x100;
constexpr int kRows = 32;  // of a wave

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
typedef __attribute__((address_space(3))) bf16x8 lds_bf16x8;
typedef __attribute__((address_space(3))) char lds_char;
__device__ __forceinline__ u32x2v tr16(lds_char* p) {
  return __builtin_bit_cast(u32x2v, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)p));
}
__device__ __forceinline__ bf16x8 read16(lds_char* p) {
  const bf16x8 r = *(lds_bf16x8*)p;
  return r;
}
__device__ __forceinline__ f32x16 mma32(const bf16x8& a, const bf16x8& b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// Position of 16-byte chunk c of a row in LDS: c ^ swz(row).  The 16 rows that a read of the keys takes in a
// cycle, and the four rows and four chunks of a transposing read, fall on different banks.
template <int D>
__device__ __forceinline__ int swz(int row) {
  if constexpr (D == 64) return ((row >> 1) & 1) << 2 | ((row >> 2) & 1) << 1 | ((row >> 3) & 1);
  else return (row & 3) << 2 | ((row >> 2) & 1) << 1 | ((row >> 3) & 1);
}

template <bool Q8, int D, int NW>
struct Many {
  static constexpr int ROWS = kRows * NW;
  static constexpr int RB = D * 2;
  static constexpr int TILE = kTile * RB;  // bytes of a tile of keys or values in LDS
  static constexpr int SCALES = Q8 ? 2 * kTile * 4 : 0;
  static constexpr int STAGE = 2 * TILE + SCALES;
  static constexpr int LDS = 2 * STAGE;
};

template <bool Q8, int D, int NW>
__global__ __launch_bounds__(64 * NW) void attn_many_kernel(AttnParams p) {
  using M = Many<Q8, D, NW>;
  constexpr int RB = M::RB, CB = Q8 ? D : 2 * D;  // bytes of a row in LDS and in the cache
  constexpr int KS = D / 16;                      // contraction steps of the scores
  constexpr int DB = D / 32;                      // blocks of output columns
  constexpr int TR = kTile * CB / 1024;           // 1 KB transfers of a tile of keys
  constexpr int NI = (TR + NW - 1) / NW;          // of a wave
  static_assert(TR % NI == 0, "a wave takes NI transfers or none");
  constexpr int RPL = 1024 / CB;                  // rows of one
  __shared__ __attribute__((aligned(1024))) char lds[M::LDS];
  const int lane = threadIdx.x & 63, wv = uni(threadIdx.x >> 6), col = lane & 31, half = lane >> 5;
  const int h = blockIdx.x % p.Hk;
  // descending: a causal sequence's last rows see the most keys
  const int id = p.plan.units + p.plan.spare - 1 - blockIdx.x / p.Hk;
  Unit u;
  if (!find_unit<true>(p, id, lane, &u)) return;

  const int row = u.row0 + kRows * wv + col;
  const bool live = row < u.row0 + u.nrows;
  const int last = last_key(p, u, row), first = first_key(p, last);
  // of this wave's rows: keys up to all_last and from all_first on are seen by all, beyond any_last by none
  const int r0 = u.row0 + kRows * wv, r1 = min(r0 + kRows, u.row0 + u.nrows) - 1;
  const int all_last = uni(last_key(p, u, r0)), any_last = uni(r1 >= r0 ? last_key(p, u, r1) : -1);
  const int all_first = uni(first_key(p, any_last)), any_first = uni(first_key(p, all_last));
  bf16x8 q[KS];
  {
    const int t = row / p.G;
    const bf16* from = static_cast<const bf16*>(p.q.p) + (int64_t)(u.begin + t) * p.q.pitch +
                       (h * p.G + row - t * p.G) * p.q.head + 8 * half;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
#pragma unroll
      for (int j = 0; j < 8; ++j) q[s][j] = (bf16)0.f;
      if (live) {
        if (p.q_vec) {
          q[s] = *reinterpret_cast<const bf16x8*>(from + 16 * s);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) q[s][j] = from[16 * s + j];
        }
      }
    }
  }

  f32x16 o[DB];
#pragma unroll
  for (int b = 0; b < DB; ++b)
#pragma unroll
    for (int r = 0; r < 16; ++r) o[b][r] = 0.f;
  float m = -__builtin_inff(), l = 0.f;  // the maximum is of products, before the scale

  const uint32_t base = dma::lds_addr(lds);
  // keys: row col (and 32 more), chunk 2 s + half
  lds_char* kp[KS];
#pragma unroll
  for (int s = 0; s < KS; ++s)
    kp[s] = (lds_char*)(uintptr_t)(base + col * RB + 16 * ((2 * s + half) ^ swz<D>(col)));
  // values, transposing: rows 4 half + (lane & 15) / 4 of each 8, columns 16 ((lane >> 4) & 1) + 4 (lane & 3)
  lds_char* vp[2][DB];
#pragma unroll
  for (int e = 0; e < 2; ++e)
#pragma unroll
    for (int b = 0; b < DB; ++b) {
      const int r = 8 * e + 4 * half + ((lane & 15) >> 2), c = 4 * b + 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
      vp[e][b] = (lds_char*)(uintptr_t)(base + M::TILE + r * RB + 16 * (c ^ swz<D>(r)) + 8 * (lane & 1));
    }

  // Transfers.  A wave has kTile / NW rows of a tile, which lie in one page; the page of the tile after the next
  // is asked for with the next tile's rows.
  constexpr int WR = NI * RPL;  // rows
  const int nt = (u.hi - u.lo + kTile - 1) / kTile;
  const bool carries = wv * NI < TR;
  const __amdgpu_buffer_rsrc_t pages =
      dma::store_rsrc(const_cast<int*>(p.table) + u.seq * p.table_pitch, (uint32_t)p.width * 4);
  auto page_of = [&](int t) {
    const int key = u.lo + kTile * t + wv * WR;
    return (int)__builtin_amdgcn_raw_buffer_load_b32(pages, (key >> p.pshift) * 4, 0, 0);
  };
  int page_v = carries ? page_of(0) : 0;
  u32x4v kn[Q8 ? NI : 1], vn[Q8 ? NI : 1];
  float sn = 0.f;

  auto ask = [&](int t, int stage) {
    if (carries) {
      const int key = u.lo + kTile * t + wv * WR, page = uni(page_v);
      const Window w = page_rows(p, page, h, key, WR, u.hi, CB);
      const char *kb = static_cast<const char*>(p.k) + w.at, *vb = static_cast<const char*>(p.v) + w.at;
      if constexpr (Q8) {
        const __amdgpu_buffer_rsrc_t rk = dma::store_rsrc(const_cast<char*>(kb), w.bytes);
        const __amdgpu_buffer_rsrc_t rv = dma::store_rsrc(const_cast<char*>(vb), w.bytes);
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          kn[i] = __builtin_bit_cast(u32x4v, __builtin_amdgcn_raw_buffer_load_b128(rk, 1024 * i + 16 * lane, 0, 0));
          vn[i] = __builtin_bit_cast(u32x4v, __builtin_amdgcn_raw_buffer_load_b128(rv, 1024 * i + 16 * lane, 0, 0));
        }
      } else {
        const dma::i32x4 rk = dma::make_rsrc(kb, w.bytes), rv = dma::make_rsrc(vb, w.bytes);
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const int r = RPL * i + lane / (RB / 16), c = (lane % (RB / 16)) ^ swz<D>(wv * WR + r);
          const uint32_t to = uni(base + stage * M::STAGE + (wv * WR + RPL * i) * RB);
          dma::dma16(rk, r * RB + 16 * c, 0, to);
          dma::dma16(rv, r * RB + 16 * c, 0, to + M::TILE);
        }
      }
      if (t + 1 < nt) page_v = page_of(t + 1);
    }
    if constexpr (Q8) {
      // scales: the first wave the keys', the second the values'
      if (wv < 2) {
        sn = 0.f;
        const int key = u.lo + kTile * t + lane;
        if (key < u.hi) {
          const int page = p.table[u.seq * p.table_pitch + (key >> p.pshift)];
          if (page >= 0 && page < p.pages)
            sn = (wv ? p.vs : p.ks)[((int64_t)page * p.Hk + h) * p.P + (key & (p.P - 1))];
        }
      }
    }
  };
  // 8-bit tiles: from registers into LDS, as bf16
  auto land = [&](int stage) {
    char* to = lds + stage * M::STAGE;
    if (carries)
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int r = (wv * NI + i) * RPL + lane / (D / 16), c = 2 * (lane % (D / 16)), x = swz<D>(r);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int at = r * RB + 16 * ((c + e) ^ x);
          *reinterpret_cast<bf16x8*>(to + at) = q8_bf16(u32x2v{kn[i][2 * e], kn[i][2 * e + 1]});
          *reinterpret_cast<bf16x8*>(to + M::TILE + at) = q8_bf16(u32x2v{vn[i][2 * e], vn[i][2 * e + 1]});
        }
      }
    if (wv < 2) reinterpret_cast<float*>(to + 2 * M::TILE)[wv * kTile + lane] = sn;
  };

  // Maxima are kept while a new one is less than 2^8 times the old one's weight: outputs and sum are then as
  // exact, and most tiles change nothing.
  const float slack = 8.f / p.scale;

  // One tile.  EDGE: some of its keys are not seen by some of the wave's rows.
  auto tile = [&](int t, int stage, auto edge_t) {
    constexpr bool EDGE = decltype(edge_t)::value;
    const int key = u.lo + kTile * t;
    if constexpr (Q8) land(stage);
    dma::wait_vm0();
    __syncthreads();  // this tile is there, and the other stage's readers are done
    if (t + 1 < nt) ask(t + 1, stage ^ 1);
    if constexpr (EDGE)
      if (key > any_last || key + kTile <= any_first) return;  // nothing of it is seen by this wave's rows
    const int at = stage * M::STAGE;
    f32x16 z[2];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
#pragma unroll
      for (int r = 0; r < 16; ++r) z[kb][r] = 0.f;
#pragma unroll
      for (int s = 0; s < KS; ++s) z[kb] = mma32(read16(kp[s] + at + 32 * kb * RB), q[s], z[kb]);
    }
    if constexpr (!EDGE) {
      // four operands ahead of the products
      __builtin_amdgcn_sched_group_barrier(kDsRead, 4, 0);
#pragma unroll
      for (int i = 0; i < 2 * KS - 4; ++i) {
        __builtin_amdgcn_sched_group_barrier(kMfma, 1, 0);
        __builtin_amdgcn_sched_group_barrier(kDsRead, 1, 0);
      }
      __builtin_amdgcn_sched_group_barrier(kMfma, 4, 0);
    }
    float top = -__builtin_inff();
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        f32x4 ks;
        if constexpr (Q8)
          ks = *reinterpret_cast<const f32x4*>(lds + at + 2 * M::TILE + 4 * (32 * kb + 8 * g + 4 * half));
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          float x = z[kb][4 * g + r];
          if constexpr (Q8) x *= ks[r];
          if constexpr (EDGE) {
            const int k = key + 32 * kb + 8 * g + 4 * half + r;
            x = k < u.hi && k <= last && k >= first ? x : -__builtin_inff();
          }
          z[kb][4 * g + r] = x;
          top = fmaxf(top, x);
        }
      }
    top = max_halves(top);
    if (__ballot(top > m + slack)) {
      const float now = fmaxf(m, top), a = part_weight(m * p.scale, now * p.scale);
      m = now;
      l *= a;
#pragma unroll
      for (int b = 0; b < DB; ++b) o[b] *= a;
    }
    const float off = m == -__builtin_inff() ? 0.f : -m * p.scale;
    bf16x8 pf[4];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        f32x4 vs;
        if constexpr (Q8)
          vs = *reinterpret_cast<const f32x4*>(lds + at + 2 * M::TILE + 4 * (kTile + 32 * kb + 8 * g + 4 * half));
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float x = z[kb][4 * g + r];
          float e = __builtin_amdgcn_exp2f(__builtin_fmaf(x, p.scale, off));
          l += e;
          // (a hidden key's scale may be anything)
          if constexpr (Q8) e = EDGE && x == -__builtin_inff() ? 0.f : e * vs[r];
          // Weights enter the product as bf16: each is off by 2^-8 of itself at most, in either direction,
          // where the output's own rounding is as large.
          pf[2 * kb + g / 2][4 * (g & 1) + r] = (bf16)e;
        }
      }
    auto values = [&](int s, int b) {
      const u32x2v lo = tr16(vp[0][b] + at + 16 * s * RB), hi = tr16(vp[1][b] + at + 16 * s * RB);
      return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3));
    };
    bool odd = false;  // infinities or NaN among values that some rows do not see
    if constexpr (EDGE) {
#pragma unroll 1
      for (int i = 0; i < M::TILE; i += 1024)
        odd |= not_finite(*reinterpret_cast<const bf16x8*>(lds + at + M::TILE + i + 16 * lane));
      odd = __ballot(odd) != 0;
    }
    if (!EDGE || !odd) {
#pragma unroll
      for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int b = 0; b < DB; ++b) o[b] = mma32(values(s, b), pf[s], o[b]);
      if constexpr (!EDGE && !Q8) {
        __builtin_amdgcn_sched_group_barrier(kDsRead, 4, 1);
        __builtin_amdgcn_sched_group_barrier(kValu, 24, 1);
#pragma unroll
        for (int i = 0; i < 4 * DB; ++i) {
          __builtin_amdgcn_sched_group_barrier(kMfma, 1, 1);
          __builtin_amdgcn_sched_group_barrier(kDsRead, 2, 1);
          __builtin_amdgcn_sched_group_barrier(kValu, 24 / DB, 1);
        }
      }
    } else {
      // a product with a weight of 0 would not be 0: such values are added where they are seen, and taken out
#pragma unroll
      for (int b = 0; b < DB; ++b) {
#pragma unroll 1
        for (int j = 0; j < kTile; ++j) {
          const int k = key + j;
          const bool seen = k < u.hi && k <= last && k >= first;
          const char* from = lds + at + M::TILE + j * RB + 8 * half;
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const u32x2v w = *reinterpret_cast<const u32x2v*>(from + 16 * ((4 * b + g) ^ swz<D>(j)));
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const float x = __uint_as_float(r & 1 ? w[r / 2] & 0xffff0000u : w[r / 2] << 16);
              o[b][4 * g + r] += seen && (__float_as_uint(x) & 0x7f800000u) == 0x7f800000u ? x : 0.f;
            }
          }
        }
        __builtin_amdgcn_sched_barrier(0);  // (rare: few registers before speed)
      }
#pragma unroll
      for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int b = 0; b < DB; ++b) {
          o[b] = mma32(finite_part(values(s, b)), pf[s], o[b]);
          __builtin_amdgcn_sched_barrier(0);
        }
    }
  };

  // Tiles [in0, in1) are seen whole by all of the wave's rows; the others, first and last, are masked.
  int in0 = nt, in1 = nt;
  if (r1 >= r0) {
    in0 = min(nt, max(0, all_first - u.lo + kTile - 1) / kTile);
    in1 = min(nt, max(0, min(all_last + 1, u.hi) - u.lo) / kTile);
    in0 = (in0 + 1) & ~1;  // (two at a time, in their stages)
    if (in1 - in0 < 2) in0 = in1 = nt;
  }
  if (nt) {
    dma::wait_vm0();
    ask(0, 0);
  }
  int t = 0;
  for (int end = in0;; end = nt) {
#pragma unroll 1
    for (; t < end; ++t) tile(t, t & 1, std::true_type{});
    if (t >= nt) break;
#pragma unroll 1
    for (; t + 2 <= in1; t += 2) {
      tile(t, 0, std::false_type{});
      tile(t + 1, 1, std::false_type{});
    }
  }
  m *= p.scale;

  l = add_halves(l);
  if (!live) return;
  // lane: columns 32 b + 8 g + 4 half + r of its row
  if (u.pieces == 1) {
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int64_t to = out_row(p, u, h, row);
    bf16* out = static_cast<bf16*>(p.o) + to * D + 4 * half;
#pragma unroll
    for (int b = 0; b < DB; ++b)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const float r[4] = {o[b][4 * g] * inv, o[b][4 * g + 1] * inv, o[b][4 * g + 2] * inv, o[b][4 * g + 3] * inv};
        storev<bf16, 4>(out + 32 * b + 8 * g, r);
      }
    if (p.lse && half == 0) p.lse[to] = row_lse(m, l);
  } else {
    const int at = row - u.row0;
    float* out = part_outputs(p, u.slot, h) + (int64_t)at * D + 4 * half;
#pragma unroll
    for (int b = 0; b < DB; ++b)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const float r[4] = {o[b][4 * g], o[b][4 * g + 1], o[b][4 * g + 2], o[b][4 * g + 3]};
        storev<float, 4>(out + 32 * b + 8 * g, r);
      }
    if (half == 0) {
      float* s = part_sums(p, u.slot, h) + 2 * at;
      s[0] = m;
      s[1] = l;
    }
  }
}

template <bool Q8, int D>
hipError_t launch(const AttnParams& p, hipStream_t st) {
  constexpr int NW = many_rows(D) / kRows;
  const int64_t groups = ((int64_t)p.plan.units + p.plan.spare) * p.Hk;
  attn_many_kernel<Q8, D, NW><<<dim3((unsigned)groups), 64 * NW, 0, st>>>(p);
  return hipGetLastError();
}

template <bool Q8>
hipError_t by_width(const AttnParams& p, hipStream_t st) {
  return p.D == 64 ? launch<Q8, 64>(p, st) : (p.D == 128 ? launch<Q8, 128>(p, st) : launch<Q8, 256>(p, st));
}

}  // namespace

hipError_t launch_attn_many(const AttnParams& p, bool q8, hipStream_t st) {
  return q8 ? by_width<true>(p, st) : by_width<false>(p, st);
}

}  // namespace gdn
