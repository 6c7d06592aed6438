// gdn_attn_few.hip -- attention of few rows (single tokens, short drafts: at most 32 rows a kv head) over a
// paged cache.
//
//   z_j = scale q . k_j over the keys that the row sees,  o = sum_j e^{z_j - m} v_j / sum_j e^{z_j - m}
//
// in one pass with a running maximum m and sum.  The G query heads of a kv head and the sequence's new tokens
// are the rows of one 16- or 32-row tile, so keys and values are read once for all of them.  Bound by memory:
// each of a workgroup's four waves takes every fourth 32 keys by itself, without barriers: keys come into
// registers as matrix operands (rows of 16 keys), values into the wave's own part of LDS, and the next 32 are
// under way while these are worked on.  The transposed scores' accumulators are the second product's operand
// as they are: lane (lq, li) has keys 4 lq + r of each 16, for row li.
//
// One token after 131071 keys of 8 heads of 128 columns, bf16 (537 MB): 94 us, 5.7 TB/s, and 5 for the join; 32
// single tokens over 8-bit caches (321 MB, contexts up to 20000): 67 + 5 us, 4.8 TB/s.  Page numbers are a load
// before the loads: asked for a tile ahead they took 125 us to 113 and 89 to 71.  Of 256 columns, 16 query and 2 key
// heads, which leave one wave a SIMD: one token after 131071 62 us (268 MB, 4.3 TB/s), over 8 bits 53 (136 MB, 2.6
// TB/s); 32 single tokens after 0 .. 18600 121 us (610 MB, 5 TB/s), over 8 bits 77 (310 MB, 4 TB/s).
#include "../../include/gdn.h"
#include "gdn_attn_device.h"
#include "gdn_q8.h"

namespace gdn {

namespace {

constexpr int kWaves = 4;
constexpr int kTile = 32;  // keys that a wave takes at a time

typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
__device__ __forceinline__ u32x2v tr16(uint32_t lds) {
  return __builtin_bit_cast(u32x2v, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(uintptr_t)lds));
}

// Position of 16-byte chunk c of a value row in LDS: an XOR that lets the eight rows and two chunks that a
// transposing read takes in a cycle, and the rows that are written, fall on different banks.
template <int D>
__device__ __forceinline__ int swz(int row) {
  if constexpr (D == 64) return ((row >> 1) & 1) << 2 | ((row >> 2) & 1) << 1 | ((row >> 3) & 1);
  else return (row & 3) << 2 | ((row >> 2) & 1) << 1 | ((row >> 3) & 1);
}

template <bool Q8, int D, int MT>
struct Few {
  static constexpr int ROWS = 16 * MT;
  static constexpr int RB = D * 2;                     // bytes of a value row in LDS
  static constexpr int STAGES = Q8 ? 1 : 2;            // 8-bit values are converted on their way into LDS
  static constexpr int VBYTES = kTile * RB * STAGES;   // of a wave
  static constexpr int OBYTES = ROWS * (D + 4) * 4;    // of a wave, at the end
  static constexpr int WAVE = VBYTES > OBYTES ? VBYTES : OBYTES;
  static constexpr int LDS = kWaves * (WAVE + ROWS * 8);
};

template <bool Q8, int D, int MT>
__global__ __launch_bounds__(256) void attn_few_kernel(AttnParams p) {
  using F = Few<Q8, D, MT>;
  constexpr int RB = F::RB, CB = Q8 ? D : 2 * D;  // CB: bytes of a cache row
  constexpr int KS = D / 32;                      // contraction steps of the scores
  constexpr int DB = D / 16;                      // blocks of output columns
  constexpr int KL = Q8 ? KS / 2 : KS;            // 16-byte loads of a key a lane
  constexpr int VL = kTile * CB / 1024;           // 1 KB transfers of a tile of values
  constexpr int RPL = 1024 / CB;                  // rows of one
  __shared__ __attribute__((aligned(1024))) char lds[F::LDS];
  const int lane = threadIdx.x & 63, wv = uni(threadIdx.x >> 6), li = lane & 15, lq = lane >> 4;
  const int id = quotient(blockIdx.x, p.by_heads), h = blockIdx.x - id * p.Hk;
  Unit u;
  if (!find_unit<true>(p, id, lane, &u)) return;

  // queries: column li of a 16-row tile; the columns of the head that meet a key's (see below)
  bf16x8 q[MT][KS];
  int last[MT], first[MT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    const int row = u.row0 + 16 * mt + li;
    last[mt] = last_key(p, u, row);
    first[mt] = first_key(p, last[mt]);
    const int t = quotient(row, p.by_group);
    const bf16* from = static_cast<const bf16*>(p.q.p) + (int64_t)(u.begin + t) * p.q.pitch +
                       (h * p.G + row - t * p.G) * p.q.head;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const int d = Q8 ? 64 * (s / 2) + 16 * lq + 8 * (s & 1) : 32 * s + 8 * lq;
#pragma unroll
      for (int j = 0; j < 8; ++j) q[mt][s][j] = (bf16)0.f;
      if (16 * mt + li < u.nrows) {
        if (p.q_vec) {
          q[mt][s] = *reinterpret_cast<const bf16x8*>(from + d);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) q[mt][s][j] = from[d + j];
        }
      }
    }
  }
  // keys below `all_last` and from `all_first` on are seen by every row of the unit
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

  char* mine = lds + wv * F::WAVE;
  const uint32_t vlds = dma::lds_addr(mine);
  // transposing read: rows 4 lq + li / 4 (and 16 more), columns 4 (li % 4) of a block of 16
  const int trow = 4 * lq + (li >> 2);
  const uint32_t tr0 = vlds + trow * RB + 8 * (li & 1);
  const int trc = ((li & 3) >> 1) ^ swz<D>(trow);

  u32x4v kn[2][KL];
  f32x4 ksn[2], vsn[2];
  u32x4v vn[Q8 ? VL : 1];

  // Pages of a tile's two times 16 keys (one page holds 16): asked for a tile before its keys and values.
  const __amdgpu_buffer_rsrc_t pages =
      dma::store_rsrc(const_cast<int*>(p.table) + u.seq * p.table_pitch, (uint32_t)p.width * 4);
  int page_v[2];
  auto ask_pages = [&](int key) {
#pragma unroll
    for (int kt = 0; kt < 2; ++kt)
      page_v[kt] = (int)__builtin_amdgcn_raw_buffer_load_b32(pages, ((key + 16 * kt) >> p.pshift) * 4, 0, 0);
  };
  // Asks for a tile's keys, values and scales, and for the next tile's pages.
  auto ask = [&](int key, int stage) {
    const int page[2] = {uni(page_v[0]), uni(page_v[1])};
#pragma unroll
    for (int kt = 0; kt < 2; ++kt) {
      const Window w = page_rows(p, page[kt], h, key + 16 * kt, 16, u.hi, CB);
      const __amdgpu_buffer_rsrc_t rk = dma::store_rsrc(const_cast<char*>(static_cast<const char*>(p.k)) + w.at, w.bytes);
#pragma unroll
      for (int s = 0; s < KL; ++s)
        kn[kt][s] = __builtin_bit_cast(u32x4v, __builtin_amdgcn_raw_buffer_load_b128(rk, li * CB + 64 * s + 16 * lq, 0, 0));
      const char* vb = static_cast<const char*>(p.v) + w.at;
      if constexpr (Q8) {
        const int64_t at = w.at / CB;
        const int rows = w.bytes / CB;
        const __amdgpu_buffer_rsrc_t r1 = dma::store_rsrc(const_cast<float*>(p.ks) + at, rows * 4);
        const __amdgpu_buffer_rsrc_t r2 = dma::store_rsrc(const_cast<float*>(p.vs) + at, rows * 4);
        // (dwords: a window may end inside four rows)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          ksn[kt][r] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r1, 16 * lq + 4 * r, 0, 0));
          vsn[kt][r] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r2, 16 * lq + 4 * r, 0, 0));
        }
        const __amdgpu_buffer_rsrc_t rv = dma::store_rsrc(const_cast<char*>(vb), w.bytes);
#pragma unroll
        for (int i = 0; i < VL / 2; ++i)
          vn[kt * (VL / 2) + i] = __builtin_bit_cast(u32x4v, __builtin_amdgcn_raw_buffer_load_b128(rv, 1024 * i + 16 * lane, 0, 0));
      } else {
        const dma::i32x4 rv = dma::make_rsrc(vb, w.bytes);
#pragma unroll
        for (int i = 0; i < VL / 2; ++i) {
          // lane's place in LDS is linear; it takes the chunk that belongs there
          const int row = RPL * i + lane / (RB / 16), c = (lane % (RB / 16)) ^ swz<D>(row);
          dma::dma16(rv, row * RB + 16 * c, 0, uni(vlds + stage * kTile * RB + (16 * kt + RPL * i) * RB));
        }
      }
    }
    ask_pages(key + kTile * kWaves);
  };

  int key = u.lo + kTile * wv, stage = 0;
  if (key < u.hi) {
    ask_pages(key);
    ask(key, 0);
  }
  for (; key < u.hi; key += kTile * kWaves, stage ^= F::STAGES - 1) {
    dma::wait_vm0();
    u32x4v kc[2][KL];
    f32x4 ks[2], vs[2];
#pragma unroll
    for (int kt = 0; kt < 2; ++kt) {
#pragma unroll
      for (int s = 0; s < KL; ++s) kc[kt][s] = kn[kt][s];
      if constexpr (Q8) {
        ks[kt] = ksn[kt];
        vs[kt] = vsn[kt];
      }
    }
    if constexpr (Q8) {
      // values into LDS as bf16: 16 bytes are two chunks
#pragma unroll
      for (int i = 0; i < VL; ++i) {
        const int row = RPL * i + lane / (D / 16), c = 2 * (lane % (D / 16)), x = swz<D>(row);
#pragma unroll
        for (int e = 0; e < 2; ++e)
          *reinterpret_cast<bf16x8*>(mine + row * RB + 16 * ((c + e) ^ x)) =
              q8_bf16(u32x2v{vn[i][2 * e], vn[i][2 * e + 1]});
      }
    }
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): the other stage's reads are done
    asm volatile("" ::: "memory");
    if (key + kTile * kWaves < u.hi) ask(key + kTile * kWaves, stage ^ 1);

    // scores (transposed): rows keys, columns rows of the unit
    f32x4 z[MT][2];
#pragma unroll
    for (int kt = 0; kt < 2; ++kt) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) z[mt][kt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        bf16x8 kf;
        if constexpr (Q8) {
          kf = q8_bf16(u32x2v{kc[kt][s / 2][2 * (s & 1)], kc[kt][s / 2][2 * (s & 1) + 1]});
        } else {
          kf = __builtin_bit_cast(bf16x8, kc[kt][s]);
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) z[mt][kt] = mma16(kf, q[mt][s], z[mt][kt]);
      }
    }
    const bool part = key + kTile - 1 > all_last || key < all_first;  // not all rows see all keys
    const bool edge = part || key + kTile > u.hi;
    bf16x8 pf[MT], pl[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      float top = -__builtin_inff();
#pragma unroll
      for (int kt = 0; kt < 2; ++kt) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          float x = z[mt][kt][r] * p.scale;
          if constexpr (Q8) x *= ks[kt][r];
          if (edge) {
            const int k = key + 16 * kt + 4 * lq + r;
            x = k < u.hi && k <= last[mt] && k >= first[mt] ? x : -__builtin_inff();
          }
          z[mt][kt][r] = x;
          top = fmaxf(top, x);
        }
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
      f32x4 e[2];
#pragma unroll
      for (int kt = 0; kt < 2; ++kt) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          e[kt][r] = __builtin_amdgcn_exp2f(z[mt][kt][r] - base);
          l[mt] += e[kt][r];
          // (a hidden key's scale may be anything)
          if constexpr (Q8) e[kt][r] = edge && z[mt][kt][r] == -__builtin_inff() ? 0.f : e[kt][r] * vs[kt][r];
        }
      }
      // Weights enter the product as two bf16: the upper bits, and what is left, rounded: off by 2^-16 of itself at
      // most.  (As one they are off by 2^-8, as much as the output's own rounding; the times are the same, 101 us for
      // one token after 131071, 75 for 32 over 8 bits.)
      u32x4v upper;
      f32x4 left[2];
#pragma unroll
      for (int kt = 0; kt < 2; ++kt) {
        unsigned up[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float x = e[kt][r];
          // (8-bit values are finite or NaN, and their weights of either sign)
          if constexpr (Q8) up[r] = __float_as_uint(x) & 0xffff0000u;
          else up[r] = upper_bf16(x);
          left[kt][r] = x - __uint_as_float(up[r]);
          // (an infinite scale)
          if constexpr (Q8) left[kt][r] = __builtin_fabsf(x) == __builtin_inff() ? 0.f : left[kt][r];
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) upper[2 * kt + i] = __builtin_amdgcn_perm(up[2 * i + 1], up[2 * i], 0x07060302u);
      }
      pf[mt] = __builtin_bit_cast(bf16x8, upper);
      pl[mt] = pack8<bf16>(left[0], left[1]);
    }
    const uint32_t tr = tr0 + stage * kTile * RB;
    auto values = [&](int b) {
      const uint32_t a = tr + 16 * ((2 * b) ^ trc);
      const u32x2v lo = tr16(a), hi = tr16(a + 16 * RB);
      return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3));
    };
    bool odd = false;  // infinities or NaN among values that some rows do not see
    if (part) {
      unsigned any = 0;
#pragma unroll 4
      for (int i = 0; i < kTile * RB; i += 1024)
        any |= not_finite_bits(*reinterpret_cast<const u32x4v*>(mine + stage * kTile * RB + i + 16 * lane));
      odd = __ballot(any) != 0;
    }
    if (!odd) {
#pragma unroll
      for (int b = 0; b < DB; ++b) {
        const bf16x8 v = values(b);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) o[mt][b] = mma16(v, pl[mt], mma16(v, pf[mt], o[mt][b]));
      }
    } else {
      // a product with a weight of 0 would not be 0: such values are added where they are seen, and taken out
#pragma unroll 1
      for (int j = 0; j < kTile; ++j) {
        const int k = key + j;
        const char* from = mine + stage * kTile * RB + j * RB + 8 * (lq & 1);
#pragma unroll
        for (int b = 0; b < DB; ++b) {
          const u32x2v w = *reinterpret_cast<const u32x2v*>(from + 16 * ((2 * b + (lq >> 1)) ^ swz<D>(j)));
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float x = __uint_as_float(r & 1 ? w[r / 2] & 0xffff0000u : w[r / 2] << 16);
            const bool is = (__float_as_uint(x) & 0x7f800000u) == 0x7f800000u;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
              o[mt][b][r] += is && k < u.hi && k <= last[mt] && k >= first[mt] ? x : 0.f;
          }
        }
      }
#pragma unroll
      for (int b = 0; b < DB; ++b) {
        const bf16x8 v = finite_part(values(b));
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) o[mt][b] = mma16(v, pl[mt], mma16(v, pf[mt], o[mt][b]));
        __builtin_amdgcn_sched_barrier(0);  // (rare: few registers before speed)
      }
    }
  }

  // what the waves have, joined in LDS
  float* ml = reinterpret_cast<float*>(lds + kWaves * F::WAVE);
  float* ol = reinterpret_cast<float*>(lds);
  __syncthreads();
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    const float sum = add_halves(add_rows16(l[mt]));
    const int col = wv * F::ROWS + 16 * mt + li;
    if (lq == 0) {
      ml[2 * col] = m[mt];
      ml[2 * col + 1] = sum;
    }
#pragma unroll
    for (int b = 0; b < DB; ++b) *reinterpret_cast<f32x4*>(ol + col * (D + 4) + 16 * b + 4 * lq) = o[mt][b];
  }
  __syncthreads();
  join_waves<bf16, D, F::ROWS, kWaves>(p, u, h, ol, ml);
}

template <bool Q8, int D, int MT>
hipError_t launch(const AttnParams& p, hipStream_t st) {
  const int64_t groups = ((int64_t)p.plan.units + p.plan.spare) * p.Hk;
  attn_few_kernel<Q8, D, MT><<<dim3((unsigned)groups), 256, 0, st>>>(p);
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

hipError_t launch_attn_few(const AttnParams& p, bool q8, hipStream_t st) {
  return q8 ? by_width<true>(p, st) : by_width<false>(p, st);
}

}  // namespace gdn
