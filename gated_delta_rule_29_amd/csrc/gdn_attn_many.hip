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
//
// 8192 tokens after 8192, 32 query and 8 key heads of 128 columns, bf16: 1370 to 1450 us by the card's clock,
// 1.14 to 1.2 PFLOP/s of the keys that are seen, where a large library product reaches 1.21.  Bound by instruction
// issue: a tile of 64 keys is 32 products of 32 cycles and some 140 other vector instructions a wave, and a product
// keeps the other wave's from issuing for about half of its time; matrix units are busy 59 to 61% of the time.
// Of 4096 tokens after 4096 (TFLOP/s): 128 columns over 8 bits 735 (two multiplications more for each score, 5
// registers in scratch, and one tile a stage); 64 columns 850, over 8 bits 690; 256 columns 700 to 750, over 8 bits 510.  Tiles of 128 rows of four waves, two groups of waves that take turns at products and
// exponentials (1552 us), and both interleaved by hand in a wave (1621) were no faster.
#include "../../include/gdn.h"
#include "gdn_attn_device.h"
#include "gdn_q8.h"

namespace gdn {

namespace {

// kinds of instructions for the scheduler
constexpr int kValu = 0x2, kMfma = 0x8, kDsRead = 0x100;
constexpr int kRows = 32;  // of a wave

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
typedef __attribute__((address_space(3))) bf16x8 lds_bf16x8;
__device__ __forceinline__ u32x2v tr16(uint32_t lds) {
  return __builtin_bit_cast(u32x2v, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(uintptr_t)lds));
}
__device__ __forceinline__ bf16x8 read16(uint32_t lds) {
  const bf16x8 r = *(lds_bf16x8*)(uintptr_t)lds;
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
  // Output columns of a workgroup.  256 columns of outputs and queries leave one wave a SIMD, whose 512 registers hold
  // them with bf16 caches but for 35 in scratch (750 TFLOP/s); 8-bit ones need more, for what is in flight and converted,
  // and are faster (520 against 380) with two workgroups that have half of the outputs each, both form the scores, and
  // run two waves a SIMD of 256 registers (29 more in scratch).
  static constexpr int DV = D == 256 && Q8 ? 128 : D;
  static constexpr int TK = DV < D ? 32 : 64;  // keys of a tile
  static constexpr int RK = D * 2, RV = DV * 2;  // bytes of a row of keys and of values in LDS
  static constexpr int KT = TK * RK, VT = TK * RV;  // and of a tile
  // Tiles that come and go together: with two, the waves meet half as often, and the two of a SIMD drift apart, so that
  // one's products run beside the other's exponentials.
  static constexpr int SUB = DV < D || D == 64 || (D == 128 && !Q8) ? 2 : 1;
  static constexpr int STAGE = SUB * (KT + VT);  // keys, then values
  static constexpr int SCALES = Q8 ? 2 * SUB * TK * 4 : 0;
  static constexpr int LDS = 2 * (STAGE + SCALES);
};

template <bool Q8, int D, int NW, bool LSE>
__global__ __launch_bounds__(64 * NW) void attn_many_kernel(AttnParams p) {
  using M = Many<Q8, D, NW>;
  constexpr int RK = M::RK, RV = M::RV, DV = M::DV, CB = Q8 ? D : 2 * D, VB = Q8 ? DV : 2 * DV;  // CB, VB: in the cache
  constexpr int KS = D / 16;                      // contraction steps of the scores
  constexpr int DB = DV / 32;                     // blocks of output columns
  constexpr int TK = M::TK, SUB = M::SUB, KEYS = SUB * TK;  // keys of a tile; tiles and keys of a stage
  constexpr int KB = TK / 32, PS = TK / 16;       // blocks of 32 keys, contraction steps of the outputs
  constexpr int NI = KEYS * CB / 1024 / NW, NV = KEYS * VB / 1024 / NW;  // 1 KB transfers of a wave for a stage
  constexpr int WR = KEYS / NW;                                           // and its rows
  static_assert(NI >= 1 && NV >= 1 && WR <= 16, "a wave's rows lie in one page");
  __shared__ __attribute__((aligned(1024))) char lds[M::LDS];
  const int lane = threadIdx.x & 63, wv = uni(threadIdx.x >> 6), col = lane & 31, half = lane >> 5;
  constexpr int HV = D / DV;
  const int uh = blockIdx.x / HV, up = quotient(uh, p.by_heads);
  const int h = uh - up * p.Hk, c0 = blockIdx.x % HV * DV;  // c0: the first output column
  Unit u;
  if (!find_unit<true>(p, up, lane, &u)) return;

  const int row = u.row0 + kRows * wv + col;
  const bool live = row < u.row0 + u.nrows;
  const int last = last_key(p, u, row), first = first_key(p, last);
  const unsigned seen_n = (unsigned)max(0, min(last, u.hi - 1) - first + 1);  // keys of this piece from `first` on
  bf16x8 q[KS];
  {
    const int t = quotient(row, p.by_group);
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
  float m = -__builtin_inff();  // of products, before the scale
  // l, which outputs are divided by, sums the weights as they enter the product: an error that all terms of a result
  // share drops out, and a row that one key dominates gets that key's value, whatever its weight (with the weights
  // before their rounding it was off by up to 2^-8, the same in every column).  8-bit rows enter with their scale, of
  // which a sum of weights has no part.  le sums the weights themselves, for lse: both take 1420 us where one takes 1400
  // (8192 tokens after 8192), so calls without lse leave it out.
  constexpr bool AS_THEY_ENTER = !Q8;
  float l = 0.f, le = 0.f;

  const uint32_t base = dma::lds_addr(lds);
  // where a stage's operands are read; the other stage is `hop` away
  constexpr int KP = D == 256 ? 1 : KS;  // (256 columns: an XOR with 32 s leads from chunk to chunk)
  constexpr int VP = DV == 256 ? 1 : DB;
  uint32_t kp[KP], vp[2][VP];
  int hop = M::STAGE;
  // keys: row col (and 32 more), chunk 2 s + half
#pragma unroll
  for (int s = 0; s < KP; ++s) kp[s] = base + col * RK + 16 * ((2 * s + half) ^ swz<D>(col));
  // values, transposing: rows 4 half + (lane & 15) / 4 of each 8, columns 16 ((lane >> 4) & 1) + 4 (lane & 3)
#pragma unroll
  for (int e = 0; e < 2; ++e)
#pragma unroll
    for (int b = 0; b < VP; ++b) {
      const int r = 8 * e + 4 * half + ((lane & 15) >> 2), c = 4 * b + 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
      vp[e][b] = base + SUB * M::KT + r * RV + 16 * (c ^ swz<DV>(r)) + 8 * (lane & 1);
    }

  // Transfers.  A wave's rows lie in one page, whose number is asked for a stage ahead, as a scalar.
  typedef __attribute__((address_space(4))) const int const_int;
  const int nt = (u.hi - u.lo + TK - 1) / TK, ns = (nt + SUB - 1) / SUB;  // tiles and stages
  const_int* table = (const_int*)(uintptr_t)(p.table + u.seq * p.table_pitch);
  const int64_t page_bytes = (int64_t)p.Hk * p.P * CB;
  const char *khead = static_cast<const char*>(p.k) + (int64_t)h * p.P * CB,
             *vhead = static_cast<const char*>(p.v) + (int64_t)h * p.P * CB + c0 * (CB / D);
  auto page_of = [&](int t) { return table[min(u.lo + KEYS * t + wv * WR, u.hi - 1) >> p.pshift]; };
  int page = nt ? page_of(0) : 0;
  u32x4v kn[Q8 ? NI : 1], vn[Q8 ? NV : 1];
  float sn = 0.f;
  constexpr int SG = KEYS / 64;  // waves that fetch a stage's key scales
  auto page_of_key = [&](int t) {
    return p.table[u.seq * p.table_pitch + (min(u.lo + KEYS * t + 64 * (wv % SG) + lane, u.hi - 1) >> p.pshift)];
  };
  int key_page = Q8 && nt && wv < 2 * SG ? page_of_key(0) : 0;

  // Lane's part of transfer i of rows of `row` bytes in the cache (of which a transfer takes `part`).
  auto place = [&](int i, auto part_c, auto row_c) {
    constexpr int PART = decltype(part_c)::value, LPR = PART / 16;  // lanes of a row
    return (uint32_t)((1024 / PART * i + lane / LPR) * decltype(row_c)::value + 16 * (lane % LPR));
  };
  // The same with the chunk that belongs at lane's place in LDS.
  auto place_swz = [&](int i, auto d_c, auto row_c) {
    constexpr int DD = decltype(d_c)::value, LPR = DD / 8;
    const int r = 512 / DD * i + lane / LPR;
    return (uint32_t)(r * decltype(row_c)::value + 16 * ((lane % LPR) ^ swz<DD>(wv * WR + r)));
  };
  typedef std::integral_constant<int, CB> cb_c;
  auto ask = [&](int t, int stage) {
    {
      const int key = u.lo + KEYS * t + wv * WR;
      const bool there = key < u.hi && (unsigned)page < (unsigned)p.pages;
      const int64_t from = there ? page * page_bytes + (key & (p.P - 1)) * CB : 0;
      const uint32_t bytes = there ? (uint32_t)(min(WR, u.hi - key) * CB) : 0;
      const char *kb = khead + from, *vb = vhead + from;
      const uint32_t v_bytes = DV == D || !bytes ? bytes : bytes - c0 * (CB / D);  // (vb is c0 columns in)
      if constexpr (Q8) {
        const __amdgpu_buffer_rsrc_t rk = dma::store_rsrc(const_cast<char*>(kb), bytes);
        const __amdgpu_buffer_rsrc_t rv = dma::store_rsrc(const_cast<char*>(vb), v_bytes);
#pragma unroll
        for (int i = 0; i < NI; ++i)
          kn[i] = __builtin_bit_cast(u32x4v, __builtin_amdgcn_raw_buffer_load_b128(rk, place(i, cb_c{}, cb_c{}), 0, 0));
#pragma unroll
        for (int i = 0; i < NV; ++i)
          vn[i] = __builtin_bit_cast(u32x4v, __builtin_amdgcn_raw_buffer_load_b128(
                                                 rv, place(i, std::integral_constant<int, VB>{}, cb_c{}), 0, 0));
      } else {
        const dma::i32x4 rk = dma::make_rsrc(kb, bytes), rv = dma::make_rsrc(vb, v_bytes);
        const uint32_t to = uni(base + stage * M::STAGE);
#pragma unroll
        for (int i = 0; i < NI; ++i)
          dma::dma16(rk, place_swz(i, std::integral_constant<int, D>{}, cb_c{}), 0, to + wv * WR * RK + 1024 * i);
#pragma unroll
        for (int i = 0; i < NV; ++i)
          dma::dma16(rv, place_swz(i, std::integral_constant<int, DV>{}, cb_c{}), 0,
                     to + SUB * M::KT + wv * WR * RV + 1024 * i);
      }
      page = page_of(t + 1);
    }
    if constexpr (Q8) {
      // scales: the first wave (or two) the keys', the next the values'; a key's page, too, is asked for a stage ahead
      if (wv < 2 * SG) {
        const int key = u.lo + KEYS * t + 64 * (wv % SG) + lane;
        sn = 0.f;
        if (key < u.hi && (unsigned)key_page < (unsigned)p.pages)
          sn = (wv < SG ? p.ks : p.vs)[((int64_t)key_page * p.Hk + h) * p.P + (key & (p.P - 1))];
        key_page = page_of_key(t + 1);
      }
    }
  };
  // 8-bit tiles: from registers into LDS, as bf16
  auto land_rows = [&](char* to, u32x4v x, int i, auto d_c) {
    constexpr int DD = decltype(d_c)::value, LPR = DD / 16;
    const int r = wv * WR + 1024 / DD * i + lane / LPR, c = 2 * (lane % LPR);
#pragma unroll
    for (int e = 0; e < 2; ++e)
      *reinterpret_cast<bf16x8*>(to + r * 2 * DD + 16 * ((c + e) ^ swz<DD>(r))) = q8_bf16(u32x2v{x[2 * e], x[2 * e + 1]});
  };
  auto land = [&](int stage) {
    char* to = lds + stage * M::STAGE;
#pragma unroll
    for (int i = 0; i < NI; ++i) land_rows(to, kn[i], i, std::integral_constant<int, D>{});
#pragma unroll
    for (int i = 0; i < NV; ++i) land_rows(to + SUB * M::KT, vn[i], i, std::integral_constant<int, DV>{});
    if (wv < 2 * SG) reinterpret_cast<float*>(lds + 2 * M::STAGE + stage * M::SCALES)[wv * 64 + lane] = sn;
  };

  // Tiles [see0, see1) have keys that some of this wave's rows see; all rows see all of tiles [in0, in1).
  int see0 = nt, see1 = nt, in0 = nt, in1 = nt;
  {
    const int r0 = u.row0 + kRows * wv, r1 = min(r0 + kRows, u.row0 + u.nrows) - 1;
    if (r1 >= r0) {
      const int last0 = uni(last_key(p, u, r0)), last1 = uni(last_key(p, u, r1));
      const int first0 = uni(first_key(p, last0)), first1 = uni(first_key(p, last1));
      see0 = min(nt, max(0, first0 - u.lo) / TK);
      see1 = max(see0, min(nt, max(0, last1 - u.lo + TK) / TK));
      in0 = min(nt, max(0, first1 - u.lo + TK - 1) / TK);
      in1 = max(in0, min(nt, max(0, min(last0 + 1, u.hi) - u.lo) / TK));
    }
  }

  // Infinities or NaN among a tile's values: where some rows do not see all of its keys, a product with a weight
  // of 0 would not be 0.  Such tiles (`odd`: of the masked ones, see0 .. in0 - 1, in1 .. see1 - 1, of which there are
  // few) are left out and added in the end, key by key.
  unsigned long long odd = 0;

  // Maxima are kept while a new one is less than 2^8 times the old one's weight: most tiles change nothing.  fp32 sums
  // and the weights' relative roundings are as exact with weights up to 2^8; only the largest weight, which would be 1,
  // is rounded as the others are.
  // (Finite for the smallest scales, too: a sum of infinities of both signs would compare as false for ever.)
  const float slack = fminf(8.f / p.scale, 0x1.fffffep127f);

  auto key_rows = [&](int s, int off) { return read16((KP == 1 ? kp[0] ^ (32 * s) : kp[s % KP]) + off); };
  // One tile, number t, the stage's number `sub`.  EDGE: some of its keys are not seen by some of the wave's rows.
  auto tile = [&](int t, int stage, int sub, auto edge_t) {
    constexpr bool EDGE = decltype(edge_t)::value;
    const int key = u.lo + TK * t;
    const float* scales = reinterpret_cast<const float*>(lds + 2 * M::STAGE + stage * M::SCALES) + sub * TK + 4 * half;
    f32x16 z[KB];
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
      for (int r = 0; r < 16; ++r) z[kb][r] = 0.f;
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
      for (int s = 0; s < KS; ++s) z[kb] = mma32(key_rows(s, sub * M::KT + 32 * kb * RK), q[s], z[kb]);
    if constexpr (!EDGE) {
      // four operands ahead of the products
      __builtin_amdgcn_sched_group_barrier(kDsRead, 4, 0);
#pragma unroll
      for (int i = 0; i < KB * KS - 4; ++i) {
        __builtin_amdgcn_sched_group_barrier(kMfma, 1, 0);
        __builtin_amdgcn_sched_group_barrier(kDsRead, 1, 0);
      }
      __builtin_amdgcn_sched_group_barrier(kMfma, 4, 0);
    }
    const unsigned from0 = (unsigned)(key + 4 * half - first);
    float top = -__builtin_inff();
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        f32x4 ks;
        if constexpr (Q8)
          ks = *reinterpret_cast<const f32x4*>(scales + 32 * kb + 8 * g);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          float x = z[kb][4 * g + r];
          if constexpr (Q8) x *= ks[r];
          if constexpr (EDGE) x = from0 + (unsigned)(32 * kb + 8 * g + r) < seen_n ? x : -__builtin_inff();
          z[kb][4 * g + r] = x;
          top = fmaxf(top, x);
        }
      }
    top = max_halves(top);
    if (__ballot(top > m + slack)) {
      const float now = fmaxf(m, top), a = part_weight(m * p.scale, now * p.scale);
      m = now;
      l *= a;
      if constexpr (LSE) le *= a;
#pragma unroll
      for (int b = 0; b < DB; ++b) o[b] *= a;
    }
    const float off = m == -__builtin_inff() ? 0.f : -m * p.scale;
    bf16x8 pf[PS];
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        f32x4 vs;
        if constexpr (Q8)
          vs = *reinterpret_cast<const f32x4*>(scales + KEYS + 32 * kb + 8 * g);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float x = z[kb][4 * g + r];
          float e = __builtin_amdgcn_exp2f(__builtin_fmaf(x, p.scale, off));
          if constexpr (EDGE || !AS_THEY_ENTER) l += e;
          if constexpr (LSE) le += e;
          // (a hidden key's scale may be anything)
          if constexpr (Q8) e = EDGE && x == -__builtin_inff() ? 0.f : e * vs[r];
          // Weights enter the product as bf16: each is off by 2^-8 of itself at most, in either direction, where the
          // output's own rounding is as large (8192 tokens after 8192: 0.0023 of the outputs' norm from 64 bits, 0.0017
          // of it that rounding).  What is left, as a second product for every tile, would take half as many matrix
          // instructions more: 229 -> 319 us for 4096 tokens after 4096 with 64 columns, 227 -> 274 for 1024 after 8000
          // with 256, and 128 columns have no registers for it.  At the edges, where rows may see a few keys only, it is
          // done (2% of a serving step's chunks, nothing of a long prompt).
          bf16 w = (bf16)e;
          // (8-bit values are finite or NaN, and their weights of either sign)
          if constexpr (EDGE && !Q8) w = __builtin_bit_cast(bf16, (unsigned short)(upper_bf16(e) >> 16));
          pf[2 * kb + g / 2][4 * (g & 1) + r] = w;
          if constexpr (EDGE) {
            z[kb][4 * g + r] = e - (float)w;
            if constexpr (Q8) z[kb][4 * g + r] = __builtin_fabsf((float)w) == __builtin_inff() ? 0.f : z[kb][4 * g + r];
          }
        }
      }
    if constexpr (!EDGE && AS_THEY_ENTER) {
      // (two weights and the sum are rounded once, to nearest)
      typedef bf16 bf16x2 __attribute__((ext_vector_type(2)));
      const bf16x2 one = {(bf16)1.f, (bf16)1.f};
#pragma unroll
      for (int s = 0; s < PS; ++s)
#pragma unroll
        for (int j = 0; j < 8; j += 2)
          l = __builtin_amdgcn_fdot2_f32_bf16(bf16x2{pf[s][j], pf[s][j + 1]}, one, l, false);
    }
    auto values = [&](int s, int b) {
      const int x = VP == 1 ? 64 * b : 0, off = sub * M::VT + 16 * s * RV;
      const u32x2v lo = tr16((vp[0][b % VP] ^ x) + off), hi = tr16((vp[1][b % VP] ^ x) + off);
      return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3));
    };
    if (EDGE && (t < in0 || t >= in1)) {
      unsigned any = 0;
      const char* v = lds + stage * M::STAGE + SUB * M::KT + sub * M::VT + 16 * lane;
#pragma unroll 4
      for (int i = 0; i < M::VT; i += 1024) any |= not_finite_bits(*reinterpret_cast<const u32x4v*>(v + i));
      if (__ballot(any)) {
        odd |= 1ull << (t < in0 ? t - see0 : t - in1 + (in0 - see0));
        return;
      }
    }
#pragma unroll
    for (int s = 0; s < PS; ++s)
#pragma unroll
      for (int b = 0; b < DB; ++b) o[b] = mma32(values(s, b), pf[s], o[b]);
    if constexpr (EDGE) {
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int s = 0; s < PS; ++s) {
#pragma unroll
        for (int j = 0; j < 8; ++j) pf[s][j] = (bf16)z[s / 2][8 * (s & 1) + j];
#pragma unroll
        for (int b = 0; b < DB; ++b) o[b] = mma32(values(s, b), pf[s], o[b]);
      }
    }
    if constexpr (!EDGE) {
      __builtin_amdgcn_sched_group_barrier(kDsRead, Q8 ? 6 : 4, 1);
      __builtin_amdgcn_sched_group_barrier(kValu, Q8 ? 32 : 24, 1);
#pragma unroll
      for (int i = 0; i < PS * DB; ++i) {
        __builtin_amdgcn_sched_group_barrier(kMfma, 1, 1);
        __builtin_amdgcn_sched_group_barrier(kDsRead, 2, 1);
        __builtin_amdgcn_sched_group_barrier(kValu, 24 / DB, 1);
      }
    }
  };

  if (nt) {
    dma::wait_vm0();
    ask(0, 0);
  }
  // The start of stage n: its tiles are there, and the other stage's readers are done.
  auto arrive = [&](int n) {
    if constexpr (Q8) land(n & 1);
    dma::wait_vm0();
    __syncthreads();
    if (n + 1 < ns) ask(n + 1, (n + 1) & 1);
  };
  auto leave = [&] {
#pragma unroll
    for (int s = 0; s < KP; ++s) kp[s] += hop;
#pragma unroll
    for (int b = 0; b < VP; ++b) {
      vp[0][b] += hop;
      vp[1][b] += hop;
    }
    hop = -hop;
  };
  int n = 0;
  const int n0 = (in0 + SUB - 1) / SUB, n1 = in1 / SUB;  // stages of tiles that all rows see whole
  for (int end = min(n0, ns);; end = ns) {
#pragma unroll 1
    for (; n < end; ++n) {
      arrive(n);
#pragma unroll 1
      for (int sub = 0; sub < SUB; ++sub) {
        const int t = n * SUB + sub;
        if (t >= see0 && t < see1) tile(t, n & 1, sub, std::true_type{});
      }
      leave();
    }
    if (n >= ns) break;
#pragma unroll 1
    for (; n < n1; ++n) {
      arrive(n);
      static_for<SUB>([&](auto sub) { tile(n * SUB + sub(), n & 1, sub(), std::false_type{}); });
      leave();
    }
  }
  if (odd) {
    const float off = m == -__builtin_inff() ? 0.f : -m * p.scale;
    for (unsigned long long left = odd; left; left &= left - 1) {
      const int e = __builtin_ctzll(left), t = e < in0 - see0 ? see0 + e : in1 + e - (in0 - see0);
#pragma unroll 1
      for (int j = 0; j < TK; ++j) {
        const int key = u.lo + TK * t + j;
        if (key >= u.hi) break;
        const Window w = page_rows(p, p.table[u.seq * p.table_pitch + (key >> p.pshift)], h, key, 1, u.hi, CB);
        const char *kr = static_cast<const char*>(p.k) + w.at, *vr = static_cast<const char*>(p.v) + w.at;
        if (!w.bytes) continue;  // a page that the cache does not have: values of 0
        const int64_t place = w.at / CB;
        float x = 0.f;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          const bf16x8 k8 = Q8 ? q8_bf16(*reinterpret_cast<const u32x2v*>(kr + 16 * s + 8 * half))
                               : *reinterpret_cast<const bf16x8*>(kr + 32 * s + 16 * half);
#pragma unroll
          for (int i = 0; i < 8; ++i) x = __builtin_fmaf((float)q[s][i], (float)k8[i], x);
        }
        x = add_halves(x);
        if constexpr (Q8) x *= p.ks[place];
        float weight = __builtin_amdgcn_exp2f(__builtin_fmaf(x, p.scale, off));
        if constexpr (Q8) weight *= p.vs[place];
        const bool seen = (unsigned)(key - first) < seen_n;
#pragma unroll
        for (int b = 0; b < DB; ++b)
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const int c = c0 + 32 * b + 8 * g + 4 * half;
            float v[4];
            if constexpr (Q8) {
              const int w4 = *reinterpret_cast<const int*>(vr + c);
              const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(w4, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(w4, true);
              v[0] = lo[0], v[1] = lo[1], v[2] = hi[0], v[3] = hi[1];
            } else {
              loadv<bf16, 4>(reinterpret_cast<const bf16*>(vr) + c, v);
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) o[b][4 * g + r] += seen ? weight * v[r] : 0.f;
          }
      }
    }
  }
  m *= p.scale;

  l = add_halves(l);
  if constexpr (LSE) le = add_halves(le);
  if (!live) return;
  // lane: columns 32 b + 8 g + 4 half + r of its row
  if (u.pieces == 1) {
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int64_t to = out_row(p, u, h, row);
    bf16* out = static_cast<bf16*>(p.o) + to * D + c0 + 4 * half;
#pragma unroll
    for (int b = 0; b < DB; ++b)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const float r[4] = {o[b][4 * g] * inv, o[b][4 * g + 1] * inv, o[b][4 * g + 2] * inv, o[b][4 * g + 3] * inv};
        storev<bf16, 4>(out + 32 * b + 8 * g, r);
      }
    if (p.lse && half == 0 && c0 == 0) p.lse[to] = row_lse(m, LSE ? le : l);
  } else {
    const int at = row - u.row0;
    // (one sum a piece: outputs are scaled to it)
    const float f = !LSE || l == 0.f ? 1.f : le / l;
    float* out = part_outputs(p, u.slot, h) + (int64_t)at * D + c0 + 4 * half;
#pragma unroll
    for (int b = 0; b < DB; ++b)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const float r[4] = {o[b][4 * g] * f, o[b][4 * g + 1] * f, o[b][4 * g + 2] * f, o[b][4 * g + 3] * f};
        storev<float, 4>(out + 32 * b + 8 * g, r);
      }
    if (half == 0 && c0 == 0) {
      float* s = part_sums(p, u.slot, h) + 2 * at;
      s[0] = m;
      s[1] = LSE ? le : l;
    }
  }
}

template <bool Q8, int D>
hipError_t launch(const AttnParams& p, hipStream_t st) {
  constexpr int NW = many_rows(D, Q8) / kRows;
  const int64_t groups = ((int64_t)p.plan.units + p.plan.spare) * p.Hk * (D / Many<Q8, D, NW>::DV);
  if (!Q8 && p.lse) attn_many_kernel<Q8, D, NW, !Q8><<<dim3((unsigned)groups), 64 * NW, 0, st>>>(p);
  else attn_many_kernel<Q8, D, NW, false><<<dim3((unsigned)groups), 64 * NW, 0, st>>>(p);
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
