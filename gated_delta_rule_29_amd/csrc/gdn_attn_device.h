// gdn_attn_device.h -- device-side pieces shared by the attention kernels: the unit of work that a workgroup
// takes, the keys that a row sees, and what a workgroup's waves leave behind.
#pragma once

#include "gdn_attn.h"
#include "gdn_dma.h"
#include "gdn_layer_device.h"

namespace gdn {

// A piece of a unit's keys.
struct Unit {
  int seq, tile;        // tile: row0 / rows of a tile
  int piece, pieces;    // of the unit
  int slot;             // number of the piece among the pieces of all cut units; those of a unit are `apart`
  int apart;
  int begin, n;         // the sequence's first row in the batch and its tokens
  int len;              // its keys
  int row0, nrows;      // the unit's rows
  int lo, hi;           // the piece's keys; lo is a multiple of 64
};

__device__ __forceinline__ int attn_len(const AttnParams& p, int i) {
  return min(max(p.lens[i], 0), p.width << p.pshift);
}
// New tokens of sequence i (offsets on the device that are not the host's may decrease).
__device__ __forceinline__ int attn_tokens(const AttnParams& p, int i) {
  return max(seq_begin(p.s, i + 1) - seq_begin(p.s, i), 0);
}
// Tiles of a sequence in the launch's class, and an upper bound of a tile's keys.
__device__ __forceinline__ int attn_tiles(const AttnParams& p, int rows) {
  if (p.cls != kAllRows && (rows <= kFewRows) != (p.cls == kFew)) return 0;
  return (rows + p.plan.rows - 1) >> p.plan.row_bits;
}
__device__ __forceinline__ int attn_span(const AttnParams& p, int len) {
  return p.window ? (int)min((uint32_t)len, (uint32_t)p.window + p.plan.rows + 64) : len;  // (2^31 + 2^9 at most)
}

__device__ __forceinline__ int uni(int x) { return __builtin_amdgcn_readfirstlane(x); }

__device__ __forceinline__ int quotient(int n, const Divisor& d) { return (int)(((uint64_t)(uint32_t)n * d.mul) >> d.shift); }

// Inclusive prefix sum over the wave's lanes: shifts within rows of 16 lanes, then each row's and half's last lane into
// the next ones.
template <int CTRL, int ROWS>
__device__ __forceinline__ int add_shifted(int x) {
  return x + __builtin_amdgcn_update_dpp(0, x, CTRL, ROWS, 0xf, false);
}
__device__ __forceinline__ int wave_prefix(int x) {
  x = add_shifted<0x111, 0xf>(x);
  x = add_shifted<0x112, 0xf>(x);
  x = add_shifted<0x114, 0xf>(x);
  x = add_shifted<0x118, 0xf>(x);
  x = add_shifted<0x142, 0xa>(x);
  return add_shifted<0x143, 0xc>(x);
}

// Keys of a piece, about: so many that the units are cut into at most `spare` pieces more than there are units (a
// unit of n keys into n / keys, rounded: sum of tiles * (pieces - 1) <= sum of tiles * span / keys).  Every wave of every workgroup finds
// the same number, by itself; this is its reciprocal.
__device__ __forceinline__ float attn_pieces_a_key(const AttnParams& p, int lane) {
  // (in fp32, every wave in the same order; 2^-7 more keys than that, which 2^23 sequences can be off)
  float sum = 0.f;
  for (int i = lane; i < p.s.n; i += 64)
    sum += (float)attn_tiles(p, attn_tokens(p, i) * p.G) * (float)attn_span(p, attn_len(p, i));
  const float keys = fmaxf(wave_sum(sum) * (1.f + 0x1p-7f) * __builtin_amdgcn_rcpf((float)p.plan.spare),
                           (float)p.plan.min_piece);
  return __uint_as_float((unsigned)uni((int)__float_as_uint(__builtin_amdgcn_rcpf(keys))));
}

// Pieces of n keys, each of about 1 / inv.
__device__ __forceinline__ int attn_pieces(int n, float inv) { return max(1, (int)__builtin_fmaf((float)n, inv, 0.5f)); }

// Finds piece number `id` (PIECES), or unit number `id` of those that may be cut; false where there is nothing to do.
// Numbers go from the last sequence to the first, in a sequence by pieces and then from its last tile, whose rows see
// the most keys, to its first; sequences whose tiles all have many keys go before those whose first tiles have few.
// So what is long starts early (9 chunks of a serving step, 7 .. 2048 tokens: 130 -> 117 us), and numbers that stand
// for no piece (a causal sequence's first tiles have fewer) come in runs: where they alternate with others, those
// fall on half of the chip (the same with twice the pieces: 114 us instead of 80).
template <bool PIECES>
__device__ __forceinline__ bool find_unit(const AttnParams& p, int id, int lane, Unit* u) {
  const float inv = p.plan.spare ? attn_pieces_a_key(p, lane) : 0.f;
  int before = 0, before_cut = 0;  // what is counted, and cut units' pieces, of the sequences looked at
  int seq, at, cut_at = 0, per_tile = 1, tiles;
  if (p.plan.spare == 0 && !p.s.cu) {  // sequences alike
    const int e = quotient(id, p.by_tiles);
    if (e >= p.s.n) return false;
    seq = p.s.n - 1 - e;
    tiles = p.by_tiles.by;
    at = e * tiles;
  } else {
    const bool alike = p.plan.rows <= kFewRows || !p.causal || p.window;  // (few new tokens: one pass)
    bool level = true;
    for (int base = 0;; base += 64) {
      if (base >= p.s.n) {
        if (!level || alike) return false;
        level = false;
        base = 0;
      }
      const int i = p.s.n - 1 - (base + lane);
      int mine_tiles = 0, k = 1;
      if (i >= 0) {
        const int n = attn_tokens(p, i), len = attn_len(p, i);
        if (alike || (n <= len / 2) == level) mine_tiles = attn_tiles(p, n * p.G);
        if (p.plan.spare) k = attn_pieces(attn_span(p, len), inv);
      }
      const int cut = k > 1 ? mine_tiles * k : 0, mine = PIECES ? mine_tiles * k : (k > 1 ? mine_tiles : 0);
      const int sum = wave_prefix(mine), sum_cut = wave_prefix(cut);
      const unsigned long long m = __ballot(id < before + sum && id >= before + sum - mine);
      if (m) {
        const int l = __builtin_ctzll(m);
        seq = i + lane - l;
        tiles = __builtin_amdgcn_readlane(mine_tiles, l);
        per_tile = __builtin_amdgcn_readlane(k, l);
        at = before + __builtin_amdgcn_readlane(sum - mine, l);
        cut_at = before_cut + __builtin_amdgcn_readlane(sum_cut - cut, l);
        break;
      }
      before += __builtin_amdgcn_readlane(sum, 63);
      before_cut += __builtin_amdgcn_readlane(sum_cut, 63);
    }
  }
  seq = uni(seq);
  const int off = id - at, turn = !PIECES ? per_tile - 1 : (per_tile == 1 ? 0 : off / tiles);
  u->seq = seq;
  u->tile = tiles - 1 - (PIECES ? off - turn * tiles : off);
  u->piece = per_tile - 1 - turn;
  u->slot = cut_at + turn * tiles + (tiles - 1 - u->tile);
  u->apart = -tiles;
  u->begin = uni(seq_begin(p.s, seq));
  u->n = uni(attn_tokens(p, seq));
  u->len = uni(attn_len(p, seq));
  u->row0 = u->tile * p.plan.rows;
  u->nrows = min(p.plan.part_rows, u->n * p.G - u->row0);  // (part_rows: the most that a tile has)
  // the keys that any of the rows sees, and this piece's share of them
  int base = 0, end = u->len;
  if (p.causal) {
    end = max(0, min(end, u->len - u->n + quotient(u->row0 + u->nrows - 1, p.by_group) + 1));
    if (p.window) base = min(end, max(0, u->len - u->n + quotient(u->row0, p.by_group) - p.window + 1)) & ~63;
  }
  // (a causal sequence's first tiles see fewer keys than its last one, and may have fewer pieces)
  u->pieces = p.plan.spare ? uni(min(per_tile, attn_pieces(end - base, inv))) : 1;
  if (PIECES ? u->piece >= u->pieces : u->pieces == 1) return false;
  const int share = u->pieces == 1 ? (end - base + 63) & ~63 : ((end - base + u->pieces - 1) / u->pieces + 63) & ~63;
  const int64_t lo = base + (int64_t)u->piece * share;
  u->lo = (int)min(lo, (int64_t)end);
  u->hi = (int)min(lo + share, (int64_t)end);
  return true;
}

// The last key that row `row` of the unit's sequence sees, and the first.
__device__ __forceinline__ int last_key(const AttnParams& p, const Unit& u, int row) {
  return p.causal ? min(u.len - 1, u.len - u.n + quotient(row, p.by_group)) : u.len - 1;
}
__device__ __forceinline__ int first_key(const AttnParams& p, int last) {
  return p.window ? max(0, last - p.window + 1) : 0;  // (an empty row's last key is negative)
}

// A cache's rows [key, key + rows) of a head, which lie in this page, as a bounds-checked window: rows at or
// behind `end`, and pages that the cache does not have, read as zeros.  `row`: bytes.
struct Window {
  int64_t at;      // byte offset in the cache
  uint32_t bytes;
};
__device__ __forceinline__ Window page_rows(const AttnParams& p, int page, int h, int key, int rows, int end,
                                            int row) {
  Window w{0, 0};
  if (key < end && page >= 0 && page < p.pages) {
    w.at = (((int64_t)page * p.Hk + h) * p.P + (key & (p.P - 1))) * row;
    w.bytes = (uint32_t)(min(rows, end - key) * row);
  }
  return w;
}

__device__ __forceinline__ float max_rows16(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
  const auto q = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(q[0]), __uint_as_float(q[1]));
}
__device__ __forceinline__ float max_halves(float x) {
  const auto q = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(q[0]), __uint_as_float(q[1]));
}

// Which of 8 bf16 values are infinite or NaN, and those values with them set to 0.
typedef unsigned short u16x8 __attribute__((ext_vector_type(8)));
// (an exponent of all ones carries into the sign's place when a one is added to it)
__device__ __forceinline__ unsigned not_finite_bits(const u32x4v& v) {
  unsigned r = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) r |= ((v[i] & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
  return r;
}
__device__ __forceinline__ bf16x8 finite_part(const bf16x8& v) {
  u16x8 b = __builtin_bit_cast(u16x8, v);
#pragma unroll
  for (int i = 0; i < 8; ++i) b[i] = (b[i] & 0x7f80) == 0x7f80 ? 0 : b[i];
  return __builtin_bit_cast(bf16x8, b);
}
// A weight w of a bf16 cache's values as two bf16, upper (exact in bf16, as fp32 bits) and what is left, which is
// rounded to bf16: off by 2^-16 of w at most.  From w = 2^-102 on both are positive (upper is cut from the number below
// w, so that something is left of 1, too, which the key of a row's maximum has): products of 0, or of both signs, with
// an infinite value that is seen would make its column NaN.
__device__ __forceinline__ unsigned upper_bf16(float w) {
  const unsigned b = __float_as_uint(w);
  return (max(b, 1u) - 1u) & 0xffff0000u;
}
// Weight of a partial result whose maximum is m in a whole whose maximum is top (both may be -infinity).
__device__ __forceinline__ float part_weight(float m, float top) {
  return m == -__builtin_inff() ? 0.f : __builtin_amdgcn_exp2f(m - top);
}
__device__ __forceinline__ float row_lse(float m, float l) {
  return l > 0.f || l != l ? (m + __builtin_amdgcn_logf(l)) * kLn2 : -__builtin_inff();
}

// Index of output row (token of the batch, query head) of the unit's row.
__device__ __forceinline__ int64_t out_row(const AttnParams& p, const Unit& u, int h, int row) {
  const int t = quotient(row, p.by_group);
  return (int64_t)(u.begin + t) * p.Hq + h * p.G + (row - t * p.G);
}
// Partial results of a piece: its rows' outputs, and their maxima and sums.
__device__ __forceinline__ float* part_outputs(const AttnParams& p, int slot, int h) {
  return p.part + ((int64_t)slot * p.Hk + h) * p.plan.part_rows * p.D;
}
__device__ __forceinline__ float* part_sums(const AttnParams& p, int slot, int h) {
  const int64_t before = 2 * (int64_t)p.plan.spare * p.Hk * p.plan.part_rows * p.D;
  return p.part + before + ((int64_t)slot * p.Hk + h) * p.plan.part_rows * 2;
}

// The end of a workgroup of WV waves that each have their own keys: col (0 .. ROWS - 1) of wave w has outputs
// o[w][col][D] (a pitch of D + 4), maximum ml[w][col][0] and sum ml[w][col][1].  Called by all threads,
// with the waves' values in LDS.
template <typename T, int D, int ROWS, int WV>
__device__ __forceinline__ void join_waves(const AttnParams& p, const Unit& u, int h, const float* o,
                                           const float* ml) {
  constexpr int LP = D / 4;
  const bool whole = u.pieces == 1;
  float* part = whole ? nullptr : part_outputs(p, u.slot, h);
  float* sums = whole ? nullptr : part_sums(p, u.slot, h);
  for (int i = threadIdx.x; i < u.nrows * LP; i += blockDim.x) {
    const int col = i / LP, c = (i % LP) * 4;
    float m[WV], top = -__builtin_inff(), l = 0.f;
#pragma unroll
    for (int w = 0; w < WV; ++w) {
      m[w] = ml[(w * ROWS + col) * 2];
      top = fmaxf(top, m[w]);
    }
    float r[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < WV; ++w) {
      const float a = part_weight(m[w], top);
      const float* from = o + (w * ROWS + col) * (D + 4) + c;
      l += a * ml[(w * ROWS + col) * 2 + 1];
#pragma unroll
      for (int e = 0; e < 4; ++e) r[e] += a * from[e];
    }
    if (whole) {
      const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
      for (int e = 0; e < 4; ++e) r[e] *= inv;
      const int64_t row = out_row(p, u, h, u.row0 + col);
      storev<T, 4>(static_cast<T*>(p.o) + row * D + c, r);
      if (p.lse && c == 0) p.lse[row] = row_lse(top, l);
    } else {
      storev<float, 4>(part + (int64_t)col * D + c, r);
      if (c == 0) {
        sums[2 * col] = top;
        sums[2 * col + 1] = l;
      }
    }
  }
}

}  // namespace gdn
