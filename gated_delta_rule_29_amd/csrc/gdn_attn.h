// gdn_attn.h -- host-side launch interface of the operators of a full-attention layer: rotary positions,
// the paged cache (written and read back) and the attention of new tokens over it.
//
// Head tensors [tokens, H, D] are addressed as base + token * pitch + head * head_pitch.  A cache is
// [pages, Hk, P, D]; place s of it (a slot) is row s % P of page s / P.
#pragma once

#include "gdn_layer.h"

namespace gdn {

// A head tensor that is read.
struct Heads {
  const void* p;
  int64_t pitch, head;
};

struct RopeParams {
  Heads x;
  const int* pos;           // [T]
  const uint64_t* table;    // [R / 2] turns a position, in 2^-64 turns
  float magnitude;
  void* y;                  // [T, H, D]
  int T, H, D, R;
  bool inter;               // pairs (2i, 2i + 1); otherwise (i, i + R / 2)
  bool back;                // the transpose: turned backwards
};
hipError_t launch_rope(const RopeParams& p, int dtype, hipStream_t st);

struct Cache {
  void *k, *v;              // [pages, H, P, D]
  float *ks, *vs;           // [pages, H, P] with an 8-bit cache, or nullptr
  int pages, P, H, D;
};

struct CacheRowsParams {
  Cache c;
  Heads k, v;               // written: [T, H, D]
  void *ko, *vo;            // read: [T, H, D]
  const int* slots;         // [T]
  int T;
};
constexpr int kCacheMaxD = 512;
hipError_t launch_cache_write(const CacheRowsParams& p, int dtype, bool q8, hipStream_t st);
hipError_t launch_cache_read(const CacheRowsParams& p, int dtype, bool q8, hipStream_t st);

// n / d for n < 2^31 as a product: with 2^(s-1) < d <= 2^s and mul = ceil(2^(31+s) / d), n mul / 2^(31+s) is above
// n / d by less than 1 / d.  (A kernel of a few microseconds is bound by the instructions that it fetches: a division
// is 25 of them.)
struct Divisor {
  uint32_t mul, shift, by;
};
inline Divisor divisor(uint32_t d) {
  uint32_t s = 0;
  while ((uint64_t{1} << s) < d) ++s;
  return Divisor{(uint32_t)(((uint64_t{1} << (31 + s)) + d - 1) / d), 31 + s, d};
}

// The rows of a sequence and a kv head: its n new tokens times the G query heads that share the head, row
// token * G + g.  Tiles of rows are the units of work; a unit's keys may be cut into pieces that run at
// once and are joined.
struct AttnPlan {
  int rows;        // of a tile: 2^row_bits
  int row_bits;
  int units;       // tiles of all sequences of the class
  int spare;       // pieces beyond one a unit, at most (0: no unit is cut; cut units have 2 * spare at most)
  int min_piece;   // keys
  int part_rows;   // rows of a tile that exist (the pitch of partial results)
};

// A call's sequences fall into two classes: with at most kFewRows rows (each wave takes its own keys) and
// with more (each wave takes its own rows).  A sequence after 32768 keys, 8 key heads of 128 columns, us as few / as
// many: 17 rows 43 / 39 over bf16 and 43 / 54 over 8 bits, 32 rows 45 / 39 and 44 / 54, 40 rows 58 / 40 and 63 / 54, 64
// rows 60 / 40 and 63 / 56; eight of them: 32 rows 209 / 188 and 177 / 276, 40 rows 275 / 188 and 320 / 281; eight after
// 1000 keys: 32 rows 26 / 24 and 25 / 39, 40 rows 32 / 24 and 32 / 40.  (17 to 32 rows over bf16 keep the class
// whose weights are two bf16, for a tenth of their time.)
constexpr int kFewRows = 32;
// Rows of a tile of the second class.  256 bf16 columns take twice the registers: one wave a SIMD instead of two.
constexpr int many_rows(int D, bool q8) { return D == 256 && !q8 ? 128 : 256; }
enum AttnClass { kAllRows = 0, kFew = 1, kMany = 2 };

struct AttnParams {
  Heads q;                  // [rows, Hq, D]
  const void *k, *v;        // caches
  const float *ks, *vs;
  const int* table;         // [n, width], rows of table_pitch
  int64_t table_pitch;
  const int* lens;          // [n]
  Seqs s;
  void* o;                  // [rows, Hq, D]
  float* lse;               // [rows, Hq] or nullptr
  int Hq, Hk, G, D, pages, P, pshift, width;  // G: query heads of a kv head
  bool q_vec;               // rows of q are aligned to 16 bytes
  float scale;              // of the scores, times log2 e
  bool causal;
  int window;               // 0: none
  int cls;
  AttnPlan plan;
  Divisor by_heads, by_group, by_tiles;  // kv heads; G; tiles of a sequence of a dense batch
  float* part;              // workspace: outputs [2 * spare][Hk][part_rows][D], then maxima and sums [..][2]
};

struct AttnPlans {
  AttnPlan few, many;       // units 0: the class is empty.  fp32: all rows are in `few`
};
// window: 0 leaves at least as many pieces as any.
AttnPlans attn_plans(const int* cu, int n, int T, int G, int Hk, int D, int dtype, bool q8, int64_t max_keys, int window);
size_t attn_ws_bytes(const AttnPlans& pl, int Hk, int D);
hipError_t launch_attn(AttnParams p, const AttnPlans& pl, int dtype, bool q8, void* ws, hipStream_t st);

// One launch for the sequences of p.cls, by p.plan.
hipError_t launch_attn_few(const AttnParams& p, bool q8, hipStream_t st);
hipError_t launch_attn_many(const AttnParams& p, bool q8, hipStream_t st);
hipError_t launch_attn_f32(const AttnParams& p, bool q8, hipStream_t st);
hipError_t launch_attn_join(const AttnParams& p, int dtype, hipStream_t st);

}  // namespace gdn
