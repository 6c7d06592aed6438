// gdn_attn_plan.hip -- how a call of the attention is cut into tiles of rows and pieces of keys, and the
// kernel that joins the pieces.
#include "../../include/gdn.h"
#include "gdn_attn_device.h"

namespace gdn {

namespace {

// Rows of units whose keys were cut, joined from their pieces: out = sum_i w_i o_i / sum_i w_i l_i with
// w_i = 2^{m_i - max m}, with a running maximum.  RPW rows at a time, 256 / RPW threads each: D / 4 columns of
// four times groups that take every so-many-th piece, joined in LDS in a fixed order.  A workgroup takes `rows`
// rows of a unit: most workgroups of a call that cuts little find nothing to do, so they are few.
template <typename T, int D, int RPW>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnParams p, Divisor per_unit, int rows) {
  constexpr int TEAM = 256 / RPW, LP = D / 4, GR = TEAM / LP;
  __shared__ float acc[RPW][GR][D + 2];
  const int lane = threadIdx.x & 63;
  const int sub = threadIdx.x / TEAM, tid = threadIdx.x % TEAM, g = tid / LP, c = (tid % LP) * 4;
  const int rest = quotient(blockIdx.x, p.by_heads), h = blockIdx.x - rest * p.Hk, id = quotient(rest, per_unit);
  Unit u;
  if (!find_unit<false>(p, id, lane, &u)) return;
  const int pieces = u.pieces;
  const int64_t step = (int64_t)u.apart * p.Hk * p.plan.part_rows;  // rows from piece to piece
  const int first = (rest - id * (int)per_unit.by) * rows, end = min(first + rows, u.nrows);
  for (int at0 = first; at0 < end; at0 += RPW) {
    const int at = at0 + sub;
    const float* part = part_outputs(p, u.slot, h) + (int64_t)at * D + c;
    const float* ml = part_sums(p, u.slot, h) + 2 * at;
    float top = -__builtin_inff(), l = 0.f;
    float r[4] = {0.f, 0.f, 0.f, 0.f};
    if (at < end) {
#pragma unroll 4
      for (int i = g; i < pieces; i += GR) {
        float x[4], s[2];
        loadv<float, 4>(part + i * step * D, x);
        loadv<float, 2>(ml + 2 * i * step, s);
        const float now = fmaxf(top, s[0]), a = part_weight(top, now), w = part_weight(s[0], now);
        top = now;
        l = l * a + w * s[1];
#pragma unroll
        for (int e = 0; e < 4; ++e) r[e] = r[e] * a + w * x[e];
      }
    }
    __syncthreads();  // the last rows' readers are done
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[sub][g][c + e] = r[e];
    if (c == 0) {
      acc[sub][g][D] = top;
      acc[sub][g][D + 1] = l;
    }
    __syncthreads();
    if (at >= end || g) continue;
    float all = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < GR; ++i) all = fmaxf(all, acc[sub][i][D]);
    l = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) r[e] = 0.f;
#pragma unroll
    for (int i = 0; i < GR; ++i) {
      const float w = part_weight(acc[sub][i][D], all);
      l += w * acc[sub][i][D + 1];
#pragma unroll
      for (int e = 0; e < 4; ++e) r[e] += w * acc[sub][i][c + e];
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int e = 0; e < 4; ++e) r[e] *= inv;
    const int64_t row = out_row(p, u, h, u.row0 + at);
    storev<T, 4>(static_cast<T*>(p.o) + row * D + c, r);
    if (p.lse && c == 0) p.lse[row] = row_lse(all, l);
  }
}

template <typename T, int D>
hipError_t launch_join(const AttnParams& p, hipStream_t st) {
  // one row a workgroup where rows are few and pieces many
  const bool few = p.plan.part_rows <= kFewRows;
  constexpr int RPW = 1024 / D;  // rows at a time, a group of threads each
  const int rows = few ? 1 : 2 * RPW, per_unit = (p.plan.part_rows + rows - 1) / rows;
  // (there are at most `spare` cut units)
  const int64_t groups = (int64_t)(p.plan.units < p.plan.spare ? p.plan.units : p.plan.spare) * p.Hk * per_unit;
  if (groups > kMaxGroups) return hipErrorInvalidConfiguration;
  if (few) attn_join_kernel<T, D, 1><<<dim3((unsigned)groups), 256, 0, st>>>(p, divisor(per_unit), rows);
  else attn_join_kernel<T, D, RPW><<<dim3((unsigned)groups), 256, 0, st>>>(p, divisor(per_unit), rows);
  return hipGetLastError();
}
template <typename T>
hipError_t join_width(const AttnParams& p, hipStream_t st) {
  return p.D == 64 ? launch_join<T, 64>(p, st) : (p.D == 128 ? launch_join<T, 128>(p, st) : launch_join<T, 256>(p, st));
}

// Pieces beyond one a unit, so that a piece has about a `fill`-th of all keys of all heads' units.  least: tiles of
// the sequence that has the fewest; if they are as many as the pieces, none is long enough to be cut.  (A call that
// cuts nothing has no join to launch, 5 to 9 us.)
int spare_pieces(const AttnPlan& pl, int Hk, int64_t max_keys, int window, int fill, int64_t least) {
  if (window && max_keys > (int64_t)window + pl.rows + 64) max_keys = (int64_t)window + pl.rows + 64;
  if (!pl.units || 2 * max_keys < 3 * pl.min_piece) return 0;
  const int spare = (fill + Hk - 1) / Hk;
  return least >= spare ? 0 : spare;
}

}  // namespace

AttnPlans attn_plans(const int* cu, int n, int T, int G, int Hk, int D, int dtype, bool q8, int64_t max_keys,
                     int window) {
  AttnPlans a{};
  const bool f32 = dtype == GDN_DTYPE_F32;
  const int64_t few_limit = f32 ? INT64_MAX : kFewRows;
  const int many = many_rows(D, q8);
  // (a dense batch's sequences are alike: the first stands for all)
  const int seqs = cu ? n : 1, times = cu ? 1 : n;
  const auto rows_of = [&](int i) { return (int64_t)(cu ? cu[i + 1] - cu[i] : T) * G; };
  int64_t most_few = 0, units_many = 0, most_many = 0, least_many = INT64_MAX;
  for (int i = 0; i < seqs; ++i) {
    const int64_t rows = rows_of(i);
    if (rows <= few_limit) {
      if (rows > most_few) most_few = rows;
    } else {
      const int64_t tiles = (rows + many - 1) / many;
      units_many += tiles * times;
      if (rows > most_many) most_many = rows;
      if (tiles < least_many) least_many = tiles;
    }
  }
  // 32-row tiles of 256 columns would not fit into registers
  a.few.row_bits = most_few <= 16 || D == 256 ? 4 : 5;
  a.few.rows = 1 << a.few.row_bits;
  int64_t units_few = 0, least_few = INT64_MAX;
  for (int i = 0; most_few && i < seqs; ++i) {
    const int64_t rows = rows_of(i);
    if (rows > few_limit) continue;
    const int64_t tiles = (rows + a.few.rows - 1) / a.few.rows;
    units_few += tiles * times;
    if (tiles < least_few) least_few = tiles;
  }
  const int64_t most = INT32_MAX / 2;
  a.few.units = (int)(units_few < most ? units_few : most);
  a.few.part_rows = (int)(most_few < a.few.rows ? most_few : a.few.rows);
  // Pieces fill the chip once or twice.  Few rows, 256 / 512 / 1024 / 2048 pieces: one token after 131071 98 / 101 / 111 /
  // 131 us, the same over 8 bits 58 / 52 / 59; 32 tokens after 0 .. 18600 241 / 227 / 221, over 8 bits 157 / 135 / 131;
  // of 256 columns, 8 bits, 69 / 74 / 91.  Shortest piece 256 / 512 / 1024 keys: one token after 8191 18 / 16 / 20.
  // Many rows, 256 / 384 / 512 pieces: 256 tokens after 32768 161 / 193 / 178, 2048 after 6000 235 / 241 / 305, 9 chunks
  // of a serving step 122 / 114 / 123: pieces that are no whole number of rounds, and 128 KB written and read a
  // piece, cost more than what they even out.
  a.few.min_piece = 512;
  a.few.spare = spare_pieces(a.few, Hk, max_keys, window, 512, least_few);
  a.many.rows = many;
  a.many.row_bits = __builtin_ctz((unsigned)many);
  a.many.units = (int)(units_many < most ? units_many : most);
  a.many.part_rows = (int)(most_many < many ? most_many : many);
  a.many.min_piece = 1024;
  a.many.spare = spare_pieces(a.many, Hk, max_keys, window, 256, least_many);
  return a;
}

static size_t part_bytes(const AttnPlan& pl, int Hk, int D) {
  if (!pl.units || !pl.spare) return 0;
  const size_t n = 2 * (size_t)pl.spare * Hk * pl.part_rows * (D + 2) * sizeof(float);
  return (n + 255) & ~size_t{255};
}
size_t attn_ws_bytes(const AttnPlans& pl, int Hk, int D) { return part_bytes(pl.few, Hk, D) + part_bytes(pl.many, Hk, D); }

hipError_t launch_attn_join(const AttnParams& p, int dtype, hipStream_t st) {
  return dtype == GDN_DTYPE_BF16 ? join_width<bf16>(p, st) : join_width<float>(p, st);
}

hipError_t launch_attn(AttnParams p, const AttnPlans& pl, int dtype, bool q8, void* ws, hipStream_t st) {
  char* at = static_cast<char*>(ws);
  p.by_heads = divisor((uint32_t)p.Hk);
  p.by_group = divisor((uint32_t)p.G);
  for (int many = 1; many >= 0; --many) {  // the class with more work goes first
    p.plan = many ? pl.many : pl.few;
    if (!p.plan.units) continue;
    // (T is 0 in a packed batch, whose tiles are looked for)
    p.by_tiles = divisor(p.s.cu ? 1u : (uint32_t)(((int64_t)p.s.T * p.G + p.plan.rows - 1) >> p.plan.row_bits));
    p.cls = dtype == GDN_DTYPE_F32 || !(many ? pl.few : pl.many).units ? kAllRows : (many ? kMany : kFew);
    p.part = reinterpret_cast<float*>(at);
    at += part_bytes(p.plan, p.Hk, p.D);
    hipError_t e = dtype == GDN_DTYPE_F32 ? launch_attn_f32(p, q8, st)
                                          : (many ? launch_attn_many(p, q8, st) : launch_attn_few(p, q8, st));
    if (e == hipSuccess && p.plan.spare) e = launch_attn_join(p, dtype, st);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace gdn
