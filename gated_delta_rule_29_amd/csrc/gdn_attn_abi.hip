// gdn_attn_abi.hip -- the extern "C" boundary of a full-attention layer's operators (rotary positions, paged
// cache, attention): argument validation and dispatch.  The contract of every entry point is in
// include/gdn.h; errors as in gdn_abi.hip.
#include "../../include/gdn.h"
#include "gdn_attn.h"

using gdn::check_workspace;
using gdn::fail;
using gdn::hip_fail;
using gdn::ok;

namespace {

#define GDN_TRY(expr)          \
  do {                         \
    const int rc_ = (expr);    \
    if (rc_) return rc_;       \
  } while (0)

constexpr int64_t kMaxStride = int64_t{1} << 32;  // elements from token to token or head to head

int check_dtype(int dtype) {
  if (dtype != GDN_DTYPE_F32 && dtype != GDN_DTYPE_BF16)
    return fail(GDN_ERR_INVALID, "dtype must be GDN_DTYPE_F32 (0) or GDN_DTYPE_BF16 (1), got %d", dtype);
  return GDN_OK;
}

int check_heads(const char* name, const void* p, int64_t pitch, int64_t head, int D) {
  if (!p) return fail(GDN_ERR_INVALID, "%s must be a non-null device pointer", name);
  if (pitch < D || head < D)
    return fail(GDN_ERR_INVALID, "%s's pitches (%lld, %lld) are less than a head's %d columns", name, (long long)pitch,
                (long long)head, D);
  if (pitch > kMaxStride || head > kMaxStride)
    return fail(GDN_ERR_UNSUPPORTED, "%s's pitches (%lld, %lld) exceed 2^32", name, (long long)pitch, (long long)head);
  return GDN_OK;
}

int check_tokens(int T, int H, int D) {
  if (T <= 0 || H <= 0 || D <= 0) return fail(GDN_ERR_INVALID, "T, H and D must be positive (got %d, %d, %d)", T, H, D);
  if (T > GDN_MAX_TOKENS) return fail(GDN_ERR_INVALID, "T = %d exceeds %d", T, GDN_MAX_TOKENS);
  if (H > 4096) return fail(GDN_ERR_UNSUPPORTED, "H must be <= 4096, got %d", H);
  return GDN_OK;
}

int rope(const void* x, int64_t pitch, int64_t head, const int* pos, const uint64_t* table, float magnitude, void* y,
         int T, int H, int D, int R, int inter, int dtype, bool back, void* stream) {
  GDN_TRY(check_tokens(T, H, D));
  GDN_TRY(check_dtype(dtype));
  GDN_TRY(check_heads(back ? "dy" : "x", x, pitch, head, D));
  if (!pos || !table || !y)
    return fail(GDN_ERR_INVALID, "positions, table and the output must be non-null device pointers");
  if (D > 1024) return fail(GDN_ERR_UNSUPPORTED, "D must be <= 1024, got %d", D);
  if (R < 2 || R % 2 || R > D) return fail(GDN_ERR_INVALID, "R must be even and in 2 .. D = %d, got %d", D, R);
  // (a workgroup has 256 items, of one column each at the least)
  if ((int64_t)T * (((int64_t)H * D + 255) / 256) > gdn::kMaxGroups)
    return fail(GDN_ERR_INVALID, "%d tokens of %d heads of %d columns exceed the grid limit", T, H, D);
  const gdn::RopeParams p{{x, pitch, head}, pos, table, magnitude, y, T, H, D, R, inter != 0, back};
  const hipError_t e = gdn::launch_rope(p, dtype, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? ok() : hip_fail(e, back ? "rope_bwd launch" : "rope_fwd launch");
}

// A cache of `pages` pages; *q8: held in 8 bits.
int check_cache(const void* k, const void* v, const float* ks, const float* vs, int pages, int P, int H, int D,
                int dtype, int cache_dtype, bool* q8) {
  if (!k || !v) return fail(GDN_ERR_INVALID, "k_cache and v_cache must be non-null device pointers");
  GDN_TRY(check_dtype(dtype));
  *q8 = cache_dtype == GDN_DTYPE_E4M3;
  if (!*q8 && cache_dtype != dtype)
    return fail(GDN_ERR_INVALID, "the cache's dtype must be the activations' (%d) or GDN_DTYPE_E4M3 (2), got %d", dtype,
                cache_dtype);
  if (*q8 && (!ks || !vs)) return fail(GDN_ERR_INVALID, "an 8-bit cache needs k_scale and v_scale");
  if (!*q8 && (ks || vs)) return fail(GDN_ERR_INVALID, "k_scale and v_scale are of an 8-bit cache");
  if (pages <= 0 || H <= 0 || D <= 0)
    return fail(GDN_ERR_INVALID, "pages, heads and columns must be positive (got %d, %d, %d)", pages, H, D);
  if (P < 16 || P > 1024 || (P & (P - 1)))
    return fail(GDN_ERR_UNSUPPORTED, "a page must have 16, 32, .. 1024 places, got %d", P);
  if ((int64_t)pages * P > INT32_MAX)
    return fail(GDN_ERR_INVALID, "%d pages of %d places exceed 2^31 - 1", pages, P);
  return GDN_OK;
}

int check_rows(const gdn::CacheRowsParams& p) {
  GDN_TRY(check_tokens(p.T, p.c.H, p.c.D));
  if (!p.slots) return fail(GDN_ERR_INVALID, "slots must be a non-null device pointer");
  if (p.c.D > gdn::kCacheMaxD) return fail(GDN_ERR_UNSUPPORTED, "D must be <= %d, got %d", gdn::kCacheMaxD, p.c.D);
  if ((int64_t)p.T * p.c.H > gdn::kMaxGroups)
    return fail(GDN_ERR_INVALID, "%d tokens of %d heads exceed the grid limit", p.T, p.c.H);
  return GDN_OK;
}

struct Attn {
  const void* q;
  int64_t q_pitch, q_head;
  const void *k, *v;
  const float *ks, *vs;
  const int* table;
  int64_t table_pitch;
  int width;
  const int* lens;
  float scale;
  int causal, window;
  void* o;
  float* lse;
  int Hq, Hk, D, pages, P, dtype, cache_dtype;
};

int check_attn_sizes(int Hq, int Hk, int D, int P, int width, int dtype) {
  GDN_TRY(check_dtype(dtype));
  if (Hq <= 0 || Hk <= 0 || Hq % Hk)
    return fail(GDN_ERR_INVALID, "Hq must be a positive multiple of Hk (got %d, %d)", Hq, Hk);
  if (Hq > 4096) return fail(GDN_ERR_UNSUPPORTED, "Hq must be <= 4096, got %d", Hq);
  if (D != 64 && D != 128 && D != 256) return fail(GDN_ERR_UNSUPPORTED, "D must be 64, 128 or 256, got %d", D);
  if (P < 16 || P > 1024 || (P & (P - 1)))
    return fail(GDN_ERR_UNSUPPORTED, "a page must have 16, 32, .. 1024 places, got %d", P);
  if (width <= 0) return fail(GDN_ERR_INVALID, "block_table must have columns (got %d)", width);
  if ((int64_t)width * P > GDN_MAX_TOKENS)
    return fail(GDN_ERR_INVALID, "%d pages of %d places a sequence exceed %d", width, P, GDN_MAX_TOKENS);
  return GDN_OK;
}

// The most rows of a sequence and kv head.
int check_attn_rows(const gdn::Seqs& s, const int* cu_host, int G) {
  int64_t n = s.T;
  for (int i = 0; cu_host && i < s.n; ++i) n = n > cu_host[i + 1] - cu_host[i] ? n : cu_host[i + 1] - cu_host[i];
  if (n * G > GDN_MAX_TOKENS)
    return fail(GDN_ERR_INVALID, "%lld tokens of %d query heads a key head exceed %d", (long long)n, G, GDN_MAX_TOKENS);
  return GDN_OK;
}

gdn::AttnPlans plans(const gdn::Seqs& s, const int* cu_host, int Hq, int Hk, int D, int P, int width, int dtype,
                     int cache_dtype, int window) {
  return gdn::attn_plans(cu_host, s.n, s.T, Hq / Hk, Hk, D, dtype, cache_dtype == GDN_DTYPE_E4M3, (int64_t)width * P,
                         window);
}

bool odd16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 != 0; }

int attn(const gdn::Seqs& s, const int* cu_host, const Attn& a, void* ws, size_t ws_bytes, const char* what,
         void* stream) {
  bool q8;
  GDN_TRY(check_attn_sizes(a.Hq, a.Hk, a.D, a.P, a.width, a.dtype));
  GDN_TRY(check_cache(a.k, a.v, a.ks, a.vs, a.pages, a.P, a.Hk, a.D, a.dtype, a.cache_dtype, &q8));
  GDN_TRY(check_heads("q", a.q, a.q_pitch, a.q_head, a.D));
  if (!a.table || !a.lens || !a.o)
    return fail(GDN_ERR_INVALID, "block_table, seq_lens and o must be non-null device pointers");
  if (odd16(a.k) || odd16(a.v) || odd16(a.o))
    return fail(GDN_ERR_INVALID, "k_cache, v_cache and o must be 16-byte aligned");
  if (a.table_pitch < a.width)
    return fail(GDN_ERR_INVALID, "block_table's pitch %lld is less than its %d columns", (long long)a.table_pitch, a.width);
  if (a.table_pitch > kMaxStride) return fail(GDN_ERR_UNSUPPORTED, "block_table's pitch exceeds 2^32");
  if (!(a.scale > 0.f) || a.scale > 1e30f)
    return fail(GDN_ERR_INVALID, "scale must be positive and finite (got %g)", (double)a.scale);
  if (a.window < 0 || (a.window && !a.causal))
    return fail(GDN_ERR_INVALID, "window must be 0 or, in a causal call, positive (got %d)", a.window);
  GDN_TRY(check_attn_rows(s, cu_host, a.Hq / a.Hk));
  // A window of all keys that a sequence may have hides none; differences of positions and windows fit 32 bits.
  const int window = a.window >= (int64_t)a.width * a.P ? 0 : a.window;
  const gdn::AttnPlans pl = plans(s, cu_host, a.Hq, a.Hk, a.D, a.P, a.width, a.dtype, a.cache_dtype, window);
  // (512 threads a workgroup at most, and two workgroups for 256 columns)
  for (const gdn::AttnPlan& q : {pl.few, pl.many})
    if (((int64_t)q.units + q.spare) * a.Hk > gdn::kMaxGroups / 4 ||
        (int64_t)q.spare * a.Hk * q.part_rows > gdn::kMaxGroups)
      return fail(GDN_ERR_INVALID, "%s of these sizes exceeds the grid limit", what);
  GDN_TRY(check_workspace(ws, ws_bytes, gdn::attn_ws_bytes(pl, a.Hk, a.D)));
  gdn::AttnParams p{};
  p.q = {a.q, a.q_pitch, a.q_head};
  p.k = a.k; p.v = a.v; p.ks = a.ks; p.vs = a.vs;
  p.table = a.table; p.table_pitch = a.table_pitch; p.width = a.width; p.lens = a.lens;
  p.s = s; p.o = a.o; p.lse = a.lse;
  p.Hq = a.Hq; p.Hk = a.Hk; p.G = a.Hq / a.Hk; p.D = a.D; p.pages = a.pages; p.P = a.P;
  p.pshift = __builtin_ctz((unsigned)a.P);
  p.q_vec = !odd16(a.q) && a.q_pitch % 8 == 0 && a.q_head % 8 == 0;
  p.scale = a.scale * 1.4426950408889634f;
  p.causal = a.causal != 0;
  p.window = window;
  const hipError_t e = gdn::launch_attn(p, pl, a.dtype, q8, ws, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? ok() : hip_fail(e, what);
}

int dense(int B, int T, gdn::Seqs* s) {
  if (B <= 0 || T <= 0) return fail(GDN_ERR_INVALID, "B and T must be positive (got %d, %d)", B, T);
  if ((int64_t)B * T > GDN_MAX_TOKENS)
    return fail(GDN_ERR_INVALID, "B*T = %lld exceeds %d", (long long)B * T, GDN_MAX_TOKENS);
  *s = gdn::Seqs{nullptr, B, T, B * T};
  return GDN_OK;
}

int packed(const int* cu, const int* cu_host, int N, int T_total, gdn::Seqs* s) {
  if (!cu || !cu_host) return fail(GDN_ERR_INVALID, "cu_seqlens (device) and cu_seqlens_host must be non-null");
  if (N < 1 || T_total < 1) return fail(GDN_ERR_INVALID, "N and T_total must be positive (got %d, %d)", N, T_total);
  if (T_total > GDN_MAX_TOKENS) return fail(GDN_ERR_INVALID, "T_total = %d exceeds %d", T_total, GDN_MAX_TOKENS);
  if (cu_host[0] != 0) return fail(GDN_ERR_INVALID, "cu_seqlens[0] must be 0 (got %d)", cu_host[0]);
  for (int i = 0; i < N; ++i)
    if (cu_host[i + 1] <= cu_host[i])
      return fail(GDN_ERR_INVALID, "cu_seqlens must be strictly increasing (sequence %d is empty or negative)", i);
  if (cu_host[N] != T_total)
    return fail(GDN_ERR_INVALID, "cu_seqlens[N] = %d differs from T_total = %d", cu_host[N], T_total);
  *s = gdn::Seqs{cu, N, 0, T_total};
  return GDN_OK;
}

}  // namespace

extern "C" {

int rope_fwd(const void* x, int64_t x_pitch, int64_t x_head, const int* positions, const uint64_t* table,
             float magnitude, void* y, int T, int H, int D, int R, int interleaved, int dtype, void* stream) {
  return rope(x, x_pitch, x_head, positions, table, magnitude, y, T, H, D, R, interleaved, dtype, false, stream);
}

int rope_bwd(const void* dy, int64_t dy_pitch, int64_t dy_head, const int* positions, const uint64_t* table,
             float magnitude, void* dx, int T, int H, int D, int R, int interleaved, int dtype, void* stream) {
  return rope(dy, dy_pitch, dy_head, positions, table, magnitude, dx, T, H, D, R, interleaved, dtype, true, stream);
}

int kv_cache_write(const void* k, int64_t k_pitch, int64_t k_head, const void* v, int64_t v_pitch, int64_t v_head,
                   const int* slots, void* k_cache, void* v_cache, float* k_scale, float* v_scale, int T, int pages,
                   int P, int H, int D, int dtype, int cache_dtype, void* stream) {
  bool q8;
  GDN_TRY(check_cache(k_cache, v_cache, k_scale, v_scale, pages, P, H, D, dtype, cache_dtype, &q8));
  GDN_TRY(check_heads("k", k, k_pitch, k_head, D));
  GDN_TRY(check_heads("v", v, v_pitch, v_head, D));
  const gdn::CacheRowsParams p{{k_cache, v_cache, k_scale, v_scale, pages, P, H, D},
                               {k, k_pitch, k_head}, {v, v_pitch, v_head}, nullptr, nullptr, slots, T};
  GDN_TRY(check_rows(p));
  const hipError_t e = gdn::launch_cache_write(p, dtype, q8, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "kv_cache_write launch");
}

int kv_cache_read(const void* k_cache, const void* v_cache, const float* k_scale, const float* v_scale,
                  const int* slots, void* k, void* v, int T, int pages, int P, int H, int D, int dtype,
                  int cache_dtype, void* stream) {
  bool q8;
  GDN_TRY(check_cache(k_cache, v_cache, k_scale, v_scale, pages, P, H, D, dtype, cache_dtype, &q8));
  if (!k || !v) return fail(GDN_ERR_INVALID, "k and v must be non-null device pointers");
  const gdn::CacheRowsParams p{{const_cast<void*>(k_cache), const_cast<void*>(v_cache), const_cast<float*>(k_scale),
                                const_cast<float*>(v_scale), pages, P, H, D},
                               {nullptr, 0, 0}, {nullptr, 0, 0}, k, v, slots, T};
  GDN_TRY(check_rows(p));
  const hipError_t e = gdn::launch_cache_read(p, dtype, q8, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "kv_cache_read launch");
}

size_t paged_attn_workspace_bytes(int B, int T, int Hq, int Hk, int D, int P, int max_pages, int dtype,
                                  int cache_dtype) {
  gdn::Seqs s;
  if (dense(B, T, &s) || check_attn_sizes(Hq, Hk, D, P, max_pages, dtype) || check_attn_rows(s, nullptr, Hq / Hk)) return 0;
  return gdn::attn_ws_bytes(plans(s, nullptr, Hq, Hk, D, P, max_pages, dtype, cache_dtype, 0), Hk, D);
}

size_t paged_attn_varlen_workspace_bytes(const int* cu_seqlens_host, int N, int Hq, int Hk, int D, int P,
                                         int max_pages, int dtype, int cache_dtype) {
  gdn::Seqs s;
  if (!cu_seqlens_host || N < 1 || packed(cu_seqlens_host, cu_seqlens_host, N, cu_seqlens_host[N], &s) ||
      check_attn_sizes(Hq, Hk, D, P, max_pages, dtype) || check_attn_rows(s, cu_seqlens_host, Hq / Hk))
    return 0;
  return gdn::attn_ws_bytes(plans(s, cu_seqlens_host, Hq, Hk, D, P, max_pages, dtype, cache_dtype, 0), Hk, D);
}

int paged_attn_fwd(const void* q, int64_t q_pitch, int64_t q_head, const void* k_cache, const void* v_cache,
                   const float* k_scale, const float* v_scale, const int* block_table, int64_t table_pitch,
                   int max_pages, const int* seq_lens, float scale, int causal, int window, void* o, float* lse, int B,
                   int T, int Hq, int Hk, int D, int pages, int P, int dtype, int cache_dtype, void* workspace,
                   size_t workspace_bytes, void* stream) {
  gdn::Seqs s;
  GDN_TRY(dense(B, T, &s));
  const Attn a{q, q_pitch, q_head, k_cache, v_cache, k_scale, v_scale, block_table, table_pitch, max_pages, seq_lens,
               scale, causal, window, o, lse, Hq, Hk, D, pages, P, dtype, cache_dtype};
  return attn(s, nullptr, a, workspace, workspace_bytes, "paged_attn_fwd", stream);
}

int paged_attn_fwd_varlen(const void* q, int64_t q_pitch, int64_t q_head, const void* k_cache, const void* v_cache,
                          const float* k_scale, const float* v_scale, const int* block_table, int64_t table_pitch,
                          int max_pages, const int* seq_lens, const int* cu_seqlens, const int* cu_seqlens_host, int N,
                          float scale, int causal, int window, void* o, float* lse, int T_total, int Hq, int Hk, int D,
                          int pages, int P, int dtype, int cache_dtype, void* workspace, size_t workspace_bytes,
                          void* stream) {
  gdn::Seqs s;
  GDN_TRY(packed(cu_seqlens, cu_seqlens_host, N, T_total, &s));
  const Attn a{q, q_pitch, q_head, k_cache, v_cache, k_scale, v_scale, block_table, table_pitch, max_pages, seq_lens,
               scale, causal, window, o, lse, Hq, Hk, D, pages, P, dtype, cache_dtype};
  return attn(s, cu_seqlens_host, a, workspace, workspace_bytes, "paged_attn_fwd_varlen", stream);
}

int paged_attn_step(const void* q, int64_t q_pitch, int64_t q_head, const void* k_cache, const void* v_cache,
                    const float* k_scale, const float* v_scale, const int* block_table, int64_t table_pitch,
                    int max_pages, const int* seq_lens, float scale, int window, void* o, int B, int Hq, int Hk, int D,
                    int pages, int P, int dtype, int cache_dtype, void* workspace, size_t workspace_bytes,
                    void* stream) {
  gdn::Seqs s;
  GDN_TRY(dense(B, 1, &s));
  const Attn a{q, q_pitch, q_head, k_cache, v_cache, k_scale, v_scale, block_table, table_pitch, max_pages, seq_lens,
               scale, 1, window, o, nullptr, Hq, Hk, D, pages, P, dtype, cache_dtype};
  return attn(s, nullptr, a, workspace, workspace_bytes, "paged_attn_step", stream);
}

}  // extern "C"
