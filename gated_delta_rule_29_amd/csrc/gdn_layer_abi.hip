// gdn_layer_abi.hip -- the extern "C" boundary of the layer operators (short causal convolution,
// selective scan, residual RMS norm): argument validation and dispatch.  The contract of every
// entry point is in include/gdn.h; errors as in gdn_abi.hip.
#include "../../include/gdn.h"
#include "gdn_layer.h"

using gdn::check_workspace;
using gdn::fail;
using gdn::hip_fail;
using gdn::ok;

namespace {

static_assert(GDN_SSM_CHUNK == gdn::kSsmChunk, "the header's chunk is the kernels'");

int check_dtype(int dtype) {
  if (dtype != GDN_DTYPE_F32 && dtype != GDN_DTYPE_BF16)
    return fail(GDN_ERR_INVALID, "dtype must be GDN_DTYPE_F32 (0) or GDN_DTYPE_BF16 (1), got %d", dtype);
  return GDN_OK;
}

int check_pitch(const char* name, const void* p, int64_t pitch, int width) {
  if (p && pitch < width)
    return fail(GDN_ERR_INVALID, "%s's pitch %lld is less than its row of %d", name, (long long)pitch, width);
  if (p && pitch > GDN_MAX_PITCH)
    return fail(GDN_ERR_UNSUPPORTED, "%s's pitch %lld exceeds %d", name, (long long)pitch, GDN_MAX_PITCH);
  return GDN_OK;
}

int check_state(const char* name, const void* p, int N) {
  if (N % 4 == 0 && reinterpret_cast<uintptr_t>(p) % 16)
    return fail(GDN_ERR_INVALID, "%s must be 16-byte aligned", name);
  return GDN_OK;
}

#define GDN_TRY(expr)          \
  do {                         \
    const int rc_ = (expr);    \
    if (rc_) return rc_;       \
  } while (0)

// The sequences of a dense call.
int dense_seqs(int B, int T, gdn::Seqs* s) {
  if (B <= 0 || T <= 0) return fail(GDN_ERR_INVALID, "B and T must be positive (got %d, %d)", B, T);
  if ((int64_t)B * T > GDN_MAX_TOKENS)
    return fail(GDN_ERR_INVALID, "B*T = %lld exceeds %d", (long long)B * T, GDN_MAX_TOKENS);
  *s = gdn::Seqs{nullptr, B, T, B * T};
  return GDN_OK;
}

// The sequences of a packed call, from the host offsets.
int packed_seqs(const int* cu, const int* cu_host, int N, int T_total, gdn::Seqs* s) {
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

// ------------------------------------------------------------------------------- convolution

int check_conv(const void* x, int64_t pitch, const float* w, int D, int W, int dtype) {
  if (!x || !w) return fail(GDN_ERR_INVALID, "x and w must be non-null device pointers");
  GDN_TRY(check_dtype(dtype));
  if (D <= 0 || W <= 0) return fail(GDN_ERR_INVALID, "D and W must be positive (got %d, %d)", D, W);
  if (W < 2 || W > 4) return fail(GDN_ERR_UNSUPPORTED, "W must be 2, 3 or 4, got %d", W);
  return check_pitch("x", x, pitch, D);
}

int check_grid(int64_t groups, const char* what) {
  if (groups > gdn::kMaxGroups)
    return fail(GDN_ERR_INVALID, "%s of these sizes exceeds the grid limit", what);
  return GDN_OK;
}

// One thread a channel and 32 tokens in the smallest instance (fewer tokens in small calls only).
int check_conv_grid(const gdn::Seqs& s, int D, const char* what) {
  return check_grid(((int64_t)((s.rows + 31) / 32) * D + 255) / 256, what);
}

int conv_fwd(const gdn::Seqs& s, const void* x, int64_t x_pitch, const float* w, const float* bias,
             const void* init, void* y, void* last, int D, int W, int silu, int dtype, void* stream) {
  GDN_TRY(check_conv(x, x_pitch, w, D, W, dtype));
  if (!y) return fail(GDN_ERR_INVALID, "y must be a non-null device pointer");
  GDN_TRY(check_conv_grid(s, D, "causal_conv_fwd"));
  const gdn::ConvParams p{x, x_pitch, w, bias, init, y, last, s, D, W, silu != 0};
  const hipError_t e = gdn::launch_conv_fwd(p, dtype, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "causal_conv_fwd launch");
}

int conv_bwd(const gdn::Seqs& s, const void* dy, int64_t dy_pitch, const void* x, int64_t x_pitch,
             const float* w, const float* bias, const void* init, const void* dlast, void* dx,
             void* dinit, float* dw, float* dbias, int D, int W, int silu, int dtype, void* ws,
             size_t ws_bytes, void* stream) {
  GDN_TRY(check_conv(x, x_pitch, w, D, W, dtype));
  if (!dy || !dx || !dw) return fail(GDN_ERR_INVALID, "dy, dx and dw must be non-null device pointers");
  GDN_TRY(check_pitch("dy", dy, dy_pitch, D));
  GDN_TRY(check_conv_grid(s, D, "causal_conv_bwd"));
  GDN_TRY(check_workspace(ws, ws_bytes, gdn::conv_bwd_ws_bytes(s.rows, D, W)));
  gdn::ConvBwdParams p{};
  p.f = gdn::ConvParams{x, x_pitch, w, bias, init, nullptr, nullptr, s, D, W, silu != 0};
  p.dy = dy; p.dy_pitch = dy_pitch; p.dlast = dlast; p.dx = dx; p.dinit = dinit; p.dw = dw;
  p.dbias = dbias; p.part = static_cast<float*>(ws);
  const hipError_t e = gdn::launch_conv_bwd(p, dtype, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "causal_conv_bwd launch");
}

// -------------------------------------------------------------------------------------- scan

struct Scan {
  const void *x, *dt, *z, *Bm, *Cm;
  int64_t x_pitch, dt_pitch, z_pitch, b_pitch, c_pitch;
  const float *A, *skip, *dt_bias;
};

int check_scan(const Scan& a, int D, int N, int dtype) {
  if (!a.x || !a.dt || !a.A || !a.Bm || !a.Cm)
    return fail(GDN_ERR_INVALID, "x, dt, A, Bm and Cm must be non-null device pointers");
  GDN_TRY(check_dtype(dtype));
  if (D <= 0 || N <= 0) return fail(GDN_ERR_INVALID, "D and N must be positive (got %d, %d)", D, N);
  if (N > gdn::kSsmMaxN) return fail(GDN_ERR_UNSUPPORTED, "N must be <= %d, got %d", gdn::kSsmMaxN, N);
  GDN_TRY(check_pitch("x", a.x, a.x_pitch, D));
  GDN_TRY(check_pitch("dt", a.dt, a.dt_pitch, D));
  GDN_TRY(check_pitch("z", a.z, a.z_pitch, D));
  GDN_TRY(check_pitch("Bm", a.Bm, a.b_pitch, N));
  GDN_TRY(check_state("A", a.A, N));
  return check_pitch("Cm", a.Cm, a.c_pitch, N);
}

using Split = gdn::SsmSplit;

Split dense_split(bool bwd, int B, int T, int D, int N) { return gdn::ssm_split(bwd, nullptr, B, T, D, N); }
Split packed_split(bool bwd, const int* cu, int n, int D, int N) { return gdn::ssm_split(bwd, cu, n, 0, D, N); }

// Whether the offsets can be sized at all (the calls check them in full).
bool sizable(const int* cu, int n, int D, int N) {
  if (!cu || n < 1 || D <= 0 || N <= 0 || N > gdn::kSsmMaxN || cu[0] != 0) return false;
  for (int i = 0; i < n; ++i)
    if (cu[i + 1] <= cu[i]) return false;
  return cu[n] <= GDN_MAX_TOKENS;
}

gdn::SsmParams scan_params(const gdn::Seqs& s, const Split& sp, const int* cu_host, const Scan& a, int D, int N,
                           int softplus) {
  gdn::SsmParams p{};
  p.x = a.x; p.dt = a.dt; p.z = a.z; p.Bm = a.Bm; p.Cm = a.Cm;
  p.x_pitch = a.x_pitch; p.dt_pitch = a.dt_pitch; p.z_pitch = a.z_pitch;
  p.b_pitch = a.b_pitch; p.c_pitch = a.c_pitch;
  p.A = a.A; p.skip = a.skip; p.dt_bias = a.dt_bias;
  p.s = s; p.D = D; p.N = N; p.softplus = softplus != 0; p.split = sp;
  p.chunks = cu_host ? ssm_scan_num_chunks(cu_host, s.n) : (int64_t)s.n * ((s.T + GDN_SSM_CHUNK - 1) / GDN_SSM_CHUNK);
  return p;
}

// (The joins, of 256 states a workgroup, run where sequences times channels are few.)
int check_scan_grid(const Split& sp, int D, int N) {
  const int ch = gdn::ssm_channels(N);
  return check_grid((int64_t)sp.nseg * ((D + ch - 1) / ch), "ssm_scan");
}

int scan_fwd(const gdn::Seqs& s, const Split& sp, const int* cu_host, const Scan& a, const float* h0, void* y, float* ht,
             float* h, int D, int N, int softplus, int dtype, void* ws, size_t ws_bytes, void* stream) {
  if (!y) return fail(GDN_ERR_INVALID, "y must be a non-null device pointer");
  GDN_TRY(check_state("h0", h0, N));
  GDN_TRY(check_state("ht", ht, N));
  GDN_TRY(check_state("h", h, N));
  GDN_TRY(check_scan_grid(sp, D, N));
  GDN_TRY(check_workspace(ws, ws_bytes, gdn::ssm_fwd_ws_bytes(sp, s.n, D, N)));
  gdn::SsmParams p = scan_params(s, sp, cu_host, a, D, N, softplus);
  p.h0 = h0; p.y = y; p.ht = ht; p.h = h;
  const hipError_t e = gdn::launch_ssm_fwd(p, dtype, ws, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "ssm_scan_fwd launch");
}

struct ScanGrads {
  void *dx, *ddt, *dBm, *dCm, *dz;
  float *dA, *dskip, *ddt_bias, *dh0;
};

int scan_bwd(const gdn::Seqs& s, const Split& sp, const int* cu_host, const Scan& a, const void* dy, int64_t dy_pitch,
             const float* h, const float* dht, const ScanGrads& o, int D, int N, int softplus, int dtype,
             void* ws, size_t ws_bytes, void* stream) {
  if (!dy || !h) return fail(GDN_ERR_INVALID, "dy and h must be non-null device pointers");
  if (!o.dx || !o.ddt || !o.dA || !o.dBm || !o.dCm)
    return fail(GDN_ERR_INVALID, "dx, ddt, dA, dBm and dCm must be non-null device pointers");
  if ((a.z != nullptr) != (o.dz != nullptr)) return fail(GDN_ERR_INVALID, "dz is given if and only if z is");
  GDN_TRY(check_pitch("dy", dy, dy_pitch, D));
  GDN_TRY(check_state("h", h, N));
  GDN_TRY(check_state("dht", dht, N));
  GDN_TRY(check_state("dh0", o.dh0, N));
  GDN_TRY(check_scan_grid(sp, D, N));
  GDN_TRY(check_workspace(ws, ws_bytes, gdn::ssm_bwd_ws_bytes(sp, s.rows, D, N)));
  gdn::SsmBwdParams p{};
  p.f = scan_params(s, sp, cu_host, a, D, N, softplus);
  p.f.h = const_cast<float*>(h);
  p.dy = dy; p.dy_pitch = dy_pitch; p.dht = dht;
  p.dx = o.dx; p.ddt = o.ddt; p.dz = o.dz; p.dB = o.dBm; p.dC = o.dCm;
  p.dA = o.dA; p.dskip = o.dskip; p.ddt_bias = o.ddt_bias; p.dh0 = o.dh0;
  const hipError_t e = gdn::launch_ssm_bwd(p, dtype, ws, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "ssm_scan_bwd launch");
}

// ch: channels of a workgroup in a large call's smallest instance.
int check_step(int B, int S, const int* slots, int D, int ch) {
  if (B <= 0 || S <= 0) return fail(GDN_ERR_INVALID, "B and S must be positive (got %d, %d)", B, S);
  if (!slots && S < B) return fail(GDN_ERR_INVALID, "without slots the cache needs a slot a row (S = %d, B = %d)", S, B);
  return check_grid((int64_t)B * ((D + ch - 1) / ch), "a step");
}

// -------------------------------------------------------------------------------------- norm

int check_norm(const void* x, int64_t x_pitch, const void* residual, int64_t r_pitch, const float* w, float eps,
               int M, int D, int dtype, int rdtype) {
  if (!x || !w) return fail(GDN_ERR_INVALID, "x and w must be non-null device pointers");
  GDN_TRY(check_dtype(dtype));
  GDN_TRY(check_dtype(rdtype));
  if (dtype == GDN_DTYPE_F32 && rdtype != GDN_DTYPE_F32)
    return fail(GDN_ERR_UNSUPPORTED, "fp32 activations with a bf16 residual");
  if (M <= 0 || D <= 0) return fail(GDN_ERR_INVALID, "M and D must be positive (got %d, %d)", M, D);
  if (M > GDN_MAX_TOKENS) return fail(GDN_ERR_INVALID, "M = %d exceeds %d", M, GDN_MAX_TOKENS);
  if (D > gdn::kNormMaxD) return fail(GDN_ERR_UNSUPPORTED, "D must be <= %d, got %d", gdn::kNormMaxD, D);
  if (!(eps > 0.f)) return fail(GDN_ERR_INVALID, "eps must be positive (got %g)", (double)eps);
  GDN_TRY(check_pitch("x", x, x_pitch, D));
  return check_pitch("residual", residual, r_pitch, D);
}

int norm_fwd(gdn::NormParams p, int dtype, int rdtype, const char* what, void* stream) {
  GDN_TRY(check_norm(p.x, p.x_pitch, p.residual, p.r_pitch, p.w, p.eps, p.M, p.D, dtype, rdtype));
  if (!p.y) return fail(GDN_ERR_INVALID, "the output must be a non-null device pointer");
  if (p.sum && !p.residual) return fail(GDN_ERR_INVALID, "sum is written with a residual only");
  const hipError_t e = gdn::launch_norm_fwd(p, dtype, rdtype, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? ok() : hip_fail(e, what);
}

}  // namespace

extern "C" {

int causal_conv_fwd(const void* x, int64_t x_pitch, const float* w, const float* bias, const void* init, void* y,
                    void* last, int B, int T, int D, int W, int silu, int dtype, void* stream) {
  gdn::Seqs s;
  GDN_TRY(dense_seqs(B, T, &s));
  return conv_fwd(s, x, x_pitch, w, bias, init, y, last, D, W, silu, dtype, stream);
}

int causal_conv_fwd_varlen(const void* x, int64_t x_pitch, const float* w, const float* bias, const int* cu_seqlens,
                           const int* cu_seqlens_host, int N, const void* init, void* y, void* last, int T_total,
                           int D, int W, int silu, int dtype, void* stream) {
  gdn::Seqs s;
  GDN_TRY(packed_seqs(cu_seqlens, cu_seqlens_host, N, T_total, &s));
  return conv_fwd(s, x, x_pitch, w, bias, init, y, last, D, W, silu, dtype, stream);
}

size_t causal_conv_bwd_workspace_bytes(int T_total, int D, int W) {
  if (T_total <= 0 || D <= 0 || W < 2 || W > 4) return 0;
  return gdn::conv_bwd_ws_bytes(T_total, D, W);
}

int causal_conv_bwd(const void* dy, int64_t dy_pitch, const void* x, int64_t x_pitch, const float* w,
                    const float* bias, const void* init, const void* dlast, void* dx, void* dinit, float* dw,
                    float* dbias, int B, int T, int D, int W, int silu, int dtype, void* workspace,
                    size_t workspace_bytes, void* stream) {
  gdn::Seqs s;
  GDN_TRY(dense_seqs(B, T, &s));
  return conv_bwd(s, dy, dy_pitch, x, x_pitch, w, bias, init, dlast, dx, dinit, dw, dbias, D, W, silu, dtype,
                  workspace, workspace_bytes, stream);
}

int causal_conv_bwd_varlen(const void* dy, int64_t dy_pitch, const void* x, int64_t x_pitch, const float* w,
                           const float* bias, const int* cu_seqlens, const int* cu_seqlens_host, int N,
                           const void* init, const void* dlast, void* dx, void* dinit, float* dw, float* dbias,
                           int T_total, int D, int W, int silu, int dtype, void* workspace, size_t workspace_bytes,
                           void* stream) {
  gdn::Seqs s;
  GDN_TRY(packed_seqs(cu_seqlens, cu_seqlens_host, N, T_total, &s));
  return conv_bwd(s, dy, dy_pitch, x, x_pitch, w, bias, init, dlast, dx, dinit, dw, dbias, D, W, silu, dtype,
                  workspace, workspace_bytes, stream);
}

int causal_conv_step(const void* x, int64_t x_pitch, const float* w, const float* bias, void* state, const int* slots,
                     void* y, int B, int S, int D, int W, int silu, int dtype, void* stream) {
  GDN_TRY(check_conv(x, x_pitch, w, D, W, dtype));
  if (!state || !y) return fail(GDN_ERR_INVALID, "state and y must be non-null device pointers");
  GDN_TRY(check_step(B, S, slots, D, 256));
  const gdn::ConvStepParams p{x, x_pitch, w, bias, state, slots, y, B, S, D, W, silu != 0};
  const hipError_t e = gdn::launch_conv_step(p, dtype, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "causal_conv_step launch");
}

int ssm_scan_num_chunks(const int* cu_seqlens_host, int N_seq) {
  if (!sizable(cu_seqlens_host, N_seq, 1, 1)) return -1;
  int64_t total = 0;
  for (int i = 0; i < N_seq; ++i)
    total += ((int64_t)cu_seqlens_host[i + 1] - cu_seqlens_host[i] + GDN_SSM_CHUNK - 1) / GDN_SSM_CHUNK;
  return total > INT32_MAX ? -1 : (int)total;
}

size_t ssm_scan_fwd_workspace_bytes(int B, int T, int D, int N) {
  if (B <= 0 || T <= 0 || D <= 0 || N <= 0 || N > gdn::kSsmMaxN || (int64_t)B * T > GDN_MAX_TOKENS) return 0;
  return gdn::ssm_fwd_ws_bytes(dense_split(false, B, T, D, N), B, D, N);
}

size_t ssm_scan_fwd_varlen_workspace_bytes(const int* cu_seqlens_host, int N_seq, int D, int N) {
  if (!sizable(cu_seqlens_host, N_seq, D, N)) return 0;
  return gdn::ssm_fwd_ws_bytes(packed_split(false, cu_seqlens_host, N_seq, D, N), N_seq, D, N);
}

size_t ssm_scan_bwd_workspace_bytes(int B, int T, int D, int N) {
  if (B <= 0 || T <= 0 || D <= 0 || N <= 0 || N > gdn::kSsmMaxN || (int64_t)B * T > GDN_MAX_TOKENS) return 0;
  return gdn::ssm_bwd_ws_bytes(dense_split(true, B, T, D, N), B * T, D, N);
}

size_t ssm_scan_bwd_varlen_workspace_bytes(const int* cu_seqlens_host, int N_seq, int D, int N) {
  if (!sizable(cu_seqlens_host, N_seq, D, N)) return 0;
  return gdn::ssm_bwd_ws_bytes(packed_split(true, cu_seqlens_host, N_seq, D, N), cu_seqlens_host[N_seq], D, N);
}

int ssm_scan_fwd(const void* x, int64_t x_pitch, const void* dt, int64_t dt_pitch, const float* A, const void* Bm,
                 int64_t b_pitch, const void* Cm, int64_t c_pitch, const float* skip, const void* z, int64_t z_pitch,
                 const float* dt_bias, const float* h0, void* y, float* ht, float* h, int B, int T, int D, int N,
                 int softplus, int dtype, void* workspace, size_t workspace_bytes, void* stream) {
  const Scan a{x, dt, z, Bm, Cm, x_pitch, dt_pitch, z_pitch, b_pitch, c_pitch, A, skip, dt_bias};
  gdn::Seqs s;
  GDN_TRY(check_scan(a, D, N, dtype));
  GDN_TRY(dense_seqs(B, T, &s));
  return scan_fwd(s, dense_split(false, B, T, D, N), nullptr, a, h0, y, ht, h, D, N, softplus, dtype, workspace,
                  workspace_bytes, stream);
}

int ssm_scan_fwd_varlen(const void* x, int64_t x_pitch, const void* dt, int64_t dt_pitch, const float* A,
                        const void* Bm, int64_t b_pitch, const void* Cm, int64_t c_pitch, const int* cu_seqlens,
                        const int* cu_seqlens_host, int N_seq, const float* skip, const void* z, int64_t z_pitch,
                        const float* dt_bias, const float* h0, void* y, float* ht, float* h, int T_total, int D,
                        int N, int softplus, int dtype, void* workspace, size_t workspace_bytes, void* stream) {
  const Scan a{x, dt, z, Bm, Cm, x_pitch, dt_pitch, z_pitch, b_pitch, c_pitch, A, skip, dt_bias};
  gdn::Seqs s;
  GDN_TRY(check_scan(a, D, N, dtype));
  GDN_TRY(packed_seqs(cu_seqlens, cu_seqlens_host, N_seq, T_total, &s));
  return scan_fwd(s, packed_split(false, cu_seqlens_host, N_seq, D, N), cu_seqlens_host, a, h0, y, ht, h, D, N, softplus, dtype,
                  workspace, workspace_bytes, stream);
}

int ssm_scan_bwd(const void* dy, int64_t dy_pitch, const float* h, const void* x, int64_t x_pitch, const void* dt,
                 int64_t dt_pitch, const float* A, const void* Bm, int64_t b_pitch, const void* Cm, int64_t c_pitch,
                 const float* skip, const void* z, int64_t z_pitch, const float* dt_bias, const float* dht, void* dx,
                 void* ddt, float* dA, void* dBm, void* dCm, float* dskip, void* dz, float* ddt_bias, float* dh0,
                 int B, int T, int D, int N, int softplus, int dtype, void* workspace, size_t workspace_bytes,
                 void* stream) {
  const Scan a{x, dt, z, Bm, Cm, x_pitch, dt_pitch, z_pitch, b_pitch, c_pitch, A, skip, dt_bias};
  const ScanGrads o{dx, ddt, dBm, dCm, dz, dA, dskip, ddt_bias, dh0};
  gdn::Seqs s;
  GDN_TRY(check_scan(a, D, N, dtype));
  GDN_TRY(dense_seqs(B, T, &s));
  return scan_bwd(s, dense_split(true, B, T, D, N), nullptr, a, dy, dy_pitch, h, dht, o, D, N, softplus, dtype, workspace,
                  workspace_bytes, stream);
}

int ssm_scan_bwd_varlen(const void* dy, int64_t dy_pitch, const float* h, const void* x, int64_t x_pitch,
                        const void* dt, int64_t dt_pitch, const float* A, const void* Bm, int64_t b_pitch,
                        const void* Cm, int64_t c_pitch, const int* cu_seqlens, const int* cu_seqlens_host, int N_seq,
                        const float* skip, const void* z, int64_t z_pitch, const float* dt_bias, const float* dht,
                        void* dx, void* ddt, float* dA, void* dBm, void* dCm, float* dskip, void* dz, float* ddt_bias,
                        float* dh0, int T_total, int D, int N, int softplus, int dtype, void* workspace,
                        size_t workspace_bytes, void* stream) {
  const Scan a{x, dt, z, Bm, Cm, x_pitch, dt_pitch, z_pitch, b_pitch, c_pitch, A, skip, dt_bias};
  const ScanGrads o{dx, ddt, dBm, dCm, dz, dA, dskip, ddt_bias, dh0};
  gdn::Seqs s;
  GDN_TRY(check_scan(a, D, N, dtype));
  GDN_TRY(packed_seqs(cu_seqlens, cu_seqlens_host, N_seq, T_total, &s));
  return scan_bwd(s, packed_split(true, cu_seqlens_host, N_seq, D, N), cu_seqlens_host, a, dy, dy_pitch, h, dht, o, D, N, softplus,
                  dtype, workspace, workspace_bytes, stream);
}

int ssm_step(const void* x, int64_t x_pitch, const void* dt, int64_t dt_pitch, const float* A, const void* Bm,
             int64_t b_pitch, const void* Cm, int64_t c_pitch, const float* skip, const void* z, int64_t z_pitch,
             const float* dt_bias, float* state, const int* slots, void* y, int B, int S, int D, int N, int softplus,
             int dtype, void* stream) {
  const Scan a{x, dt, z, Bm, Cm, x_pitch, dt_pitch, z_pitch, b_pitch, c_pitch, A, skip, dt_bias};
  GDN_TRY(check_scan(a, D, N, dtype));
  if (!state || !y) return fail(GDN_ERR_INVALID, "state and y must be non-null device pointers");
  GDN_TRY(check_state("state", state, N));
  GDN_TRY(check_step(B, S, slots, D, 4 * gdn::ssm_channels(N)));
  const gdn::SsmStepParams p{x, dt, z, Bm, Cm, x_pitch, dt_pitch, z_pitch, b_pitch, c_pitch, A, skip, dt_bias,
                             state, slots, y, B, S, D, N, softplus != 0};
  const hipError_t e = gdn::launch_ssm_step(p, dtype, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "ssm_step launch");
}

int rms_norm_fwd(const void* x, int64_t x_pitch, const void* residual, int64_t r_pitch, const float* w, float eps,
                 void* y, void* sum, float* rstd, int M, int D, int dtype, int rdtype, void* stream) {
  const gdn::NormParams p{x, residual, x_pitch, r_pitch, w, eps, y, sum, rstd, nullptr, M, D, 0};
  return norm_fwd(p, dtype, rdtype, "rms_norm_fwd launch", stream);
}

int rms_norm_q8_fwd(const void* x, int64_t x_pitch, const void* residual, int64_t r_pitch, const float* w, float eps,
                    int block, void* q, float* scale, void* sum, int M, int D, int dtype, int rdtype, void* stream) {
  if (!scale) return fail(GDN_ERR_INVALID, "scale must be a non-null device pointer");
  if (block != 0 && block != 128) return fail(GDN_ERR_UNSUPPORTED, "block must be 0 (a row) or 128, got %d", block);
  const gdn::NormParams p{x, residual, x_pitch, r_pitch, w, eps, q, sum, nullptr, scale, M, D, block};
  return norm_fwd(p, dtype, rdtype, "rms_norm_q8_fwd launch", stream);
}

size_t rms_norm_bwd_workspace_bytes(int M, int D) {
  if (M <= 0 || D <= 0 || D > gdn::kNormMaxD) return 0;
  return gdn::norm_bwd_ws_bytes(M, D);
}

int rms_norm_bwd(const void* dy, int64_t dy_pitch, const void* s, int64_t s_pitch, const float* w, const float* rstd,
                 const void* dsum, int64_t dsum_pitch, void* ds, void* dx, float* dw, int M, int D, int dtype,
                 int sdtype, void* workspace, size_t workspace_bytes, void* stream) {
  GDN_TRY(check_norm(dy, dy_pitch, nullptr, 0, w, 1.f, M, D, dtype, sdtype));
  if (!s || !rstd || !ds || !dw) return fail(GDN_ERR_INVALID, "s, rstd, ds and dw must be non-null device pointers");
  GDN_TRY(check_pitch("s", s, s_pitch, D));
  GDN_TRY(check_pitch("dsum", dsum, dsum_pitch, D));
  GDN_TRY(check_workspace(workspace, workspace_bytes, gdn::norm_bwd_ws_bytes(M, D)));
  const gdn::NormBwdParams p{dy, s, dsum, dy_pitch, s_pitch, dsum_pitch, w, rstd, ds, dx, dw,
                             static_cast<float*>(workspace), M, D};
  const hipError_t e = gdn::launch_norm_bwd(p, dtype, sdtype, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "rms_norm_bwd launch");
}

}  // extern "C"
