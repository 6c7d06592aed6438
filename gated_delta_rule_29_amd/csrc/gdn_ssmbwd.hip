// gdn_ssmbwd.hip -- gradient of the selective state space scan, from the states that the forward saved
// every 32 tokens.
//
// With y' the gradient of the ungated output (dy silu(z), or dy), a_t = e^{de_t A} and g_t the
// gradient of h_t:
//   g_t = C_t y'_t + a_{t+1} g_{t+1}                (the last token's a g: dht)
//   dC_t = sum_d y'_t h_t,   dB_t = sum_d g_t de_t x_t,   dx_t = de_t (g_t . B_t) + skip y'_t
//   dde_t = x_t (g_t . B_t) + sum_n A g_t a_t h_{t-1},   dA = sum_t de_t g_t a_t h_{t-1}
//   ddt_t = dde_t softplus'(dt_t + dt_bias),   dz_t = dy_t y_t silu'(z_t),   dh0 = a_0 g_0
//
// Lanes as in the forward (gdn_ssm.hip).  A workgroup walks the 32-token chunks of its segment from
// the last to the first: it forms the chunk's a_t h_{t-1} from the saved state into registers, then
// walks the tokens backwards.  dB and dC are sums over all channels: each wave adds up its
// channels' shares in registers, the workgroup its waves' in LDS, and a last kernel the workgroups'
// in a fixed order.
#include "../../include/gdn.h"
#include "gdn_ssm_device.h"

namespace gdn {

namespace {

constexpr int kDppRor8 = 0x128, kDppQuadReverse = 0x1B;

__device__ __forceinline__ float fold32(float a, float b) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float fold16(float a, float b) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Adds a lane's shares db[i], dc[i] of one token over the wave's channels and writes the sums to
// out[2][NP] (dB, then dC).  Each exchange also halves the number of values: the lower half wave
// goes on with dB, the upper with dC, then even and odd rows of 16 with even and odd i.
template <int LN, int NPL>
__device__ __forceinline__ void add_channels(const float (&db)[NPL], const float (&dc)[NPL], float* out, int lane) {
  constexpr int NP = LN * NPL;
  float u[NPL / 2];
#pragma unroll
  for (int i = 0; i < NPL / 2; ++i)
    u[i] = fold16(fold32(db[2 * i], dc[2 * i]), fold32(db[2 * i + 1], dc[2 * i + 1]));
  float* q = out + (lane >> 5) * NP;
  const int odd = (lane >> 4) & 1;
  if constexpr (LN == 16) {
#pragma unroll
    for (int i = 0; i < NPL / 2; ++i) q[(lane & 15) * NPL + 2 * i + odd] = u[i];
  } else {
    static_assert(LN == 4 && NPL == 4, "four lanes hold four states each");
    const bool b3 = lane & 8;
    float r = (b3 ? u[1] : u[0]) + dpp<kDppRor8>(b3 ? u[0] : u[1]);
    r += dpp<kDppHalfMirror>(dpp<kDppQuadReverse>(r));  // lane ^ 4
    if (!(lane & 4)) q[(lane & 3) * 4 + (b3 ? 2 : 0) + odd] = r;
  }
}

// A token's step size, its derivative by the raw one, and the gradient of the ungated output.
struct Token {
  float de, sig, gy;
};
__device__ __forceinline__ Token token_of(bool v, bool softplus, bool gate, float raw, float dout, float z) {
  Token k;
  k.de = raw;
  k.sig = 1.f;
  if (softplus) k.de = softplus_f(raw, &k.sig);
  if (!v) k.de = 0.f;
  k.gy = gate ? dout * z * sigmoid_f(z) : dout;
  return k;
}

// Gradient of the state before a segment from its own tokens alone, and its summed step sizes.
template <typename T, int LN, int NPL>
__global__ __launch_bounds__(256) void ssm_bwd_summary_kernel(SsmBwdParams p, int groups) {
  constexpr int NP = LN * NPL, CH = 64 / LN, TL = kSsmChunk / LN;
  __shared__ __align__(16) float bc[kSsmChunk * NP * 2];
  const SsmParams& f = p.f;
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int j = lane % LN, seg = blockIdx.x / groups;
  const int c = ((blockIdx.x - seg * groups) * 4 + wv) * CH + lane / LN;
  const bool cv = c < f.D;
  const int cc = cv ? c : f.D - 1;
  const Piece pc = find_piece(f.s, seg, f.seg, lane);
  if (pc.seq < 0 || pc.k == 0) return;  // nothing is before the first segment
  const int t0 = pc.begin + pc.k * f.seg, t1 = min(t0 + f.seg, pc.end);
  float A2[NPL], g[NPL] = {};
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const int n = j * NPL + i;
    A2[i] = n < f.N ? f.A[(int64_t)cc * f.N + n] * kLog2e : 0.f;
  }
  const float bias = f.dt_bias ? f.dt_bias[cc] : 0.f;
  float dsum = 0.f;
  for (int tb = t0 + (t1 - t0 - 1) / kSsmChunk * kSsmChunk; tb >= t0; tb -= kSsmChunk) {
    __syncthreads();
    stage_bc<T, NP>(f, tb, t1, bc);
    Token tk[TL];
#pragma unroll
    for (int q = 0; q < TL; ++q) {
      const int t = tb + q * LN + j;
      const bool v = t < t1;
      const float raw = (v ? to_f(static_cast<const T*>(f.dt)[t * f.dt_pitch + cc]) : 0.f) + bias;
      const float dout = v ? to_f(static_cast<const T*>(p.dy)[t * p.dy_pitch + cc]) : 0.f;
      const float z = f.z && v ? to_f(static_cast<const T*>(f.z)[t * f.z_pitch + cc]) : 0.f;
      tk[q] = token_of(v, f.softplus, f.z != nullptr, raw, dout, z);
      dsum += tk[q].de;
    }
    __syncthreads();
#pragma unroll
    for (int q = TL - 1; q >= 0; --q) {
      static_for<LN>([&](auto r) {
        constexpr int k = LN - 1 - r();
        const float dk = lane_of<LN, k>(tk[q].de), gk = lane_of<LN, k>(tk[q].gy);
        float b[NPL], cf[NPL];
        read_bc<NPL>(bc + ((q * LN + k) * NP + j * NPL) * 2, b, cf);
#pragma unroll
        for (int i = 0; i < NPL; ++i)
          g[i] = __builtin_fmaf(cf[i], gk, g[i]) * __builtin_amdgcn_exp2f(dk * A2[i]);
      });
    }
  }
  if (cv) store_state<NPL>(f.seg_state + (int64_t)seg * f.D * f.N, c, j, f.N, g);
  dsum = group_sum<LN>(dsum);
  if (cv && j == 0) f.seg_sum[(int64_t)seg * f.D + c] = dsum;
}

// A sequence's segments from the last to the first: seg_state becomes the gradient that reaches each
// segment's last state from behind it.
__global__ __launch_bounds__(256) void ssm_bwd_join_kernel(SsmBwdParams p, int per_seq) {
  const SsmParams& f = p.f;
  const int seq = blockIdx.x / per_seq;
  const int64_t e = (int64_t)(blockIdx.x - seq * per_seq) * 256 + threadIdx.x;
  const int64_t DN = (int64_t)f.D * f.N;
  const SeqPieces sp = pieces_of(f.s, seq, f.seg, threadIdx.x & 63);
  if (e >= DN) return;
  const int64_t d = e / f.N;
  const float a = f.A[e] * kLog2e;
  float g = p.dht ? p.dht[seq * DN + e] : 0.f;
  for (int i = sp.count - 1; i >= 0; --i) {
    const int64_t s = sp.first + i;
    const float own = i ? f.seg_state[s * DN + e] : 0.f, sum = i ? f.seg_sum[s * f.D + d] : 0.f;
    f.seg_state[s * DN + e] = g;
    g = __builtin_fmaf(__builtin_amdgcn_exp2f(a * sum), g, own);
  }
}

template <typename T, int LN, int NPL>
__global__ __launch_bounds__(256, 2) void ssm_bwd_kernel(SsmBwdParams p, int groups) {
  constexpr int NP = LN * NPL, CH = 64 / LN, TL = kSsmChunk / LN;
  __shared__ __align__(16) float bc[kSsmChunk * NP * 2];
  __shared__ __align__(16) float red[4][kSsmChunk][2 * NP];
  const SsmParams& f = p.f;
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int j = lane % LN, seg = blockIdx.x / groups, grp = blockIdx.x - seg * groups;
  const int c = (grp * 4 + wv) * CH + lane / LN;
  const bool cv = c < f.D;
  const int cc = cv ? c : f.D - 1;
  const Piece pc = find_piece(f.s, seg, f.seg, lane);
  if (pc.seq < 0) return;
  const int t0 = pc.begin + pc.k * f.seg, t1 = min(t0 + f.seg, pc.end);
  const int64_t DN = (int64_t)f.D * f.N;
  const int64_t chunk0 = find_piece_before(f.s, pc, kSsmChunk, lane) + (t0 - pc.begin) / kSsmChunk;

  float A2[NPL], g[NPL], dA[NPL] = {};
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const int n = j * NPL + i;
    A2[i] = n < f.N ? f.A[(int64_t)cc * f.N + n] * kLog2e : 0.f;
  }
  load_state<NPL>(f.seg_state ? f.seg_state + seg * DN : p.dht ? p.dht + pc.seq * DN : nullptr, cc, j, f.N, g);
  const float bias = f.dt_bias ? f.dt_bias[cc] : 0.f, skip = f.skip ? f.skip[cc] : 0.f;
  float dskip = 0.f, dbias = 0.f;

  for (int tb = t0 + (t1 - t0 - 1) / kSsmChunk * kSsmChunk; tb >= t0; tb -= kSsmChunk) {
    __syncthreads();
    stage_bc<T, NP>(f, tb, t1, bc);
    float h[NPL], ph[kSsmChunk][NPL];
    load_state<NPL>(f.h + (chunk0 + (tb - t0) / kSsmChunk) * DN, cc, j, f.N, h);
    float x[TL], z[TL], dout[TL];
    Token tk[TL];
#pragma unroll
    for (int q = 0; q < TL; ++q) {
      const int t = tb + q * LN + j;
      const bool v = t < t1;
      x[q] = v ? to_f(static_cast<const T*>(f.x)[t * f.x_pitch + cc]) : 0.f;
      const float raw = (v ? to_f(static_cast<const T*>(f.dt)[t * f.dt_pitch + cc]) : 0.f) + bias;
      dout[q] = v && cv ? to_f(static_cast<const T*>(p.dy)[t * p.dy_pitch + cc]) : 0.f;
      z[q] = f.z && v ? to_f(static_cast<const T*>(f.z)[t * f.z_pitch + cc]) : 0.f;
      tk[q] = token_of(v, f.softplus, f.z != nullptr, raw, dout[q], z[q]);
    }
    if (!cv) {  // lanes past the last channel give nothing to the sums over channels
#pragma unroll
      for (int i = 0; i < NPL; ++i) g[i] = 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < TL; ++q) {
      const float dx = tk[q].de * x[q];
      static_for<LN>([&](auto k) {
        const float dk = lane_of<LN, k()>(tk[q].de), xk = lane_of<LN, k()>(dx);
        float b[NPL], cf[NPL];
        read_bc<NPL>(bc + ((q * LN + k()) * NP + j * NPL) * 2, b, cf);
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
          const float ah = __builtin_amdgcn_exp2f(dk * A2[i]) * h[i];
          ph[q * LN + k()][i] = ah;
          h[i] = __builtin_fmaf(xk, b[i], ah);
        }
      });
    }
#pragma unroll
    for (int q = TL - 1; q >= 0; --q) {
      const float dx = tk[q].de * x[q];
      float yv[LN], gb[LN], ga[LN];
      static_for<LN>([&](auto r) {
        constexpr int k = LN - 1 - r();
        const float dk = lane_of<LN, k>(tk[q].de), xk = lane_of<LN, k>(dx), gk = lane_of<LN, k>(tk[q].gy);
        float b[NPL], cf[NPL], db[NPL], dc[NPL];
        read_bc<NPL>(bc + ((q * LN + k) * NP + j * NPL) * 2, b, cf);
        float sy = 0.f, sb = 0.f, sa = 0.f;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
          const float ah = ph[q * LN + k][i], ht = __builtin_fmaf(xk, b[i], ah);
          sy = __builtin_fmaf(cf[i], ht, sy);
          g[i] = __builtin_fmaf(cf[i], gk, g[i]);
          dc[i] = gk * ht;
          db[i] = xk * g[i];
          sb = __builtin_fmaf(g[i], b[i], sb);
          const float gah = g[i] * ah;
          sa = __builtin_fmaf(gah, A2[i], sa);
          dA[i] = __builtin_fmaf(gah, dk, dA[i]);
          g[i] *= __builtin_amdgcn_exp2f(dk * A2[i]);
        }
        yv[k] = sy;
        gb[k] = sb;
        ga[k] = sa;
        add_channels<LN, NPL>(db, dc, red[wv][q * LN + k], lane);
      });
      const float y = reduce_scatter<LN>(yv, j), sb = reduce_scatter<LN>(gb, j), sa = reduce_scatter<LN>(ga, j);
      const int t = tb + q * LN + j;
      const float ddt = (x[q] * sb + sa * kLn2) * tk[q].sig;
      if (t < t1 && cv) {
        const int64_t o = (int64_t)t * f.D + c;
        static_cast<T*>(p.dx)[o] = to_t<T>(tk[q].de * sb + skip * tk[q].gy);
        static_cast<T*>(p.ddt)[o] = to_t<T>(ddt);
        if (f.z) {
          const float s = sigmoid_f(z[q]);
          static_cast<T*>(p.dz)[o] = to_t<T>(dout[q] * (y + skip * x[q]) * s * (1.f + z[q] * (1.f - s)));
        }
        dbias += ddt;
        dskip = __builtin_fmaf(tk[q].gy, x[q], dskip);
      }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < kSsmChunk * 2 * NP; e += 256) {
      const int tk_ = e / (2 * NP), m = e % (2 * NP), n = m % NP, t = tb + tk_;
      if (t < t1 && n < f.N) {
        const float s = red[0][tk_][m] + red[1][tk_][m] + red[2][tk_][m] + red[3][tk_][m];
        p.part_bc[(((int64_t)grp * f.s.rows + t) * 2 + m / NP) * f.N + n] = s;
      }
    }
  }
  if (cv) {
    float* pa = p.part_a + ((int64_t)seg * f.D + c) * (f.N + 2);
#pragma unroll
    for (int i = 0; i < NPL; ++i)
      if (j * NPL + i < f.N) pa[j * NPL + i] = dA[i];
    dskip = group_sum<LN>(dskip);
    dbias = group_sum<LN>(dbias);
    if (j == 0) {
      pa[f.N] = dskip;
      pa[f.N + 1] = dbias;
    }
    if (p.dh0 && pc.k == 0) store_state<NPL>(p.dh0 + pc.seq * DN, c, j, f.N, g);
  }
}

template <typename T>
struct BcOut {
  T *dB, *dC;
  int N;
  __device__ void operator()(int64_t c, float s) const {
    const int64_t t = c / (2 * N);
    const int m = (int)(c - t * (2 * N));
    if (m < N) dB[t * N + m] = to_t<T>(s);
    else dC[t * N + m - N] = to_t<T>(s);
  }
};

struct ParamOut {
  float *dA, *dskip, *dbias;
  int N;
  __device__ void operator()(int64_t c, float s) const {
    const int64_t d = c / (N + 2);
    const int m = (int)(c - d * (N + 2));
    if (m < N) dA[d * N + m] = s;
    else if (m == N) { if (dskip) dskip[d] = s; }
    else if (dbias) dbias[d] = s;
  }
};

int bwd_channels(int N) { return N <= 16 ? 64 : 16; }  // of a workgroup

size_t al256(size_t x) { return (x + 255) & ~(size_t)255; }

struct BwdWs {
  size_t state, sum, bc, a, total;
};
BwdWs bwd_ws(int nseg, int rows, int D, int N) {
  BwdWs w;
  const size_t groups = (D + bwd_channels(N) - 1) / bwd_channels(N);
  w.state = 0;
  w.sum = al256((size_t)nseg * D * N * 4);
  w.bc = w.sum + al256((size_t)nseg * D * 4);
  w.a = w.bc + al256(groups * rows * 2 * N * 4);
  w.total = w.a + al256((size_t)nseg * D * (N + 2) * 4);
  return w;
}

}  // namespace

size_t ssm_bwd_ws_bytes(int nseg, int rows, int D, int N) { return bwd_ws(nseg, rows, D, N).total; }

hipError_t launch_ssm_bwd(SsmBwdParams p, int dtype, void* ws, hipStream_t st) {
  SsmParams& f = p.f;
  const BwdWs w = bwd_ws(f.nseg, f.s.rows, f.D, f.N);
  char* base = static_cast<char*>(ws);
  const bool split = f.nseg > f.s.n;
  f.seg_state = split ? reinterpret_cast<float*>(base + w.state) : nullptr;
  f.seg_sum = split ? reinterpret_cast<float*>(base + w.sum) : nullptr;
  p.part_bc = reinterpret_cast<float*>(base + w.bc);
  p.part_a = reinterpret_cast<float*>(base + w.a);
  return ssm_dispatch(dtype, f.N, [&](auto t, auto ln, auto npl) {
    using T = decltype(t);
    constexpr int LN = decltype(ln)::value, NPL = decltype(npl)::value;
    const int ch = 4 * (64 / LN), groups = (f.D + ch - 1) / ch;
    const dim3 grid((unsigned)(groups * f.nseg));
    hipError_t e;
    if (split) {
      ssm_bwd_summary_kernel<T, LN, NPL><<<grid, 256, 0, st>>>(p, groups);
      if ((e = hipGetLastError()) != hipSuccess) return e;
      const int per_seq = (int)(((int64_t)f.D * f.N + 255) / 256);
      ssm_bwd_join_kernel<<<dim3((unsigned)(per_seq * f.s.n)), 256, 0, st>>>(p, per_seq);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    ssm_bwd_kernel<T, LN, NPL><<<grid, 256, 0, st>>>(p, groups);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    int64_t cols = (int64_t)f.s.rows * 2 * f.N;
    column_sum_kernel<<<dim3((unsigned)((cols + 63) / 64)), 1024, 0, st>>>(
        p.part_bc, groups, cols, BcOut<T>{static_cast<T*>(p.dB), static_cast<T*>(p.dC), f.N});
    if ((e = hipGetLastError()) != hipSuccess) return e;
    cols = (int64_t)f.D * (f.N + 2);
    column_sum_kernel<<<dim3((unsigned)((cols + 63) / 64)), 1024, 0, st>>>(
        p.part_a, f.nseg, cols, ParamOut{p.dA, p.dskip, p.ddt_bias, f.N});
    return hipGetLastError();
  });
}

}  // namespace gdn
