// gdn_ssmbwd.hip -- gradient of the selective state space scan, from the states that the forward saved
// every 16 tokens.
//
// With y' the gradient of the ungated output (dy silu(z), or dy), a_t = e^{de_t A} and g_t the
// gradient of h_t:
//   g_t = C_t y'_t + a_{t+1} g_{t+1}                (the last token's a g: dht)
//   dC_t = sum_d y'_t h_t,   dB_t = sum_d g_t de_t x_t,   dx_t = de_t (g_t . B_t) + skip y'_t
//   dde_t = x_t (g_t . B_t) + sum_n A g_t a_t h_{t-1},   dA = sum_t de_t g_t a_t h_{t-1}
//   ddt_t = dde_t softplus'(dt_t + dt_bias),   dz_t = dy_t y_t silu'(z_t),   dh0 = a_0 g_0
//
// Lanes as in the forward (gdn_ssm.hip).  A workgroup walks the 16-token chunks of its segment from
// the last to the first: it forms the chunk's a_t and a_t h_{t-1} from the saved state into registers
// (16 tokens of both are what they hold), then walks the tokens backwards.  dB and dC are sums
// over all channels: each wave adds up its channels' shares through LDS, the workgroup its waves',
// and a last kernel the workgroups', in a fixed order.
#include "../../include/gdn.h"
#include "gdn_ssm_device.h"

namespace gdn {

namespace {

__device__ __forceinline__ float fold32(float a, float b) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float fold16(float a, float b) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Adds the shares of dB and dC over a wave's channels.  put() takes a lane's shares of token k of a group
// of LN tokens, done() leaves the group's sums in out[token][dB: NP, dC: NP].
//
// 16 lanes a channel (4 channels): by lane exchanges that halve the values too; the lower half
// wave goes on with dB, the upper with dC, then even and odd rows of 16 lanes with even and odd i.
template <int LN, int NPL>
struct AddChannels {
  static constexpr int NP = LN * NPL, LDS = 4;
  float* out;
  int lane;
  __device__ __forceinline__ AddChannels(float*, int l) : lane(l) {}
  __device__ __forceinline__ void put(int k, const float (&db)[NPL], const float (&dc)[NPL]) {
    float* q = out + k * 2 * NP + (lane >> 5) * NP + (lane & 15) * NPL + ((lane >> 4) & 1);
#pragma unroll
    for (int i = 0; i < NPL / 2; ++i)
      q[2 * i] = fold16(fold32(db[2 * i], dc[2 * i]), fold32(db[2 * i + 1], dc[2 * i + 1]));
  }
  __device__ __forceinline__ void done() {}
};
// Four lanes a channel (16 channels): exchanges would cost as much as the gradient itself (17
// instructions a token, half of them at a third of the rate), so the shares go through the
// wave's own LDS: [token][dB, dC][channel][16], each lane then adds two columns of one token.
template <>
struct AddChannels<4, 4> {
  static constexpr int WHICH = 16 * 16 + 16;  // padded: dB and dC of a token on different banks
  static constexpr int LDS = 4 * 2 * WHICH;
  float *buf, *out;
  int lane;
  __device__ __forceinline__ AddChannels(float* b, int l) : buf(b), lane(l) {}
  __device__ __forceinline__ void put(int k, const float (&db)[4], const float (&dc)[4]) {
    float* q = buf + k * 2 * WHICH + lane * 4;
    *reinterpret_cast<f32x4*>(q) = f32x4{db[0], db[1], db[2], db[3]};
    *reinterpret_cast<f32x4*>(q + WHICH) = f32x4{dc[0], dc[1], dc[2], dc[3]};
  }
  __device__ __forceinline__ void done() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    const int tok = lane >> 4, which = (lane >> 3) & 1, n = (lane & 7) * 2;
    const float* q = buf + (tok * 2 + which) * WHICH + n;
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int c = 0; c < 16; ++c) {
      const float2 v = *reinterpret_cast<const float2*>(q + c * 16);
      s0 += v.x;
      s1 += v.y;
    }
    *reinterpret_cast<float2*>(out + tok * 32 + which * 16 + n) = make_float2(s0, s1);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
};

// A thread's dA, dskip and ddt_bias over a piece, which may be a whole sequence: a running fp32 sum would
// lose up to half a unit of 2^-24 for each of its tokens where the terms have one sign, so the registers'
// sums of kFold tokens are added up here.  Kept in LDS by four lanes a channel, whose registers are all
// taken (8 of them would spill), in registers by 16, whose LDS is.
constexpr int kFold = 256;
template <int LN, int K>
struct PieceSums {
  static constexpr int LDS = 1;
  float s[K] = {};
  __device__ __forceinline__ PieceSums(float*) {}
  __device__ __forceinline__ void add(int i, float v) { s[i] += v; }
  __device__ __forceinline__ float get(int i) const { return s[i]; }
};
template <int K>
struct PieceSums<4, K> {
  static constexpr int LDS = K * 256;
  float* s;  // [K][256 threads], each thread its own
  __device__ __forceinline__ PieceSums(float* lds) : s(lds + threadIdx.x) {
#pragma unroll
    for (int i = 0; i < K; ++i) s[i * 256] = 0.f;
  }
  __device__ __forceinline__ void add(int i, float v) { s[i * 256] += v; }
  __device__ __forceinline__ float get(int i) const { return s[i * 256]; }
};

// A chunk's x, dt, z and dy as a lane owns them: the j-th of every LN tokens of channel cc; 0 behind the
// end.  (Without a gate z is read as x and not used.)
template <typename T, int LN>
struct ChunkIn {
  static constexpr int TL = kSsmChunk / LN;
  unsigned x[TL], dt[TL], z[TL], dy[TL];
  __device__ __forceinline__ void ask(const SsmBwdParams& p, int tb, int rows, int j, int cc) {
    const SsmParams& f = p.f;
    const void* zp = f.z ? f.z : f.x;
    const int64_t zpitch = f.z ? f.z_pitch : f.x_pitch;
    const auto rx = window<T>(f.x, f.x_pitch, tb, rows, f.D), rd = window<T>(f.dt, f.dt_pitch, tb, rows, f.D),
               rz = window<T>(zp, zpitch, tb, rows, f.D), ry = window<T>(p.dy, p.dy_pitch, tb, rows, f.D);
    auto at = [&](int64_t pitch) { return (unsigned)(j * (int)pitch + cc) * (unsigned)sizeof(T); };
    const unsigned vx = at(f.x_pitch), vd = at(f.dt_pitch), vz = at(zpitch), vy = at(p.dy_pitch);
#pragma unroll
    for (int q = 0; q < TL; ++q) {
      const unsigned s = q * LN * sizeof(T);
      x[q] = load_bits<T>(rx, vx + s * (unsigned)f.x_pitch);
      dt[q] = load_bits<T>(rd, vd + s * (unsigned)f.dt_pitch);
      z[q] = load_bits<T>(rz, vz + s * (unsigned)zpitch);
      dy[q] = load_bits<T>(ry, vy + s * (unsigned)p.dy_pitch);
    }
  }
};

// A token's step size, its derivative by the raw one, and the gradient of the ungated output.
struct Token {
  float de, sig, gy;
};
__device__ __forceinline__ Token token_of(bool v, bool softplus, bool gate, float raw, float dout, float z) {
  Token k;
  float sig;
  const float sp = softplus_f(raw, &sig), s = z * sigmoid_f(z);
  k.de = v ? (softplus ? sp : raw) : 0.f;
  k.sig = softplus ? sig : 1.f;
  k.gy = dout * (gate ? s : 1.f);
  return k;
}

// Gradient of the state before a segment from its own tokens alone, and its summed step sizes.
template <typename T, int LN, int NPL>
__global__ __launch_bounds__(256) void ssm_bwd_summary_kernel(SsmBwdParams p, int groups) {
  constexpr int NP = LN * NPL, TL = kSsmChunk / LN;
  __shared__ __align__(16) float bc[kSsmChunk * NP * 2];
  const SsmParams& f = p.f;
  const Place<LN> w(f, groups, f.split.seg, f.split.nseg);
  if (w.pc.seq < 0 || w.pc.k < f.split.main / f.split.seg) return;  // nothing is before the first piece
  const int j = w.j, cc = w.cc, t0 = w.t0, t1 = w.t1;
  float A2[NPL], g[NPL] = {};
  load_decay<NPL>(f, cc, j, A2);
  const float bias = f.dt_bias ? f.dt_bias[cc] : 0.f;
  float dsum = 0.f;
  for (int tb = t0 + (t1 - t0 - 1) / kSsmChunk * kSsmChunk; tb >= t0; tb -= kSsmChunk) {
    ChunkIn<T, LN> in;
    StageBC<T, NP, kSsmChunk, 256> st;
    const int rows = min(t1 - tb, kSsmChunk);
    in.ask(p, tb, rows, j, cc);
    st.load(f, tb, rows);
    __syncthreads();
    st.store(bc);
    __syncthreads();
#pragma unroll
    for (int q = TL - 1; q >= 0; --q) {
      const Token tk = token_of(tb + q * LN + j < t1, f.softplus, f.z != nullptr, of_bits<T>(in.dt[q]) + bias,
                                of_bits<T>(in.dy[q]), of_bits<T>(in.z[q]));
      dsum += tk.de;
      static_for<LN>([&](auto r) {
        constexpr int k = LN - 1 - r();
        const float dk = shared_lane<LN, k>(tk.de), gk = shared_lane<LN, k>(tk.gy);
        float b[NPL], cf[NPL];
        read_bc<NPL>(bc + ((q * LN + k) * NP + j * NPL) * 2, b, cf);
#pragma unroll
        for (int i = 0; i < NPL; ++i)
          g[i] = __builtin_fmaf(cf[i], gk, g[i]) * decay(dk, A2[i]);
      });
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  if (w.cv) store_state<NPL>(f.seg_state + (int64_t)w.seg * f.D * f.N, w.c, j, f.N, g);
  dsum = group_sum<LN>(dsum);
  if (w.cv && j == 0) f.seg_sum[(int64_t)w.seg * f.D + w.c] = dsum;
}

// A sequence's segments from the last to the last one of its first piece (of its only one where it is
// shorter than a piece): seg_state becomes the gradient that reaches each segment's last state from behind it.
__global__ __launch_bounds__(256) void ssm_bwd_join_kernel(SsmBwdParams p, int per_seq) {
  const SsmParams& f = p.f;
  const int seq = blockIdx.x / per_seq;
  const int64_t e = (int64_t)(blockIdx.x - seq * per_seq) * 256 + threadIdx.x;
  const int64_t DN = (int64_t)f.D * f.N;
  const SeqPieces sp = pieces_of(f.s, seq, f.split.seg, f.split.nseg, threadIdx.x & 63);
  if (e >= DN) return;
  const int64_t d = e / f.N;
  const float a = f.A[e] * kLog2e;
  float g = p.dht ? p.dht[seq * DN + e] : 0.f;
  const int first = f.split.main / f.split.seg, stop = min(first, sp.count) - 1;
  for (int i = sp.count - 1; i >= stop && i >= 0; --i) {
    const int64_t s = sp.first + i;
    const bool summed = i >= first;
    const float own = summed ? f.seg_state[s * DN + e] : 0.f, sum = summed ? f.seg_sum[s * f.D + d] : 0.f;
    f.seg_state[s * DN + e] = g;
    g = __builtin_fmaf(__builtin_amdgcn_exp2f(a * sum), g, own);
  }
}

// The gradient proper.  Bound by vector instructions: 56 of the 94 a token and wave are its own (4 states
// a lane, 14 operations each, one of them an exponential).  4 x 2048 tokens x 4096 channels x 16 states,
// bf16: 520 us, vector units busy 69% of the time.  What the layout costs and gains there:
//  - 16 tokens' a and a h in registers (128 of the 255) leave two waves a SIMD.  32 tokens of a h with
//    the exponential taken again spilled 61 registers: 1290 us.
//  - the channel sums through LDS: 640 us with two barriers a chunk, 572 with one.
//  - the next chunk's inputs asked for in the middle of the walk, when the last group's a and a h are
//    done with (no spills): 497; at its start (12 spills): 572.
template <typename T, int LN, int NPL>
__global__ __launch_bounds__(256, 2) void ssm_bwd_kernel(SsmBwdParams p, int groups) {
  constexpr int NP = LN * NPL, TL = kSsmChunk / LN;
  __shared__ __align__(16) float bc[2][kSsmChunk * NP * 2];
  __shared__ __align__(16) float red[2][4][kSsmChunk * 2 * NP];
  __shared__ __align__(16) float shares[4][AddChannels<LN, NPL>::LDS];
  __shared__ float far[PieceSums<LN, NPL + 2>::LDS];
  const SsmParams& f = p.f;
  const Place<LN> w(f, groups, f.split.main, f.split.nmain);
  if (w.pc.seq < 0) return;
  const int j = w.j, c = w.c, cc = w.cc, t0 = w.t0, t1 = w.t1;
  const bool cv = w.cv, gate = f.z;
  const int64_t DN = (int64_t)f.D * f.N;
  int tb = t0 + (t1 - t0 - 1) / kSsmChunk * kSsmChunk;

  // a chunk's inputs are asked for while the one behind it is computed
  ChunkIn<T, LN> in;
  StageBC<T, NP, kSsmChunk, 256> st;
  float hs[NPL];
  int64_t chunk = min(find_piece_before(f.s, w.pc, kSsmChunk, w.lane) + (tb - w.pc.begin) / kSsmChunk, f.chunks - 1);
  in.ask(p, tb, min(t1 - tb, kSsmChunk), j, cc);
  st.load(f, tb, min(t1 - tb, kSsmChunk));
  load_state<NPL>(f.h + chunk * DN, cc, j, f.N, hs);

  float A2[NPL], g[NPL], dA[NPL] = {};
  load_decay<NPL>(f, cc, j, A2);
  const int64_t last_seg =
      min(find_piece_before(f.s, w.pc, f.split.seg, w.lane) + (t1 - 1 - w.pc.begin) / f.split.seg, (int64_t)f.split.nseg - 1);
  load_state<NPL>(f.seg_state ? f.seg_state + last_seg * DN : p.dht ? p.dht + w.pc.seq * DN : nullptr, cc, j, f.N, g);
  if (!cv) {  // lanes without a channel give nothing to the sums over channels
#pragma unroll
    for (int i = 0; i < NPL; ++i) g[i] = 0.f;
  }
  const float bias = f.dt_bias ? f.dt_bias[cc] : 0.f, skip = f.skip ? f.skip[cc] : 0.f;
  float dskip = 0.f, dbias = 0.f;
  PieceSums<LN, NPL + 2> sums(far);
  const unsigned vo = cv ? (unsigned)(j * f.D + c) * sizeof(T) : kNowhere;
  AddChannels<LN, NPL> add(shares[w.wv], w.lane);
  st.store(bc[0]);
  __syncthreads();

  for (int buf = 0; tb >= t0; tb -= kSsmChunk, buf ^= 1) {
    float h[NPL], a[kSsmChunk][NPL], ah[kSsmChunk][NPL], x[TL], z[TL], dout[TL];
    Token tk[TL];
#pragma unroll
    for (int i = 0; i < NPL; ++i) h[i] = hs[i];
#pragma unroll
    for (int q = 0; q < TL; ++q) {
      x[q] = of_bits<T>(in.x[q]);
      z[q] = of_bits<T>(in.z[q]);
      dout[q] = cv ? of_bits<T>(in.dy[q]) : 0.f;
      tk[q] = token_of(tb + q * LN + j < t1, f.softplus, gate, of_bits<T>(in.dt[q]) + bias, dout[q], z[q]);
    }
    const bool more = tb > t0;
#pragma unroll
    for (int q = 0; q < TL; ++q) {
      const float dx = tk[q].de * x[q];
      static_for<LN>([&](auto k) {
        const float dk = lane_of<LN, k()>(tk[q].de), xk = lane_of<LN, k()>(dx);
        float b[NPL], cf[NPL];
        read_bc<NPL>(bc[buf] + ((q * LN + k()) * NP + j * NPL) * 2, b, cf);
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
          const float e = decay(dk, A2[i]);
          a[q * LN + k()][i] = e;
          ah[q * LN + k()][i] = e * h[i];
          h[i] = __builtin_fmaf(xk, b[i], e * h[i]);
        }
      });
    }
    const int rows = min(t1 - tb, kSsmChunk);
    const auto rx = window<T>(p.dx, f.D, tb, rows, f.D), rd = window<T>(p.ddt, f.D, tb, rows, f.D),
               rz = window<T>(gate ? p.dz : p.dx, f.D, tb, gate ? rows : 0, f.D);
#pragma unroll
    for (int q = TL - 1; q >= 0; --q) {
      if (q == (TL > 1 ? TL - 2 : 0)) {  // the next chunk's inputs, once the last group's a and a h are done with
        const int left = more ? kSsmChunk : 0;
        chunk -= more && chunk > 0;
        in.ask(p, tb - kSsmChunk, left, j, cc);
        st.load(f, tb - kSsmChunk, left);
        load_state<NPL>(f.h + chunk * DN, cc, j, f.N, hs);
      }
      const float dx = tk[q].de * x[q];
      float yv[LN], gb[LN], ga[LN];
      add.out = red[buf][w.wv] + q * LN * 2 * NP;
      static_for<LN>([&](auto r) {
        constexpr int k = LN - 1 - r();
        const float dk = lane_of<LN, k>(tk[q].de), xk = lane_of<LN, k>(dx), gk = lane_of<LN, k>(tk[q].gy);
        float b[NPL], cf[NPL], db[NPL], dc[NPL];
        read_bc<NPL>(bc[buf] + ((q * LN + k) * NP + j * NPL) * 2, b, cf);
        float sy = 0.f, sb = 0.f, sa = 0.f;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
          const float p_ = ah[q * LN + k][i], ht = __builtin_fmaf(xk, b[i], p_);
          sy = __builtin_fmaf(cf[i], ht, sy);
          g[i] = __builtin_fmaf(cf[i], gk, g[i]);
          dc[i] = gk * ht;
          db[i] = xk * g[i];
          sb = __builtin_fmaf(g[i], b[i], sb);
          const float gah = g[i] * p_;
          sa = __builtin_fmaf(gah, A2[i], sa);
          dA[i] = __builtin_fmaf(gah, dk, dA[i]);
          g[i] *= a[q * LN + k][i];
        }
        yv[k] = sy;
        gb[k] = sb;
        ga[k] = sa;
        add.put(k, db, dc);
      });
      const float y = reduce_scatter<LN>(yv, j), sb = reduce_scatter<LN>(gb, j), sa = reduce_scatter<LN>(ga, j);
      const float ddt = (x[q] * sb + sa * kLn2) * tk[q].sig, s = sigmoid_f(z[q]);
      const unsigned so = q * LN * (unsigned)f.D * sizeof(T);  // stores behind the end are dropped
      store_bits<T>(rx, to_t<T>(tk[q].de * sb + skip * tk[q].gy), vo + so);
      store_bits<T>(rd, to_t<T>(ddt), vo + so);
      store_bits<T>(rz, to_t<T>(dout[q] * (y + skip * x[q]) * s * (1.f + z[q] * (1.f - s))), vo + so);
      dbias += tb + q * LN + j < t1 ? ddt : 0.f;
      dskip = __builtin_fmaf(tk[q].gy, x[q], dskip);
      add.done();
    }
    if (more) st.store(bc[buf ^ 1]);
    // one barrier a chunk: what is read here is written again two chunks on
    __syncthreads();
    for (int e = threadIdx.x; e < kSsmChunk * 2 * NP; e += 256) {
      const int k = e / (2 * NP), m = e % (2 * NP), n = m % NP;
      if (k < rows && n < f.N)
        p.part_bc[(((int64_t)w.grp * f.s.rows + tb + k) * 2 + m / NP) * f.N + n] =
            red[buf][0][e] + red[buf][1][e] + red[buf][2][e] + red[buf][3][e];
    }
    if ((tb - t0) % kFold == 0) {
#pragma unroll
      for (int i = 0; i < NPL; ++i) {
        sums.add(i, dA[i]);
        dA[i] = 0.f;
      }
      sums.add(NPL, dskip);
      sums.add(NPL + 1, dbias);
      dskip = dbias = 0.f;
    }
  }
  if (cv) {
    float* pa = p.part_a + ((int64_t)w.seg * f.D + c) * (f.N + 2);
#pragma unroll
    for (int i = 0; i < NPL; ++i)
      if (j * NPL + i < f.N) pa[j * NPL + i] = sums.get(i);
    dskip = group_sum<LN>(sums.get(NPL));
    dbias = group_sum<LN>(sums.get(NPL + 1));
    if (j == 0) {
      pa[f.N] = dskip;
      pa[f.N + 1] = dbias;
    }
    if (p.dh0 && w.pc.k == 0) store_state<NPL>(p.dh0 + w.pc.seq * DN, c, j, f.N, g);
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
BwdWs bwd_ws(const SsmSplit& sp, int rows, int D, int N) {
  BwdWs w;
  const size_t groups = (D + bwd_channels(N) - 1) / bwd_channels(N);
  w.state = 0;
  w.sum = al256((size_t)sp.nseg * D * N * 4);
  w.bc = w.sum + al256((size_t)sp.nseg * D * 4);
  w.a = w.bc + al256(groups * rows * 2 * N * 4);
  w.total = w.a + al256((size_t)sp.nmain * D * (N + 2) * 4);
  return w;
}

}  // namespace

size_t ssm_bwd_ws_bytes(const SsmSplit& sp, int rows, int D, int N) { return bwd_ws(sp, rows, D, N).total; }

hipError_t launch_ssm_bwd(SsmBwdParams p, int dtype, void* ws, hipStream_t st) {
  SsmParams& f = p.f;
  const BwdWs w = bwd_ws(f.split, f.s.rows, f.D, f.N);
  char* base = static_cast<char*>(ws);
  const bool split = f.split.nmain > f.s.n;  // (a sequence of one piece needs no summary)
  f.seg_state = split ? reinterpret_cast<float*>(base + w.state) : nullptr;
  f.seg_sum = split ? reinterpret_cast<float*>(base + w.sum) : nullptr;
  p.part_bc = reinterpret_cast<float*>(base + w.bc);
  p.part_a = reinterpret_cast<float*>(base + w.a);
  return ssm_dispatch(dtype, f.N, [&](auto t, auto ln, auto npl) {
    using T = decltype(t);
    constexpr int LN = decltype(ln)::value, NPL = decltype(npl)::value;
    const int ch = 4 * (64 / LN), groups = (f.D + ch - 1) / ch;
    hipError_t e;
    if (split) {
      ssm_bwd_summary_kernel<T, LN, NPL><<<dim3((unsigned)(groups * f.split.nseg)), 256, 0, st>>>(p, groups);
      if ((e = hipGetLastError()) != hipSuccess) return e;
      const int per_seq = (int)(((int64_t)f.D * f.N + 255) / 256);
      ssm_bwd_join_kernel<<<dim3((unsigned)(per_seq * f.s.n)), 256, 0, st>>>(p, per_seq);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    ssm_bwd_kernel<T, LN, NPL><<<dim3((unsigned)(groups * f.split.nmain)), 256, 0, st>>>(p, groups);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    int64_t cols = (int64_t)f.s.rows * 2 * f.N;
    e = column_sum(p.part_bc, groups, cols, BcOut<T>{static_cast<T*>(p.dB), static_cast<T*>(p.dC), f.N}, st);
    if (e != hipSuccess) return e;
    cols = (int64_t)f.D * (f.N + 2);
    return column_sum(p.part_a, f.split.nmain, cols, ParamOut{p.dA, p.dskip, p.ddt_bias, f.N}, st);
  });
}

}  // namespace gdn
