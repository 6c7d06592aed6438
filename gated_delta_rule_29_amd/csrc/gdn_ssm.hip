// gdn_ssm.hip -- the selective state space scan: for prompts (dense or packed sequences, initial and
// final states, states saved for the backward pass) and for single tokens on a cache of states.
//
//   de_t = softplus(dt_t + dt_bias)   (or dt_t + dt_bias)
//   h_t[d,n] = e^{de_t[d] A[d,n]} h_{t-1}[d,n] + de_t[d] x_t[d] B_t[n]
//   y_t[d] = (sum_n C_t[n] h_t[d,n] + skip[d] x_t[d]) * (z_t[d] sigmoid(z_t[d]) if z)
//
// Layout.  LN lanes hold a channel's N states, NPL each (N padded to LN * NPL with zeros), so a wave
// holds 64 / LN channels.  Lane j of a channel also owns every LN-th token: it loads that token's x,
// dt and z and forms its step size, gate and output once, and the channel's other lanes read the
// two values they need through lane-exchange operands.  B and C, shared by all channels, are staged as
// fp32 in LDS.  Everything is fp32 but the inputs' and outputs' own types.
//
// Long sequences are cut into segments where there are too few channels to fill the chip: a first
// kernel forms each segment's end state from a zero start, a second joins them (a segment's whole
// decay is e^{A sum(de)}), and the scan proper then runs all segments at once.
#include "../../include/gdn.h"
#include "gdn_ssm_device.h"

namespace gdn {

namespace {

// The state from a zero start and the summed step sizes of a segment, 32 tokens at a time (97 us at the
// size below, 101 with 16): the recurrence without its outputs.
template <typename T, int LN, int NPL>
__global__ __launch_bounds__(256) void ssm_fwd_summary_kernel(SsmParams p, int groups) {
  constexpr int NP = LN * NPL, TL = kSsmBlock / LN;
  __shared__ __align__(16) float bc[kSsmBlock * NP * 2];
  const Place<LN> w(p, groups, p.split.seg, p.split.nseg);
  if (w.pc.seq < 0 || w.t1 == w.pc.end) return;  // nothing follows the last segment
  const int j = w.j, cc = w.cc;
  float A2[NPL], h[NPL] = {};
  load_decay<NPL>(p, cc, j, A2);
  const float bias = p.dt_bias ? p.dt_bias[cc] : 0.f;
  float dsum = 0.f;
  for (int tb = w.t0; tb < w.t1; tb += kSsmBlock) {  // (whole blocks: only a last segment ends inside one)
    unsigned xr[TL], dr[TL];
    StageBC<T, NP, kSsmBlock, 256> st;
    const auto rx = window<T>(p.x, p.x_pitch, tb, kSsmBlock, p.D), rd = window<T>(p.dt, p.dt_pitch, tb, kSsmBlock, p.D);
#pragma unroll
    for (int g = 0; g < TL; ++g) {
      xr[g] = load_bits<T>(rx, (unsigned)((g * LN + j) * (int)p.x_pitch + cc) * sizeof(T));
      dr[g] = load_bits<T>(rd, (unsigned)((g * LN + j) * (int)p.dt_pitch + cc) * sizeof(T));
    }
    st.load(p, tb, kSsmBlock);
    __syncthreads();
    st.store(bc);
    __syncthreads();
#pragma unroll
    for (int g = 0; g < TL; ++g) {
      float de = of_bits<T>(dr[g]) + bias;
      const float sp = softplus_f(de, nullptr);
      de = p.softplus ? sp : de;
      const float dx = de * of_bits<T>(xr[g]);
      dsum += de;
      static_for<LN>([&](auto k) {
        const float dk = shared_lane<LN, k()>(de), xk = shared_lane<LN, k()>(dx);
        float b[NPL], cf[NPL];
        read_bc<NPL>(bc + ((g * LN + k()) * NP + j * NPL) * 2, b, cf);
#pragma unroll
        for (int i = 0; i < NPL; ++i) h[i] = __builtin_fmaf(decay(dk, A2[i]), h[i], xk * b[i]);
      });
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  if (w.cv) store_state<NPL>(p.seg_state + (int64_t)w.seg * p.D * p.N, w.c, j, p.N, h);
  dsum = group_sum<LN>(dsum);
  if (w.cv && j == 0) p.seg_sum[(int64_t)w.seg * p.D + w.c] = dsum;
}

// The scan proper, a chunk of 16 tokens at a time.  Bound by vector instructions: 20 of the 33 a token
// and wave are the recurrence's own (16 channels x 4 states a lane: 2 products, an exponential and 2
// fused multiply-adds each).  Seven waves a SIMD hide the loads; asking for a 32-token block's inputs a
// block ahead took 99 registers and 177 us instead of 68 and 151 (4 x 2048 tokens x 4096 channels x
// 16 states, bf16, states saved).
template <typename T, int LN, int NPL>
__global__ __launch_bounds__(256) void ssm_fwd_kernel(SsmParams p, int groups) {
  constexpr int NP = LN * NPL, TL = kSsmChunk / LN;
  __shared__ __align__(16) float bc[kSsmChunk * NP * 2];
  const Place<LN> w(p, groups, p.split.seg, p.split.nseg);
  if (w.pc.seq < 0) return;
  const int j = w.j, cc = w.cc, t1 = w.t1;
  const bool gate = p.z;
  const void* zp = gate ? p.z : p.x;
  const int64_t zpitch = gate ? p.z_pitch : p.x_pitch;
  const unsigned vx = (unsigned)(j * (int)p.x_pitch + cc) * sizeof(T), vd = (unsigned)(j * (int)p.dt_pitch + cc) * sizeof(T),
                 vz = (unsigned)(j * (int)zpitch + cc) * sizeof(T);
  const int64_t DN = (int64_t)p.D * p.N;
  float A2[NPL], h[NPL];
  load_decay<NPL>(p, cc, j, A2);
  load_state<NPL>(p.seg_state ? p.seg_state + w.seg * DN : p.h0 ? p.h0 + w.pc.seq * DN : nullptr, cc, j, p.N, h);
  const float bias = p.dt_bias ? p.dt_bias[cc] : 0.f, skip = p.skip ? p.skip[cc] : 0.f;
  int64_t chunk = p.h ? find_piece_before(p.s, w.pc, kSsmChunk, w.lane) + (w.t0 - w.pc.begin) / kSsmChunk : 0;
  const unsigned vy = w.cv ? (unsigned)(j * p.D + w.c) * sizeof(T) : kNowhere;

  for (int tb = w.t0; tb < t1; tb += kSsmChunk) {
    const int rows = min(t1 - tb, kSsmChunk);
    const auto rx = window<T>(p.x, p.x_pitch, tb, rows, p.D), rd = window<T>(p.dt, p.dt_pitch, tb, rows, p.D),
               rz = window<T>(zp, zpitch, tb, rows, p.D), ry = window<T>(p.y, p.D, tb, rows, p.D);
    unsigned xr[TL], dr[TL], zr[TL];
#pragma unroll
    for (int g = 0; g < TL; ++g) {
      xr[g] = load_bits<T>(rx, vx + g * LN * (unsigned)p.x_pitch * sizeof(T));
      dr[g] = load_bits<T>(rd, vd + g * LN * (unsigned)p.dt_pitch * sizeof(T));
      zr[g] = load_bits<T>(rz, vz + g * LN * (unsigned)zpitch * sizeof(T));
    }
    StageBC<T, NP, kSsmChunk, 256> st;
    st.load(p, tb, rows);
    __syncthreads();
    st.store(bc);
    __syncthreads();
    if (p.h && w.cv && chunk < p.chunks) store_state<NPL>(p.h + chunk * DN, w.c, j, p.N, h);
    ++chunk;
#pragma unroll
    for (int g = 0; g < TL; ++g) {
      const float x = of_bits<T>(xr[g]), z = of_bits<T>(zr[g]);
      float de = of_bits<T>(dr[g]) + bias;
      const float sp = softplus_f(de, nullptr);
      de = p.softplus ? sp : de;
      if (g * LN + j >= rows) de = 0.f;  // a token behind the end keeps the state as it is
      const float dx = de * x;
      float yp[LN];
      static_for<LN>([&](auto k) {
        const float dk = shared_lane<LN, k()>(de), xk = shared_lane<LN, k()>(dx);
        float b[NPL], cf[NPL];
        read_bc<NPL>(bc + ((g * LN + k()) * NP + j * NPL) * 2, b, cf);
        float acc = 0.f;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
          h[i] = __builtin_fmaf(decay(dk, A2[i]), h[i], xk * b[i]);
          acc = __builtin_fmaf(cf[i], h[i], acc);
        }
        yp[k()] = acc;
      });
      float y = reduce_scatter<LN>(yp, j) + skip * x;
      const float s = z * sigmoid_f(z);
      y *= gate ? s : 1.f;
      store_bits<T>(ry, to_t<T>(y), vy + g * LN * (unsigned)p.D * sizeof(T));  // dropped behind the end
      __builtin_amdgcn_sched_barrier(0);  // keeps the exponentials of later tokens from filling the registers
    }
  }
  if (p.ht && t1 == w.pc.end && w.cv) store_state<NPL>(p.ht + w.pc.seq * DN, w.c, j, p.N, h);
}

// A sequence's segments in order: seg_state becomes the state at each segment's start.
__global__ __launch_bounds__(256) void ssm_join_kernel(SsmParams p, int per_seq) {
  const int seq = blockIdx.x / per_seq;
  const int64_t e = (int64_t)(blockIdx.x - seq * per_seq) * 256 + threadIdx.x;
  const int lane = threadIdx.x & 63;
  const int64_t DN = (int64_t)p.D * p.N;
  const SeqPieces sp = pieces_of(p.s, seq, p.split.seg, p.split.nseg, lane);
  if (e >= DN) return;
  const int64_t d = e / p.N;
  const float a = p.A[e] * kLog2e;
  float h = p.h0 ? p.h0[seq * DN + e] : 0.f;
  for (int i = 0; i < sp.count; ++i) {
    const int64_t s = sp.first + i;
    const bool last = i == sp.count - 1;
    const float own = last ? 0.f : p.seg_state[s * DN + e], sum = last ? 0.f : p.seg_sum[s * p.D + d];
    p.seg_state[s * DN + e] = h;
    h = __builtin_fmaf(__builtin_amdgcn_exp2f(a * sum), h, own);
  }
}

// One token a row.  A row whose slot is outside the cache, or is an earlier row's, changes nothing
// and gives 0.  A workgroup has U * 256 / LN channels of one row; bound by the states' bytes, so
// everything that a lane reads is asked for before anything is waited for: 256 rows x 4096 channels x 16
// states (143 MB) in 25 us, 5.7 TB/s; one set of channels a workgroup, its loads after one another,
// took 43.
template <typename T, int LN, int NPL, int U>
__global__ __launch_bounds__(256) void ssm_step_kernel(SsmStepParams p, int groups) {
  constexpr int CH = 256 / LN;
  const int b = blockIdx.x / groups, grp = blockIdx.x - b * groups, j = threadIdx.x % LN;
  const int slot = p.slots ? p.slots[b] : b;
  bool live = slot >= 0 && slot < p.S;
  const int other = p.slots && (int)threadIdx.x < b ? p.slots[threadIdx.x] : -1;
  float* st = p.state + (live ? (int64_t)slot * p.D * p.N : 0);
  float h[U][NPL], A2[U][NPL], bn[NPL], cn[NPL], x[U], dt[U], z[U], bias[U], skip[U];
  int c[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    c[u] = (grp * U + u) * CH + threadIdx.x / LN;
    const int cc = min(c[u], p.D - 1);
    load_state<NPL>(st, cc, j, p.N, h[u]);
    load_state<NPL>(p.A, cc, j, p.N, A2[u]);
    x[u] = to_f(static_cast<const T*>(p.x)[b * p.x_pitch + cc]);
    dt[u] = to_f(static_cast<const T*>(p.dt)[b * p.dt_pitch + cc]);
    z[u] = to_f(p.z ? static_cast<const T*>(p.z)[b * p.z_pitch + cc] : static_cast<const T*>(p.x)[b * p.x_pitch + cc]);
    bias[u] = p.dt_bias ? p.dt_bias[cc] : 0.f;
    skip[u] = p.skip ? p.skip[cc] : 0.f;
  }
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const int n = j * NPL + i, nn = min(n, p.N - 1);
    const float bv = to_f(static_cast<const T*>(p.Bm)[b * p.b_pitch + nn]), cv = to_f(static_cast<const T*>(p.Cm)[b * p.c_pitch + nn]);
    bn[i] = n < p.N ? bv : 0.f;
    cn[i] = n < p.N ? cv : 0.f;
  }
  if (p.slots && live) {  // slot is the workgroup's
    int taken = other == slot;
    for (int i = threadIdx.x + 256; i < b; i += 256) taken |= p.slots[i] == slot;
    live = !__syncthreads_or(taken);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float de = dt[u] + bias[u];
    const float sp = softplus_f(de, nullptr);
    de = p.softplus ? sp : de;
    const float dx = de * x[u];
    float acc = 0.f;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      h[u][i] = __builtin_fmaf(decay(de, A2[u][i] * kLog2e), h[u][i], dx * bn[i]);
      acc = __builtin_fmaf(cn[i], h[u][i], acc);
    }
    const float s = z[u] * sigmoid_f(z[u]);
    const float y = (group_sum<LN>(acc) + skip[u] * x[u]) * (p.z ? s : 1.f);
    if (c[u] < p.D) {
      if (live) store_state<NPL>(st, c[u], j, p.N, h[u]);
      if (j == 0) static_cast<T*>(p.y)[(int64_t)b * p.D + c[u]] = to_t<T>(live ? y : 0.f);
    }
  }
}

}  // namespace

// Long sequences are cut where the channels give fewer than two waves a SIMD (2048): the summary costs
// 0.65 of the scan proper, less than what too few waves cost.  Segments are then as short as gives
// eight waves a SIMD.  Sequences of 2048 tokens x 4096 channels x 16 states, bf16 (scan + summary, us): four
// of them uncut, one wave, 303; cut for two 201 + 124, for four 173 + 109, for eight 161 + 106.  Eight of them
// uncut, two waves, 398; cut for eight 307 + 194.
//
// The gradient's registers allow two waves a SIMD (three with 17 to 32 states), so that it takes pieces of
// several segments, and only what is behind the first piece has to be summarised: four of those sequences
// uncut 752 us, in two-wave segments 513 + 164, in pieces of eight-wave segments 520 + 71.
//
// The rule takes sequences for equally long.  One of 16384 tokens beside eight of one token counts as nine
// and is not cut: 2337 us, against 550 by itself.
SsmSplit ssm_split(bool backward, const int* cu, int n, int T, int D, int N) {
  const int ch = ssm_channels(N) / 4;  // channels of a wave
  const int64_t per_seg = (D + ch - 1) / ch;
  int longest = cu ? 1 : T;
  for (int i = 0; cu && i < n; ++i) longest = cu[i + 1] - cu[i] > longest ? cu[i + 1] - cu[i] : longest;
  const int64_t rows = cu ? cu[n] : (int64_t)n * T;
  auto whole = [](int64_t x, int64_t m) { return (x + m - 1) / m * m; };
  // tokens a segment for so many waves in all
  auto tokens = [&](int64_t waves) {
    const int64_t want = (waves + per_seg - 1) / per_seg;
    return whole((rows + want - 1) / want, kSsmBlock);
  };
  const int64_t uncut = whole(longest, kSsmBlock);
  int64_t seg = uncut, main = uncut;
  if (per_seg * n < 2048 && longest > 4 * kSsmBlock) {
    seg = tokens(8192) < 2 * kSsmBlock ? 2 * kSsmBlock : tokens(8192);  // (128 at least: 31.5 us against 25.8 for
                                                                       // 601 tokens x 1000 channels x 24 states)
    seg = seg < uncut ? seg : uncut;
    main = seg == uncut ? uncut : backward ? whole(tokens(2048), seg) : seg;
  }
  SsmSplit r{(int)seg, 0, (int)main, 0};
  for (int i = 0; i < (cu ? n : 1); ++i) {
    const int64_t len = cu ? cu[i + 1] - cu[i] : T, times = cu ? 1 : n;
    r.nseg += (int)(times * ((len + seg - 1) / seg));
    r.nmain += (int)(times * ((len + main - 1) / main));
  }
  return r;
}

size_t ssm_fwd_ws_bytes(const SsmSplit& sp, int n, int D, int N) {
  return sp.nseg > n ? (size_t)sp.nseg * D * (N + 1) * 4 : 0;
}

hipError_t launch_ssm_fwd(SsmParams p, int dtype, void* ws, hipStream_t st) {
  const bool split = p.split.nseg > p.s.n;
  p.seg_state = split ? static_cast<float*>(ws) : nullptr;
  p.seg_sum = split ? p.seg_state + (int64_t)p.split.nseg * p.D * p.N : nullptr;
  return ssm_dispatch(dtype, p.N, [&](auto t, auto ln, auto npl) {
    using T = decltype(t);
    constexpr int LN = decltype(ln)::value, NPL = decltype(npl)::value;
    const int groups = (p.D + 4 * (64 / LN) - 1) / (4 * (64 / LN));
    const dim3 grid((unsigned)(groups * p.split.nseg));
    hipError_t e;
    if (split) {
      ssm_fwd_summary_kernel<T, LN, NPL><<<grid, 256, 0, st>>>(p, groups);
      if ((e = hipGetLastError()) != hipSuccess) return e;
      const int per_seq = (int)(((int64_t)p.D * p.N + 255) / 256);
      ssm_join_kernel<<<dim3((unsigned)(per_seq * p.s.n)), 256, 0, st>>>(p, per_seq);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    ssm_fwd_kernel<T, LN, NPL><<<grid, 256, 0, st>>>(p, groups);
    return hipGetLastError();
  });
}

hipError_t launch_ssm_step(const SsmStepParams& p, int dtype, hipStream_t st) {
  return ssm_dispatch(dtype, p.N, [&](auto t, auto ln, auto npl) {
    using T = decltype(t);
    constexpr int LN = decltype(ln)::value, NPL = decltype(npl)::value, CH = 256 / LN;
    // Four sets of channels a workgroup where that still gives each CU eight; one where the call is
    // small and spreading it shortens it.
    const int64_t one = (int64_t)p.B * ((p.D + CH - 1) / CH);
    const int u = one >= 4 * 8 * 256 ? 4 : 1, groups = (p.D + CH * u - 1) / (CH * u);
    const dim3 grid((unsigned)(groups * p.B));
    if (u == 4) ssm_step_kernel<T, LN, NPL, 4><<<grid, 256, 0, st>>>(p, groups);
    else ssm_step_kernel<T, LN, NPL, 1><<<grid, 256, 0, st>>>(p, groups);
    return hipGetLastError();
  });
}

}  // namespace gdn
