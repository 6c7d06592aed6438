// gdn_conv.hip -- the short causal convolution in front of a recurrent scan: one filter of W
// (2..4) taps a channel, a bias and SiLU, over dense or packed sequences, its gradient, and its
// single-token form on a cache of the last W - 1 tokens.
//
//   u_t = bias + sum_{i < W} w_i x_{t-(W-1)+i},   y_t = u_t or u_t / (1 + e^{-u_t})
//
// Rows before a sequence's first token are the initial rows init[0 .. W-2] (oldest first).
#include "../../include/gdn.h"
#include "gdn_layer_device.h"

namespace gdn {

namespace {

// Both passes are bound by memory (2 or 3 values a token and channel, some 10 operations each).  One
// thread walks the tokens of a tile for V channels, its window in registers; neighbouring threads have
// neighbouring channels, so that a wave reads a row in one stretch.  V is 4 (one access of 8 or 16
// bytes), or 1 where widths, pitches or addresses do not allow that.  Eight bf16 channels a thread
// were slower: their taps, window and tokens take 150 registers (forward over 16384 x 4096 bf16
// with a 32-token tile 64 us against 53, which is 5.1 TB/s; gradient 100 against 90).
//
// Tokens whose loads are asked for together; they have to hide the memory's latency.  (Forward with
// 4: 61 us.  The gradient's other registers leave room for 4: 90 us against 104 with 8.)
constexpr int kFwdBatch = 8, kBwdBatch = 4;
constexpr int kBwdTile = 64;  // (the first tokens' window and the last ones' du are read twice)

template <typename T, int W, int V>
struct Filter {
  float w[W][V], b[V];
  __device__ void load(const ConvParams& p, int d0) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
      for (int k = 0; k < W; ++k) w[k][v] = p.w[(int64_t)(d0 + v) * W + k];
      b[v] = p.bias ? p.bias[d0 + v] : 0.f;
    }
  }
  // u of the token whose window is win[0 .. W-2], x
  __device__ float u(const float (&win)[W - 1][V], const float (&x)[V], int v) const {
    float s = b[v];
#pragma unroll
    for (int k = 0; k < W - 1; ++k) s = __builtin_fmaf(w[k][v], win[k][v], s);
    return __builtin_fmaf(w[W - 1][v], x[v], s);
  }
};

// Initial rows of sequence `seq` (zero where there are none).
template <typename T, int W, int V>
__device__ __forceinline__ void load_init(const ConvParams& p, int seq, int d0, int k, float (&x)[V]) {
  if (p.init) {
    loadv<T, V>(static_cast<const T*>(p.init) + ((int64_t)seq * (W - 1) + k) * p.D + d0, x);
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] = 0.f;
  }
}

// The offsets of a packed batch in LDS, where there are not too many: finding a tile's sequence is a chain
// of dependent reads, each of which waits for the memory otherwise.  Called by the whole workgroup.
constexpr int kLdsOffsets = 1024;
__device__ __forceinline__ Seqs offsets_in_lds(const Seqs& s, int (&cu)[kLdsOffsets + 1]) {
  Seqs r = s;
  if (s.cu && s.n <= kLdsOffsets) {
    for (int i = threadIdx.x; i <= s.n; i += blockDim.x) cu[i] = s.cu[i];
    __syncthreads();
    r.cu = cu;
  }
  return r;
}

// The window of token t: rows t-(W-1) .. t-1 of its sequence, which starts at row `begin`.
template <typename T, int W, int V>
__device__ __forceinline__ void load_window(const ConvParams& p, int seq, int begin, int t, int d0,
                                            float (&win)[W - 1][V]) {
#pragma unroll
  for (int k = 0; k < W - 1; ++k) {
    const int r = t - (W - 1) + k;
    if (r >= begin) loadv<T, V>(static_cast<const T*>(p.x) + r * p.x_pitch + d0, win[k]);
    else load_init<T, W, V>(p, seq, d0, r - begin + W - 1, win[k]);
  }
}

template <int W, int V>
__device__ __forceinline__ void shift(float (&win)[W - 1][V], const float (&x)[V]) {
#pragma unroll
  for (int v = 0; v < V; ++v) {
#pragma unroll
    for (int k = 0; k < W - 2; ++k) win[k][v] = win[k + 1][v];
    win[W - 2][v] = x[v];
  }
}

template <typename T, int W, int V>
__global__ __launch_bounds__(256) void conv_fwd_kernel(ConvParams p, int groups, int tile) {
  __shared__ int cu[kLdsOffsets + 1];
  p.s = offsets_in_lds(p.s, cu);
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t tl = id / groups;
  const int d0 = (int)(id - tl * groups) * V;
  if (tl * tile >= p.s.rows) return;
  const int t0 = (int)tl * tile, t1 = min(t0 + tile, p.s.rows);
  const T* x = static_cast<const T*>(p.x);
  T* y = static_cast<T*>(p.y);
  Filter<T, W, V> f;
  f.load(p, d0);
  int seq = seq_of_row(p.s, t0);
  int begin = min(seq_begin(p.s, seq), t0), end = seq_begin(p.s, seq + 1);
  float win[W - 1][V];
  load_window<T, W, V>(p, seq, begin, t0, d0, win);
  auto token = [&](int t, const float (&xt)[V]) {
    float o[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float u = f.u(win, xt, v);
      o[v] = p.silu ? u * sigmoid_f(u) : u;
    }
    storev<T, V>(y + (int64_t)t * p.D + d0, o);
    shift<W, V>(win, xt);
  };
  for (int t = t0; t < t1;) {
    if (t >= end && seq + 1 < p.s.n) {
      ++seq;
      begin = end;
      end = seq_begin(p.s, seq + 1);
      load_window<T, W, V>(p, seq, t, t, d0, win);
    }
    if (t + kFwdBatch <= min(end, t1)) {
      float xt[kFwdBatch][V];
#pragma unroll
      for (int i = 0; i < kFwdBatch; ++i) loadv<T, V>(x + (t + i) * p.x_pitch + d0, xt[i]);
#pragma unroll
      for (int i = 0; i < kFwdBatch; ++i) token(t + i, xt[i]);
      t += kFwdBatch;
    } else {
      float xt[V];
      loadv<T, V>(x + t * p.x_pitch + d0, xt);
      token(t, xt);
      ++t;
    }
    if (p.last && t == end) {
#pragma unroll
      for (int k = 0; k < W - 1; ++k)
        storev<T, V>(static_cast<T*>(p.last) + ((int64_t)seq * (W - 1) + k) * p.D + d0, win[k]);
    }
  }
}

// Gradient.  du_t = dy_t act'(u_t);  dx_r = sum_k w_k du_{r+(W-1)-k} over the tokens of r's
// sequence, plus dlast for its last W - 1 rows;  dw_k = sum_t du_t x_{t-(W-1)+k};  dbias = sum du.
// A tile's thread walks its tokens and up to W - 1 more of the same sequence, whose du its last
// rows need; acc[k] gathers row t-(W-1)+k.  Rows before the sequence's first token are the initial
// rows, written by the tile that holds that token.
template <typename T, int W, int V>
__global__ __launch_bounds__(256) void conv_bwd_kernel(ConvBwdParams p, int groups, int tile) {
  __shared__ int cu[kLdsOffsets + 1];
  p.f.s = offsets_in_lds(p.f.s, cu);
  const ConvParams& f = p.f;
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t tl = id / groups;
  const int d0 = (int)(id - tl * groups) * V;
  if (tl * tile >= f.s.rows) return;
  const int t0 = (int)tl * tile, t1 = min(t0 + tile, f.s.rows);
  const T* x = static_cast<const T*>(f.x);
  const T* dy = static_cast<const T*>(p.dy);
  Filter<T, W, V> w;
  w.load(f, d0);
  int seq = seq_of_row(f.s, t0);
  int begin = min(seq_begin(f.s, seq), t0), end = seq_begin(f.s, seq + 1);
  float win[W - 1][V], acc[W][V] = {}, dw[W + 1][V] = {};
  load_window<T, W, V>(f, seq, begin, t0, d0, win);

  auto emit = [&](int r, const float (&a)[V]) {
    if (r >= begin) {
      if (r >= t0 && r < t1) storev<T, V>(static_cast<T*>(p.dx) + (int64_t)r * f.D + d0, a);
    } else if (begin >= t0 && p.dinit) {
      storev<T, V>(static_cast<T*>(p.dinit) + ((int64_t)seq * (W - 1) + r - begin + W - 1) * f.D + d0, a);
    }
  };

  // mine: the token is the tile's own (its du counts in dw and dbias)
  auto token = [&](int t, const float (&xt)[V], const float (&g)[V], bool mine) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float du = g[v];
      if (f.silu) {
        const float u = w.u(win, xt, v), s = sigmoid_f(u);
        du *= s * (1.f + u * (1.f - s));
      }
#pragma unroll
      for (int k = 0; k < W; ++k) acc[k][v] = __builtin_fmaf(w.w[k][v], du, acc[k][v]);
      if (mine) {
#pragma unroll
        for (int k = 0; k < W - 1; ++k) dw[k][v] = __builtin_fmaf(du, win[k][v], dw[k][v]);
        dw[W - 1][v] = __builtin_fmaf(du, xt[v], dw[W - 1][v]);
        dw[W][v] += du;
      }
    }
    emit(t - (W - 1), acc[0]);
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
      for (int k = 0; k < W - 1; ++k) acc[k][v] = acc[k + 1][v];
      acc[W - 1][v] = 0.f;
    }
    shift<W, V>(win, xt);
  };

  for (int t = t0; t < t1 + W - 1;) {
    if (t >= end) {
      if (t >= t1 || seq + 1 >= f.s.n) break;
      ++seq;
      begin = end;
      end = seq_begin(f.s, seq + 1);
      load_window<T, W, V>(f, seq, t, t, d0, win);
    }
    if (t + kBwdBatch <= min(end, t1)) {
      float xt[kBwdBatch][V], g[kBwdBatch][V];
#pragma unroll
      for (int i = 0; i < kBwdBatch; ++i) {
        loadv<T, V>(x + (t + i) * f.x_pitch + d0, xt[i]);
        loadv<T, V>(dy + (t + i) * p.dy_pitch + d0, g[i]);
      }
#pragma unroll
      for (int i = 0; i < kBwdBatch; ++i) token(t + i, xt[i], g[i], true);
      t += kBwdBatch;
    } else {
      float xt[V], g[V];
      loadv<T, V>(x + t * f.x_pitch + d0, xt);
      loadv<T, V>(dy + t * p.dy_pitch + d0, g);
      token(t, xt, g, t < t1);
      ++t;
    }
    if (t == end) {  // acc[k] is row end - (W-1) + k
#pragma unroll
      for (int k = 0; k < W - 1; ++k) {
        if (p.dlast) {
          float l[V];
          loadv<T, V>(static_cast<const T*>(p.dlast) + ((int64_t)seq * (W - 1) + k) * f.D + d0, l);
#pragma unroll
          for (int v = 0; v < V; ++v) acc[k][v] += l[v];
        }
        emit(end - (W - 1) + k, acc[k]);
#pragma unroll
        for (int v = 0; v < V; ++v) acc[k][v] = 0.f;
      }
    }
  }
#pragma unroll
  for (int k = 0; k <= W; ++k)
#pragma unroll
    for (int v = 0; v < V; ++v) p.part[(tl * (W + 1) + k) * f.D + d0 + v] = dw[k][v];
}

struct ConvWeightOut {
  float *dw, *dbias;
  int D, W;
  __device__ void operator()(int64_t c, float s) const {
    const int k = (int)(c / D), d = (int)(c - (int64_t)k * D);
    if (k < W) dw[(int64_t)d * W + k] = s;
    else if (dbias) dbias[d] = s;
  }
};

// One token a row: the window is the row's slot of the cache, which then moves on by one token.
// A row whose slot is outside the cache, or is an earlier row's, changes nothing and gives 0.
template <typename T, int W, int V>
__global__ __launch_bounds__(256) void conv_step_kernel(ConvStepParams p, int groups) {
  const int per_row = (groups + 255) / 256;
  const int b = blockIdx.x / per_row, g = (blockIdx.x - b * per_row) * 256 + threadIdx.x;
  const int slot = p.slots ? p.slots[b] : b;
  bool live = slot >= 0 && slot < p.S;
  if (p.slots && live) live = !slot_taken(p.slots, b, slot);  // slot is the workgroup's
  if (g >= groups) return;
  const int d0 = g * V;
  T* y = static_cast<T*>(p.y) + (int64_t)b * p.D + d0;
  float o[V] = {};
  if (live) {
    ConvParams f{};
    f.w = p.w;
    f.bias = p.bias;
    Filter<T, W, V> w;
    w.load(f, d0);
    T* st = static_cast<T*>(p.state) + (int64_t)slot * (W - 1) * p.D + d0;
    float win[W - 1][V], xt[V];
#pragma unroll
    for (int k = 0; k < W - 1; ++k) loadv<T, V>(st + (int64_t)k * p.D, win[k]);
    loadv<T, V>(static_cast<const T*>(p.x) + b * p.x_pitch + d0, xt);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float u = w.u(win, xt, v);
      o[v] = p.silu ? u * sigmoid_f(u) : u;
    }
    shift<W, V>(win, xt);
#pragma unroll
    for (int k = 0; k < W - 1; ++k) storev<T, V>(st + (int64_t)k * p.D, win[k]);
  }
  storev<T, V>(y, o);
}

bool aligned(std::initializer_list<const void*> ps, int dtype) {
  for (const void* q : ps)
    if (reinterpret_cast<uintptr_t>(q) % (dtype == GDN_DTYPE_BF16 ? 8 : 16)) return false;
  return true;
}

// f(T{}, W, V): the instance for these types and widths; vec: four channels at once are possible.
template <typename F>
hipError_t dispatch(int dtype, int W, bool vec, F&& f) {
  using std::integral_constant;
  auto taps = [&](auto t, auto v) {
    switch (W) {
      case 2: return f(t, integral_constant<int, 2>{}, v);
      case 3: return f(t, integral_constant<int, 3>{}, v);
      default: return f(t, integral_constant<int, 4>{}, v);
    }
  };
  auto width = [&](auto t) {
    return vec ? taps(t, integral_constant<int, 4>{}) : taps(t, integral_constant<int, 1>{});
  };
  return dtype == GDN_DTYPE_BF16 ? width(bf16{}) : width(float{});
}

// Tokens of a forward tile: 32, or fewer where that would leave the chip without 4 waves a SIMD (8189 packed
// tokens x 4096 channels: 32 tokens 35.9 us, 16 37.1, 8 41.1).
int fwd_tile(int rows, int groups) {
  int tile = 32;
  while (tile > kFwdBatch && (int64_t)((rows + tile - 1) / tile) * groups < 4096 * 64) tile /= 2;
  return tile;
}

}  // namespace

size_t conv_bwd_ws_bytes(int rows, int D, int W) {
  return (size_t)((rows + kBwdTile - 1) / kBwdTile) * (W + 1) * D * 4;
}

hipError_t launch_conv_fwd(const ConvParams& p, int dtype, hipStream_t st) {
  const bool vec = p.D % 4 == 0 && p.x_pitch % 4 == 0 && aligned({p.x, p.init, p.y, p.last}, dtype);
  return dispatch(dtype, p.W, vec, [&](auto t, auto w, auto v) {
    const int groups = p.D / v;
    const int tile = fwd_tile(p.s.rows, groups);
    const int64_t threads = (int64_t)((p.s.rows + tile - 1) / tile) * groups;
    conv_fwd_kernel<decltype(t), w(), v()><<<dim3((unsigned)((threads + 255) / 256)), 256, 0, st>>>(p, groups, tile);
    return hipGetLastError();
  });
}

hipError_t launch_conv_bwd(const ConvBwdParams& p, int dtype, hipStream_t st) {
  const ConvParams& f = p.f;
  const bool vec = f.D % 4 == 0 && f.x_pitch % 4 == 0 && p.dy_pitch % 4 == 0 &&
                   aligned({f.x, f.init, p.dy, p.dlast, p.dx, p.dinit}, dtype);
  return dispatch(dtype, f.W, vec, [&](auto t, auto w, auto v) {
    const int groups = f.D / v;
    const int tiles = (f.s.rows + kBwdTile - 1) / kBwdTile;
    const int64_t threads = (int64_t)tiles * groups;
    conv_bwd_kernel<decltype(t), w(), v()><<<dim3((unsigned)((threads + 255) / 256)), 256, 0, st>>>(p, groups, kBwdTile);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t cols = (int64_t)(f.W + 1) * f.D;
    return column_sum(p.part, tiles, cols, ConvWeightOut{p.dw, p.dbias, f.D, f.W}, st);
  });
}

hipError_t launch_conv_step(const ConvStepParams& p, int dtype, hipStream_t st) {
  const bool vec = p.D % 4 == 0 && p.x_pitch % 4 == 0 && aligned({p.x, p.state, p.y}, dtype);
  return dispatch(dtype, p.W, vec, [&](auto t, auto w, auto v) {
    const int groups = p.D / v;
    const int per_row = (groups + 255) / 256;
    conv_step_kernel<decltype(t), w(), v()><<<dim3((unsigned)(p.B * per_row)), 256, 0, st>>>(p, groups);
    return hipGetLastError();
  });
}

}  // namespace gdn
