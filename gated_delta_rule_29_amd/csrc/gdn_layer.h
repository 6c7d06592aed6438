// gdn_layer.h -- host-side launch interface of the layer operators around the recurrent scans:
// the short causal convolution, the selective state space scan and the residual RMS norm.
//
// Row tensors are addressed as rows of `pitch` elements: row r of a [tokens, C] tensor starts
// at base + r * pitch.  A dense batch of B sequences of T tokens has rows b * T + t; a packed
// one has its sequences' tokens in order, sequence i covering rows [cu[i], cu[i + 1]).
#pragma once

#include <stdint.h>

#include <hip/hip_runtime.h>

namespace gdn {

// Error reporting shared by the files of the C boundary (defined in gdn_abi.hip): they set the
// calling thread's message and return the status code.
int fail(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
int ok();
int hip_fail(hipError_t e, const char* what);
int check_workspace(const void* ws, size_t bytes, size_t need);

// The sequences of a call: dense (cu null) or packed.
struct Seqs {
  const int* cu;  // device offsets [n + 1] of a packed batch, or nullptr
  int n;          // sequences
  int T;          // tokens of each sequence of a dense batch
  int rows;       // tokens in all
};

struct ConvParams {
  const void* x;
  int64_t x_pitch;
  const float* w;      // [D, W]
  const float* bias;   // [D] or nullptr
  const void* init;    // [n, W-1, D] or nullptr (zero)
  void* y;             // [rows, D]
  void* last;          // [n, W-1, D] or nullptr
  Seqs s;
  int D, W;
  bool silu;
};

struct ConvBwdParams {
  ConvParams f;        // the forward's inputs (y, last unused)
  const void* dy;
  int64_t dy_pitch;
  const void* dlast;   // [n, W-1, D] or nullptr (zero)
  void* dx;            // [rows, D]
  void* dinit;         // [n, W-1, D] or nullptr
  float* dw;           // [D, W]
  float* dbias;        // [D] or nullptr
  float* part;         // workspace: [tiles][W + 1][D]
};

struct ConvStepParams {
  const void* x;
  int64_t x_pitch;
  const float* w;
  const float* bias;
  void* state;         // [S, W-1, D]
  const int* slots;    // [B] or nullptr (row b uses slot b)
  void* y;             // [B, D]
  int B, S, D, W;
  bool silu;
};

size_t conv_bwd_ws_bytes(int rows, int D, int W);
hipError_t launch_conv_fwd(const ConvParams& p, int dtype, hipStream_t st);
hipError_t launch_conv_bwd(const ConvBwdParams& p, int dtype, hipStream_t st);
hipError_t launch_conv_step(const ConvStepParams& p, int dtype, hipStream_t st);

// Tokens between two saved states of the selective scan (and of a step of its kernels); tokens that a
// segment's summary takes at a time, of which segments have a multiple.
constexpr int kSsmChunk = 16;
constexpr int kSsmBlock = 32;
constexpr int kSsmMaxN = 64;
inline int ssm_channels(int N) { return N <= 16 ? 64 : 16; }  // of a workgroup

// Workgroups of 256 threads that a launch can have: it takes fewer than 2^32 threads.
constexpr int64_t kMaxGroups = (1 << 24) - 1;

// How long sequences are cut: segments of `seg` tokens (a multiple of kSsmBlock), nseg in all, are
// summarised and joined; the pass proper takes `main` tokens (a multiple of seg) at a time, nmain in all.
struct SsmSplit {
  int seg, nseg, main, nmain;
};

struct SsmParams {
  const void* x;        // rows of D
  const void* dt;
  const void* z;        // or nullptr
  const void* Bm;       // rows of N
  const void* Cm;
  int64_t x_pitch, dt_pitch, z_pitch, b_pitch, c_pitch;
  const float* A;       // [D, N]
  const float* skip;    // [D] or nullptr
  const float* dt_bias; // [D] or nullptr
  const float* h0;      // [n, D, N] or nullptr (zero)
  void* y;              // [rows, D]
  float* ht;            // [n, D, N] or nullptr
  float* h;             // saved states [chunks, D, N] or nullptr
  int64_t chunks;
  Seqs s;
  int D, N;
  bool softplus;
  SsmSplit split;
  float* seg_state;     // workspace [nseg, D, N]: a segment's end from a zero start, then its start
  float* seg_sum;       // workspace [nseg, D]: the segment's summed step sizes
};

struct SsmBwdParams {
  SsmParams f;          // the forward's inputs; h: the states that it saved
  const void* dy;
  int64_t dy_pitch;
  const float* dht;     // [n, D, N] or nullptr (zero)
  void *dx, *ddt, *dz;  // [rows, D]
  void *dB, *dC;        // [rows, N]
  float *dA;            // [D, N]
  float *dskip;         // [D] or nullptr
  float *ddt_bias;      // [D] or nullptr
  float *dh0;           // [n, D, N] or nullptr
  float* part_bc;       // workspace [channel groups][rows][2][N]
  float* part_a;        // workspace [nmain][D][N + 2]
};

struct SsmStepParams {
  const void *x, *dt, *z, *Bm, *Cm;
  int64_t x_pitch, dt_pitch, z_pitch, b_pitch, c_pitch;
  const float *A, *skip, *dt_bias;
  float* state;         // [S, D, N]
  const int* slots;     // [B] or nullptr
  void* y;              // [B, D]
  int B, S, D, N;
  bool softplus;
};

// The split of a call over n sequences: from their offsets on the host, or (cu null) of T tokens each.
SsmSplit ssm_split(bool backward, const int* cu, int n, int T, int D, int N);
size_t ssm_fwd_ws_bytes(const SsmSplit& sp, int n, int D, int N);
size_t ssm_bwd_ws_bytes(const SsmSplit& sp, int rows, int D, int N);
hipError_t launch_ssm_fwd(SsmParams p, int dtype, void* ws, hipStream_t st);
hipError_t launch_ssm_bwd(SsmBwdParams p, int dtype, void* ws, hipStream_t st);
hipError_t launch_ssm_step(const SsmStepParams& p, int dtype, hipStream_t st);

struct NormParams {
  const void* x;         // rows of D
  const void* residual;  // or nullptr
  int64_t x_pitch, r_pitch;
  const float* w;        // [D]
  float eps;
  void* y;               // [M, D] dtype, or e4m3 bytes with `scale`
  void* sum;             // [M, D] residual type, or nullptr
  float* rstd;           // [M] or nullptr
  float* scale;          // [M, ceil(D / block)] or nullptr
  int M, D, block;       // block: columns that share a scale (0: the row)
};

struct NormBwdParams {
  const void* dy;        // rows of D
  const void* s;         // the normalised values, rows of D
  const void* dsum;      // or nullptr
  int64_t dy_pitch, s_pitch, dsum_pitch;
  const float* w;
  const float* rstd;
  void* dres;            // [M, D] in the type of s
  void* dx;              // [M, D] in the type of dy, or nullptr
  float* dw;             // [D]
  float* part;           // workspace [groups][D]
  int M, D;
};

constexpr int kNormMaxD = 32768;
size_t norm_bwd_ws_bytes(int M, int D);
hipError_t launch_norm_fwd(const NormParams& p, int dtype, int rdtype, hipStream_t st);
hipError_t launch_norm_bwd(const NormBwdParams& p, int dtype, int sdtype, hipStream_t st);

}  // namespace gdn
