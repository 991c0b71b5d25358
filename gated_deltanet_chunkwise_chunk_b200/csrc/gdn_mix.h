// Host-side declarations of the mixing-layer operators (short convolution, selective scan, layer
// norm): problem descriptions and launchers.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace gdn {
namespace mix {

// Sequences of one call: B of T tokens each, or n packed ones (cu, device).
struct Seqs {
  const int64_t* cu;
  int* status;  // the workspace's status word
  int64_t T;    // tokens of a dense sequence, or of the whole packed batch
  int n;        // sequences
};

inline int64_t max_units(const Seqs& s, int lg) {
  if (s.cu) return (s.T >> lg) + s.n;
  return (s.T == 0 ? 1 : ((s.T - 1) >> lg) + 1) * s.n;
}

// Validates a packing (cu[0] = 0, non-decreasing, cu[n] = T) and writes the status word.
cudaError_t check_packing(const Seqs& s, cudaStream_t stream);

struct Conv {
  Seqs seqs;
  int64_t D, ld;
  int W, dtype;
  bool silu;
  const void* x;
  const float* weight;
  const float* bias;
  const void* init;
  void* y;
  void* final;
  // backward
  const void* dy;
  const void* dfinal;
  void* dx;
  float* dweight;
  float* dbias;
  void* dinit;
  float* part;  // [units][W + 1][D]
};
constexpr int kConvMaxW = 8;
int64_t conv_bwd_units(const Seqs& s, int64_t D);
cudaError_t conv_forward(const Conv& c, cudaStream_t s);
cudaError_t conv_backward(const Conv& c, cudaStream_t s);
cudaError_t conv_step(const Conv& c, cudaStream_t s);

struct Norm {
  int64_t rows, D;
  int64_t inner_x, ld_x, inner_z, ld_z;
  int dtype;
  bool rms;
  float eps;
  const void* x;
  const float* weight;
  const float* bias;
  const void* gate;
  void* y;
  float* stats;
  // backward
  const void* dy;
  void* dx;
  void* dgate;
  float* dweight;
  float* dbias;
  float* part;
};
size_t norm_bwd_part_floats(int64_t rows, int64_t D);
cudaError_t norm_forward(const Norm& c, cudaStream_t s);
cudaError_t norm_backward(const Norm& c, cudaStream_t s);

struct Ssm {
  Seqs seqs;
  int64_t D, ld_x, ld_dt, ld_b, ld_c;
  int N, G, dtype;
  int lg;    // log2 of a segment's tokens, in the direction that runs
  bool cut;  // whether a sequence may have several segments
  // accesses that the per-channel tensors, and B and C, take: 2 of 16 bytes, 1 of 4, 0 of single elements
  int vec, vec_bc;
  const void* x;
  const void* dt;
  const float* A_log;
  const void* Bm;
  const void* Cm;
  const float* skip;
  const float* dt_bias;
  const float* init;
  void* y;
  float* final;
  // workspace
  float* starts;  // [units][D][NP]  state (backward: gradient) at a segment's open end
  float* sums;    // [units][D]      sum of delta over a segment
  float* ckpt;    // [16-token units][D][NP]  states entering every 16th token, or null
  // backward
  const void* dy;
  const float* dfinal;
  void* dx;
  void* ddt;
  void* dB;
  void* dC;
  float* dA_log;
  float* dskip;
  float* ddt_bias;
  float* dinit;
  float* part_bc;   // [channel tiles of a group][tokens][G][2][NP]
  float* part_par;  // [units of at most 256 tokens][D][N + 2]
};

// What a call needs besides the status word; offsets are the caller's.
struct SsmSizes {
  int lg[2];    // forward, backward
  bool cut[2];
  int64_t starts, sums, ckpt, part_bc, part_par;  // floats
};
int ssm_padded(int N);
SsmSizes ssm_sizes(const Seqs& s, int64_t tokens, int64_t D, int N, int G);
cudaError_t ssm_forward(const Ssm& c, cudaStream_t s);
cudaError_t ssm_backward(const Ssm& c, cudaStream_t s);
cudaError_t ssm_step(const Ssm& c, cudaStream_t s);

// Strands of rows that a sum of n partial rows is split into, by n alone.
inline int sum_strands(int64_t n) { return n <= 8 ? 1 : n <= 128 ? 8 : 32; }

// Column sums of partial rows part[r * ld + c], r < n, in a fixed order: column j D + d of a row [W + 1][D] goes
// to out[d W + j], the last D to out2; either may be null.  With packed sequences nothing is written where their
// boundaries were found invalid (and the rows never were).
cudaError_t column_sums(const char* name, const Seqs& seqs, const float* part, int64_t n, int64_t ld, int64_t width, float* out,
                        float* out2, int W, int64_t D, cudaStream_t s);

}  // namespace mix
}  // namespace gdn
