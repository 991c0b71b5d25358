// Selective state space scan: what its kernels share.
//   delta[t,d] = softplus(dt[t,d] + dt_bias[d]),   A[d,n] = -exp(A_log[d,n]),
//   h[t,d,n] = exp(delta A) h[t-1,d,n] + delta x[t,d] B[t,g,n],   y[t,d] = sum_n C[t,g,n] h[t,d,n] + Dskip[d] x[t,d],
// g = d / (D / G) the channel's group.
//
// The states of a channel never mix with another channel's, so the work of a token is D x N independent
// recurrences, each an exponential and about four multiply-adds: no matrix product has these entries (the
// decay differs in t, d and n), and the exponentials bound it: 16 per clock and multiprocessor.
//
// A warp walks over the tokens of a piece of a sequence with one channel and four states to a lane: lane
// (cl, nl) holds states 4 nl .. 4 nl + 3 of channel cl, NL = NP / 4 lanes to a channel (NP: N rounded up to a
// power of two) and CW = 32 / NL channels to a warp.  So few states to a lane (instead of, say, four channels
// by four states) make as many warps as there are, and one sequence of a wide layer then fills the card
// without being cut along time, which would cost a second pass of exponentials.
// Tiles of 32 tokens are staged in shared memory: a lane fetches one token's CW channels of x and dt, applies
// the softplus once and leaves them token-contiguous, so that a state lane reads four tokens with one load;
// B and C are shared by the block's warps.  Tokens past the piece's end are staged as delta = x = 0, which
// leaves every state as it is.
#pragma once

#include "kda_gate_math.cuh"
#include "mix_common.cuh"

namespace gdn {
namespace mix {

constexpr int kTile = 32;        // tokens of a staged tile: one a lane
constexpr int kRow = kTile + 4;  // its padded row: 16-byte aligned quads, CW rows on distinct banks
constexpr int kWarps = 4;        // warps of a block
constexpr int kCkpt = 16;        // tokens between the states that the forward keeps for the backward
constexpr int kCkptLog = 4;
constexpr float kLog2e = 1.44269504088896341f;
constexpr float kLn2 = 0.693147180559945309f;

template <int NP>
struct Shape {
  static constexpr int NL = NP / 4;        // lanes of a channel
  static constexpr int CW = 32 / NL;       // channels of a warp
  static constexpr int CC = CW * kWarps;   // and of a block
};

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// softplus with the framework's pass-through above 20
__device__ __forceinline__ float softplus_acc(float x) {
  return x > 20.f ? x : fmaxf(x, 0.f) + log1p_unit(exp_acc(-fabsf(x)));
}

// Sums M values over the lanes (lane / STRIDE) % LANES.  While a lane has several values, each step
// halves them: a lane keeps one half and hands over the other.  Afterwards a lane has M / LANES values,
// the first of them number M / LANES * (its index in bit-reversed order), or one that LANES / M lanes share.
template <int M, int LANES, int STRIDE>
__device__ __forceinline__ void lane_sums(float* v, int lane) {
  if constexpr (LANES > 1) {
    if constexpr (M > 1) {
      const bool up = lane & STRIDE;
#pragma unroll
      for (int i = 0; i < M / 2; ++i) {
        const float keep = up ? v[M / 2 + i] : v[i], give = up ? v[i] : v[M / 2 + i];
        v[i] = keep + __shfl_xor_sync(0xffffffffu, give, STRIDE);
      }
      lane_sums<M / 2, LANES / 2, STRIDE * 2>(v, lane);
    } else {
      v[0] += __shfl_xor_sync(0xffffffffu, v[0], STRIDE);
      lane_sums<1, LANES / 2, STRIDE * 2>(v, lane);
    }
  }
}

// The number of the first value that lane_sums<M, LANES, 1> leaves with lane index l.
template <int M, int LANES>
__device__ __forceinline__ int lane_slot(int l) {
  int at = 0;
#pragma unroll
  for (int m = M, k = LANES; m > 1 && k > 1; m /= 2, k /= 2, l >>= 1) at += (l & 1) * (m / 2);
  return at;
}

// A warp's tile of one per-channel input, as fetched: lane = token.
template <typename T, int CW>
struct Cols {
  static constexpr int V = CW * (int)sizeof(T) > 16 ? 16 / (int)sizeof(T) : CW;
  Pack<T, V> r[CW / V];

  // row: the token's first element of the warp's channels; n: how many of them exist
  __device__ __forceinline__ void fetch(const T* row, bool in, bool vec, int n) {
    if (vec) {
#pragma unroll
      for (int i = 0; i < CW / V; ++i) {
        if (in && n > 0)
          r[i].load(row + i * V);
        else
          r[i].zero();
      }
    } else {
#pragma unroll
      for (int i = 0; i < CW; ++i) r[i / V].v[i % V] = in && i < n ? row[i] : down<T>(0.f);
    }
  }
  __device__ __forceinline__ float get(int i) const { return up<T>(r[i / V].v[i % V]); }
  __device__ __forceinline__ void put(int i, float f) { r[i / V].v[i % V] = down<T>(f); }
  __device__ __forceinline__ void store(T* row, bool in, bool vec, int n) const {
    if (!in) return;
    if (vec) {
      if (n > 0) {
#pragma unroll
        for (int i = 0; i < CW / V; ++i) r[i].store(row + i * V);
      }
    } else {
#pragma unroll
      for (int i = 0; i < CW; ++i)
        if (i < n) row[i] = r[i / V].v[i % V];
    }
  }
};

// A block's tile of B or C: [kTile][NP] floats in shared memory, zero past N and past the piece.
template <typename T, int NP>
struct Mat {
  static constexpr int PER = kTile * NP / (kWarps * 32);
  T r[PER];

  // m: element (first token of the tile, state 0)
  __device__ __forceinline__ void fetch(const T* m, int64_t ld, int N, int tokens) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = i * kWarps * 32 + threadIdx.x, t = e / NP, n = e % NP;
      r[i] = t < tokens && n < N ? m[t * ld + n] : down<T>(0.f);
    }
  }
  __device__ __forceinline__ void stage(float* s) const {
#pragma unroll
    for (int i = 0; i < PER; ++i) s[i * kWarps * 32 + threadIdx.x] = up<T>(r[i]);
  }
};

// Where a block and a warp are: unit, group and channels.
template <int NP>
struct Place {
  using S = Shape<NP>;
  Piece p;
  int g, warp, lane, nl, cl, n;  // n: channels that exist of the warp's
  int64_t c0, ch;                // the warp's first channel, the lane's
  bool live;

  // whether the unit exists; the channels are set either way
  __device__ __forceinline__ bool find(const Ssm& s, int lg) {
    warp = threadIdx.x >> 5;
    lane = threadIdx.x & 31;
    nl = lane % S::NL;
    cl = lane / S::NL;
    const int64_t Dg = s.D / s.G, tiles = (Dg + S::CC - 1) / S::CC;
    g = (int)(blockIdx.y / tiles);
    const int64_t local = (blockIdx.y - g * tiles) * S::CC + warp * S::CW, rest = Dg - local;
    n = rest <= 0 ? 0 : rest < S::CW ? (int)rest : S::CW;
    c0 = g * Dg + local;
    ch = c0 + cl;
    live = cl < n;
    return find_piece(s.seqs, blockIdx.x, lg, p);
  }
};

// Four states of a lane from and to [...][D][N] and the padded [...][D][NP] workspace.
__device__ __forceinline__ void load_states(const float* p, int N, int n0, float (&h)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) h[j] = n0 + j < N ? p[n0 + j] : 0.f;
}
__device__ __forceinline__ void store_states(float* p, int N, int n0, const float (&h)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (n0 + j < N) p[n0 + j] = h[j];
}

// A log2(e), kept finite so that a token of delta = 0 past the piece's end keeps the state
__device__ __forceinline__ float decay_rate(float A_log) {
  const float a = -expf(A_log) * kLog2e;
  return a < -3.4e38f ? -3.4e38f : a;
}

// that of a lane's four states (0 for states that do not exist: their decay is 1, their input 0)
__device__ __forceinline__ void load_decay(const Ssm& s, int64_t ch, bool live, int n0, float (&a)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) a[j] = live && n0 + j < s.N ? decay_rate(s.A_log[ch * s.N + n0 + j]) : 0.f;
}

template <int NP>
__device__ __forceinline__ int64_t state_at(const Ssm& s, int64_t unit, int64_t ch, int n0) {
  return (unit * s.D + ch) * NP + n0;
}

}  // namespace mix
}  // namespace gdn
