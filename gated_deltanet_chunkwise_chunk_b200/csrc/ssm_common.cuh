// Selective state space scan: what its kernels share.
//   delta[t,d] = softplus(dt[t,d] + dt_bias[d]),   A[d,n] = -exp(A_log[d,n]),
//   h[t,d,n] = exp(delta A) h[t-1,d,n] + delta x[t,d] B[t,g,n],   y[t,d] = sum_n C[t,g,n] h[t,d,n] + Dskip[d] x[t,d],
// g = d / (D / G) the channel's group.
//
// The states of a channel never mix with another channel's, so the work of a token is D x N independent
// recurrences, each an exponential and about four multiply-adds: no matrix product has these entries (the
// decay differs in t, d and n).  Exponentials (16 per clock and multiprocessor) and instruction issue bound it.
//
// A warp walks over the tokens of a segment with one channel and SPL states to a lane: lane (cl, nl) holds
// states SPL nl .. of channel cl, NL = NP / SPL lanes to a channel (NP: N rounded up to a power of two) and
// CW = 32 / NL channels to a warp; a block has CC = 512 / NP channels in 16 / SPL such warps, and four more
// warps that feed them.  Tiles of 32 tokens arrive in shared memory three deep by asynchronous copies; the
// feeding warps widen them to fp32 (the softplus applied once) with the tokens of a channel (of a state, for B
// and C) contiguous, so that a lane reads four tokens with one load and pairs of tokens go through packed
// multiply-adds, and write the results out.  A tile is widened while the one before it is worked on: one
// barrier a tile.  Tokens past the segment's end are staged as delta = x = 0, which leaves every state as it is.
#pragma once

#include "mix_common.cuh"

namespace gdn {
namespace mix {

constexpr int kTile = 32;        // tokens of a staged tile
constexpr int kRow = kTile + 4;  // a widened row: rows of a warp, or of its lanes, are on distinct banks
constexpr int kFeed = 128;       // feeding threads: a lane has a token, a warp a quarter of the channels
// Raw tiles in flight; two where the widest tiles would not fit otherwise.
template <typename T, int NP>
constexpr int kRing = sizeof(T) == 4 && NP == 64 ? 2 : 3;
constexpr int kCkpt = 16;  // tokens between the states that the forward keeps for the backward
constexpr int kCkptLog = 4;
constexpr int kParLog = 8;  // tokens that a partial sum of the parameters' gradients has at most
constexpr float kLog2e = 1.44269504088896341f;
constexpr float kLn2 = 0.693147180559945309f;

template <int NP, int SPL>
struct Shape {
  static constexpr int NL = NP / SPL;       // lanes of a channel
  static constexpr int CW = 32 / NL;        // channels of a warp
  static constexpr int CC = 512 / NP;       // channels of a block
  static constexpr int WORK = 32 * CC / CW; // threads that hold states; the feeding threads follow
  static constexpr int NT = WORK + kFeed;
  static constexpr int FC = CC / 4;         // channels of a feeding thread
};

// The row of state n in a widened [NP][kRow] array: the rows that lanes read together are neighbours.
template <int NP, int SPL>
__device__ __forceinline__ int state_row(int n) { return (n % SPL * (NP / SPL) + n / SPL) * kRow; }

__device__ __forceinline__ float4 ld4(const float* p) { return *reinterpret_cast<const float4*>(p); }

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// 2^t for t <= 0 of two values on the multiply-add pipe: t = n + f, f in [-1/2, 1/2], a polynomial of degree 6 in f
// (a least-squares fit of the relative error; at most 1.6e-8), times 2^n.  Evaluated, it is off by half of a half ulp on
// average and 1.9 at most, without a bias (1e-9), where the hardware's exponential is off by up to 2 ulp and to one side:
// a state that remembers a thousand tokens multiplies a thousand of them.  Below 2^-126.5 it is 0, as the decay of a rate
// past fp32 has to be: its product with the rate is no gradient.  A NaN stays a NaN: the maximum keeps it, and 2^n is a
// factor (an integer added to the exponent would make a number of a NaN's bits).
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 ex2_exact(float2 t) {
  t = {max_nan(t.x, -127.f), max_nan(t.y, -127.f)};
  constexpr float big = 12583039.f;  // 1.5 2^23 + 127: the low bits of m are n + 127, the exponent of 2^n
  const float2 m = __fadd2_rn(t, {big, big}), f = __ffma2_rn(__fadd2_rn(m, {-big, -big}), {-1.f, -1.f}, t);
  constexpr float c[7] = {1.f,           0.693147182f,  0.240226477f,   0.0555033237f,
                          0.00961843692f, 0.00133988739f, 0.00015353362f};
  float2 p = {c[6], c[6]};
#pragma unroll
  for (int k = 5; k >= 0; --k) p = __ffma2_rn(p, f, {c[k], c[k]});
  return __fmul2_rn(p, {__int_as_float(__float_as_int(m.x) << 23), __int_as_float(__float_as_int(m.y) << 23)});
}

// The decays exp(delta A) of two tokens, a = A log2(e), on the way forward and in the backward's first pass over segments.
// Tensors of 16 bits take the hardware's exponential, since the polynomial costs as many instructions as all the rest
// (forward of 8 x 1024 x 4096 x 16 237 against 364 us, that first pass 82 against 132).  It is low on average: by 5e-9 to
// 8e-9 (relative) for -2^-8 < t < 0, 1.6e-8 to 2.7e-8 down to -1, 5e-8 below (2^20 arguments in each octave), and a state
// that remembers a thousand tokens multiplies a thousand of them.  So t gets an offset, in the product's own rounding,
// that takes out 9.7e-9: errors of the fp32 outputs against 64 bits (2 x 4096 x 2048 x 16 bf16, root mean square
// relative) without it, with it and of the formulas in fp32 by elementary torch operations: state 5.1e-7, 2.9e-7 and
// 3.6e-7; dA_log 9.0e-7, 5.0e-7 and 1.5e-6; the initial state's gradient 4.2e-7, 3.7e-7 and 2.8e-6.  A step of 0 still
// decays by exactly 1.
constexpr float kOffset = 1.4e-8f;
template <typename T>
__device__ __forceinline__ float2 decays(float2 delta, float2 a) {
  if constexpr (sizeof(T) == 4) return ex2_exact(__fmul2_rn(delta, a));
  const float2 t = __ffma2_rn(delta, a, {kOffset, kOffset});
  return {ex2(t.x), ex2(t.y)};
}

// The framework's softplus (v above 20 passes through) of two values, and e = exp(-|v|) for their slope.
// softplus = max(v, 0) + log(1 + e).  The exponent's product is carried with its remainder, as in exp_acc;
// log(1 + e) / e on [0, 1] is a polynomial of degree 9 (a least-squares fit of the relative error; at most 3.4e-8).
__device__ __forceinline__ float2 softplus2(float2 v, float2& e) {
  const float2 a = {fminf(fabsf(v.x), 100.f), fminf(fabsf(v.y), 100.f)};
  const float2 t = __fmul2_rn(a, {-kLog2e, -kLog2e});
  float2 r = __ffma2_rn(a, {-kLog2e, -kLog2e}, {-t.x, -t.y});
  r = __ffma2_rn(a, {-1.92596299e-8f, -1.92596299e-8f}, r);
  e = {ex2(t.x), ex2(t.y)};
  e = __ffma2_rn(__fmul2_rn(e, r), {kLn2, kLn2}, e);
  constexpr float c[10] = {1.f,          -0.499999017f, 0.333299637f, -0.249541342f, 0.196759388f,
                           -0.153055906f, 0.106036514f,  -0.0569594987f, 0.0198514443f, -0.00324402121f};
  float2 p = {c[9], c[9]};
#pragma unroll
  for (int k = 8; k >= 0; --k) p = __ffma2_rn(p, e, {c[k], c[k]});
  // comparisons that are false for NaN leave it in the result
  float2 o = {v.x < 0.f ? 0.f : v.x, v.y < 0.f ? 0.f : v.y};
  o = __ffma2_rn(p, e, o);
  return {v.x > 20.f ? v.x : o.x, v.y > 20.f ? v.y : o.y};
}
// softplus' = 1 / (1 + exp(-v)), 1 above 20
__device__ __forceinline__ float softplus_slope(float v, float e) {
  const float r = rcp(1.f + e);
  return v > 20.f ? 1.f : v < 0.f ? e * r : r + (v - v);
}

// Sums M values over the lanes (lane / STRIDE) % LANES.  While a lane has several values, each step
// halves them: a lane keeps one half and hands over the other.  Afterwards a lane has M / LANES values,
// the first of them number lane_slot, or one that LANES / M lanes share.
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

// A feeding thread's share of a tile where rows do not come in 16-byte words: 4 bytes at a time (every fp32 tensor,
// and with WORDS the even widths of the others), or half words through registers, all of a thread's loads under way
// before the first is stored.
template <typename T, int WIDTH, int PITCH, bool WORDS>
__device__ __forceinline__ void fetch_narrow(T* dst, int f, const T* base, int64_t ld, int tokens, int width, int vec) {
  if (sizeof(T) == 4 || (WORDS && vec == 1)) {
    constexpr int V = 4 / (int)sizeof(T), PER = WIDTH / V;
#pragma unroll(WORDS ? 4 : 1)
    for (int i = 0; i < kTile * PER / kFeed; ++i) {
      const int e = i * kFeed + f, t = e / PER, c = e % PER * V;
      const bool in = t < tokens && c < width;
      const T* src = in ? base + t * ld + c : base;
      const unsigned d = (unsigned)__cvta_generic_to_shared(dst + t * PITCH + c);
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(d), "l"(src), "r"(in ? 4 : 0));
    }
  } else {
    constexpr int ALL = kTile * WIDTH / kFeed, B = WORDS || ALL < 4 ? ALL : 4;
#pragma unroll 1
    for (int i0 = 0; i0 < ALL; i0 += B) {
      T v[B];
#pragma unroll
      for (int i = 0; i < B; ++i) {
        const int e = (i0 + i) * kFeed + f, t = e / WIDTH, c = e % WIDTH;
        v[i] = down<T>(0.f);
        if (t < tokens && c < width) v[i] = base[t * ld + c];
      }
#pragma unroll
      for (int i = 0; i < B; ++i) {
        const int e = (i0 + i) * kFeed + f;
        dst[e / WIDTH * PITCH + e % WIDTH] = v[i];
      }
    }
  }
}

// The same as a call, so that the usual path keeps its registers; not for warps that have given registers up, of
// which a called function does not know.
template <typename T, int WIDTH, int PITCH>
__device__ __noinline__ void fetch_narrow_call(T* dst, int f, const T* base, int64_t ld, int tokens, int width, int vec) {
  fetch_narrow<T, WIDTH, PITCH, true>(dst, f, base, ld, tokens, width, vec);
}

// A feeding thread's share of the asynchronous copies of a [kTile][WIDTH] tile of rows with a token stride, to rows
// of PITCH elements.  What does not exist is zero.
template <typename T, int WIDTH, int PITCH>
struct Feed {
  static constexpr int V = 16 / (int)sizeof(T), PER = WIDTH / V, ALL = kTile * PER, N = (ALL + kFeed - 1) / kFeed;
  const T* base;
  int64_t ld;
  int width, vec;

  template <bool CALL = true>
  __device__ __forceinline__ void fetch(T* dst, int f, int64_t t0, int tokens) const {
    if (vec == 2) {
      const int c = f % PER * V;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int t = i * (kFeed / PER) + f / PER;
        if (ALL % kFeed != 0 && t >= kTile) break;
        const bool in = t < tokens && c < width;
        const T* src = in ? base + (t0 + t) * ld + c : base;
        const unsigned d = (unsigned)__cvta_generic_to_shared(dst + t * PITCH + c);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(in ? 16 : 0));
      }
    } else if constexpr (CALL) {
      fetch_narrow_call<T, WIDTH, PITCH>(dst, f, base + t0 * ld, ld, tokens, width, vec);
    } else {
      fetch_narrow<T, WIDTH, PITCH, false>(dst, f, base + t0 * ld, ld, tokens, width, vec);
    }
  }
};
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int PENDING>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory"); }

// B or C of a raw tile [kTile][NP] to fp32 [NP][kRow]: a feeding thread takes four tokens of a state.
template <typename T, int NP, int SPL>
__device__ __forceinline__ void widen_states(float* to, const T* raw, int f) {
#pragma unroll
  for (int i = 0; i < (NP * 8 + kFeed - 1) / kFeed; ++i) {
    const int e = i * kFeed + f, n = e % NP, q = e / NP;
    if (NP * 8 % kFeed != 0 && q >= 8) break;
    const T* r = raw + q * 4 * NP + n;
    *reinterpret_cast<float4*>(to + state_row<NP, SPL>(n) + 4 * q) = make_float4(up<T>(r[0]), up<T>(r[NP]), up<T>(r[2 * NP]), up<T>(r[3 * NP]));
  }
}

// CW channels of a token in registers, as they are in memory.
template <typename T, int CW>
struct Cols {
  static constexpr int V = CW * (int)sizeof(T) > 16 ? 16 / (int)sizeof(T) : CW;
  Pack<T, V> r[CW / V];

  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < CW / V; ++i) r[i].load(p + i * V);
  }
  __device__ __forceinline__ float get(int i) const { return r[i / V].f(i % V); }
  // elements i and i + 1, i even
  __device__ __forceinline__ void put2(int i, float2 f) {
    if constexpr (V == 1) {
      r[i].set_pair(0, {f.x, 0.f});
      r[i + 1].set_pair(0, {f.y, 0.f});
    } else {
      r[i / V].set_pair(i % V / 2, f);
    }
  }
  // n: how many of them exist (whole accesses of them)
  __device__ __forceinline__ void store(T* p, int vec, int n) const {
    if (vec == 2) {
#pragma unroll
      for (int i = 0; i < CW / V; ++i)
        if (i * V < n) r[i].store(p + i * V);
    } else if (sizeof(T) == 2 && V > 1 && vec == 1) {
#pragma unroll
      for (int i = 0; i < CW; i += 2)
        if (i < n) *reinterpret_cast<unsigned*>(p + i) = r[i / V].u[i % V / 2];
    } else {
#pragma unroll
      for (int i = 0; i < CW; ++i)
        if (i < n) p[i] = reinterpret_cast<const T*>(&r[i / V])[i % V];
    }
  }
};

// Where a block and a thread are.
template <int NP, int SPL>
struct Place {
  using S = Shape<NP, SPL>;
  Piece p;
  int g;           // group
  int64_t tile;    // the block's channel tile in the group
  int lane, nl, cl, warp;
  int c, n0;       // working threads: the lane's channel in the block and its first state
  bool feeds, live;
  int f, tok, sc;  // feeding threads: their number, token and first channel
  int width;       // channels of the block that exist
  int64_t c0, ch;  // the block's first channel, the lane's

  // whether the unit exists; the channels are set either way
  __device__ __forceinline__ bool find(const Ssm& s, int lg) {
    warp = threadIdx.x >> 5;
    lane = threadIdx.x & 31;
    nl = lane % S::NL;
    cl = lane / S::NL;
    c = warp * S::CW + cl;
    n0 = nl * SPL;
    feeds = threadIdx.x >= S::WORK;
    f = (int)threadIdx.x - S::WORK;
    tok = lane;
    sc = (f >> 5) * S::FC;
    const int64_t Dg = s.D / s.G, tiles = (Dg + S::CC - 1) / S::CC;
    g = (int)(blockIdx.y / tiles);
    tile = blockIdx.y - g * tiles;
    const int64_t local = tile * S::CC, rest = Dg - local;
    c0 = g * Dg + local;
    ch = c0 + c;
    live = !feeds && c < rest;
    width = rest < S::CC ? (int)rest : S::CC;
    return find_piece(s.seqs, blockIdx.x, lg, p);
  }
};

// The block's raw tiles of one per-channel input; a row is padded so that lanes on neighbouring tokens read
// distinct banks.
template <typename T, int NP>
struct RawRows {
  static constexpr int CC = 512 / NP, PITCH = CC + 16 / (int)sizeof(T);
  T v[kRing<T, NP>][kTile * PITCH];
};

// A block's view of the inputs of its segment.
template <typename T, int NP, int SPL>
struct Inputs {
  static constexpr int CC = 512 / NP;
  Feed<T, CC, RawRows<T, NP>::PITCH> x, dt, dy;
  Feed<T, NP, NP> B, C;

  __device__ __forceinline__ Inputs(const Ssm& s, const Place<NP, SPL>& at) {
    const int64_t t0 = at.p.t0, n = (int64_t)at.g * s.N;
    x = {static_cast<const T*>(s.x) + t0 * s.ld_x + at.c0, s.ld_x, at.width, s.vec};
    dt = {static_cast<const T*>(s.dt) + t0 * s.ld_dt + at.c0, s.ld_dt, at.width, s.vec};
    dy = {static_cast<const T*>(s.dy) + t0 * s.D + at.c0, s.D, at.width, s.vec};
    B = {static_cast<const T*>(s.Bm) + t0 * s.ld_b + n, s.ld_b, s.N, s.vec_bc};
    C = {static_cast<const T*>(s.Cm) + t0 * s.ld_c + n, s.ld_c, s.N, s.vec_bc};
  }
};

// The states of a lane from and to [...][D][N] ...
template <int SPL>
__device__ __forceinline__ void load_states(const float* p, int N, int n0, float (&h)[SPL]) {
#pragma unroll
  for (int j = 0; j < SPL; ++j) h[j] = n0 + j < N ? p[n0 + j] : 0.f;
}
template <int SPL>
__device__ __forceinline__ void store_states(float* p, int N, int n0, const float (&h)[SPL]) {
#pragma unroll
  for (int j = 0; j < SPL; ++j)
    if (n0 + j < N) p[n0 + j] = h[j];
}
// ... and the workspace's padded [...][D][NP]
template <int SPL>
__device__ __forceinline__ void load_padded(const float* p, float (&h)[SPL]) {
  Pack<float, SPL> v;
  v.load(p);
  v.get(h);
}
template <int SPL>
__device__ __forceinline__ void store_padded(float* p, const float (&h)[SPL]) {
  Pack<float, SPL> v;
  v.set(h);
  v.store(p);
}

// exp(A_log) and A log2(e), kept finite so that a token of delta = 0 past the piece's end keeps the state, and a decay of 0
// has no gradient
constexpr float kMost = 3.4e38f;
__device__ __forceinline__ float rate_of(float A_log) {
  const float e = expf(A_log);
  return e > kMost ? kMost : e;  // (false for NaN)
}
__device__ __forceinline__ float decay_rate(float A_log) {
  const float a = -expf(A_log) * kLog2e;
  return a < -kMost ? -kMost : a;
}

// that of a lane's states (0 for states that do not exist: their decay is 1, their input 0)
template <int SPL>
__device__ __forceinline__ void load_decay(const Ssm& s, int64_t ch, bool live, int n0, float (&a)[SPL]) {
#pragma unroll
  for (int j = 0; j < SPL; ++j) a[j] = live && n0 + j < s.N ? decay_rate(s.A_log[ch * s.N + n0 + j]) : 0.f;
}

template <int NP>
__device__ __forceinline__ int64_t state_at(const Ssm& s, int64_t unit, int64_t ch, int n0) {
  return (unit * s.D + ch) * NP + n0;
}

}  // namespace mix
}  // namespace gdn
