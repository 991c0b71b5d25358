// Shared device code of the mixing-layer operators (short convolution, selective scan, layer
// norm): typed vector loads and stores, the sigmoid family, and the division of packed sequences
// into pieces.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "gdn.h"
#include "gdn_common.cuh"
#include "gdn_launch.h"
#include "gdn_mix.h"

namespace gdn {
namespace mix {

template <typename T>
__device__ __forceinline__ float up(T x);
template <>
__device__ __forceinline__ float up<float>(float x) { return x; }
template <>
__device__ __forceinline__ float up<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <>
__device__ __forceinline__ float up<__half>(__half x) { return __half2float(x); }

template <typename T>
__device__ __forceinline__ T down(float x);
template <>
__device__ __forceinline__ float down<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 down<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half down<__half>(float x) { return __float2half_rn(x); }

// V consecutive elements moved as one access of V * sizeof(T) bytes (a power of two up to 16; the
// address has that alignment).
template <int BYTES>
struct Word;
template <>
struct Word<2> { using type = unsigned short; };
template <>
struct Word<4> { using type = unsigned int; };
template <>
struct Word<8> { using type = uint2; };
template <>
struct Word<16> { using type = uint4; };

// Two neighbouring elements of a 16-bit type, from and to the word that holds them.
__device__ __forceinline__ float2 widen2(unsigned w, __nv_bfloat16) {
  return {__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)};
}
__device__ __forceinline__ float2 widen2(unsigned w, __half) {
  __half2 h;
  *reinterpret_cast<unsigned*>(&h) = w;
  return __half22float2(h);
}
__device__ __forceinline__ unsigned narrow2(float2 f, __nv_bfloat16) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
  return *reinterpret_cast<const unsigned*>(&h);
}
__device__ __forceinline__ unsigned narrow2(float2 f, __half) {
  const __half2 h = __floats2half2_rn(f.x, f.y);
  return *reinterpret_cast<const unsigned*>(&h);
}

template <typename T, int V>
struct Pack {
  using W = typename Word<sizeof(T) * V>::type;
  static constexpr int WORDS = (int)sizeof(T) * V / 4;  // 0: a single half word
  union {
    W w;
    unsigned u[WORDS > 0 ? WORDS : 1];
    T one;
  };
  __device__ __forceinline__ Pack() {}
  __device__ __forceinline__ void load(const T* p) { w = *reinterpret_cast<const W*>(p); }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < (WORDS > 0 ? WORDS : 1); ++i) u[i] = 0u;
  }
  __device__ __forceinline__ void store(T* p) const { *reinterpret_cast<W*>(p) = w; }
  // elements 2 i and 2 i + 1 (V = 1: the element and 0)
  __device__ __forceinline__ float2 pair(int i) const {
    if constexpr (V == 1)
      return {up<T>(one), 0.f};
    else if constexpr (sizeof(T) == 4)
      return {__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1])};
    else
      return widen2(u[i], T{});
  }
  __device__ __forceinline__ void set_pair(int i, float2 f) {
    if constexpr (V == 1) {
      one = down<T>(f.x);
    } else if constexpr (sizeof(T) == 4) {
      u[2 * i] = __float_as_uint(f.x);
      u[2 * i + 1] = __float_as_uint(f.y);
    } else {
      u[i] = narrow2(f, T{});
    }
  }
  __device__ __forceinline__ float f(int i) const {
    const float2 v = pair(i / 2);
    return i % 2 ? v.y : v.x;
  }
  __device__ __forceinline__ void get(float (&o)[V]) const {
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = f(i);
  }
  __device__ __forceinline__ void set(const float (&o)[V]) {
#pragma unroll
    for (int i = 0; i < V; i += 2) set_pair(i / 2, {o[i], i + 1 < V ? o[i + 1 < V ? i + 1 : 0] : 0.f});
  }
};

// e^x for the gates and the softplus.  x log2(e) is formed as a rounded product and its exact
// remainder, and the remainder enters as the factor 1 + r ln 2, so the only error beyond the
// hardware's 2^t (2 ulp) is the last product's: no growth with |x|.  Outside [-126, 126] (in
// powers of two) the result is 0 or infinity as for any fp32 exponential that flushes.
__device__ __forceinline__ float exp_acc(float x) {
  constexpr float kLog2e = 1.44269504088896341f;
  constexpr float kLow = 1.92596299112661746887e-8f;  // log2(e) - kLog2e
  const float t = x * kLog2e;
  const float r = fmaf(x, kLow, fmaf(x, kLog2e, -t));
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
  // |t| large makes e 0 or inf (x infinite: r is NaN), and then the remainder says nothing
  return fabsf(t) < 126.f ? fmaf(e, r * 0.693147180559945309f, e) : e;
}

__device__ __forceinline__ float rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// 1 / (1 + e^-x); 0 and 1 in the limits, NaN for NaN.  For 16-bit tensors the exponential without
// the remainder is enough: its relative error (2 + 1.2 |x|) 2^-23 is far below the result's rounding.
template <typename T>
__device__ __forceinline__ float sigmoid(float x) {
  if constexpr (sizeof(T) == 4) return rcp(1.f + exp_acc(-x));
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * -1.44269504088896341f));
  return rcp(1.f + e);
}

// A piece of one sequence: `len` tokens from flat token `t0`, which is token `pos` of sequence `seq`
// (of `slen` tokens).
struct Piece {
  int seq, idx, pos, len, slen;
  int64_t t0;
};

// Pieces of at most 2^lg tokens.  Packed: sequence n owns the units floor(cu[n] / 2^lg) + n up to
// floor(cu[n+1] / 2^lg) + n, one more than its full pieces at most, so a unit finds its sequence by
// one binary search without a table; units past a sequence's end are idle.  Every sequence has a
// piece 0, an empty one too (its states pass through).
__device__ __forceinline__ bool find_piece(const Seqs& s, int64_t unit, int lg, Piece& p) {
  int64_t bos, len, first;
  int n;
  if (s.cu) {
    int lo = 0, hi = s.n - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if ((s.cu[mid] >> lg) + mid <= unit)
        lo = mid;
      else
        hi = mid - 1;
    }
    n = lo;
    bos = s.cu[n];
    len = s.cu[n + 1] - bos;
    first = (bos >> lg) + n;
  } else {
    const int64_t per = s.T == 0 ? 1 : ((s.T - 1) >> lg) + 1;
    n = (int)(unit / per);
    bos = (int64_t)n * s.T;
    len = s.T;
    first = n * per;
  }
  const int64_t pos = (unit - first) << lg;
  if (pos > 0 && pos >= len) return false;
  p.seq = n;
  p.idx = (int)(unit - first);
  p.pos = (int)pos;
  p.slen = (int)len;
  const int64_t rest = len - pos, most = (int64_t)1 << lg;
  p.len = (int)(rest < most ? rest : most);
  p.t0 = bos + pos;
  return true;
}

// The unit of sequence n's piece 0.
__device__ __forceinline__ int64_t first_unit(const Seqs& s, int n, int lg) {
  if (s.cu) return (s.cu[n] >> lg) + n;
  return (int64_t)n * (s.T == 0 ? 1 : ((s.T - 1) >> lg) + 1);
}

// Whether the packing was found invalid by the kernel before this one; a dense call's status word
// (which has no such kernel) is cleared here.
__device__ __forceinline__ bool bad_call(const Seqs& s) {
  if (s.cu) return *((volatile const int*)s.status) != 0;
  if (s.status && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0 && threadIdx.y == 0) s.status[0] = (int)GDN_OK;
  return false;
}

// The sum over rows r < n of part[r * ld + c]: STR strands of rows for each column, each in row order, the strands
// in a fixed tree.  Returns it with its column c to one thread a column, c = -1 to the others.
template <int STR>
__device__ __forceinline__ float strand_sums(const float* __restrict__ part, int64_t n, int64_t ld, int64_t width, int64_t& c) {
  if constexpr (STR == 1) {
    c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    float a = 0.f;
    if (c < width) {
#pragma unroll 4
      for (int64_t r = 0; r < n; ++r) a += part[r * ld + c];
    } else {
      c = -1;
    }
    return a;
  } else {
    __shared__ float red[32][STR + 1];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int64_t from = (int64_t)blockIdx.x * 32 + tx;
    float a = 0.f;
    if (from < width) {
#pragma unroll 4
      for (int64_t r = ty; r < n; r += STR) a += part[r * ld + from];
    }
    red[tx][ty] = a;
    __syncthreads();
    const int col = threadIdx.x / STR, strand = threadIdx.x % STR;
    float v = red[col][strand];
#pragma unroll
    for (int o = STR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    c = (int64_t)blockIdx.x * 32 + col;
    if (strand != 0 || c >= width) c = -1;
    return v;
  }
}

// A kernel's dynamic shared memory, asked for where it is over the default.
template <typename K>
inline cudaError_t allow_shared(K* kernel, size_t bytes) {
  return bytes > 48 * 1024 ? cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) : cudaSuccess;
}

}  // namespace mix
}  // namespace gdn
