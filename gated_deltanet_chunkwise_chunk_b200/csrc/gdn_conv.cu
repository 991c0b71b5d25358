// Short causal convolution along the sequence, channel by channel, with its silu:
//   pre[t, d] = bias[d] + sum_{j < W} w[d, j] x[t - (W-1) + j, d],   y = silu(pre) or pre,
// t counted inside the sequence; inputs before its first token come from the state (the last W - 1
// inputs) or are zero.  Backward, with dpre = dy silu'(pre) (pre is recomputed):
//   dx[t] = sum_j w[d, j] dpre[t + (W-1) - j],  dw[d, j] = sum_t dpre[t] x[t - (W-1) + j],
//   dbias = sum_t dpre[t].
// All three directions move bytes: the taps are kept in registers and every input row is read from
// HBM once (neighbouring strips of tokens meet in L1 and L2).
#include <algorithm>

#include "mix_common.cuh"

namespace gdn {
namespace mix {

__global__ void __launch_bounds__(256) k_check_packing(Seqs s) {
  __shared__ int bad;
  if (threadIdx.x == 0) bad = 0;
  __syncthreads();
  for (int n = threadIdx.x; n < s.n; n += 256) {
    const int64_t a = s.cu[n], b = s.cu[n + 1];
    if (a < 0 || b < a || b > s.T || (n == 0 && a != 0) || (n == s.n - 1 && b != s.T)) bad = 1;
  }
  __syncthreads();
  if (threadIdx.x == 0) s.status[0] = bad ? (int)GDN_ERR_INVALID_ARG : (int)GDN_OK;
}

cudaError_t check_packing(const Seqs& s, cudaStream_t stream) {
  ProfScope ps("check_packing", stream);
  k_check_packing<<<1, 256, 0, stream>>>(s);
  return cudaGetLastError();
}

// Columns x STR strands of rows; each strand in row order, the strands in a fixed tree.
template <int STR>
__global__ void __launch_bounds__(STR == 1 ? 256 : 32 * STR) k_column_sums(const float* __restrict__ part, int64_t n, int64_t ld,
                                                                          int64_t width, float* __restrict__ out,
                                                                          float* __restrict__ out2, int W, int64_t D) {
  int64_t c;
  const float v = strand_sums<STR>(part, n, ld, width, c);
  if (c < 0) return;
  const int64_t j = c / D, d = c - j * D;
  if (j < W) {
    if (out) out[d * W + j] = v;
  } else if (out2) {
    out2[d] = v;
  }
}

cudaError_t column_sums(const char* name, const float* part, int64_t n, int64_t ld, int64_t width, float* out,
                        float* out2, int W, int64_t D, cudaStream_t s) {
  ProfScope ps(name, s);
  switch (sum_strands(n)) {
    case 1: k_column_sums<1><<<(unsigned)((width + 255) / 256), 256, 0, s>>>(part, n, ld, width, out, out2, W, D); break;
    case 8: k_column_sums<8><<<(unsigned)((width + 31) / 32), 256, 0, s>>>(part, n, ld, width, out, out2, W, D); break;
    default: k_column_sums<32><<<(unsigned)((width + 31) / 32), 1024, 0, s>>>(part, n, ld, width, out, out2, W, D);
  }
  return cudaGetLastError();
}

namespace {

constexpr int FS = 8;   // tokens of a thread's strip, forward
constexpr int BS = 16;  // and backward
constexpr int NT = 256;

// Row p (place in the sequence, may be negative) of the sequence's inputs.
template <typename T, int V>
__device__ __forceinline__ void load_row(const Conv& c, const Piece& p, int at, int64_t ch, Pack<T, V>& r) {
  if (at >= 0)
    r.load(static_cast<const T*>(c.x) + (p.t0 - p.pos + at) * c.ld + ch);
  else if (c.init)
    r.load(static_cast<const T*>(c.init) + ((int64_t)p.seq * (c.W - 1) + at + c.W - 1) * c.D + ch);
  else
    r.zero();
}

template <typename T, int V, int W>
__device__ __forceinline__ void load_taps(const Conv& c, int64_t ch, float (&w)[W][V]) {
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int j = 0; j < W; ++j) w[j][i] = c.weight[(ch + i) * W + j];
}

// Block (lanes over channel vectors, strips of tokens); all of a strip's rows are requested before
// the first is used.
template <typename T, int V, int W>
__global__ void __launch_bounds__(NT) k_conv_fwd(Conv c, int lg) {
  if (bad_call(c.seqs)) return;
  Piece p;
  if (!find_piece(c.seqs, blockIdx.x, lg, p)) return;
  const int64_t ch = ((int64_t)blockIdx.y * blockDim.x + threadIdx.x) * V;
  if (ch >= c.D) return;
  const int s0 = p.pos + threadIdx.y * FS;
  const int end = p.pos + p.len;
  if (s0 < end) {
    Pack<T, V> rows[FS + W - 1];
#pragma unroll
    for (int i = 0; i < FS + W - 1; ++i) {
      const int at = s0 + i - (W - 1);
      if (at < end) load_row<T, V>(c, p, at, ch, rows[i]);
    }
    float w[W][V], bias[V];
    load_taps<T, V, W>(c, ch, w);
#pragma unroll
    for (int i = 0; i < V; ++i) bias[i] = c.bias ? c.bias[ch + i] : 0.f;
    T* y = static_cast<T*>(c.y) + (p.t0 - p.pos + s0) * c.D + ch;
#pragma unroll
    for (int t = 0; t < FS; ++t) {
      if (s0 + t >= end) break;
      float o[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float a = bias[i];
#pragma unroll
        for (int j = 0; j < W; ++j) a = fmaf(w[j][i], up<T>(rows[t + j].v[i]), a);
        o[i] = c.silu ? a * sigmoid<T>(a) : a;
      }
      Pack<T, V> r;
      r.set(o);
      r.store(y + (int64_t)t * c.D);
    }
  }
  if (c.final && end == p.slen && (int)threadIdx.y < W - 1) {
    Pack<T, V> r;
    load_row<T, V>(c, p, p.slen - (W - 1) + (int)threadIdx.y, ch, r);
    r.store(static_cast<T*>(c.final) + ((int64_t)p.seq * (W - 1) + threadIdx.y) * c.D + ch);
  }
}

// A strip slides over its tokens and the W - 1 after them: dpre of a token completes dx of the token
// W - 1 before it.  The next four rows of x and dy are in flight while four are worked on.
template <typename T, int V, int W>
__global__ void __launch_bounds__(NT) k_conv_bwd(Conv c, int lg) {
  __shared__ float red[NT * V];
  if (bad_call(c.seqs)) return;
  Piece p;
  const bool some = find_piece(c.seqs, blockIdx.x, lg, p);
  const int64_t ch = ((int64_t)blockIdx.y * blockDim.x + threadIdx.x) * V;
  const bool live = ch < c.D;
  float dw[W][V], db[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    db[i] = 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) dw[j][i] = 0.f;
  }
  const int s0 = some ? p.pos + (int)threadIdx.y * BS : 0;
  if (some && live && (s0 < p.pos + p.len || s0 == 0)) {
    float w[W][V], bias[V], xw[W][V], dp[W][V];
    load_taps<T, V, W>(c, ch, w);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      bias[i] = c.bias ? c.bias[ch + i] : 0.f;
#pragma unroll
      for (int j = 0; j < W; ++j) dp[j][i] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      Pack<T, V> r;
      load_row<T, V>(c, p, s0 + j - (W - 1), ch, r);
      r.get(xw[j + 1]);
    }
    const int64_t bos = p.t0 - p.pos;
    const T* dy = static_cast<const T*>(c.dy) + bos * c.D + ch;
    T* dx = static_cast<T*>(c.dx) + bos * c.D + ch;
    constexpr int STEPS = BS + W - 1, GR = 4;
    Pack<T, V> xb[GR], yb[GR];
    auto fetch = [&](int i, Pack<T, V>& x, Pack<T, V>& g) {
      const int at = s0 + i;
      if (i < STEPS && at < p.slen) {
        load_row<T, V>(c, p, at, ch, x);
        g.load(dy + (int64_t)at * c.D);
      } else {
        x.zero();
        g.zero();
      }
    };
#pragma unroll
    for (int k = 0; k < GR; ++k) fetch(k, xb[k], yb[k]);
#pragma unroll
    for (int i0 = 0; i0 < STEPS; i0 += GR) {
      Pack<T, V> xc[GR], yc[GR];
#pragma unroll
      for (int k = 0; k < GR; ++k) {
        xc[k] = xb[k];
        yc[k] = yb[k];
      }
#pragma unroll
      for (int k = 0; k < GR; ++k) fetch(i0 + GR + k, xb[k], yb[k]);
#pragma unroll
      for (int k = 0; k < GR; ++k) {
        const int i = i0 + k;
        if (i >= STEPS) break;
        const int at = s0 + i;
        const bool in = at < p.slen;
        float xn[V], g[V];
        xc[k].get(xn);
        yc[k].get(g);
#pragma unroll
        for (int v = 0; v < V; ++v) {
#pragma unroll
          for (int j = 0; j < W - 1; ++j) {
            xw[j][v] = xw[j + 1][v];
            dp[j][v] = dp[j + 1][v];
          }
          xw[W - 1][v] = xn[v];
          float d = g[v];
          if (c.silu) {
            float a = bias[v];
#pragma unroll
            for (int j = 0; j < W; ++j) a = fmaf(w[j][v], xw[j][v], a);
            const float sg = sigmoid<T>(a);
            d *= sg * fmaf(a, 1.f - sg, 1.f);
          }
          dp[W - 1][v] = in ? d : 0.f;
          if (i < BS && in) {
            db[v] += d;
#pragma unroll
            for (int j = 0; j < W; ++j) dw[j][v] = fmaf(d, xw[j][v], dw[j][v]);
          }
        }
        const int q = at - (W - 1);  // the token whose gradient is now complete
        const bool own = i >= W - 1 && q < p.slen;
        const bool before = q < 0 && s0 == 0;
        if ((own || before) && (own ? c.dx != nullptr : c.dinit != nullptr)) {
          float o[V];
#pragma unroll
          for (int v = 0; v < V; ++v) {
            o[v] = 0.f;
#pragma unroll
            for (int j = 0; j < W; ++j) o[v] = fmaf(w[j][v], dp[W - 1 - j][v], o[v]);
          }
          const int slot = q - p.slen + (W - 1);  // its place in the final state
          if (c.dfinal && slot >= 0) {
            Pack<T, V> r;
            r.load(static_cast<const T*>(c.dfinal) + ((int64_t)p.seq * (W - 1) + slot) * c.D + ch);
#pragma unroll
            for (int v = 0; v < V; ++v) o[v] += up<T>(r.v[v]);
          }
          Pack<T, V> r;
          r.set(o);
          if (own)
            r.store(dx + (int64_t)q * c.D);
          else
            r.store(static_cast<T*>(c.dinit) + ((int64_t)p.seq * (W - 1) + i) * c.D + ch);
        }
      }
    }
  }
  if (!c.part) return;
  // the block's strips in order, one tap at a time
  float* part = c.part + (int64_t)blockIdx.x * (W + 1) * c.D + ch;
#pragma unroll
  for (int j = 0; j <= W; ++j) {
    __syncthreads();
#pragma unroll
    for (int v = 0; v < V; ++v) red[(threadIdx.y * blockDim.x + threadIdx.x) * V + v] = j < W ? dw[j < W ? j : 0][v] : db[v];
    __syncthreads();
    if (threadIdx.y == 0 && live) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float a = 0.f;
        for (int s = 0; s < (int)blockDim.y; ++s) a += red[(s * blockDim.x + threadIdx.x) * V + v];
        part[(int64_t)j * c.D + v] = a;
      }
    }
  }
}

// One token for each sequence; the state moves up by one input.  state and final may be one buffer:
// a thread reads its channels' slots before it writes them.
template <typename T, int V, int W>
__global__ void __launch_bounds__(NT) k_conv_step(Conv c) {
  const int64_t per = c.D / V, at = (int64_t)blockIdx.x * NT + threadIdx.x;
  const int64_t n = at / per, ch = (at - n * per) * V;
  if (n >= c.seqs.n) return;
  Pack<T, V> rows[W];
  const T* st = static_cast<const T*>(c.init) + n * (W - 1) * c.D + ch;
#pragma unroll
  for (int j = 0; j < W - 1; ++j) rows[j].load(st + (int64_t)j * c.D);
  rows[W - 1].load(static_cast<const T*>(c.x) + n * c.ld + ch);
  float w[W][V], o[V];
  load_taps<T, V, W>(c, ch, w);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float a = c.bias ? c.bias[ch + i] : 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) a = fmaf(w[j][i], up<T>(rows[j].v[i]), a);
    o[i] = c.silu ? a * sigmoid<T>(a) : a;
  }
  Pack<T, V> r;
  r.set(o);
  r.store(static_cast<T*>(c.y) + n * c.D + ch);
  T* nx = static_cast<T*>(c.final) + n * (W - 1) * c.D + ch;
#pragma unroll
  for (int j = 0; j < W - 1; ++j) rows[j + 1].store(nx + (int64_t)j * c.D);
}

// Lanes over channel vectors (a power of two up to 32) so that narrow tensors still fill the block.
int lanes_of(int64_t D, int V) {
  int l = 32;
  while (l > 1 && (int64_t)(l / 2) * V >= D) l /= 2;
  return l;
}

int log2i(int x) {
  int l = 0;
  while ((1 << l) < x) ++l;
  return l;
}

// Whole 16-byte (backward: four-element) vectors need widths, strides and bases that are multiples.
bool vec_ok(const Conv& c, int es, int V) {
  const uintptr_t b = (uintptr_t)es * V;
  if (c.D % V || c.ld % V) return false;
  const void* ps[] = {c.x, c.init, c.y, c.final, c.dy, c.dfinal, c.dx, c.dinit};
  for (const void* p : ps)
    if (reinterpret_cast<uintptr_t>(p) % b) return false;
  return true;
}

// The backward's block: lanes and the log of a piece's tokens, the same for both vector widths so
// that the partial rows' count is a function of the sizes alone.
int bwd_lg(int64_t D) { return log2i(BS * NT / lanes_of(D, 4)); }

template <typename T, int V, int W>
cudaError_t fwd_w(const Conv& c, cudaStream_t s) {
  const int lanes = lanes_of(c.D, V), lg = log2i(FS * NT / lanes);
  const dim3 grid((unsigned)max_units(c.seqs, lg), (unsigned)((c.D + (int64_t)lanes * V - 1) / ((int64_t)lanes * V)));
  k_conv_fwd<T, V, W><<<grid, dim3(lanes, NT / lanes), 0, s>>>(c, lg);
  return cudaGetLastError();
}

template <typename T, int V, int W>
cudaError_t bwd_w(const Conv& c, cudaStream_t s) {
  const int lanes = lanes_of(c.D, 4), lg = bwd_lg(c.D);
  const dim3 grid((unsigned)max_units(c.seqs, lg), (unsigned)((c.D + (int64_t)lanes * V - 1) / ((int64_t)lanes * V)));
  k_conv_bwd<T, V, W><<<grid, dim3(lanes, NT / lanes), 0, s>>>(c, lg);
  return cudaGetLastError();
}

template <typename T, int V, int W>
cudaError_t step_w(const Conv& c, cudaStream_t s) {
  const int64_t n = c.seqs.n * (c.D / V);
  k_conv_step<T, V, W><<<(unsigned)((n + NT - 1) / NT), NT, 0, s>>>(c);
  return cudaGetLastError();
}

enum { FWD, BWD, STEP };

template <int WHAT, typename T, int V>
cudaError_t by_width(const Conv& c, cudaStream_t s) {
  switch (c.W) {
#define GDN_CONV_W(w)                                        \
  case w:                                                    \
    return WHAT == FWD   ? fwd_w<T, V, w>(c, s)              \
           : WHAT == BWD ? bwd_w<T, (V > 4 ? 4 : V), w>(c, s) \
                         : step_w<T, V, w>(c, s);
    GDN_CONV_W(1)
    GDN_CONV_W(2)
    GDN_CONV_W(3)
    GDN_CONV_W(4)
    GDN_CONV_W(5)
    GDN_CONV_W(6)
    GDN_CONV_W(7)
    GDN_CONV_W(8)
#undef GDN_CONV_W
  }
  return cudaErrorInvalidValue;
}

template <int WHAT>
cudaError_t dispatch(const Conv& c, cudaStream_t s) {
  if (c.dtype == GDN_DTYPE_FP32)
    return vec_ok(c, 4, 4) ? by_width<WHAT, float, 4>(c, s) : by_width<WHAT, float, 1>(c, s);
  const bool v = vec_ok(c, 2, WHAT == BWD ? 4 : 8);
  if (c.dtype == GDN_DTYPE_BF16)
    return v ? by_width<WHAT, __nv_bfloat16, 8>(c, s) : by_width<WHAT, __nv_bfloat16, 1>(c, s);
  return v ? by_width<WHAT, __half, 8>(c, s) : by_width<WHAT, __half, 1>(c, s);
}

}  // namespace

int64_t conv_bwd_units(const Seqs& s, int64_t D) { return max_units(s, bwd_lg(D)); }

cudaError_t conv_forward(const Conv& c, cudaStream_t s) {
  ProfScope ps("conv_fwd", s);
  return dispatch<FWD>(c, s);
}

cudaError_t conv_backward(const Conv& c, cudaStream_t s) {
  {
    ProfScope ps("conv_bwd", s);
    const cudaError_t e = dispatch<BWD>(c, s);
    if (e != cudaSuccess) return e;
  }
  if (!c.part) return cudaSuccess;
  return column_sums("conv_bwd_sums", c.part, conv_bwd_units(c.seqs, c.D), (c.W + 1) * c.D, (c.W + 1) * c.D, c.dweight,
                     c.dbias, c.W, c.D, s);
}

cudaError_t conv_step(const Conv& c, cudaStream_t s) {
  ProfScope ps("conv_step", s);
  return dispatch<STEP>(c, s);
}

}  // namespace mix
}  // namespace gdn
