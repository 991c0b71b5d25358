// Short causal convolution along the sequence, channel by channel, with its silu:
//   pre[t, d] = bias[d] + sum_{j < W} w[d, j] x[t - (W-1) + j, d],   y = silu(pre) or pre,
// t counted inside the sequence; inputs before its first token come from the state (the last W - 1
// inputs) or are zero.  Backward, with dpre = dy silu'(pre) (pre is recomputed):
//   dx[t] = sum_j w[d, j] dpre[t + (W-1) - j],  dw[d, j] = sum_t dpre[t] x[t - (W-1) + j],
//   dbias = sum_t dpre[t].
// All three directions move bytes: the taps are kept in registers and every input row is read from
// HBM once (neighbouring strips of tokens meet in L1 and L2).  What it takes to move them at speed: rows on
// their way ahead of their use (asynchronous copies into rings of the thread's own), taps read in memory
// order through shared memory (32 strided loads a thread cost more than the rows: 204 us instead of 68
// forward), and packed multiply-adds.  Measured at 2 x 8192 x 4096 bf16 with four taps and the silu: forward
// 68 us for 268 MB (4.0 TB/s), bound by latency at two blocks a multiprocessor and by the exponentials and
// reciprocals (half their pipe); backward 139 us for 403 MB (2.9 TB/s), bound by latency too (issue 51%, DRAM 34% of
// their peaks with 24% of the warps; 36 instructions an element); 256 single tokens of 4096 channels 10 us.
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
__global__ void __launch_bounds__(STR == 1 ? 256 : 32 * STR) k_column_sums(Seqs seqs, const float* __restrict__ part, int64_t n,
                                                                          int64_t ld, int64_t width, float* __restrict__ out,
                                                                          float* __restrict__ out2, int W, int64_t D) {
  if (bad_call(seqs)) return;
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

cudaError_t column_sums(const char* name, const Seqs& seqs, const float* part, int64_t n, int64_t ld, int64_t width, float* out,
                        float* out2, int W, int64_t D, cudaStream_t s) {
  ProfScope ps(name, s);
  switch (sum_strands(n)) {
    case 1: k_column_sums<1><<<(unsigned)((width + 255) / 256), 256, 0, s>>>(seqs, part, n, ld, width, out, out2, W, D); break;
    case 8: k_column_sums<8><<<(unsigned)((width + 31) / 32), 256, 0, s>>>(seqs, part, n, ld, width, out, out2, W, D); break;
    default: k_column_sums<32><<<(unsigned)((width + 31) / 32), 1024, 0, s>>>(seqs, part, n, ld, width, out, out2, W, D);
  }
  return cudaGetLastError();
}

namespace {

constexpr int BS = 32;  // tokens of a thread's strip, backward
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

// The taps and the bias of the block's channels to shared memory, [W + 1][cols + 4]: read in memory order (a
// thread's own W V taps are far from the next lane's), left with the channels next to one another.
template <int W>
__device__ __forceinline__ void stage_taps(const Conv& c, float* taps, int64_t c0, int cols) {
  const int n = threadIdx.y * blockDim.x + threadIdx.x;
  const int have = (int)min((int64_t)cols, c.D - c0);
  for (int e = n; e < have * W; e += NT) taps[e % W * (cols + 4) + e / W] = c.weight[c0 * W + e];
  for (int e = n; e < have; e += NT) taps[W * (cols + 4) + e] = c.bias ? c.bias[c0 + e] : 0.f;
}

// Pairs of channels, for packed multiply-adds; a single channel leaves the second lane of its pair empty.
template <int V>
struct Pairs {
  static constexpr int N = (V + 1) / 2;
  float2 v[N];
  template <typename T>
  __device__ __forceinline__ void from(const Pack<T, V>& p) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = p.pair(i);
  }
  template <typename T>
  __device__ __forceinline__ void to(Pack<T, V>& p) const {
#pragma unroll
    for (int i = 0; i < N; ++i) p.set_pair(i, v[i]);
  }
  __device__ __forceinline__ void load(const float* p) {
    if constexpr (V == 1) {
      v[0] = {p[0], 0.f};
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = *reinterpret_cast<const float2*>(p + 2 * i);
    }
  }
};

template <typename T>
__device__ __forceinline__ float2 sigmoid2(float2 a) {
  return {sigmoid<T>(a.x), sigmoid<T>(a.y)};
}

// A thread's own rows on their way through shared memory: two halves of kHalf rows, one under way while the other
// is worked on.  Nobody else touches them, so they need no barrier.  Single half words, which have no asynchronous
// copy, go through registers.
constexpr int kHalf = 8;

template <typename T, int V>
struct Ring {
  static constexpr int BYTES = V * (int)sizeof(T), SLOT = NT * (BYTES < 4 ? 4 : BYTES), HALF = kHalf * SLOT;
  static constexpr size_t bytes = 2 * HALF;
  unsigned to, from;  // this thread's first slot of the half to fill and of the half to read

  __device__ __forceinline__ Ring(const char* shared, int n) {
    from = (unsigned)__cvta_generic_to_shared(shared) + n * (SLOT / NT);
    to = from;
  }
  // the next row of the half to fill, its k-th
  __device__ __forceinline__ void ask(int k, const T* src, bool in) const {
    if constexpr (BYTES == 16) {
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + k * SLOT), "l"(src), "r"(in ? 16 : 0) : "memory");
    } else if constexpr (BYTES >= 4) {
      asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(to + k * SLOT), "l"(src), "n"(BYTES), "r"(in ? BYTES : 0) : "memory");
    }
  }
  // the k-th row of a half word, loaded by the caller (all of a half's before the first is put)
  __device__ __forceinline__ void put(int k, unsigned v) const { asm volatile("st.shared.u32 [%0], %1;" ::"r"(to + k * SLOT), "r"(v) : "memory"); }
  __device__ __forceinline__ Pack<T, V> get(int k) const {
    Pack<T, V> r;
    const unsigned at = from + k * SLOT;
    if constexpr (BYTES == 16)
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.u[0]), "=r"(r.u[1]), "=r"(r.u[2]), "=r"(r.u[3]) : "r"(at) : "memory");
    else if constexpr (BYTES == 8)
      asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(r.u[0]), "=r"(r.u[1]) : "r"(at) : "memory");
    else
      asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r.u[0]) : "r"(at) : "memory");
    return r;
  }
  // go on to the other half, to fill (`way` = HALF, -HALF in turn) or to read
  __device__ __forceinline__ void filled(int way) { to += way; }
  __device__ __forceinline__ void read(int way) { from += way; }
  static __device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
  template <int PENDING>
  static __device__ __forceinline__ void wait() { asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory"); }
};

// Block (lanes over channel vectors, strips of `strip` tokens).  The window of the last W inputs is a ring whose
// places repeat every W tokens, so a round of GR tokens (a multiple of W) is one copy of the code.
template <typename T, int V, int W>
__global__ void __launch_bounds__(NT, W <= 4 ? 2 : 1) k_conv_fwd(Conv c, int lg, int strip) {
  extern __shared__ __align__(16) char shared[];
  if (bad_call(c.seqs)) return;
  Piece p{};
  if (!find_piece(c.seqs, blockIdx.x, lg, p)) return;
  const int cols = blockDim.x * V;
  const int64_t c0 = (int64_t)blockIdx.y * cols, ch = c0 + threadIdx.x * V;
  Ring<T, V> ring(shared, threadIdx.y * blockDim.x + threadIdx.x);
  float* taps = reinterpret_cast<float*>(shared + Ring<T, V>::bytes);
  const bool live = ch < c.D;
  const int end = p.pos + p.len, s0 = p.pos + threadIdx.y * strip, s1 = live ? min(end, s0 + strip) : s0;
  constexpr int N = Pairs<V>::N, GR = kHalf / W * W, HALF = Ring<T, V>::HALF;
  const T* x = static_cast<const T*>(c.x) + (p.t0 - p.pos + s0) * c.ld + ch;  // the next row to ask for
  int left = s1 - s0;
  auto ask = [&](int way) {
    if constexpr (Ring<T, V>::BYTES >= 4) {
#pragma unroll
      for (int k = 0; k < GR; ++k, x += c.ld) ring.ask(k, x, k < left);
    } else {
      unsigned v[GR];
#pragma unroll
      for (int k = 0; k < GR; ++k, x += c.ld) v[k] = k < left ? *reinterpret_cast<const unsigned short*>(x) : 0u;
#pragma unroll
      for (int k = 0; k < GR; ++k) ring.put(k, v[k]);
    }
    left -= GR;
    ring.commit();
    ring.filled(way);
  };
  ask(HALF);
  ask(-HALF);
  stage_taps<W>(c, taps, c0, cols);
  __syncthreads();
  if (s0 < s1) {
    Pairs<V> w[W], bias;
#pragma unroll
    for (int j = 0; j < W; ++j) w[j].load(taps + j * (cols + 4) + threadIdx.x * V);
    bias.load(taps + W * (cols + 4) + threadIdx.x * V);
    Pairs<V> xw[W];  // before the strip's first token, the token j - W before it is at place j
#pragma unroll
    for (int j = 0; j < W; ++j) {
      Pack<T, V> r;
      if (j > 0)
        load_row<T, V>(c, p, s0 + j - W, ch, r);
      else
        r.zero();
      xw[j].from(r);
    }
    T* y = static_cast<T*>(c.y) + (p.t0 - p.pos + s0) * c.D + ch;
    int way = HALF;
#pragma unroll 1
    for (int n = s1 - s0; n > 0; n -= GR, way = -way) {
      ring.template wait<1>();
#pragma unroll
      for (int k = 0; k < GR; ++k, y += c.D) {
        const int here = k % W;
        xw[here].from(ring.get(k));
        Pairs<V> o = bias;
#pragma unroll
        for (int j = 0; j < W; ++j)
#pragma unroll
          for (int i = 0; i < N; ++i) o.v[i] = __ffma2_rn(w[j].v[i], xw[(here + 1 + j) % W].v[i], o.v[i]);
        if (c.silu) {
#pragma unroll
          for (int i = 0; i < N; ++i) o.v[i] = __fmul2_rn(o.v[i], sigmoid2<T>(o.v[i]));
        }
        Pack<T, V> r;
        o.to(r);
        if (k < n) r.store(y);
      }
      ring.read(way);
      ask(way);
    }
  }
  ring.template wait<0>();
  if (live && c.final && end == p.slen && (int)threadIdx.y < W - 1) {
    Pack<T, V> r;
    load_row<T, V>(c, p, p.slen - (W - 1) + (int)threadIdx.y, ch, r);
    r.store(static_cast<T*>(c.final) + ((int64_t)p.seq * (W - 1) + threadIdx.y) * c.D + ch);
  }
}

// A strip slides over its tokens and the W - 1 after them: dpre of a token completes dx of the token W - 1 before
// it.  The windows of the last W inputs and dpre are rings whose places repeat every W tokens, so a round of GR
// tokens (a multiple of W) is one copy of the code; the rows of the round ahead are in flight meanwhile.
template <typename T, int V, int W>
__global__ void __launch_bounds__(NT, W <= 4 ? 2 : 1) k_conv_bwd(Conv c, int lg) {
  extern __shared__ __align__(16) char shared[];
  __shared__ float red[NT * V];
  constexpr int N = Pairs<V>::N, GR = kHalf / W * W, STEPS = BS + W - 1;
  if (bad_call(c.seqs)) return;
  Piece p{};
  const bool some = find_piece(c.seqs, blockIdx.x, lg, p);
  const int cols = blockDim.x * V;
  const int64_t c0 = (int64_t)blockIdx.y * cols, ch = c0 + threadIdx.x * V;
  const bool live = ch < c.D;
  const int me = threadIdx.y * blockDim.x + threadIdx.x;
  Ring<T, V> xs(shared, me), gs(shared + Ring<T, V>::bytes, me);
  float* taps = reinterpret_cast<float*>(shared + 2 * Ring<T, V>::bytes);
  const int s0 = some ? p.pos + (int)threadIdx.y * BS : 0;
  const bool busy = some && live && (s0 < p.pos + p.len || s0 == 0);
  const int64_t bos = p.t0 - p.pos;
  constexpr int HALF = Ring<T, V>::HALF;
  const T* x = static_cast<const T*>(c.x) + (bos + s0) * c.ld + ch;  // the next rows to ask for
  const T* dy = static_cast<const T*>(c.dy) + (bos + s0) * c.D + ch;
  int left = busy ? min(STEPS, p.slen - s0) : 0;
  auto ask = [&](int way) {
    if constexpr (Ring<T, V>::BYTES >= 4) {
#pragma unroll
      for (int k = 0; k < GR; ++k, x += c.ld, dy += c.D) {
        xs.ask(k, x, k < left);
        gs.ask(k, dy, k < left);
      }
    } else {
      unsigned v[GR], g[GR];
#pragma unroll
      for (int k = 0; k < GR; ++k, x += c.ld, dy += c.D) {
        v[k] = k < left ? *reinterpret_cast<const unsigned short*>(x) : 0u;
        g[k] = k < left ? *reinterpret_cast<const unsigned short*>(dy) : 0u;
      }
#pragma unroll
      for (int k = 0; k < GR; ++k) xs.put(k, v[k]), gs.put(k, g[k]);
    }
    left -= GR;
    xs.commit();
    xs.filled(way);
    gs.filled(way);
  };
  ask(HALF);
  ask(-HALF);
  stage_taps<W>(c, taps, c0, cols);
  __syncthreads();
  Pairs<V> dw[W], db;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    db.v[i] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < W; ++j) dw[j].v[i] = {0.f, 0.f};
  }
  if (busy) {
    Pairs<V> w[W], bias, xw[W], dp[W];
#pragma unroll
    for (int j = 0; j < W; ++j) w[j].load(taps + j * (cols + 4) + threadIdx.x * V);
    bias.load(taps + W * (cols + 4) + threadIdx.x * V);
    // step i's values are at place i % W; before step 0, step j - W's at place j
#pragma unroll
    for (int j = 0; j < W; ++j) {
#pragma unroll
      for (int i = 0; i < N; ++i) dp[j].v[i] = {0.f, 0.f};
      Pack<T, V> r;
      if (j > 0)
        load_row<T, V>(c, p, s0 + j - W, ch, r);
      else
        r.zero();
      xw[j].from(r);
    }
    T* dx = static_cast<T*>(c.dx) + (bos + s0 - (W - 1)) * c.D + ch;  // of the token that a step completes
    int way = HALF;
#pragma unroll 1
    for (int i0 = 0; i0 < STEPS; i0 += GR, way = -way) {
      xs.template wait<1>();
#pragma unroll
      for (int k = 0; k < GR; ++k, dx += c.D) {
        const int i = i0 + k, at = s0 + i;
        if (i >= STEPS) break;
        constexpr int L = W - 1;
        const int here = k % W;
        const bool in = at < p.slen;
        xw[here].from(xs.get(k));
        Pairs<V> g;
        g.from(gs.get(k));
        if (c.silu) {
#pragma unroll
          for (int v = 0; v < N; ++v) {
            float2 a = bias.v[v];
#pragma unroll
            for (int j = 0; j < W; ++j) a = __ffma2_rn(w[j].v[v], xw[(here + 1 + j) % W].v[v], a);
            const float2 sg = sigmoid2<T>(a), one = {1.f, 1.f};
            const float2 rest = __ffma2_rn(sg, {-1.f, -1.f}, one);
            g.v[v] = __fmul2_rn(g.v[v], __fmul2_rn(sg, __ffma2_rn(a, rest, one)));
          }
        }
#pragma unroll
        for (int v = 0; v < N; ++v) {
          if (!in) g.v[v] = {0.f, 0.f};
          dp[here].v[v] = g.v[v];
        }
        if (i < BS && in) {
#pragma unroll
          for (int v = 0; v < N; ++v) {
            db.v[v] = __fadd2_rn(db.v[v], g.v[v]);
#pragma unroll
            for (int j = 0; j < W; ++j) dw[j].v[v] = __ffma2_rn(g.v[v], xw[(here + 1 + j) % W].v[v], dw[j].v[v]);
          }
        }
        const int q = at - L;  // the token whose gradient is now complete
        const bool own = i >= L && q < p.slen;
        const bool before = q < 0 && s0 == 0;
        if ((own || before) && (own ? c.dx != nullptr : c.dinit != nullptr)) {
          Pairs<V> o;
#pragma unroll
          for (int v = 0; v < N; ++v) {
            o.v[v] = __fmul2_rn(w[L].v[v], dp[(here + 1) % W].v[v]);
#pragma unroll
            for (int j = 1; j < W; ++j) o.v[v] = __ffma2_rn(w[L - j].v[v], dp[(here + 1 + j) % W].v[v], o.v[v]);
          }
          const int slot = q - p.slen + L;  // its place in the final state
          if (c.dfinal && slot >= 0) {
            Pack<T, V> r;
            r.load(static_cast<const T*>(c.dfinal) + ((int64_t)p.seq * L + slot) * c.D + ch);
            Pairs<V> f;
            f.from(r);
#pragma unroll
            for (int v = 0; v < N; ++v) o.v[v] = __fadd2_rn(o.v[v], f.v[v]);
          }
          Pack<T, V> r;
          o.to(r);
          if (own)
            r.store(dx);
          else
            r.store(static_cast<T*>(c.dinit) + ((int64_t)p.seq * L + i) * c.D + ch);
        }
      }
      xs.read(way);
      gs.read(way);
      ask(way);
    }
  }
  xs.template wait<0>();
  if (!c.part) return;
  // the block's strips in order, one tap at a time
  float* part = c.part + (int64_t)blockIdx.x * (W + 1) * c.D + ch;
#pragma unroll
  for (int j = 0; j <= W; ++j) {
    __syncthreads();
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float2 f = j < W ? dw[j < W ? j : 0].v[v / 2] : db.v[v / 2];
      red[(threadIdx.y * blockDim.x + threadIdx.x) * V + v] = v % 2 ? f.y : f.x;
    }
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

// One token for each sequence, two channels to a thread (more would put a thread's taps far from the next
// lane's); the state moves up by one input.  state and final may be one buffer:
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
  float o[V], w[V * W];
  if constexpr (V * W % 4 == 0) {  // (ch is a multiple of V)
#pragma unroll
    for (int i = 0; i < V * W; i += 4) {
      const float4 f = *reinterpret_cast<const float4*>(c.weight + ch * W + i);
      w[i] = f.x, w[i + 1] = f.y, w[i + 2] = f.z, w[i + 3] = f.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V * W; ++i) w[i] = c.weight[ch * W + i];
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float a = c.bias ? c.bias[ch + i] : 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) a = fmaf(w[i * W + j], rows[j].f(i), a);
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

// Vectors of V elements need widths, strides and bases that are multiples: 16 bytes forward, four elements backward,
// or else the 4-byte words of an even width.
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

size_t taps_bytes(int lanes, int V, int W) { return (size_t)(W + 1) * (lanes * V + 4) * sizeof(float); }

template <typename T, int V, int W>
cudaError_t fwd_w(const Conv& c, cudaStream_t s) {
  const int lanes = lanes_of(c.D, V);
  const int64_t across = (c.D + (int64_t)lanes * V - 1) / ((int64_t)lanes * V);
  int strip = kHalf, lg = log2i(strip * NT / lanes);
  // strips of up to 64 tokens while eight blocks for each of 148 multiprocessors are left
  const int64_t tokens = c.seqs.cu ? c.seqs.T : c.seqs.T * c.seqs.n;
  while (strip < 64 && (tokens >> (lg + 1)) * across >= 148 * 8) strip *= 2, ++lg;
  const dim3 grid((unsigned)max_units(c.seqs, lg), (unsigned)across);
  const size_t bytes = Ring<T, V>::bytes + taps_bytes(lanes, V, W);
  if (cudaError_t e = allow_shared(k_conv_fwd<T, V, W>, bytes)) return e;
  k_conv_fwd<T, V, W><<<grid, dim3(lanes, NT / lanes), bytes, s>>>(c, lg, strip);
  return cudaGetLastError();
}

template <typename T, int V, int W>
cudaError_t bwd_w(const Conv& c, cudaStream_t s) {
  const int lanes = lanes_of(c.D, 4), lg = bwd_lg(c.D);
  const dim3 grid((unsigned)max_units(c.seqs, lg), (unsigned)((c.D + (int64_t)lanes * V - 1) / ((int64_t)lanes * V)));
  const size_t bytes = 2 * Ring<T, V>::bytes + taps_bytes(lanes, V, W);
  if (cudaError_t e = allow_shared(k_conv_bwd<T, V, W>, bytes)) return e;
  k_conv_bwd<T, V, W><<<grid, dim3(lanes, NT / lanes), bytes, s>>>(c, lg);
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
                         : step_w<T, (V > 2 ? 2 : V), w>(c, s);
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
  const int V = vec_ok(c, 2, WHAT == BWD ? 4 : 8) ? 8 : vec_ok(c, 2, 2) ? 2 : 1;
  if (c.dtype == GDN_DTYPE_BF16)
    return V == 8   ? by_width<WHAT, __nv_bfloat16, 8>(c, s)
           : V == 2 ? by_width<WHAT, __nv_bfloat16, 2>(c, s)
                    : by_width<WHAT, __nv_bfloat16, 1>(c, s);
  return V == 8 ? by_width<WHAT, __half, 8>(c, s) : V == 2 ? by_width<WHAT, __half, 2>(c, s) : by_width<WHAT, __half, 1>(c, s);
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
  return column_sums("conv_bwd_sums", c.seqs, c.part, conv_bwd_units(c.seqs, c.D), (c.W + 1) * c.D, (c.W + 1) * c.D,
                     c.dweight, c.dbias, c.W, c.D, s);
}

cudaError_t conv_step(const Conv& c, cudaStream_t s) {
  ProfScope ps("conv_step", s);
  return dispatch<STEP>(c, s);
}

}  // namespace mix
}  // namespace gdn
