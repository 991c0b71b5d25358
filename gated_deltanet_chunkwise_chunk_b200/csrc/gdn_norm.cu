// Layer norm over the last axis, with optional weight, bias and gate; the rms form keeps the mean.
//   xh = (x - mu) rstd,  n = xh w + b,  y = n  or  n silu(z)
// Backward: dn = dy silu(z), dz = dy n silu'(z), u = dn w,
//   dx = rstd (u - mean(u) - xh mean(u xh))   (rms: without mean(u)),
//   dw = sum over rows of dn xh,  db = sum over rows of dn.
// Bound by HBM: a row stays in registers between its statistics and its output, so x (z, dy) is read
// once and y (dx, dz) written once.  A row belongs to a group of 1 to 32 lanes (several rows to a
// block) or to a block of up to 512 threads; each thread holds NV vectors of it.  The variance
// is the mean of (x - mu)^2 over the registers, not a difference of sums.  The backward's blocks walk
// over many rows with the weight's and bias's sums in registers and the next rows' loads in flight;
// their partial rows are added in block order by a second kernel, so the sums do not depend on timing.
// Measured (bf16): rows of 4096, 8192 of them, with weight and bias: forward 36 us for 134 MB (3.7 TB/s), backward
// 59 us for 201 MB (3.4 TB/s); gated rms rows of 128, 262144 of them: forward 47 us for 201 MB (4.3 TB/s), backward
// 95 us for 335 MB (3.5 TB/s).  The forward of the heads is bound by issue (81% of its peak; DRAM 47%); the others wait
// for their own latencies (issue 58 to 71%, DRAM 32 to 39%): a row's sums cost its threads as much as eight elements, so
// a thread has 16 to 32 of them, which leaves sixteen warps a multiprocessor.
#include <algorithm>

#include "mix_common.cuh"

namespace gdn {
namespace mix {
namespace {

constexpr int NG = 256;  // threads of a block of lane groups

// Sum of N values over the row's threads, the same result in each: lanes of the group by butterflies,
// then the block's warps through shared memory in warp order.
template <int N, bool BLOCK>
__device__ __forceinline__ void row_sum(float (&a)[N], int lanes, float* sh) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    if (o >= lanes) continue;
#pragma unroll
    for (int i = 0; i < N; ++i) a[i] += __shfl_xor_sync(0xffffffffu, a[i], o);
  }
  if (BLOCK) {
    const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) sh[i * 32 + warp] = a[i];
    }
    __syncthreads();
    const int l = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float v = l < warps ? sh[i * 32 + l] : 0.f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      a[i] = v;
    }
  }
}

__device__ __forceinline__ int64_t row_at(int64_t r, int64_t inner, int64_t ld, int64_t D) {
  if (inner == 1) return r * ld;
  const int64_t o = r / inner;
  return o * ld + (r - o * inner) * D;
}

// A thread's own vectors of the rows to come, DEEP rows ahead, on their way through shared memory (nobody else
// touches them, so they need no barrier).  ARR tensors of NV vectors, and a row's statistics.  DEEP: four, or as
// many as leave room for a second block.  Single half words, which have no asynchronous copy, wait one row ahead in
// registers.
template <typename T, int V, int NV, int ARR, int MOST>
struct Ahead {
  static constexpr int BYTES = V * (int)sizeof(T), WIDTH = BYTES < 4 ? 4 : BYTES, ROW = ARR * NV * WIDTH + 8;
  static constexpr int FIT = 104 * 1024 / (ROW * MOST), DEEP = BYTES < 4 ? 1 : FIT < 2 ? 2 : FIT > 4 ? 4 : FIT;
  static constexpr size_t bytes(int threads) { return (size_t)DEEP * ROW * threads; }
  unsigned base;
  int threads;
  unsigned short held[BYTES < 4 ? ARR * NV : 1];

  __device__ __forceinline__ Ahead(const char* shared) : base((unsigned)__cvta_generic_to_shared(shared)), threads(blockDim.x) {}
  // thread-interleaved: vector v of a slot at [slot][v][thread], the statistics behind them
  __device__ __forceinline__ unsigned at(int slot, int v) const {
    return base + slot * ROW * threads + (v * threads + threadIdx.x) * WIDTH;
  }
  __device__ __forceinline__ unsigned stat_at(int slot) const { return base + (slot * ROW + ARR * NV * WIDTH) * threads + threadIdx.x * 8; }
  __device__ __forceinline__ void ask(int slot, int v, const T* src, bool in) {
    if constexpr (BYTES == 16)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at(slot, v)), "l"(src), "r"(in ? 16 : 0) : "memory");
    else if constexpr (BYTES >= 4)
      asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(at(slot, v)), "l"(src), "n"(BYTES), "r"(in ? BYTES : 0) : "memory");
    else {
      held[v] = 0;
      if (in) held[v] = *reinterpret_cast<const unsigned short*>(src);
    }
  }
  __device__ __forceinline__ void ask_stats(int slot, const float* src, bool in) const {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(stat_at(slot)), "l"(src), "r"(in ? 8 : 0) : "memory");
  }
  __device__ __forceinline__ Pack<T, V> get(int slot, int v) const {
    Pack<T, V> r;
    if constexpr (BYTES < 4) {
      r.u[0] = held[v];
      return r;
    }
    const unsigned a = at(slot, v);
    if constexpr (BYTES == 16)
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.u[0]), "=r"(r.u[1]), "=r"(r.u[2]), "=r"(r.u[3]) : "r"(a) : "memory");
    else
      asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r.u[0]) : "r"(a) : "memory");
    return r;
  }
  __device__ __forceinline__ float2 stats(int slot) const {
    float2 f;
    asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(f.x), "=f"(f.y) : "r"(stat_at(slot)) : "memory");
    return f;
  }
  static __device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
  template <int PENDING>
  static __device__ __forceinline__ void wait() { asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory"); }
};

// lanes: threads of a row; BLOCK: the whole block, else a power of two up to 32.
template <typename T, int V, int NV, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? 512 : NG) k_norm_fwd(Norm c, int lanes) {
  extern __shared__ __align__(16) char shared[];
  __shared__ float sh[2][2][32];
  using A = Ahead<T, V, NV, 2, BLOCK ? 512 : NG>;
  A ahead(shared);
  const int lane = BLOCK ? threadIdx.x : threadIdx.x & (lanes - 1);
  const int rpb = BLOCK ? 1 : NG / lanes;
  const int64_t step = (int64_t)gridDim.x * rpb;
  const int64_t first = (int64_t)blockIdx.x * rpb + (BLOCK ? 0 : threadIdx.x / lanes);
  const float inv = 1.f / (float)c.D;
  const T* x = static_cast<const T*>(c.x);
  const T* z = static_cast<const T*>(c.gate);
  T* y = static_cast<T*>(c.y);
  int col[NV];
  bool live[NV];
  float w[NV][V], b[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    col[i] = (i * lanes + lane) * V;
    live[i] = col[i] < c.D;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      w[i][v] = live[i] && c.weight ? c.weight[col[i] + v] : 1.f;
      b[i][v] = live[i] && c.bias ? c.bias[col[i] + v] : 0.f;
    }
  }
  auto ask = [&](int64_t r, int slot) {
    const bool row = r < c.rows;
    const T* xa = x + (row ? row_at(r, c.inner_x, c.ld_x, c.D) : 0);
#pragma unroll
    for (int i = 0; i < NV; ++i) ahead.ask(slot, i, xa + col[i], row && live[i]);
    if (z) {
      const T* za = z + (row ? row_at(r, c.inner_z, c.ld_z, c.D) : 0);
#pragma unroll
      for (int i = 0; i < NV; ++i) ahead.ask(slot, NV + i, za + col[i], row && live[i]);
    }
    ahead.commit();
  };
#pragma unroll
  for (int k = 0; k < A::DEEP; ++k) ask(first + k * step, k);
  int flip = 0, slot = 0;
  // every thread of a warp runs the same number of rounds (the butterflies need them all)
  for (int64_t base = (int64_t)blockIdx.x * rpb, r = first; base < c.rows; base += step, r += step) {
    const bool row = r < c.rows;
    Pack<T, V> xr[NV], zr[NV];
    ahead.template wait<A::DEEP - 1>();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      xr[i] = ahead.get(slot, i);
      if (z) zr[i] = ahead.get(slot, NV + i);
    }
    ask(r + A::DEEP * step, slot);
    slot = slot == A::DEEP - 1 ? 0 : slot + 1;
    float mu = 0.f;
    if (!c.rms) {
      float s[1] = {0.f};
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) s[0] += xr[i].f(v);
      row_sum<1, BLOCK>(s, lanes, sh[flip][0]);
      mu = s[0] * inv;
    }
    float q[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float d = xr[i].f(v) - mu;
        if (live[i]) q[0] = fmaf(d, d, q[0]);
      }
    row_sum<1, BLOCK>(q, lanes, sh[flip][1]);
    flip ^= 1;
    const float rstd = rsqrtf(fmaf(q[0], inv, c.eps));
    if (!row) continue;
    if (c.stats && lane == 0) {
      c.stats[2 * r] = mu;
      c.stats[2 * r + 1] = rstd;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!live[i]) continue;
      float o[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        o[v] = fmaf((xr[i].f(v) - mu) * rstd, w[i][v], b[i][v]);
        if (z) {
          const float g = zr[i].f(v);
          o[v] *= g * sigmoid<T>(g);
        }
      }
      Pack<T, V> out;
      out.set(o);
      out.store(y + r * c.D + col[i]);
    }
  }
}

template <typename T, int V, int NV, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? 512 : NG) k_norm_bwd(Norm c, int lanes) {
  extern __shared__ __align__(16) char shared[];
  __shared__ float sh[2][2][32];
  __shared__ float red[BLOCK ? 1 : NG * V];
  using A = Ahead<T, V, NV, 3, BLOCK ? 512 : NG>;
  A ahead(shared);
  const int lane = BLOCK ? threadIdx.x : threadIdx.x & (lanes - 1);
  const int rpb = BLOCK ? 1 : NG / lanes;
  const int64_t step = (int64_t)gridDim.x * rpb;
  const float inv = 1.f / (float)c.D;
  const T* x = static_cast<const T*>(c.x);
  const T* z = static_cast<const T*>(c.gate);
  const T* dy = static_cast<const T*>(c.dy);
  int col[NV];
  bool live[NV];
  float w[NV][V], b[NV][V], dw[NV][V], db[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    col[i] = (i * lanes + lane) * V;
    live[i] = col[i] < c.D;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      w[i][v] = live[i] && c.weight ? c.weight[col[i] + v] : 1.f;
      b[i][v] = live[i] && c.bias && z ? c.bias[col[i] + v] : 0.f;
      dw[i][v] = db[i][v] = 0.f;
    }
  }
  auto ask = [&](int64_t r, int slot) {
    const bool row = r < c.rows;
    const T* xa = x + (row ? row_at(r, c.inner_x, c.ld_x, c.D) : 0);
    const T* ga = dy + (row ? r * c.D : 0);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      ahead.ask(slot, i, xa + col[i], row && live[i]);
      ahead.ask(slot, NV + i, ga + col[i], row && live[i]);
    }
    if (z) {
      const T* za = z + (row ? row_at(r, c.inner_z, c.ld_z, c.D) : 0);
#pragma unroll
      for (int i = 0; i < NV; ++i) ahead.ask(slot, 2 * NV + i, za + col[i], row && live[i]);
    }
    ahead.ask_stats(slot, c.stats + (row ? 2 * r : 0), row);
    ahead.commit();
  };
  int64_t r = (int64_t)blockIdx.x * rpb + (BLOCK ? 0 : threadIdx.x / lanes);
#pragma unroll
  for (int k = 0; k < A::DEEP; ++k) ask(r + k * step, k);
  int flip = 0, slot = 0;
  for (int64_t base = (int64_t)blockIdx.x * rpb; base < c.rows; base += step, r += step) {
    const bool row = r < c.rows;
    Pack<T, V> xr[NV], zr[NV], gr[NV];
    ahead.template wait<A::DEEP - 1>();
    const float2 st = ahead.stats(slot);
    const float m = st.x, rs = st.y;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      xr[i] = ahead.get(slot, i);
      gr[i] = ahead.get(slot, NV + i);
      if (z) zr[i] = ahead.get(slot, 2 * NV + i);
    }
    ask(r + A::DEEP * step, slot);
    slot = slot == A::DEEP - 1 ? 0 : slot + 1;
    float xh[NV][V], u[NV][V];
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float dz[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float h = live[i] ? (xr[i].f(v) - m) * rs : 0.f;
        float dn = gr[i].f(v);
        if (z) {
          const float g = zr[i].f(v), sg = sigmoid<T>(g), n = fmaf(h, w[i][v], b[i][v]);
          dz[v] = dn * n * sg * fmaf(g, 1.f - sg, 1.f);
          dn *= g * sg;
        }
        if (row && live[i]) {
          dw[i][v] = fmaf(dn, h, dw[i][v]);
          db[i][v] += dn;
        }
        xh[i][v] = h;
        u[i][v] = dn * w[i][v];
        s[0] += u[i][v];
        s[1] = fmaf(u[i][v], h, s[1]);
      }
      if (z && row && live[i]) {
        Pack<T, V> out;
        out.set(dz);
        out.store(static_cast<T*>(c.dgate) + r * c.D + col[i]);
      }
    }
    row_sum<2, BLOCK>(s, lanes, sh[flip][0]);
    flip ^= 1;
    if (!row) continue;
    const float a0 = c.rms ? 0.f : s[0] * inv, a1 = s[1] * inv;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!live[i]) continue;
      float o[V];
#pragma unroll
      for (int v = 0; v < V; ++v) o[v] = rs * (u[i][v] - a0 - xh[i][v] * a1);
      Pack<T, V> out;
      out.set(o);
      out.store(static_cast<T*>(c.dx) + r * c.D + col[i]);
    }
  }
  if (!c.part) return;
  float* part = c.part + (int64_t)blockIdx.x * (c.dbias ? 2 : 1) * c.D;
  if constexpr (BLOCK) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (live[i]) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          part[col[i] + v] = dw[i][v];
          if (c.dbias) part[c.D + col[i] + v] = db[i][v];
        }
      }
  } else {
    for (int k = 0; k < (c.dbias ? 2 : 1); ++k)
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        __syncthreads();
#pragma unroll
        for (int v = 0; v < V; ++v) red[threadIdx.x * V + v] = k ? db[i][v] : dw[i][v];
        __syncthreads();
        if ((int)threadIdx.x < lanes && live[i]) {
#pragma unroll
          for (int v = 0; v < V; ++v) {
            float a = 0.f;
            for (int g = 0; g < rpb; ++g) a += red[(g * lanes + lane) * V + v];
            part[k * c.D + col[i] + v] = a;
          }
        }
      }
  }
}

// Rows too wide for the registers of a block: the same in three passes over the row, which the
// caches hold.  The sums of the block's rows stay in its partial row in memory.
template <typename T>
__global__ void __launch_bounds__(1024) k_norm_fwd_wide(Norm c) {
  __shared__ float sh[2][32];
  for (int64_t r = blockIdx.x; r < c.rows; r += gridDim.x) {
    const T* x = static_cast<const T*>(c.x) + row_at(r, c.inner_x, c.ld_x, c.D);
    const T* z = c.gate ? static_cast<const T*>(c.gate) + row_at(r, c.inner_z, c.ld_z, c.D) : nullptr;
    const float inv = 1.f / (float)c.D;
    float mu = 0.f;
    if (!c.rms) {
      float s[1] = {0.f};
      for (int64_t i = threadIdx.x; i < c.D; i += blockDim.x) s[0] += up<T>(x[i]);
      row_sum<1, true>(s, 32, sh[0]);
      mu = s[0] * inv;
    }
    float q[1] = {0.f};
    for (int64_t i = threadIdx.x; i < c.D; i += blockDim.x) {
      const float d = up<T>(x[i]) - mu;
      q[0] = fmaf(d, d, q[0]);
    }
    row_sum<1, true>(q, 32, sh[1]);
    const float rstd = rsqrtf(fmaf(q[0], inv, c.eps));
    if (c.stats && threadIdx.x == 0) {
      c.stats[2 * r] = mu;
      c.stats[2 * r + 1] = rstd;
    }
    for (int64_t i = threadIdx.x; i < c.D; i += blockDim.x) {
      float o = fmaf((up<T>(x[i]) - mu) * rstd, c.weight ? c.weight[i] : 1.f, c.bias ? c.bias[i] : 0.f);
      if (z) {
        const float g = up<T>(z[i]);
        o *= g * sigmoid<T>(g);
      }
      static_cast<T*>(c.y)[r * c.D + i] = down<T>(o);
    }
    __syncthreads();
  }
}

template <typename T>
__global__ void __launch_bounds__(1024) k_norm_bwd_wide(Norm c) {
  __shared__ float sh[2][32];
  const int parts = c.dbias ? 2 : 1;
  float* part = c.part ? c.part + (int64_t)blockIdx.x * parts * c.D : nullptr;
  bool first = true;
  for (int64_t r = blockIdx.x; r < c.rows; r += gridDim.x) {
    const T* x = static_cast<const T*>(c.x) + row_at(r, c.inner_x, c.ld_x, c.D);
    const T* z = c.gate ? static_cast<const T*>(c.gate) + row_at(r, c.inner_z, c.ld_z, c.D) : nullptr;
    const T* dy = static_cast<const T*>(c.dy) + r * c.D;
    const float mu = c.stats[2 * r], rs = c.stats[2 * r + 1], inv = 1.f / (float)c.D;
    float s[2] = {0.f, 0.f};
    for (int64_t i = threadIdx.x; i < c.D; i += blockDim.x) {
      const float h = (up<T>(x[i]) - mu) * rs, w = c.weight ? c.weight[i] : 1.f;
      float dn = up<T>(dy[i]);
      if (z) {
        const float g = up<T>(z[i]), sg = sigmoid<T>(g), n = fmaf(h, w, c.bias ? c.bias[i] : 0.f);
        static_cast<T*>(c.dgate)[r * c.D + i] = down<T>(dn * n * sg * fmaf(g, 1.f - sg, 1.f));
        dn *= g * sg;
      }
      if (part) {
        part[i] = first ? dn * h : fmaf(dn, h, part[i]);
        if (c.dbias) part[c.D + i] = first ? dn : part[c.D + i] + dn;
      }
      s[0] = fmaf(dn, w, s[0]);
      s[1] = fmaf(dn * w, h, s[1]);
    }
    first = false;
    row_sum<2, true>(s, 32, sh[0]);
    const float a0 = c.rms ? 0.f : s[0] * inv, a1 = s[1] * inv;
    for (int64_t i = threadIdx.x; i < c.D; i += blockDim.x) {
      const float h = (up<T>(x[i]) - mu) * rs;
      float dn = up<T>(dy[i]);
      if (z) {
        const float g = up<T>(z[i]);
        dn *= g * sigmoid<T>(g);
      }
      static_cast<T*>(c.dx)[r * c.D + i] = down<T>(rs * (dn * (c.weight ? c.weight[i] : 1.f) - a0 - h * a1));
    }
    __syncthreads();
  }
}

// Vectors of V elements need widths, strides and bases that are multiples.
bool vec_ok(const Norm& c, int es, int V) {
  if (c.D % V || c.ld_x % V || (c.gate && c.ld_z % V)) return false;
  const void* ps[] = {c.x, c.gate, c.y, c.dy, c.dx, c.dgate};
  for (const void* p : ps)
    if (reinterpret_cast<uintptr_t>(p) % ((uintptr_t)V * es)) return false;
  return true;
}

// How a call is launched; a function of the sizes and the vector width only.
struct Plan {
  bool wide, block;
  int nv, threads;  // vectors of a thread; threads of a row
  int64_t blocks;
};

// The backward's blocks walk over rows: up to four of 128 threads or so on each of 148 multiprocessors.
constexpr int64_t kBwdBlocks = 592;
constexpr int64_t kManyRows = 148 * 8;

// Vectors of a row that a thread may hold: 64 bytes' worth in flight, backward 16 elements in registers.
constexpr int most_vectors(int V, int es, bool bwd) { return bwd ? 16 / V : 64 / (V * es < 4 ? 4 : V * es); }

Plan make_plan(int64_t rows, int64_t D, int V, int es, bool bwd) {
  Plan p{};
  const int64_t vecs = (D + V - 1) / V;
  const int most = most_vectors(V, es, bwd);
  p.wide = vecs > 512 * (int64_t)most;
  if (p.wide) {
    p.threads = 1024;
    p.blocks = std::min(rows, bwd ? kBwdBlocks / 2 : (int64_t)148 * 2);
    return p;
  }
  // Many rows: as many vectors to a thread as it may hold, since a row's sums cost each of its threads the same,
  // while 16 lanes are left to read neighbouring vectors together.
  // Few: as many threads to a row as there are, since only its latency counts.
  p.nv = 1;
  while (p.nv < most && (rows >= kManyRows ? p.nv * 32 <= vecs : (vecs + p.nv - 1) / p.nv > 512)) p.nv *= 2;
  const int64_t threads = (vecs + p.nv - 1) / p.nv;
  p.block = threads > 32;
  if (p.block) {
    p.threads = (int)((threads + 31) / 32 * 32);
    p.blocks = std::min<int64_t>(rows, bwd ? kBwdBlocks * 128 / std::max(128, p.threads) : 148 * std::max(2, 512 / p.threads));
    return p;
  }
  p.threads = 1;
  while (p.threads < threads) p.threads *= 2;
  const int rpb = NG / p.threads;
  p.blocks = std::min((rows + rpb - 1) / rpb, bwd ? kBwdBlocks : (int64_t)148 * 8);
  return p;
}

template <typename T, int V, int NV, bool BWD>
cudaError_t launch_nv(const Norm& c, const Plan& p, cudaStream_t s) {
  if constexpr (NV <= most_vectors(V, sizeof(T), BWD)) {
    const unsigned n = (unsigned)p.blocks, threads = p.block ? p.threads : NG;
    constexpr int ARR = BWD ? 3 : 2;
    const size_t bytes = p.block ? Ahead<T, V, NV, ARR, 512>::bytes(threads) : Ahead<T, V, NV, ARR, NG>::bytes(threads);
    auto go = [&](auto* kernel) -> cudaError_t {
      if (cudaError_t e = allow_shared(kernel, bytes)) return e;
      kernel<<<n, threads, bytes, s>>>(c, p.threads);
      return cudaGetLastError();
    };
    if constexpr (BWD)
      return p.block ? go(k_norm_bwd<T, V, NV, true>) : go(k_norm_bwd<T, V, NV, false>);
    else
      return p.block ? go(k_norm_fwd<T, V, NV, true>) : go(k_norm_fwd<T, V, NV, false>);
  }
  return cudaErrorInvalidValue;
}

template <typename T, int V, bool BWD>
cudaError_t launch(const Norm& c, cudaStream_t s, int64_t* blocks) {
  const Plan p = make_plan(c.rows, c.D, V, sizeof(T), BWD);
  *blocks = p.blocks;
  if (p.wide) {
    if constexpr (BWD)
      k_norm_bwd_wide<T><<<(unsigned)p.blocks, p.threads, 0, s>>>(c);
    else
      k_norm_fwd_wide<T><<<(unsigned)p.blocks, p.threads, 0, s>>>(c);
    return cudaGetLastError();
  }
  switch (p.nv) {
    case 1: return launch_nv<T, V, 1, BWD>(c, p, s);
    case 2: return launch_nv<T, V, 2, BWD>(c, p, s);
    case 4: return launch_nv<T, V, 4, BWD>(c, p, s);
    case 8: return launch_nv<T, V, 8, BWD>(c, p, s);
    default: return launch_nv<T, V, 16, BWD>(c, p, s);
  }
}

template <bool BWD>
cudaError_t dispatch(const Norm& c, cudaStream_t s, int64_t* n) {
  if (c.dtype == GDN_DTYPE_FP32) return vec_ok(c, 4, 4) ? launch<float, 4, BWD>(c, s, n) : launch<float, 1, BWD>(c, s, n);
  const int V = vec_ok(c, 2, 8) ? 8 : vec_ok(c, 2, 2) ? 2 : 1;
  if (c.dtype == GDN_DTYPE_BF16)
    return V == 8   ? launch<__nv_bfloat16, 8, BWD>(c, s, n)
           : V == 2 ? launch<__nv_bfloat16, 2, BWD>(c, s, n)
                    : launch<__nv_bfloat16, 1, BWD>(c, s, n);
  return V == 8 ? launch<__half, 8, BWD>(c, s, n) : V == 2 ? launch<__half, 2, BWD>(c, s, n) : launch<__half, 1, BWD>(c, s, n);
}

}  // namespace

size_t norm_bwd_part_floats(int64_t rows, int64_t D) { return (size_t)std::min(rows, kBwdBlocks) * 2 * D; }

cudaError_t norm_forward(const Norm& c, cudaStream_t s) {
  if (c.rows == 0) return cudaSuccess;
  ProfScope ps("norm_fwd", s);
  int64_t blocks = 0;
  return dispatch<false>(c, s, &blocks);
}

cudaError_t norm_backward(const Norm& c, cudaStream_t s) {
  int64_t blocks = 0;
  if (c.rows > 0) {
    ProfScope ps("norm_bwd", s);
    const cudaError_t e = dispatch<true>(c, s, &blocks);
    if (e != cudaSuccess) return e;
  }
  if (!c.dweight && !c.dbias) return cudaSuccess;
  return column_sums("norm_bwd_sums", Seqs{}, c.part, blocks, (c.dbias ? 2 : 1) * c.D, (c.dbias ? 2 : 1) * c.D, c.dweight, c.dbias,
                     1, c.D, s);
}

}  // namespace mix
}  // namespace gdn
