// Selective state space scan: backward.  With g[t] the gradient of the state behind token t and a the decays,
//   g[t] = C[t] dy[t] + a[t+1] g[t+1]  (+ the final state's gradient at the end),   q[t] = a[t] g[t] h[t-1],
//   dx = delta sum_n g B + Dskip dy,   ddelta = x sum_n g B + sum_n A q,   ddt = ddelta softplus',
//   dB = sum_d g delta x,  dC = sum_d dy h  (over the group's channels),
//   dA_log = A sum_t delta q,  dDskip = sum_t dy x,  ddt_bias = sum_t ddt.
// The states come from the forward's every-16th-token copies: a warp goes through 16 tokens forwards with
// their states and decays left in registers (4 states to a lane, so 128 of them), then back, so each
// exponential is computed once.  The sums over n and over a warp's channels are butterflies that halve the
// values as they go; a block's warps add their dB and dC in shared memory, and the blocks of a group's
// channels leave partial rows that a second kernel adds in order.  Nothing is atomic.
#include <algorithm>

#include "ssm_common.cuh"

namespace gdn {
namespace mix {
namespace {

__device__ __forceinline__ int64_t tokens_of(const Seqs& s) { return s.cu ? s.T : s.T * s.n; }

template <int NP>
struct BwdShared {
  float d[kWarps][Shape<NP>::CW][kRow];      // delta, then ddt
  float x[kWarps][Shape<NP>::CW][kRow];      // x, then dx
  float g[kWarps][Shape<NP>::CW][kRow];      // dy
  float slope[kWarps][Shape<NP>::CW][kRow];  // softplus'
  float b[kTile * NP], c[kTile * NP];
  float red[kWarps][kTile][2 * NP];  // a warp's dB and dC of the tile
};

// The gradient that leaves a segment at its front when none enters at its end, and the sum of its deltas.
template <typename T, int NP>
__global__ void __launch_bounds__(kWarps * 32) k_ssm_bwd_ends(Ssm s) {
  using S = Shape<NP>;
  constexpr int CW = S::CW;
  __shared__ __align__(16) float sd[kWarps][CW][kRow], sg[kWarps][CW][kRow], sc[kTile * NP];
  if (bad_call(s.seqs)) return;
  Place<NP> at;
  if (!at.find(s, s.lg)) return;
  const Piece& p = at.p;
  if (p.idx == 0) return;
  const int n0 = at.nl * 4;
  float A2[4], ga[4] = {0.f, 0.f, 0.f, 0.f}, dsum[CW], bias[CW];
  load_decay(s, at.ch, at.live, n0, A2);
#pragma unroll
  for (int i = 0; i < CW; ++i) {
    dsum[i] = 0.f;
    bias[i] = i < at.n && s.dt_bias ? s.dt_bias[at.c0 + i] : 0.f;
  }
  const T* dt = static_cast<const T*>(s.dt) + p.t0 * s.ld_dt + at.c0;
  const T* dy = static_cast<const T*>(s.dy) + p.t0 * s.D + at.c0;
  const T* Cm = static_cast<const T*>(s.Cm) + p.t0 * s.ld_c + (int64_t)at.g * s.N;
  Cols<T, CW> gr, tr;
  Mat<T, NP> cr;
  auto fetch = [&](int t0) {
    const int64_t t = t0 + at.lane;
    const bool in = t < p.len;
    tr.fetch(dt + t * s.ld_dt, in, s.vec, at.n);
    gr.fetch(dy + t * s.D, in, s.vec, at.n);
    cr.fetch(Cm + t0 * s.ld_c, s.ld_c, s.N, p.len - t0);
  };
  int t0 = (p.len - 1) / kTile * kTile;
  fetch(t0);
  for (; t0 >= 0; t0 -= kTile) {
    const bool in = t0 + at.lane < p.len;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < CW; ++i) {
      const float d = in && i < at.n ? softplus_acc(tr.get(i) + bias[i]) : 0.f;
      sd[at.warp][i][at.lane] = d;
      sg[at.warp][i][at.lane] = gr.get(i);
      dsum[i] += d;
    }
    cr.stage(sc);
    __syncthreads();
    if (t0 > 0) fetch(t0 - kTile);
#pragma unroll 2
    for (int q = kTile / 4 - 1; q >= 0; --q) {
      const float4 dv = *reinterpret_cast<const float4*>(&sd[at.warp][at.cl][4 * q]);
      const float4 gv = *reinterpret_cast<const float4*>(&sg[at.warp][at.cl][4 * q]);
      const float d4[4] = {dv.x, dv.y, dv.z, dv.w}, g4[4] = {gv.x, gv.y, gv.z, gv.w};
#pragma unroll
      for (int k = 3; k >= 0; --k) {
        const float4 cv = *reinterpret_cast<const float4*>(&sc[(4 * q + k) * NP + n0]);
        const float c4[4] = {cv.x, cv.y, cv.z, cv.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) ga[j] = ex2(d4[k] * A2[j]) * fmaf(c4[j], g4[k], ga[j]);
      }
    }
  }
  float total = 0.f;
#pragma unroll
  for (int i = 0; i < CW; ++i) {
    float v = dsum[i];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (i == at.cl) total = v;
  }
  if (at.live) {
    *reinterpret_cast<float4*>(s.starts + state_at<NP>(s, blockIdx.x, at.ch, n0)) = make_float4(ga[0], ga[1], ga[2], ga[3]);
    if (at.nl == 0) s.sums[(int64_t)blockIdx.x * s.D + at.ch] = total;
  }
}

// The segments of a sequence from its end: a unit's slot becomes the gradient that enters it there.
template <int NP>
__global__ void __launch_bounds__(256) k_ssm_bwd_join(Ssm s) {
  if (bad_call(s.seqs)) return;
  const unsigned blocks = (unsigned)((s.D * NP + 255) / 256);  // of a sequence
  const int seq = (int)(blockIdx.x / blocks);
  const int64_t at = (int64_t)(blockIdx.x - seq * blocks) * 256 + threadIdx.x, ch = at / NP;
  const int n = (int)(at % NP);
  if (ch >= s.D || n >= s.N) return;
  const int64_t len = s.seqs.cu ? s.seqs.cu[seq + 1] - s.seqs.cu[seq] : s.seqs.T;
  const int64_t segs = len == 0 ? 1 : ((len - 1) >> s.lg) + 1, u0 = first_unit(s.seqs, seq, s.lg);
  const float A2 = decay_rate(s.A_log[ch * s.N + n]);
  float g = s.dfinal ? s.dfinal[((int64_t)seq * s.D + ch) * s.N + n] : 0.f;
  for (int64_t k = segs - 1; k >= 0; --k) {
    float* p = s.starts + state_at<NP>(s, u0 + k, ch, n);
    const float front = *p;
    *p = g;
    if (k > 0) g = fmaf(ex2(A2 * s.sums[(u0 + k) * s.D + ch]), g, front);
  }
}

template <typename T, int NP>
__global__ void __launch_bounds__(kWarps * 32) k_ssm_bwd(Ssm s) {
  using S = Shape<NP>;
  constexpr int NL = S::NL, CW = S::CW;
  extern __shared__ __align__(16) char raw[];
  BwdShared<NP>& m = *reinterpret_cast<BwdShared<NP>*>(raw);
  if (bad_call(s.seqs)) return;
  Place<NP> at;
  const bool unit = at.find(s, s.lg);
  const Piece& p = at.p;
  const int n0 = at.nl * 4;
  float* par = s.part_par + ((int64_t)blockIdx.x * s.D + at.ch) * (s.N + 2);
  if (!unit) {  // no such segment: its sums are empty
    if (at.live) {
      for (int j = n0; j < n0 + 4; ++j)
        if (j < s.N) par[j] = 0.f;
      if (at.nl == 0) par[s.N] = par[s.N + 1] = 0.f;
    }
    return;
  }
  float A2[4], ga[4] = {0.f, 0.f, 0.f, 0.f}, dA[4] = {0.f, 0.f, 0.f, 0.f};
  load_decay(s, at.ch, at.live, n0, A2);
  if (at.live) {
    if (s.cut && p.pos + p.len < p.slen) {
      const float4 v = *reinterpret_cast<const float4*>(s.starts + state_at<NP>(s, blockIdx.x, at.ch, n0));
      ga[0] = v.x, ga[1] = v.y, ga[2] = v.z, ga[3] = v.w;
    } else if (s.dfinal) {
      load_states(s.dfinal + ((int64_t)p.seq * s.D + at.ch) * s.N, s.N, n0, ga);
    }
  }
  const float skip = at.live && s.skip ? s.skip[at.ch] : 0.f;
  float dskip = 0.f, dbias = 0.f;
  float bias[CW];
#pragma unroll
  for (int i = 0; i < CW; ++i) bias[i] = i < at.n && s.dt_bias ? s.dt_bias[at.c0 + i] : 0.f;
  const T* x = static_cast<const T*>(s.x) + p.t0 * s.ld_x + at.c0;
  const T* dt = static_cast<const T*>(s.dt) + p.t0 * s.ld_dt + at.c0;
  const T* dy = static_cast<const T*>(s.dy) + p.t0 * s.D + at.c0;
  const T* Bm = static_cast<const T*>(s.Bm) + p.t0 * s.ld_b + (int64_t)at.g * s.N;
  const T* Cm = static_cast<const T*>(s.Cm) + p.t0 * s.ld_c + (int64_t)at.g * s.N;
  T* dx = static_cast<T*>(s.dx) + p.t0 * s.D + at.c0;
  T* ddt = static_cast<T*>(s.ddt) + p.t0 * s.D + at.c0;
  const float* ck = s.ckpt + state_at<NP>(s, first_unit(s.seqs, p.seq, kCkptLog) + p.pos / kCkpt, at.ch, n0);
  const int64_t tiles = (s.D / s.G + S::CC - 1) / S::CC;
  float* pbc = s.part_bc + (((blockIdx.y - at.g * tiles) * tokens_of(s.seqs) + p.t0) * s.G + at.g) * 2 * NP;
  const int slot = lane_slot<4, NL>(at.nl);
  constexpr int BC = CW >= 8 ? 1 : 8 / CW;  // values of dB and dC that a lane is left with
  const int bcs = lane_slot<8, CW>(at.cl), bcat = bcs / 4 * NP + n0 + bcs % 4;
  const bool bcw = at.cl < 8;

  Cols<T, CW> xr, tr, gr;
  Mat<T, NP> br, cr;
  auto fetch = [&](int t0) {
    const int64_t t = t0 + at.lane;
    const bool in = t < p.len;
    xr.fetch(x + t * s.ld_x, in, s.vec, at.n);
    tr.fetch(dt + t * s.ld_dt, in, s.vec, at.n);
    gr.fetch(dy + t * s.D, in, s.vec, at.n);
    br.fetch(Bm + t0 * s.ld_b, s.ld_b, s.N, p.len - t0);
    cr.fetch(Cm + t0 * s.ld_c, s.ld_c, s.N, p.len - t0);
  };
  int t0 = p.len > 0 ? (p.len - 1) / kTile * kTile : -1;
  if (t0 >= 0) fetch(t0);
  for (; t0 >= 0; t0 -= kTile) {
    const bool in = t0 + at.lane < p.len;
#pragma unroll
    for (int i = 0; i < CW; ++i) {
      float d = 0.f, sl = 0.f;
      if (in && i < at.n) {
        const float v = tr.get(i) + bias[i];
        d = softplus_acc(v);
        sl = v > 20.f ? 1.f : rcp(1.f + exp_acc(-v));
      }
      m.d[at.warp][i][at.lane] = d;
      m.slope[at.warp][i][at.lane] = sl;
      m.x[at.warp][i][at.lane] = xr.get(i);
      m.g[at.warp][i][at.lane] = gr.get(i);
    }
    br.stage(m.b);
    cr.stage(m.c);
    __syncthreads();
    if (t0 > 0) fetch(t0 - kTile);
    const int subs = p.len - t0 > kCkpt ? 2 : 1;
    for (int sub = subs - 1; sub >= 0; --sub) {
      float h0[4] = {0.f, 0.f, 0.f, 0.f}, h[kCkpt][4], a[kCkpt][4];
      if (at.live) {
        const float4 v = *reinterpret_cast<const float4*>(ck + (int64_t)(t0 / kCkpt + sub) * s.D * NP);
        h0[0] = v.x, h0[1] = v.y, h0[2] = v.z, h0[3] = v.w;
      }
      const int ts = sub * kCkpt;
#pragma unroll
      for (int q = 0; q < kCkpt / 4; ++q) {
        const float4 dv = *reinterpret_cast<const float4*>(&m.d[at.warp][at.cl][ts + 4 * q]);
        const float4 xv = *reinterpret_cast<const float4*>(&m.x[at.warp][at.cl][ts + 4 * q]);
        const float d4[4] = {dv.x, dv.y, dv.z, dv.w}, x4[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int t = 4 * q + k;
          const float4 bv = *reinterpret_cast<const float4*>(&m.b[(ts + t) * NP + n0]);
          const float b4[4] = {bv.x, bv.y, bv.z, bv.w};
          const float u = d4[k] * x4[k];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            a[t][j] = ex2(d4[k] * A2[j]);
            h[t][j] = fmaf(a[t][j], t > 0 ? h[t > 0 ? t - 1 : 0][j] : h0[j], u * b4[j]);
          }
        }
      }
#pragma unroll
      for (int q = kCkpt / 4 - 1; q >= 0; --q) {
        const float4 dv = *reinterpret_cast<const float4*>(&m.d[at.warp][at.cl][ts + 4 * q]);
        const float4 xv = *reinterpret_cast<const float4*>(&m.x[at.warp][at.cl][ts + 4 * q]);
        const float4 gv = *reinterpret_cast<const float4*>(&m.g[at.warp][at.cl][ts + 4 * q]);
        const float d4[4] = {dv.x, dv.y, dv.z, dv.w}, x4[4] = {xv.x, xv.y, xv.z, xv.w}, g4[4] = {gv.x, gv.y, gv.z, gv.w};
        float du[4], sq[4];
#pragma unroll
        for (int k = 3; k >= 0; --k) {
          const int t = 4 * q + k;
          const float4 bv = *reinterpret_cast<const float4*>(&m.b[(ts + t) * NP + n0]);
          const float4 cv = *reinterpret_cast<const float4*>(&m.c[(ts + t) * NP + n0]);
          const float b4[4] = {bv.x, bv.y, bv.z, bv.w}, c4[4] = {cv.x, cv.y, cv.z, cv.w};
          const float u = d4[k] * x4[k];
          float bc[8];
          du[k] = sq[k] = 0.f;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float g = fmaf(c4[j], g4[k], ga[j]);
            bc[j] = g * u;
            bc[4 + j] = g4[k] * h[t][j];
            du[k] = fmaf(g, b4[j], du[k]);
            ga[j] = a[t][j] * g;
            const float qv = ga[j] * (t > 0 ? h[t > 0 ? t - 1 : 0][j] : h0[j]);
            sq[k] = fmaf(A2[j], qv, sq[k]);
            dA[j] = fmaf(d4[k], qv, dA[j]);
          }
          lane_sums<8, CW, NL>(bc, at.lane);
          if (bcw) {
#pragma unroll
            for (int i = 0; i < BC; ++i) m.red[at.warp][ts + t][bcat + i] = bc[i];
          }
        }
        lane_sums<4, NL, 1>(du, at.lane);
        lane_sums<4, NL, 1>(sq, at.lane);
        __syncwarp();
        if (at.nl < 4) {  // the gradients take their inputs' places
          constexpr int M = NL < 4 ? 4 / NL : 1;
#pragma unroll
          for (int k = 0; k < M; ++k) {
            const int t = ts + 4 * q + slot + k;
            float &d = m.d[at.warp][at.cl][t], &xx = m.x[at.warp][at.cl][t];
            const float dyv = m.g[at.warp][at.cl][t];
            const float dd = fmaf(xx, du[k], kLn2 * sq[k]) * m.slope[at.warp][at.cl][t];
            const float dxv = fmaf(d, du[k], skip * dyv);
            dskip = fmaf(dyv, xx, dskip);
            dbias += dd;
            d = dd;
            xx = dxv;
          }
        }
      }
    }
    __syncthreads();
    {
      Cols<T, CW> ox, od;
#pragma unroll
      for (int i = 0; i < CW; ++i) {
        ox.put(i, m.x[at.warp][i][at.lane]);
        od.put(i, m.d[at.warp][i][at.lane]);
      }
      ox.store(dx + (int64_t)(t0 + at.lane) * s.D, in, s.vec, at.n);
      od.store(ddt + (int64_t)(t0 + at.lane) * s.D, in, s.vec, at.n);
    }
    const int n = min(kTile, p.len - t0) * 2 * NP;
    for (int e = threadIdx.x; e < n; e += kWarps * 32) {
      const int t = e / (2 * NP), v = e % (2 * NP);
      float r = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) r += m.red[w][t][v];
      pbc[(int64_t)(t0 + t) * s.G * 2 * NP + v] = r;
    }
    __syncwarp();
  }
#pragma unroll
  for (int o = 1; o < NL; o <<= 1) {
    dskip += __shfl_xor_sync(0xffffffffu, dskip, o);
    dbias += __shfl_xor_sync(0xffffffffu, dbias, o);
  }
  if (!at.live) return;
  for (int j = 0; j < 4; ++j)
    if (n0 + j < s.N) par[n0 + j] = dA[j];
  if (at.nl == 0) {
    par[s.N] = dskip;
    par[s.N + 1] = dbias;
  }
  if (s.dinit && p.idx == 0) store_states(s.dinit + ((int64_t)p.seq * s.D + at.ch) * s.N, s.N, n0, ga);
}

// dB and dC of a token and group: the channel tiles in order.
template <typename T>
__global__ void __launch_bounds__(256) k_ssm_bc_sums(Ssm s, int NP, int64_t tiles) {
  if (bad_call(s.seqs)) return;
  const int64_t rows = tokens_of(s.seqs) * s.G, all = rows * 2 * NP;
  for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < all; e += (int64_t)gridDim.x * 256) {
    float a = 0.f;
    for (int64_t k = 0; k < tiles; ++k) a += s.part_bc[k * all + e];
    const int64_t r = e / (2 * NP);
    const int v = (int)(e - r * 2 * NP), n = v % NP;
    if (n < s.N) static_cast<T*>(v < NP ? s.dB : s.dC)[r * s.N + n] = down<T>(a);
  }
}

// The parameters' gradients: 32 columns of [D][N + 2] by 32 strands of units, the strands in a fixed tree.
__global__ void __launch_bounds__(1024) k_ssm_par_sums(Ssm s, int64_t units) {
  __shared__ float red[32][33];
  if (bad_call(s.seqs)) return;
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int64_t width = s.D * (s.N + 2), c = (int64_t)blockIdx.x * 32 + tx;
  float a = 0.f;
  if (c < width)
    for (int64_t u = ty; u < units; u += 32) a += s.part_par[u * width + c];
  red[ty][tx] = a;
  __syncthreads();
  float v = red[tx][ty];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int64_t cc = (int64_t)blockIdx.x * 32 + ty;
  if (tx != 0 || cc >= width) return;
  const int64_t ch = cc / (s.N + 2);
  const int n = (int)(cc - ch * (s.N + 2));
  if (n < s.N) {
    if (s.dA_log) s.dA_log[ch * s.N + n] = -expf(s.A_log[ch * s.N + n]) * v;
  } else if (n == s.N) {
    if (s.dskip) s.dskip[ch] = v;
  } else if (s.ddt_bias) {
    s.ddt_bias[ch] = v;
  }
}

template <typename T, int NP>
cudaError_t backward(const Ssm& c, cudaStream_t s) {
  using S = Shape<NP>;
  const int64_t Dg = c.D / c.G, tiles = (Dg + S::CC - 1) / S::CC, units = max_units(c.seqs, c.lg);
  const dim3 grid((unsigned)units, (unsigned)(c.G * tiles));
  if (c.cut) {
    {
      ProfScope ps("ssm_bwd_ends", s);
      k_ssm_bwd_ends<T, NP><<<grid, kWarps * 32, 0, s>>>(c);
    }
    ProfScope ps("ssm_bwd_join", s);
    k_ssm_bwd_join<NP><<<(unsigned)((c.D * NP + 255) / 256 * c.seqs.n), 256, 0, s>>>(c);
  }
  cudaError_t e = cudaFuncSetAttribute(k_ssm_bwd<T, NP>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(BwdShared<NP>));
  if (e != cudaSuccess) return e;
  {
    ProfScope ps("ssm_bwd", s);
    k_ssm_bwd<T, NP><<<grid, kWarps * 32, sizeof(BwdShared<NP>), s>>>(c);
  }
  const int64_t all = (c.seqs.cu ? c.seqs.T : c.seqs.T * c.seqs.n) * c.G * 2 * NP;
  if (all > 0) {
    ProfScope ps("ssm_bwd_bc", s);
    k_ssm_bc_sums<T><<<(unsigned)std::min<int64_t>((all + 255) / 256, 148 * 32), 256, 0, s>>>(c, NP, tiles);
  }
  ProfScope ps("ssm_bwd_par", s);
  k_ssm_par_sums<<<(unsigned)((c.D * (c.N + 2) + 31) / 32), 1024, 0, s>>>(c, units);
  return cudaGetLastError();
}

template <typename T>
cudaError_t by_states(const Ssm& c, cudaStream_t s) {
  switch (ssm_padded(c.N)) {
    case 8: return backward<T, 8>(c, s);
    case 16: return backward<T, 16>(c, s);
    case 32: return backward<T, 32>(c, s);
    default: return backward<T, 64>(c, s);
  }
}

}  // namespace

cudaError_t ssm_backward(const Ssm& c, cudaStream_t s) {
  if (c.dtype == GDN_DTYPE_FP32) return by_states<float>(c, s);
  if (c.dtype == GDN_DTYPE_BF16) return by_states<__nv_bfloat16>(c, s);
  return by_states<__half>(c, s);
}

}  // namespace mix
}  // namespace gdn
