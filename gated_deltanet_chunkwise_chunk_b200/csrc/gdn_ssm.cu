// Selective state space scan: forward over sequences, and the step of one token.  The mathematics and
// the layout of the work are in ssm_common.cuh.
#include <algorithm>

#include "ssm_common.cuh"

namespace gdn {
namespace mix {
namespace {

// One segment.  END: only the state at its end from a zero state, and the sum of its deltas (the first
// pass over segments that have one before or behind them).
template <typename T, int NP, bool END>
__global__ void __launch_bounds__(kWarps * 32) k_ssm_fwd(Ssm s) {
  using S = Shape<NP>;
  constexpr int NL = S::NL, CW = S::CW;
  __shared__ __align__(16) float sd[kWarps][CW][kRow], sx[kWarps][CW][kRow];
  __shared__ __align__(16) float sb[2][kTile * NP], sc[END ? 1 : 2][END ? 4 : kTile * NP];
  if (bad_call(s.seqs)) return;
  Place<NP> at;
  if (!at.find(s, s.lg)) return;
  const Piece& p = at.p;
  if (END && p.pos + p.len == p.slen) return;  // nothing follows
  const int n0 = at.nl * 4;
  float A2[4], h[4] = {0.f, 0.f, 0.f, 0.f};
  load_decay(s, at.ch, at.live, n0, A2);
  if (!END && at.live) {
    if (s.cut && p.idx > 0) {
      const float4 v = *reinterpret_cast<const float4*>(s.starts + state_at<NP>(s, blockIdx.x, at.ch, n0));
      h[0] = v.x, h[1] = v.y, h[2] = v.z, h[3] = v.w;
    } else if (s.init) {
      load_states(s.init + ((int64_t)p.seq * s.D + at.ch) * s.N, s.N, n0, h);
    }
  }
  const float skip = !END && at.live && at.nl == 0 && s.skip ? s.skip[at.ch] : 0.f;
  float bias[CW];
#pragma unroll
  for (int i = 0; i < CW; ++i) bias[i] = i < at.n && s.dt_bias ? s.dt_bias[at.c0 + i] : 0.f;
  const T* x = static_cast<const T*>(s.x) + p.t0 * s.ld_x + at.c0;
  const T* dt = static_cast<const T*>(s.dt) + p.t0 * s.ld_dt + at.c0;
  const T* Bm = static_cast<const T*>(s.Bm) + p.t0 * s.ld_b + (int64_t)at.g * s.N;
  const T* Cm = static_cast<const T*>(s.Cm) + p.t0 * s.ld_c + (int64_t)at.g * s.N;
  T* y = static_cast<T*>(s.y) + p.t0 * s.D + at.c0;
  float* ck = nullptr;
  if (!END && s.ckpt && at.live)
    ck = s.ckpt + state_at<NP>(s, first_unit(s.seqs, p.seq, kCkptLog) + p.pos / kCkpt, at.ch, n0);
  const int slot = lane_slot<4, NL>(at.nl);
  float total = 0.f;  // END: the lane's token's deltas are summed per channel below
  float dsum[CW];
#pragma unroll
  for (int i = 0; i < CW; ++i) dsum[i] = 0.f;

  Cols<T, CW> xr, tr;
  Mat<T, NP> br, cr;
  auto fetch = [&](int t0) {
    const bool in = t0 + at.lane < p.len;
    const int64_t t = t0 + at.lane;
    xr.fetch(x + t * s.ld_x, in, s.vec, at.n);
    tr.fetch(dt + t * s.ld_dt, in, s.vec, at.n);
    br.fetch(Bm + t0 * s.ld_b, s.ld_b, s.N, p.len - t0);
    if (!END) cr.fetch(Cm + t0 * s.ld_c, s.ld_c, s.N, p.len - t0);
  };
  if (p.len > 0) fetch(0);
  int buf = 0;
  for (int t0 = 0; t0 < p.len; t0 += kTile, buf ^= 1) {
    const bool in = t0 + at.lane < p.len;
#pragma unroll
    for (int i = 0; i < CW; ++i) {
      const float d = in && i < at.n ? softplus_acc(tr.get(i) + bias[i]) : 0.f;
      sd[at.warp][i][at.lane] = d;
      sx[at.warp][i][at.lane] = xr.get(i);
      if (END) dsum[i] += d;
    }
    br.stage(sb[buf]);
    if (!END) cr.stage(sc[buf]);
    __syncthreads();
    if (t0 + kTile < p.len) fetch(t0 + kTile);
    const int quads = (min(kTile, p.len - t0) + 3) / 4;
#pragma unroll 2
    for (int q = 0; q < quads; ++q) {
      if (ck && q % (kCkpt / 4) == 0) {
        *reinterpret_cast<float4*>(ck) = make_float4(h[0], h[1], h[2], h[3]);
        ck += s.D * NP;
      }
      const float4 dv = *reinterpret_cast<const float4*>(&sd[at.warp][at.cl][4 * q]);
      const float4 xv = *reinterpret_cast<const float4*>(&sx[at.warp][at.cl][4 * q]);
      const float d4[4] = {dv.x, dv.y, dv.z, dv.w}, x4[4] = {xv.x, xv.y, xv.z, xv.w};
      float yv[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float4 bv = *reinterpret_cast<const float4*>(&sb[buf][(4 * q + k) * NP + n0]);
        const float b4[4] = {bv.x, bv.y, bv.z, bv.w};
        const float u = d4[k] * x4[k];
#pragma unroll
        for (int j = 0; j < 4; ++j) h[j] = fmaf(ex2(d4[k] * A2[j]), h[j], u * b4[j]);
        if (!END) {
          const float4 cv = *reinterpret_cast<const float4*>(&sc[buf][(4 * q + k) * NP + n0]);
          const float c4[4] = {cv.x, cv.y, cv.z, cv.w};
          float a = skip * x4[k];
#pragma unroll
          for (int j = 0; j < 4; ++j) a = fmaf(h[j], c4[j], a);
          yv[k] = a;
        }
      }
      if (!END) {
        lane_sums<4, NL, 1>(yv, at.lane);
        __syncwarp();
        if (at.nl < 4) {  // the outputs take their inputs' place
          constexpr int M = NL < 4 ? 4 / NL : 1;
#pragma unroll
          for (int k = 0; k < M; ++k) sx[at.warp][at.cl][4 * q + slot + k] = yv[k];
        }
      }
    }
    __syncwarp();
    if (!END) {
      Cols<T, CW> o;
#pragma unroll
      for (int i = 0; i < CW; ++i) o.put(i, sx[at.warp][i][at.lane]);
      o.store(y + (int64_t)(t0 + at.lane) * s.D, in, s.vec, at.n);
      __syncwarp();
    }
  }
  if (END) {
#pragma unroll
    for (int i = 0; i < CW; ++i) {
      float v = dsum[i];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (i == at.cl) total = v;
    }
    if (at.live) {
      *reinterpret_cast<float4*>(s.starts + state_at<NP>(s, blockIdx.x, at.ch, n0)) = make_float4(h[0], h[1], h[2], h[3]);
      if (at.nl == 0) s.sums[(int64_t)blockIdx.x * s.D + at.ch] = total;
    }
  } else if (s.final && at.live && p.pos + p.len == p.slen) {
    store_states(s.final + ((int64_t)p.seq * s.D + at.ch) * s.N, s.N, n0, h);
  }
}

// The segments of a sequence in order: what the first pass left at a segment's unit (its end's state
// from zero) becomes the state that enters the segment.
template <int NP>
__global__ void __launch_bounds__(256) k_ssm_join(Ssm s) {
  if (bad_call(s.seqs)) return;
  const unsigned blocks = (unsigned)((s.D * NP + 255) / 256);  // of a sequence
  const int seq = (int)(blockIdx.x / blocks);
  const int64_t at = (int64_t)(blockIdx.x - seq * blocks) * 256 + threadIdx.x, ch = at / NP;
  const int n = (int)(at % NP);
  if (ch >= s.D || n >= s.N) return;
  const int64_t len = s.seqs.cu ? s.seqs.cu[seq + 1] - s.seqs.cu[seq] : s.seqs.T;
  const int64_t segs = len == 0 ? 1 : ((len - 1) >> s.lg) + 1, u0 = first_unit(s.seqs, seq, s.lg);
  const float A2 = decay_rate(s.A_log[ch * s.N + n]);
  float h = s.init ? s.init[((int64_t)seq * s.D + ch) * s.N + n] : 0.f;
  for (int64_t k = 0; k < segs; ++k) {
    float* p = s.starts + state_at<NP>(s, u0 + k, ch, n);
    const float end = *p;
    *p = h;
    if (k + 1 < segs) h = fmaf(ex2(A2 * s.sums[(u0 + k) * s.D + ch]), h, end);
  }
}

// One token for each sequence: a thread has four states of a channel, so a state moves as 16 bytes.
// init and final may be one buffer: a thread reads its states before it writes them.
template <typename T, int NP>
__global__ void __launch_bounds__(256) k_ssm_step(Ssm s) {
  constexpr int NL = NP / 4;
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t row = at / NL;
  const int nl = (int)(at % NL), n0 = nl * 4;
  const int64_t n = row / s.D, ch = row - n * s.D;
  const bool live = n < s.seqs.n;
  float a = 0.f;
  if (live) {
    const int64_t g = ch / (s.D / s.G);
    const float* st = s.init + row * s.N;
    float* nx = s.final + row * s.N;
    const T* Bm = static_cast<const T*>(s.Bm) + n * s.ld_b + g * s.N;
    const T* Cm = static_cast<const T*>(s.Cm) + n * s.ld_c + g * s.N;
    float h[4], A2[4];
    if (s.vec) {
      const float4 v = *reinterpret_cast<const float4*>(st + n0);
      h[0] = v.x, h[1] = v.y, h[2] = v.z, h[3] = v.w;
    } else {
      load_states(st, s.N, n0, h);
    }
    load_decay(s, ch, true, n0, A2);
    const float x = up<T>(static_cast<const T*>(s.x)[n * s.ld_x + ch]);
    const float d = softplus_acc(up<T>(static_cast<const T*>(s.dt)[n * s.ld_dt + ch]) + (s.dt_bias ? s.dt_bias[ch] : 0.f));
    const float u = d * x;
    a = nl == 0 && s.skip ? s.skip[ch] * x : 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool in = n0 + j < s.N;
      h[j] = fmaf(ex2(d * A2[j]), h[j], in ? u * up<T>(Bm[n0 + j]) : 0.f);
      a = fmaf(h[j], in ? up<T>(Cm[n0 + j]) : 0.f, a);
    }
    if (s.vec)
      *reinterpret_cast<float4*>(nx + n0) = make_float4(h[0], h[1], h[2], h[3]);
    else
      store_states(nx, s.N, n0, h);
  }
#pragma unroll
  for (int o = NL / 2; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
  if (live && nl == 0) static_cast<T*>(s.y)[row] = down<T>(a);
}

template <typename T, int NP>
cudaError_t forward(const Ssm& c, cudaStream_t s) {
  using S = Shape<NP>;
  const int64_t Dg = c.D / c.G;
  const dim3 grid((unsigned)max_units(c.seqs, c.lg), (unsigned)(c.G * ((Dg + S::CC - 1) / S::CC)));
  if (c.cut) {
    {
      ProfScope ps("ssm_fwd_ends", s);
      k_ssm_fwd<T, NP, true><<<grid, kWarps * 32, 0, s>>>(c);
    }
    ProfScope ps("ssm_join", s);
    k_ssm_join<NP><<<(unsigned)((c.D * NP + 255) / 256 * c.seqs.n), 256, 0, s>>>(c);
  }
  ProfScope ps("ssm_fwd", s);
  k_ssm_fwd<T, NP, false><<<grid, kWarps * 32, 0, s>>>(c);
  return cudaGetLastError();
}

template <typename T, int NP>
cudaError_t step(const Ssm& c, cudaStream_t s) {
  const int64_t n = c.seqs.n * c.D * (NP / 4);
  ProfScope ps("ssm_step", s);
  k_ssm_step<T, NP><<<(unsigned)((n + 255) / 256), 256, 0, s>>>(c);
  return cudaGetLastError();
}

template <typename T>
cudaError_t by_states(const Ssm& c, bool one, cudaStream_t s) {
  if (c.N <= 8) return one ? step<T, 8>(c, s) : forward<T, 8>(c, s);
  if (c.N <= 16) return one ? step<T, 16>(c, s) : forward<T, 16>(c, s);
  if (c.N <= 32) return one ? step<T, 32>(c, s) : forward<T, 32>(c, s);
  return one ? step<T, 64>(c, s) : forward<T, 64>(c, s);
}

cudaError_t dispatch(const Ssm& c, bool one, cudaStream_t s) {
  if (c.dtype == GDN_DTYPE_FP32) return by_states<float>(c, one, s);
  if (c.dtype == GDN_DTYPE_BF16) return by_states<__nv_bfloat16>(c, one, s);
  return by_states<__half>(c, one, s);
}

}  // namespace

int ssm_padded(int N) { return N <= 8 ? 8 : N <= 16 ? 16 : N <= 32 ? 32 : 64; }

SsmSizes ssm_sizes(const Seqs& s, int64_t tokens, int64_t D, int N, int G) {
  SsmSizes z{};
  const int NP = ssm_padded(N), CC = 32 / (NP / 4) * kWarps;
  const int64_t Dg = D / G, tiles = (Dg + CC - 1) / CC;
  z.lg = 30;
  z.cut = false;
  const int64_t units = max_units(s, z.lg);
  if (z.cut) {
    z.starts = units * D * NP;
    z.sums = units * D;
  }
  z.ckpt = max_units(s, kCkptLog) * D * NP;
  z.part_bc = tiles * tokens * G * 2 * NP;
  z.part_par = units * D * (N + 2);
  return z;
}

cudaError_t ssm_forward(const Ssm& c, cudaStream_t s) { return dispatch(c, false, s); }
cudaError_t ssm_step(const Ssm& c, cudaStream_t s) { return dispatch(c, true, s); }

}  // namespace mix
}  // namespace gdn
