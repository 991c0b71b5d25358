// Selective state space scan: backward.  With g[t] the gradient of the state behind token t and a the decays,
//   g[t] = C[t] dy[t] + a[t+1] g[t+1]  (+ the final state's gradient at the end),   q[t] = a[t] g[t] h[t-1],
//   dx = delta sum_n g B + Dskip dy,   ddelta = x sum_n g B + sum_n A q,   ddt = ddelta softplus',
//   dB = sum_d g delta x,  dC = sum_d dy h  (over the group's channels),
//   dA_log = A sum_t delta q,  dDskip = sum_t dy x,  ddt_bias = sum_t ddt.
// The states come from the forward's every-16th-token copies: a warp goes through 16 tokens forwards with
// their states and decays left in registers (4 states to a lane, so 128 of them), then back, so each
// exponential is computed once, as a polynomial whatever the tensors' type: dA_log and the initial state's gradient
// are fp32, and the hardware exponential's bias showed in them (a tenth less time).  Only the first pass over segments takes the forward's decays.  The working warps take the registers that the feeding warps give up.
// dB and dC are sums over a warp's channels for each token and state: the lanes of neighbouring channels hold
// their four states in different orders (xor by the channel's low bits), so that what a lane keeps of a sum
// and what it hands over are always the same registers and a butterfly step is a shuffle and an addition.
// The feeding warps add the block's warps in shared memory, and the blocks of a group's channels leave
// partial rows that a second kernel adds in order.  Nothing is atomic.
// Measured at 2 x 4096 x 2048 x 16 bf16, in four segments a sequence: 425 us, 80 for the first pass over them, 19 for the
// join, 14 and 6 for the sums, 544 in all.  No unit is saturated (shared memory 59%, issue 56% of their peaks): its eight
// working warps a multiprocessor wait for the feeding warps and for their own latencies; about 110 instructions for a
// token and scheduler, a third of them the sums over a warp's channels.  With 192 and 184 registers instead of 200 for
// the working warps it is 2% and 10% slower.  A block leaves 2 NP floats of dB and dC for each token and its 512 / NP
// channels, 4 bytes a token and channel at N = 16 and 64 at N = 64: 2 x 2048 x 2048 x 64 takes 1235 us, 85 of them the
// kernel that adds these rows (DRAM 77%), and a workspace of 0.5 GB for them.
#include <algorithm>
#include <type_traits>

#include "ssm_common.cuh"

namespace gdn {
namespace mix {
namespace {

__device__ __forceinline__ int64_t tokens_of(const Seqs& s) { return s.cu ? s.T : s.T * s.n; }

constexpr int kBwd = 4;  // states of a lane

template <typename T, int NP, bool END>
struct BwdShared {
  static constexpr int X = 512 / NP * kRow, S = NP * kRow;
  float d[2][X], g[2][X], c[2][S];            // delta (then ddt), dy, C
  float x[2][END ? 4 : X], b[2][END ? 4 : S]; // x (then dx), B
  float slope[2][END ? 4 : X];                // softplus', -1 past the segment's end (where a decay is 1 and A q may overflow)
  float red[2][END ? 1 : Shape<NP, kBwd>::WORK / 32][END ? 1 : kTile][END ? 4 : 2 * NP];  // a warp's dB and dC
  // targets of 16-byte copies
  alignas(16) RawRows<T, NP> rt;
  alignas(16) RawRows<T, NP> rg;
  alignas(16) typename std::conditional<END, float, RawRows<T, NP>>::type rx;
  alignas(16) T rc[kRing<T, NP>][kTile * NP];
  alignas(16) T rb[kRing<T, NP>][END ? 8 : kTile * NP];
};

// One segment, from its end.  END: only the gradient that leaves it at its front when none enters at its end,
// and the sum of its deltas (the first pass over segments that have one before them).
template <typename T, int NP, bool END>
__global__ void __launch_bounds__(Shape<NP, kBwd>::NT, 2) k_ssm_bwd(Ssm s) {
  using S = Shape<NP, kBwd>;
  constexpr int SPL = kBwd, NL = S::NL, CW = S::CW, FC = S::FC, WW = S::WORK / 32, PITCH = RawRows<T, NP>::PITCH, R = kRing<T, NP>;
  extern __shared__ __align__(16) char raw[];
  BwdShared<T, NP, END>& m = *reinterpret_cast<BwdShared<T, NP, END>*>(raw);
  if (bad_call(s.seqs)) return;
  Place<NP, SPL> at;
  if (!at.find(s, s.lg)) return;
  const Piece& p = at.p;
  if (END && p.idx == 0) return;  // nothing precedes
  const int tiles = (p.len + kTile - 1) / kTile;

  if (at.feeds) {
    if (!END) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    const Inputs<T, NP, SPL> in(s, at);
    float bias[FC];
#pragma unroll
    for (int i = 0; i < FC; ++i) bias[i] = at.sc + i < at.width && s.dt_bias ? s.dt_bias[at.c0 + at.sc + i] : 0.f;
    const int64_t row = (p.t0 + at.tok) * s.D + at.c0 + at.sc;
    T *dx = static_cast<T*>(s.dx) + row, *ddt = static_cast<T*>(s.ddt) + row;
    float* pbc = s.part_bc + ((at.tile * tokens_of(s.seqs) + p.t0) * s.G + at.g) * 2 * NP;
    auto fetch = [&](int i, int r) {
      if (i < tiles) {
        const int t0 = (tiles - 1 - i) * kTile, n = p.len - t0;
        in.dt.template fetch<END>(m.rt.v[r], at.f, t0, n);
        in.dy.template fetch<END>(m.rg.v[r], at.f, t0, n);
        in.C.template fetch<END>(m.rc[r], at.f, t0, n);
        if constexpr (!END) {
          in.x.template fetch<END>(m.rx.v[r], at.f, t0, n);
          in.B.template fetch<END>(m.rb[r], at.f, t0, n);
        }
      }
      copy_commit();
    };
    auto widen = [&](int i, int r, int buf) {
      const bool here = (tiles - 1 - i) * kTile + at.tok < p.len;
      Cols<T, FC> xr, tr, gr;
      tr.load(m.rt.v[r] + at.tok * PITCH + at.sc);
      gr.load(m.rg.v[r] + at.tok * PITCH + at.sc);
      if constexpr (!END) xr.load(m.rx.v[r] + at.tok * PITCH + at.sc);
      const int to = at.sc * kRow + at.tok;
#pragma unroll
      for (int k = 0; k < FC; k += 2) {
        float2 e;
        const float2 v = {tr.get(k) + bias[k], tr.get(k + 1) + bias[k + 1]}, d = softplus2(v, e);
        m.d[buf][to + k * kRow] = here ? d.x : 0.f;
        m.d[buf][to + (k + 1) * kRow] = here ? d.y : 0.f;
        m.g[buf][to + k * kRow] = gr.get(k);
        m.g[buf][to + (k + 1) * kRow] = gr.get(k + 1);
        if constexpr (!END) {
          m.x[buf][to + k * kRow] = xr.get(k);
          m.x[buf][to + (k + 1) * kRow] = xr.get(k + 1);
          m.slope[buf][to + k * kRow] = here ? softplus_slope(v.x, e.x) : -1.f;
          m.slope[buf][to + (k + 1) * kRow] = here ? softplus_slope(v.y, e.y) : -1.f;
        }
      }
      widen_states<T, NP, SPL>(m.c[buf], m.rc[r], at.f);
      if constexpr (!END) widen_states<T, NP, SPL>(m.b[buf], m.rb[r], at.f);
    };
    // the gradients out of their inputs' places, and the sums over the block's channels
    auto put = [&](int i, int buf) {
      if constexpr (!END) {
        const int t0 = (tiles - 1 - i) * kTile, from = at.sc * kRow + at.tok;
        Cols<T, FC> ox, od;
        const bool here = t0 + at.tok < p.len;
#pragma unroll
        for (int k = 0; k < FC; k += 2) {
          ox.put2(k, {m.x[buf][from + k * kRow], m.x[buf][from + (k + 1) * kRow]});
          od.put2(k, {m.d[buf][from + k * kRow], m.d[buf][from + (k + 1) * kRow]});
        }
        if (here) {
          ox.store(dx + (int64_t)t0 * s.D, s.vec, at.width - at.sc);
          od.store(ddt + (int64_t)t0 * s.D, s.vec, at.width - at.sc);
        }
        const int n = min(kTile, p.len - t0) * (NP / 2);
        for (int e = at.f; e < n; e += kFeed) {
          const int t = e / (NP / 2), v = e % (NP / 2) * 4;
          float4 a = ld4(&m.red[buf][0][t][v]);
#pragma unroll
          for (int w = 1; w < WW; ++w) {
            const float4 o = ld4(&m.red[buf][w][t][v]);
            a.x += o.x, a.y += o.y, a.z += o.z, a.w += o.w;
          }
          *reinterpret_cast<float4*>(pbc + (int64_t)(t0 + t) * s.G * 2 * NP + v) = a;
        }
      }
    };
    // The feeding warps meet on a barrier of their own before they widen what all of them fetched.
    auto meet = [] { asm volatile("bar.sync 1, 128;" ::: "memory"); };
    for (int k = 0; k < R; ++k) fetch(k, k);
    int r = 0;
    for (int i = 0; i < tiles; ++i) {  // tile i (from the end) is widened while the one before it is worked on
      copy_wait<R - 1>();
      meet();
      if (i > 1) put(i - 2, i & 1);
      widen(i, r, i & 1);
      meet();
      fetch(i + R, r);
      r = r == R - 1 ? 0 : r + 1;
      __syncthreads();
    }
    copy_wait<0>();
    __syncthreads();
    if (tiles > 1) put(tiles - 2, tiles & 1);
    if (tiles > 0) put(tiles - 1, (tiles - 1) & 1);
    return;
  }

  if (!END) asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
  // register j of a lane belongs to state n0 + (j ^ pm)
  const int pm = CW >= 4 ? at.cl & 3 : at.cl & 1;
  float A2[SPL], ga[SPL];
  float2 dA[SPL];
  int row[SPL];
#pragma unroll
  for (int j = 0; j < SPL; ++j) {
    const int n = at.n0 + (j ^ pm);
    A2[j] = at.live && n < s.N ? decay_rate(s.A_log[at.ch * s.N + n]) : 0.f;
    ga[j] = 0.f;
    dA[j] = {0.f, 0.f};
    row[j] = state_row<NP, SPL>(n);
    if (!END && at.live && n < s.N) {  // nothing wrote the others
      if (s.cut && p.pos + p.len < p.slen)
        ga[j] = s.starts[state_at<NP>(s, blockIdx.x, at.ch, n)];
      else if (s.dfinal)
        ga[j] = s.dfinal[((int64_t)p.seq * s.D + at.ch) * s.N + n];
    }
  }
  const float skip = at.live && s.skip ? s.skip[at.ch] : 0.f;
  const float* ck = END ? nullptr : s.ckpt + state_at<NP>(s, first_unit(s.seqs, p.seq, kCkptLog) + p.pos / kCkpt, at.ch, at.n0);
  const int slot = lane_slot<4, NL>(at.nl);
  float total = 0.f, dskip = 0.f, dbias = 0.f;
  // The parameters' sums leave as a row for every 256 tokens (a segment of fewer), so that no running sum is longer.
  const int lgp = min(s.lg, kParLog);
  auto leave = [&](int64_t row, bool zero) {
    float* par = s.part_par + (row * s.D + at.ch) * (s.N + 2);
#pragma unroll
    for (int j = 0; j < SPL; ++j) {
      const int n = at.n0 + (j ^ pm);
      if (n < s.N) par[n] = zero ? 0.f : dA[j].x + dA[j].y;
    }
    if (at.nl == 0) {
      par[s.N] = zero ? 0.f : dskip;
      par[s.N + 1] = zero ? 0.f : dbias;
    }
  };
  // the state that enters the 16 tokens to come, asked for 16 tokens early
  int chunk = (p.len - 1) / kCkpt;
  float ahead[SPL];
  auto enter = [&](int k) {
#pragma unroll
    for (int j = 0; j < SPL; ++j) ahead[j] = at.live ? ck[(int64_t)max(k, 0) * s.D * NP + (j ^ pm)] : 0.f;
  };
  if constexpr (!END) enter(chunk);
  for (int i = 0; i < tiles; ++i) {
    const int buf = i & 1, t0 = (tiles - 1 - i) * kTile;
    __syncthreads();  // the tile is there
    float tsum = 0.f;
#pragma unroll 1
    for (int sub = p.len - t0 > kCkpt ? 1 : 0; sub >= 0; --sub) {
      float* d = m.d[buf] + at.c * kRow + sub * kCkpt;
      const float* g = m.g[buf] + at.c * kRow + sub * kCkpt;
      const float* c = m.c[buf] + sub * kCkpt;
      if constexpr (END) {
        float dq[kCkpt / 4];
#pragma unroll
        for (int q = kCkpt / 4 - 1; q >= 0; --q) {
          const float4 dv = ld4(d + 4 * q), gv = ld4(g + 4 * q);
          dq[q] = (dv.x + dv.y) + (dv.z + dv.w);
          const float2 d2[2] = {{dv.x, dv.y}, {dv.z, dv.w}}, g2[2] = {{gv.x, gv.y}, {gv.z, gv.w}};
#pragma unroll
          for (int j = 0; j < SPL; ++j) {
            const float4 cv = ld4(c + row[j] + 4 * q);
            const float2 c2[2] = {{cv.x, cv.y}, {cv.z, cv.w}};
#pragma unroll
            for (int k = 1; k >= 0; --k) {
              const float2 e = decays<T>(d2[k], {A2[j], A2[j]});
              ga[j] = e.y * fmaf(c2[k].y, g2[k].y, ga[j]);
              ga[j] = e.x * fmaf(c2[k].x, g2[k].x, ga[j]);
            }
          }
        }
        tsum += (dq[0] + dq[1]) + (dq[2] + dq[3]);
      } else {
        float* x = m.x[buf] + at.c * kRow + sub * kCkpt;
        const float* b = m.b[buf] + sub * kCkpt;
        const float* slope = m.slope[buf] + at.c * kRow + sub * kCkpt;
        float h0[SPL], h[kCkpt][SPL], a[kCkpt][SPL];
#pragma unroll
        for (int j = 0; j < SPL; ++j) h0[j] = ahead[j];
        enter(--chunk);
#pragma unroll
        for (int q = 0; q < kCkpt / 4; ++q) {
          const float4 dv = ld4(d + 4 * q), xv = ld4(x + 4 * q);
          const float2 d2[2] = {{dv.x, dv.y}, {dv.z, dv.w}}, x2[2] = {{xv.x, xv.y}, {xv.z, xv.w}};
#pragma unroll
          for (int j = 0; j < SPL; ++j) {
            const float4 bv = ld4(b + row[j] + 4 * q);
            const float2 b2[2] = {{bv.x, bv.y}, {bv.z, bv.w}};
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int t = 4 * q + 2 * k;
              const float2 e = ex2_exact(__fmul2_rn(d2[k], {A2[j], A2[j]})), u = __fmul2_rn(__fmul2_rn(d2[k], x2[k]), b2[k]);
              a[t][j] = e.x;
              a[t + 1][j] = e.y;
              h[t][j] = fmaf(a[t][j], t > 0 ? h[t > 0 ? t - 1 : 0][j] : h0[j], u.x);
              h[t + 1][j] = fmaf(a[t + 1][j], h[t][j], u.y);
            }
          }
        }
#pragma unroll
        for (int q = kCkpt / 4 - 1; q >= 0; --q) {
          const float4 dv = ld4(d + 4 * q), xv = ld4(x + 4 * q), gv = ld4(g + 4 * q);
          const float2 d2[2] = {{dv.x, dv.y}, {dv.z, dv.w}}, x2[2] = {{xv.x, xv.y}, {xv.z, xv.w}}, g2[2] = {{gv.x, gv.y}, {gv.z, gv.w}};
          float4 bv[SPL], cv[SPL];
#pragma unroll
          for (int j = 0; j < SPL; ++j) bv[j] = ld4(b + row[j] + 4 * q), cv[j] = ld4(c + row[j] + 4 * q);
          float du[4], sq[4];
#pragma unroll
          for (int k = 1; k >= 0; --k) {
            const int t = 4 * q + 2 * k;
            const float2 u = __fmul2_rn(d2[k], x2[k]);
            float2 du2 = {0.f, 0.f}, sq2 = {0.f, 0.f}, vb[SPL], vc[SPL];
#pragma unroll
            for (int j = 0; j < SPL; ++j) {
              const float2 b2 = k ? float2{bv[j].z, bv[j].w} : float2{bv[j].x, bv[j].y};
              const float2 c2 = k ? float2{cv[j].z, cv[j].w} : float2{cv[j].x, cv[j].y};
              float2 gg, q2;
              gg.y = fmaf(c2.y, g2[k].y, ga[j]);
              const float g1 = a[t + 1][j] * gg.y;
              gg.x = fmaf(c2.x, g2[k].x, g1);
              ga[j] = a[t][j] * gg.x;
              q2.y = g1 * h[t][j];
              q2.x = ga[j] * (t > 0 ? h[t > 0 ? t - 1 : 0][j] : h0[j]);
              vb[j] = __fmul2_rn(gg, u);
              vc[j] = __fmul2_rn(g2[k], {h[t][j], h[t + 1][j]});
              du2 = __ffma2_rn(gg, b2, du2);
              sq2 = __ffma2_rn({A2[j], A2[j]}, q2, sq2);
              dA[j] = __ffma2_rn(d2[k], q2, dA[j]);
            }
            du[2 * k] = du2.x, du[2 * k + 1] = du2.y;
            sq[2 * k] = sq2.x, sq[2 * k + 1] = sq2.y;
            auto step = [&](float2& keep, const float2& give, int lanes) {
              keep = __fadd2_rn(keep, {__shfl_xor_sync(0xffffffffu, give.x, lanes), __shfl_xor_sync(0xffffffffu, give.y, lanes)});
            };
            float* red = &m.red[buf][at.warp][sub * kCkpt + t][at.n0];
            if constexpr (CW >= 4) {
              step(vb[0], vb[2], 2 * NL), step(vb[1], vb[3], 2 * NL);
              step(vc[0], vc[2], 2 * NL), step(vc[1], vc[3], 2 * NL);
              step(vb[0], vb[1], NL), step(vc[0], vc[1], NL);
              if constexpr (CW >= 8) step(vb[0], vb[0], 4 * NL), step(vc[0], vc[0], 4 * NL);
              if constexpr (CW >= 16) step(vb[0], vb[0], 8 * NL), step(vc[0], vc[0], 8 * NL);
              if constexpr (CW >= 8) {  // lanes with the same sums: one writes dB, one dC
                const bool second = at.cl & 4;
                if (CW < 16 || at.cl < 8) {
                  red[(second ? NP : 0) + pm] = second ? vc[0].x : vb[0].x;
                  red[2 * NP + (second ? NP : 0) + pm] = second ? vc[0].y : vb[0].y;
                }
              } else {
                red[pm] = vb[0].x, red[NP + pm] = vc[0].x;
                red[2 * NP + pm] = vb[0].y, red[3 * NP + pm] = vc[0].y;
              }
            } else {
              step(vb[0], vb[1], NL), step(vb[2], vb[3], NL), step(vc[0], vc[1], NL), step(vc[2], vc[3], NL);
#pragma unroll
              for (int j = 0; j < 4; j += 2) {
                red[j ^ pm] = vb[j].x, red[NP + (j ^ pm)] = vc[j].x;
                red[2 * NP + (j ^ pm)] = vb[j].y, red[3 * NP + (j ^ pm)] = vc[j].y;
              }
            }
          }
          lane_sums<4, NL, 1>(du, at.lane);
          lane_sums<4, NL, 1>(sq, at.lane);
          __syncwarp();
          if (at.nl < 4) {  // the gradients take their inputs' places
            constexpr int M = NL < 4 ? 4 / NL : 1;
#pragma unroll
            for (int k = 0; k < M; ++k) {
              const int t = 4 * q + slot + k;
              const float dd = d[t], xx = x[t], gy = g[t], sl = slope[t];
              const float o = sl < 0.f ? 0.f : fmaf(xx, du[k], kLn2 * sq[k]) * sl;
              x[t] = fmaf(dd, du[k], skip * gy);
              d[t] = o;
              dskip = fmaf(gy, xx, dskip);
              dbias += o;
            }
          }
        }
      }
    }
    total += tsum;
    if (!END && (t0 & ((1 << lgp) - 1)) == 0) {  // (a segment starts on a multiple)
#pragma unroll
      for (int o = 1; o < NL; o <<= 1) {
        dskip += __shfl_xor_sync(0xffffffffu, dskip, o);
        dbias += __shfl_xor_sync(0xffffffffu, dbias, o);
      }
      if (at.live) leave(first_unit(s.seqs, p.seq, lgp) + ((p.pos + t0) >> lgp), false);
      dskip = dbias = 0.f;
#pragma unroll
      for (int j = 0; j < SPL; ++j) dA[j] = {0.f, 0.f};
    }
  }
  __syncthreads();
  if (!at.live) return;
  if constexpr (END) {
#pragma unroll
    for (int j = 0; j < SPL; ++j) s.starts[state_at<NP>(s, blockIdx.x, at.ch, at.n0 + (j ^ pm))] = ga[j];
    if (at.nl == 0) s.sums[(int64_t)blockIdx.x * s.D + at.ch] = total;
  } else {
#pragma unroll
    for (int j = 0; j < SPL; ++j) {
      const int n = at.n0 + (j ^ pm);
      if (n < s.N && s.dinit && p.idx == 0) s.dinit[((int64_t)p.seq * s.D + at.ch) * s.N + n] = ga[j];
    }
    // rows without a token: an empty sequence's, and the one that a packed sequence may have over
    if (p.pos + p.len == p.slen) {
      const int64_t end = first_unit(s.seqs, p.seq + 1, lgp);
      for (int64_t row = first_unit(s.seqs, p.seq, lgp) + ((p.slen + (1 << lgp) - 1) >> lgp); row < end; ++row) leave(row, true);
    }
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
    if (k > 0) g = fmaf(ex2_exact({A2 * s.sums[(u0 + k) * s.D + ch], 0.f}).x, g, front);
  }
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

// The parameters' gradients: columns of [D][N + 2], summed over the rows of at most 256 tokens.
template <int STR>
__global__ void __launch_bounds__(STR == 1 ? 256 : 32 * STR) k_ssm_par_sums(Ssm s, int64_t rows) {
  if (bad_call(s.seqs)) return;
  const int64_t width = s.D * (s.N + 2);
  int64_t c;
  const float v = strand_sums<STR>(s.part_par, rows, width, width, c);
  if (c < 0) return;
  const int64_t ch = c / (s.N + 2);
  const int n = (int)(c - ch * (s.N + 2));
  if (n < s.N) {
    if (s.dA_log) s.dA_log[ch * s.N + n] = -rate_of(s.A_log[ch * s.N + n]) * v;
  } else if (n == s.N) {
    if (s.dskip) s.dskip[ch] = v;
  } else if (s.ddt_bias) {
    s.ddt_bias[ch] = v;
  }
}

template <typename T, int NP>
cudaError_t backward(const Ssm& c, cudaStream_t s) {
  using S = Shape<NP, kBwd>;
  const int64_t Dg = c.D / c.G, tiles = (Dg + S::CC - 1) / S::CC, units = max_units(c.seqs, c.lg);
  const dim3 grid((unsigned)units, (unsigned)(c.G * tiles));
  if (c.cut) {
    {
      ProfScope ps("ssm_bwd_ends", s);
      constexpr size_t bytes = sizeof(BwdShared<T, NP, true>);
      if (cudaError_t e = allow_shared(k_ssm_bwd<T, NP, true>, bytes)) return e;
      k_ssm_bwd<T, NP, true><<<grid, S::NT, bytes, s>>>(c);
    }
    ProfScope ps("ssm_bwd_join", s);
    k_ssm_bwd_join<NP><<<(unsigned)((c.D * NP + 255) / 256 * c.seqs.n), 256, 0, s>>>(c);
  }
  {
    ProfScope ps("ssm_bwd", s);
    constexpr size_t bytes = sizeof(BwdShared<T, NP, false>);
    if (cudaError_t e = allow_shared(k_ssm_bwd<T, NP, false>, bytes)) return e;
    // the working warps' 200 registers and the feeding warps' 56 are the launch's 128 a thread, no more
    cudaFuncAttributes f;
    if (cudaError_t e = cudaFuncGetAttributes(&f, k_ssm_bwd<T, NP, false>)) return e;
    if (f.numRegs != 128) return cudaErrorInvalidConfiguration;
    k_ssm_bwd<T, NP, false><<<grid, S::NT, bytes, s>>>(c);
  }
  const int64_t all = (c.seqs.cu ? c.seqs.T : c.seqs.T * c.seqs.n) * c.G * 2 * NP;
  if (all > 0) {
    ProfScope ps("ssm_bwd_bc", s);
    k_ssm_bc_sums<T><<<(unsigned)std::min<int64_t>((all + 255) / 256, 148 * 32), 256, 0, s>>>(c, NP, tiles);
  }
  ProfScope ps("ssm_bwd_par", s);
  const int64_t width = c.D * (c.N + 2), rows = max_units(c.seqs, std::min(c.lg, kParLog));
  switch (sum_strands(rows)) {
    case 1: k_ssm_par_sums<1><<<(unsigned)((width + 255) / 256), 256, 0, s>>>(c, rows); break;
    case 8: k_ssm_par_sums<8><<<(unsigned)((width + 31) / 32), 256, 0, s>>>(c, rows); break;
    default: k_ssm_par_sums<32><<<(unsigned)((width + 31) / 32), 1024, 0, s>>>(c, rows);
  }
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
