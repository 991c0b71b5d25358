// Selective state space scan: forward over sequences, and the step of one token.  The mathematics and
// the layout of the work are in ssm_common.cuh.
#include <algorithm>

#include "ssm_common.cuh"

namespace gdn {
namespace mix {
namespace {

constexpr int kFwd = 4;  // states of a lane

template <typename T, int NP, bool END>
struct FwdShared {
  static constexpr int X = 512 / NP * kRow, S = NP * kRow;
  float d[2][X], x[2][X], b[2][S], c[2][END ? 4 : S];
  // targets of 16-byte copies
  alignas(16) RawRows<T, NP> rx;
  alignas(16) RawRows<T, NP> rt;
  alignas(16) T rb[kRing<T, NP>][kTile * NP];
  alignas(16) T rc[kRing<T, NP>][END ? 8 : kTile * NP];
};

// Measured (bf16, N = 16): 1 x 32768 x 4096 1.43 ms, with one block on each of 128 multiprocessors, bound by the
// latency of its four working warps (issue 40%, shared memory 54%, exponentials 39% of their peaks); 8 x 1024 x 4096
// 237 us, where shared memory binds (87%: a 16-byte load is four wavefronts however many lanes want the same
// words, 10 bytes a state and token, eight of them B and C widened).  The bytes alone would take 123 and 31 us, the
// exponentials 0.55 ms and 0.14.  fp32, with the polynomial: 376 us (issue and shared memory 61% each).
// Tried and slower: two states a lane (1.58 ms), the sums over lanes left to the feeding warps (1.54 ms), two
// channels a lane (within 15% either way).
// One segment.  END: only the state at its end from a zero state, and the sum of its deltas (the first
// pass over segments that have one behind them).
// 16 tokens at a time: their exponentials do not wait for the states, and their 16 sums over the states are
// butterflies that do not wait for one another.
template <typename T, int NP, bool END>
__global__ void __launch_bounds__(Shape<NP, kFwd>::NT, 3) k_ssm_fwd(Ssm s) {
  using S = Shape<NP, kFwd>;
  constexpr int SPL = kFwd, NL = S::NL, FC = S::FC, PITCH = RawRows<T, NP>::PITCH, R = kRing<T, NP>;
  extern __shared__ __align__(16) char raw[];
  FwdShared<T, NP, END>& m = *reinterpret_cast<FwdShared<T, NP, END>*>(raw);
  if (bad_call(s.seqs)) return;
  Place<NP, SPL> at;
  if (!at.find(s, s.lg)) return;
  const Piece& p = at.p;
  if (END && p.pos + p.len == p.slen) return;  // nothing follows
  const int tiles = (p.len + kTile - 1) / kTile;

  if (at.feeds) {
    const Inputs<T, NP, SPL> in(s, at);
    float bias[FC];
#pragma unroll
    for (int i = 0; i < FC; ++i) bias[i] = at.sc + i < at.width && s.dt_bias ? s.dt_bias[at.c0 + at.sc + i] : 0.f;
    T* y = static_cast<T*>(s.y) + (p.t0 + at.tok) * s.D + at.c0 + at.sc;
    auto fetch = [&](int tile, int r) {
      if (tile < tiles) {
        const int t0 = tile * kTile, n = p.len - t0;
        in.x.fetch(m.rx.v[r], at.f, t0, n);
        in.dt.fetch(m.rt.v[r], at.f, t0, n);
        in.B.fetch(m.rb[r], at.f, t0, n);
        if (!END) in.C.fetch(m.rc[r], at.f, t0, n);
      }
      copy_commit();
    };
    auto widen = [&](int tile, int r, int buf) {
      const bool here = tile * kTile + at.tok < p.len;
      Cols<T, FC> xr, tr;
      xr.load(m.rx.v[r] + at.tok * PITCH + at.sc);
      tr.load(m.rt.v[r] + at.tok * PITCH + at.sc);
      float *d = m.d[buf] + at.sc * kRow + at.tok, *x = m.x[buf] + at.sc * kRow + at.tok;
#pragma unroll
      for (int i = 0; i < FC; i += 2) {
        float2 e;
        const float2 v = softplus2({tr.get(i) + bias[i], tr.get(i + 1) + bias[i + 1]}, e);
        d[i * kRow] = here ? v.x : 0.f;
        d[(i + 1) * kRow] = here ? v.y : 0.f;
        x[i * kRow] = xr.get(i);
        x[(i + 1) * kRow] = xr.get(i + 1);
      }
      widen_states<T, NP, SPL>(m.b[buf], m.rb[r], at.f);
      if (!END) widen_states<T, NP, SPL>(m.c[buf], m.rc[r], at.f);
    };
    auto put = [&](int tile, int buf) {  // y, left in x's place
      const float* x = m.x[buf] + at.sc * kRow + at.tok;
      Cols<T, FC> o;
#pragma unroll
      for (int i = 0; i < FC; i += 2) o.put2(i, {x[i * kRow], x[(i + 1) * kRow]});
      if (tile * kTile + at.tok < p.len) o.store(y + (int64_t)tile * kTile * s.D, s.vec, at.width - at.sc);
    };
    // The feeding warps meet on a barrier of their own before they widen what all of them fetched.
    auto meet = [] { asm volatile("bar.sync 1, 128;" ::: "memory"); };
    for (int k = 0; k < R; ++k) fetch(k, k);
    int r = 0;
    for (int tile = 0; tile < tiles; ++tile) {  // tile is widened while the one before it is worked on
      copy_wait<R - 1>();
      meet();
      if (!END && tile > 1) put(tile - 2, tile & 1);
      widen(tile, r, tile & 1);
      meet();
      fetch(tile + R, r);
      r = r == R - 1 ? 0 : r + 1;
      __syncthreads();
    }
    copy_wait<0>();
    __syncthreads();
    if (!END) {
      if (tiles > 1) put(tiles - 2, tiles & 1);
      if (tiles > 0) put(tiles - 1, (tiles - 1) & 1);
    }
    return;
  }

  float A2[SPL], h[SPL];
  load_decay(s, at.ch, at.live, at.n0, A2);
#pragma unroll
  for (int j = 0; j < SPL; ++j) h[j] = 0.f;
  if (!END && at.live) {
    if (s.cut && p.idx > 0)
      load_states(s.starts + state_at<NP>(s, blockIdx.x, at.ch, 0), s.N, at.n0, h);  // nothing wrote the others
    else if (s.init)
      load_states(s.init + ((int64_t)p.seq * s.D + at.ch) * s.N, s.N, at.n0, h);
  }
  const float skip = !END && at.live && at.nl == 0 && s.skip ? s.skip[at.ch] : 0.f;
  float* ck = nullptr;
  if (!END && s.ckpt && at.live)
    ck = s.ckpt + state_at<NP>(s, first_unit(s.seqs, p.seq, kCkptLog) + p.pos / kCkpt, at.ch, at.n0);
  const int slot = lane_slot<kCkpt, NL>(at.nl);
  float total = 0.f;
  for (int tile = 0; tile < tiles; ++tile) {
    const int buf = tile & 1;
    __syncthreads();  // the tile is there
    const int subs = p.len - tile * kTile > kCkpt ? 2 : 1;
    float tsum = 0.f;
#pragma unroll 1
    for (int sub = 0; sub < subs; ++sub) {
      if (ck) {
        store_padded(ck, h);
        ck += s.D * NP;
      }
      const float* d = m.d[buf] + at.c * kRow + sub * kCkpt;
      float* x = m.x[buf] + at.c * kRow + sub * kCkpt;
      const float* b = m.b[buf] + state_row<NP, SPL>(at.n0) + sub * kCkpt;
      const float* c = m.c[buf] + state_row<NP, SPL>(at.n0) + sub * kCkpt;
      float yv[kCkpt], dq[kCkpt / 4];
#pragma unroll
      for (int q = 0; q < kCkpt / 4; ++q) {
        const float4 dv = ld4(d + 4 * q), xv = ld4(x + 4 * q);
        const float2 d2[2] = {{dv.x, dv.y}, {dv.z, dv.w}}, x2[2] = {{xv.x, xv.y}, {xv.z, xv.w}};
        if (END) dq[q] = (dv.x + dv.y) + (dv.z + dv.w);
        float2 u2[2], y2[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          u2[k] = __fmul2_rn(d2[k], x2[k]);
          if (!END) y2[k] = __fmul2_rn({skip, skip}, x2[k]);
        }
#pragma unroll
        for (int j = 0; j < SPL; ++j) {
          const float4 bv = ld4(b + j * NL * kRow + 4 * q);
          const float2 b2[2] = {{bv.x, bv.y}, {bv.z, bv.w}};
          float2 c2[2];
          if (!END) {
            const float4 cv = ld4(c + j * NL * kRow + 4 * q);
            c2[0] = {cv.x, cv.y}, c2[1] = {cv.z, cv.w};
          }
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float2 a = decays<T>(d2[k], {A2[j], A2[j]}), u = __fmul2_rn(u2[k], b2[k]);
            float2 hh;
            hh.x = fmaf(a.x, h[j], u.x);
            hh.y = fmaf(a.y, hh.x, u.y);
            h[j] = hh.y;
            if (!END) y2[k] = __ffma2_rn(hh, c2[k], y2[k]);
          }
        }
        if (!END) yv[4 * q] = y2[0].x, yv[4 * q + 1] = y2[0].y, yv[4 * q + 2] = y2[1].x, yv[4 * q + 3] = y2[1].y;
      }
      if (END) {
        tsum += (dq[0] + dq[1]) + (dq[2] + dq[3]);
      } else {
        lane_sums<kCkpt, NL, 1>(yv, at.lane);
        __syncwarp();
        if (NL <= kCkpt || at.nl < kCkpt) {
          constexpr int M = NL < kCkpt ? kCkpt / NL : 1;
#pragma unroll
          for (int k = 0; k < M; ++k) x[slot + k] = yv[k];
        }
      }
    }
    total += tsum;
  }
  __syncthreads();
  if (!at.live) return;
  if (END) {
    store_padded(s.starts + state_at<NP>(s, blockIdx.x, at.ch, at.n0), h);
    if (at.nl == 0) s.sums[(int64_t)blockIdx.x * s.D + at.ch] = total;
  } else if (s.final && p.pos + p.len == p.slen) {
    store_states(s.final + ((int64_t)p.seq * s.D + at.ch) * s.N, s.N, at.n0, h);
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
    if (k + 1 < segs) h = fmaf(ex2_exact({A2 * s.sums[(u0 + k) * s.D + ch], 0.f}).x, h, end);
  }
}

// One token for each sequence: a thread has four states of a channel, so a state moves as 16 bytes, and goes through
// the sequences four at a time: its decay rates serve all of them, and its lanes of a channel share out the four
// softplus and the four sums.  No unit is saturated with many requests (shared memory 65%, issue 58%, DRAM 40% of
// their peaks, 31% of the warps): it is the latency of rings whose every thread copies its own B and C.  RING: the
// states, B and C of the next two groups of four are on their way through shared memory of the thread's own
// (asynchronous 16- and 8-byte copies).  Without: plain loads, for calls of few sequences, which gain nothing from a
// ring (4 requests x 4096 x 16: 3.7 us, with the ring 4.0), and where N or the alignment of B and C does not allow the
// copies.  256 requests x 4096 x 16: 28 us for the 141 MB that they read and write (5.0 TB/s), without the ring 41; 64
// requests, below the rule's border, 10.9 without and 9.1 with it.  init and final may be one buffer: a thread reads
// its states before it writes them, and no other touches them.
template <typename T, int NP, bool RING>
__global__ void __launch_bounds__(256, 3) k_ssm_step(Ssm s) {
  constexpr int NL = NP / 4, Q = 4, OWN = NL < Q ? Q / NL : 1;  // sequences whose softplus and sum a lane has
  constexpr int MAT = 4 * (int)sizeof(T);                       // bytes of four values of B or C
  extern __shared__ __align__(16) char shared[];                // [2][Q][256] states, then B, then C
  const unsigned ring = (unsigned)__cvta_generic_to_shared(shared);
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t ch = at / NL;
  const int lane = threadIdx.x & 31, nl = (int)(at % NL), n0 = nl * 4, first = lane & ~(NL - 1);
  const bool live = ch < s.D;
  const int slot = lane_slot<Q, NL>(nl);  // of lanes that share a sum, the first writes it
  const int64_t g = live ? ch / (s.D / s.G) : 0, q0 = (int64_t)blockIdx.y * Q, step = (int64_t)gridDim.y * Q;
  const int64_t states = s.D * s.N;  // of a sequence
  const float* st = s.init + q0 * states + ch * s.N + n0;
  float* nx = s.final + q0 * states + ch * s.N + n0;
  const T* Bm = static_cast<const T*>(s.Bm) + q0 * s.ld_b + g * s.N + n0;
  const T* Cm = static_cast<const T*>(s.Cm) + q0 * s.ld_c + g * s.N + n0;
  const T* x = static_cast<const T*>(s.x) + (q0 + slot) * s.ld_x + ch;
  const T* dt = static_cast<const T*>(s.dt) + (q0 + slot) * s.ld_dt + ch;
  T* y = static_cast<T*>(s.y) + (q0 + slot) * s.D + ch;
  const bool some = live && n0 < s.N;
  int64_t left = s.seqs.n - q0, to_ask = left;
  auto at_state = [&](int half, int k) { return ring + ((half * Q + k) * 256 + threadIdx.x) * 16; };
  auto at_mat = [&](int half, int k, int which) { return ring + 2 * Q * 256 * 16 + (((which * 2 + half) * Q + k) * 256 + threadIdx.x) * MAT; };
  auto ask = [&](int half) {
    if constexpr (RING) {
#pragma unroll
      for (int k = 0; k < Q; ++k) {
        const bool in = some && k < to_ask;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at_state(half, k)), "l"(in ? st + k * states : s.init), "r"(in ? 16 : 0) : "memory");
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(at_mat(half, k, 0)), "l"(in ? static_cast<const void*>(Bm + k * s.ld_b) : s.Bm), "n"(MAT), "r"(in ? MAT : 0) : "memory");
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(at_mat(half, k, 1)), "l"(in ? static_cast<const void*>(Cm + k * s.ld_c) : s.Cm), "n"(MAT), "r"(in ? MAT : 0) : "memory");
      }
      copy_commit();
      st += step * states, Bm += step * s.ld_b, Cm += step * s.ld_c;
      to_ask -= step;
    }
  };
  T xr[OWN], tr[OWN];
  auto fetch = [&](int64_t have) {
#pragma unroll
    for (int i = 0; i < OWN; ++i) {
      xr[i] = tr[i] = down<T>(0.f);
      if (live && slot + i < have) xr[i] = x[i * s.ld_x], tr[i] = dt[i * s.ld_dt];
    }
  };
  ask(0);
  ask(1);
  fetch(left);
  float A2[4];
  load_decay(s, ch, live, n0, A2);
  const float bias = live && s.dt_bias ? s.dt_bias[ch] : 0.f, skip = live && s.skip ? s.skip[ch] : 0.f;
  for (int half = 0; left > 0; left -= step, half ^= 1) {
    float h[Q][4], xv[OWN], u[OWN], d[OWN], o[Q];
    if constexpr (!RING) {
#pragma unroll
      for (int k = 0; k < Q; ++k) {
#pragma unroll
        for (int j = 0; j < 4; ++j) h[k][j] = 0.f;
        if (some && k < left) {
          if (s.vec)
            load_padded(st + k * states, h[k]);
          else
            load_states(st + k * states, s.N - n0, 0, h[k]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < OWN; ++i) {
      xv[i] = up<T>(xr[i]);
      const float v = up<T>(tr[i]) + bias;
      float2 e;
      d[i] = softplus2({v, v}, e).x;
      u[i] = d[i] * xv[i];
    }
    x += step * s.ld_x, dt += step * s.ld_dt;
    fetch(left - step);
    if constexpr (RING) copy_wait<1>();
#pragma unroll
    for (int k = 0; k < Q; ++k) {
      // the lane whose slot covers k, and the place there
      constexpr int HAVE = NL < Q ? NL : Q;
      int owner = 0;
#pragma unroll
      for (int l = 0; l < HAVE; ++l)
        if (lane_slot<Q, NL>(l) == k / OWN * OWN) owner = l;
      const float dk = __shfl_sync(0xffffffffu, d[k % OWN], first + owner), uk = __shfl_sync(0xffffffffu, u[k % OWN], first + owner);
      float a = 0.f;
      if (some && k < left) {
        float b[4], c[4];
        if constexpr (RING) {
          asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(h[k][0]), "=f"(h[k][1]), "=f"(h[k][2]), "=f"(h[k][3]) : "r"(at_state(half, k)) : "memory");
          Pack<T, 4> pb, pc;
          if constexpr (MAT == 8) {
            asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(pb.u[0]), "=r"(pb.u[1]) : "r"(at_mat(half, k, 0)) : "memory");
            asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(pc.u[0]), "=r"(pc.u[1]) : "r"(at_mat(half, k, 1)) : "memory");
          } else {
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(pb.u[0]), "=r"(pb.u[1]), "=r"(pb.u[2]), "=r"(pb.u[3]) : "r"(at_mat(half, k, 0)) : "memory");
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(pc.u[0]), "=r"(pc.u[1]), "=r"(pc.u[2]), "=r"(pc.u[3]) : "r"(at_mat(half, k, 1)) : "memory");
          }
          pb.get(b), pc.get(c);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            b[j] = n0 + j < s.N ? up<T>(Bm[k * s.ld_b + j]) : 0.f;
            c[j] = n0 + j < s.N ? up<T>(Cm[k * s.ld_c + j]) : 0.f;
          }
        }
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
          const float2 e = decays<T>({dk, dk}, {A2[j], A2[j + 1]});
          h[k][j] = fmaf(e.x, h[k][j], uk * b[j]);
          h[k][j + 1] = fmaf(e.y, h[k][j + 1], uk * b[j + 1]);
          a = fmaf(h[k][j], c[j], a);
          a = fmaf(h[k][j + 1], c[j + 1], a);
        }
        if (RING || s.vec)
          store_padded(nx + k * states, h[k]);
        else
          store_states(nx + k * states, s.N - n0, 0, h[k]);
      }
      o[k] = a;
    }
    ask(half);
    lane_sums<Q, NL, 1>(o, lane);
#pragma unroll
    for (int i = 0; i < OWN; ++i)
      if (live && slot + i < left && nl < Q) y[i * s.D] = down<T>(fmaf(skip, xv[i], o[i]));
    nx += step * states, y += step * s.D;
    if constexpr (!RING) st += step * states, Bm += step * s.ld_b, Cm += step * s.ld_c;
  }
  copy_wait<0>();
}

template <typename T, int NP>
cudaError_t forward(const Ssm& c, cudaStream_t s) {
  using S = Shape<NP, kFwd>;
  const int64_t Dg = c.D / c.G;
  const dim3 grid((unsigned)max_units(c.seqs, c.lg), (unsigned)(c.G * ((Dg + S::CC - 1) / S::CC)));
  if (c.cut) {
    {
      ProfScope ps("ssm_fwd_ends", s);
      constexpr size_t bytes = sizeof(FwdShared<T, NP, true>);
      if (cudaError_t e = allow_shared(k_ssm_fwd<T, NP, true>, bytes)) return e;
      k_ssm_fwd<T, NP, true><<<grid, S::NT, bytes, s>>>(c);
    }
    ProfScope ps("ssm_join", s);
    k_ssm_join<NP><<<(unsigned)((c.D * NP + 255) / 256 * c.seqs.n), 256, 0, s>>>(c);
  }
  ProfScope ps("ssm_fwd", s);
  constexpr size_t bytes = sizeof(FwdShared<T, NP, false>);
  if (cudaError_t e = allow_shared(k_ssm_fwd<T, NP, false>, bytes)) return e;
  k_ssm_fwd<T, NP, false><<<grid, S::NT, bytes, s>>>(c);
  return cudaGetLastError();
}

template <typename T, int NP>
cudaError_t step(const Ssm& c, cudaStream_t s) {
  const int64_t across = (c.D * (NP / 4) + 255) / 256, groups = (c.seqs.n + 3) / 4;
  // with the ring, three blocks for each of 148 multiprocessors; without, as many as there are, up to 16
  const int64_t most = std::min<int64_t>(groups, 65535), ring = std::max<int64_t>(1, 148 * 3 / across);
  ProfScope ps("ssm_step", s);
  if (c.vec && c.vec_bc && groups >= 4 * ring) {
    constexpr size_t bytes = 2 * 4 * 256 * (16 + 8 * sizeof(T));
    if (cudaError_t e = allow_shared(k_ssm_step<T, NP, true>, bytes)) return e;
    k_ssm_step<T, NP, true><<<dim3((unsigned)across, (unsigned)ring), 256, bytes, s>>>(c);
  } else {
    const dim3 grid((unsigned)across, (unsigned)std::min(most, std::max<int64_t>(1, 148 * 16 / across)));
    k_ssm_step<T, NP, false><<<grid, 256, 0, s>>>(c);
  }
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

// Segments.  A block goes through a token in about 44 ns forward and 142 ns backward while it has a
// multiprocessor to itself, and up to three (two) blocks share one almost for free; the first pass costs 0.8
// (0.2) of a pass more and the join some 20 us.  So sequences are cut where the whole ones leave
// most of the card idle, into as many segments as make 512 blocks, of at least 128 tokens.  Measured (device time,
// bf16, N = 16, forward / backward, us, whole against cut):
//   blocks 32   1 x 8192 x 1024    365 against 131   1145 against 291
//   blocks 64   1 x 16384 x 2048   726 against 467   2328 against 1063
//   blocks 64   1 x 512 x 2048      27 against 26      78 against 52
//   blocks 64   1 x 256 x 2048      16 against 20      44 against 38
//   blocks 100  1 x 4096 x 3200    185 against 180    594 against 454
//   blocks 128  2 x 4096 x 2048    186 against 221    594 against 531
//   blocks 200  1 x 4096 x 6400    275 against 343    872 against 826
//   blocks 256  4 x 4096 x 2048    274 against 427    870 against 979
// The rule goes by sizes alone and is off for short sequences at the border (1 x 512 x 4096, 128 blocks: backward 80
// against 91) and for fp32, whose first pass has the polynomial (2 x 4096 x 2048: backward 607 against 743, 1 x 4096 x
// 3200: forward 296 against 309).
SsmSizes ssm_sizes(const Seqs& s, int64_t tokens, int64_t D, int N, int G) {
  SsmSizes z{};
  const int NP = ssm_padded(N), CC = 512 / NP;
  const int64_t Dg = D / G, tiles = (Dg + CC - 1) / CC, length = s.cu ? tokens / s.n : s.T, blocks = tiles * G * s.n;
  for (int pass = 0; pass < 2; ++pass) {
    z.lg[pass] = 30;
    z.cut[pass] = pass == 0 ? blocks <= 100 && length >= 768 : blocks <= 200 && length >= 256;
    if (z.cut[pass]) {
      const int64_t segments = (512 + blocks - 1) / blocks;
      z.lg[pass] = 7;
      while (z.lg[pass] < 30 && ((int64_t)1 << z.lg[pass]) * segments < length) ++z.lg[pass];
    }
    const int64_t u = max_units(s, z.lg[pass]);
    if (z.cut[pass]) {
      z.starts = std::max(z.starts, u * D * NP);
      z.sums = std::max(z.sums, u * D);
    }
  }
  z.ckpt = max_units(s, kCkptLog) * D * NP;
  z.part_bc = tiles * tokens * G * 2 * NP;
  z.part_par = max_units(s, std::min(z.lg[1], kParLog)) * D * (N + 2);
  return z;
}

cudaError_t ssm_forward(const Ssm& c, cudaStream_t s) { return dispatch(c, false, s); }
cudaError_t ssm_step(const Ssm& c, cudaStream_t s) { return dispatch(c, true, s); }

}  // namespace mix
}  // namespace gdn
