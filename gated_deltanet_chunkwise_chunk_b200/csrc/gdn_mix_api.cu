// C-ABI entry points of the mixing-layer operators: argument validation and workspace layout.
#include <cmath>
#include <cstdint>

#include "gdn.h"
#include "gdn_mix.h"

using namespace gdn::mix;

namespace {

constexpr size_t kAlign = 256;
constexpr int64_t kMaxTokens = (int64_t)1 << 30, kMaxWidth = (int64_t)1 << 20, kMaxGrid = 2147483647, kMaxGridY = 65535;

size_t up256(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
bool dtype_ok(int32_t t) { return t == GDN_DTYPE_FP32 || t == GDN_DTYPE_BF16 || t == GDN_DTYPE_FP16; }
size_t esize(int32_t t) { return t == GDN_DTYPE_FP32 ? 4 : 2; }
bool misaligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }
int status_of(cudaError_t e) { return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA; }

template <size_t K>
bool any_misaligned(const void* const (&ps)[K], size_t a) {
  for (const void* p : ps)
    if (misaligned(p, a)) return true;
  return false;
}
template <size_t K>
bool any_null(const void* const (&ps)[K]) {
  for (const void* p : ps)
    if (!p) return true;
  return false;
}
// Whether two buffers share bytes (null buffers share none).
bool overlap(const void* a, size_t an, const void* b, size_t bn) {
  if (!a || !b || !an || !bn) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + bn && y < x + an;
}
size_t extent(int64_t rows, int64_t ld, int64_t width, size_t es) { return rows ? ((rows - 1) * ld + width) * es : 0; }

// A buffer of a call.
struct Span {
  const void* p;
  size_t bytes;
};
// Whether an output shares bytes with an input or with another output (the workspace counts as one).
template <size_t O, size_t I>
bool clash(const Span (&outs)[O], const Span (&ins)[I]) {
  for (size_t o = 0; o < O; ++o) {
    for (const Span& i : ins)
      if (overlap(outs[o].p, outs[o].bytes, i.p, i.bytes)) return true;
    for (size_t q = 0; q < o; ++q)
      if (overlap(outs[o].p, outs[o].bytes, outs[q].p, outs[q].bytes)) return true;
  }
  return false;
}
size_t cu_bytes(int64_t n) { return (size_t)(n + 1) * sizeof(int64_t); }

bool workspace_ok(const void* ws, size_t have, size_t need) { return ws && !misaligned(ws, kAlign) && have >= need; }

// B sequences of T tokens, or N packed into T tokens (varlen)
int check_sequences(int64_t B, int64_t T, int64_t N, bool varlen) {
  if (B <= 0 || T < 0 || T > kMaxTokens || B > kMaxTokens || B * T > kMaxTokens) return GDN_ERR_INVALID_ARG;
  if (varlen && (B != 1 || N <= 0 || N > kMaxTokens)) return GDN_ERR_INVALID_ARG;
  return GDN_OK;
}

Seqs sequences(int64_t B, int64_t T, int64_t N, const int64_t* cu, bool varlen, void* status) {
  Seqs s{};
  s.cu = varlen ? cu : nullptr;
  s.status = static_cast<int*>(status);
  s.T = T;
  s.n = (int)(varlen ? N : B);
  return s;
}

// a non-null stand-in for sizes asked without the boundaries at hand
const int64_t* some_cu() { return reinterpret_cast<const int64_t*>(kAlign); }

// ------------------------------------------------------------------------------ convolution

int check_conv(const gdn_conv_dims* d, bool varlen) {
  if (!d) return GDN_ERR_INVALID_ARG;
  if (int rc = check_sequences(d->B, d->T, d->N, varlen)) return rc;
  if (d->D <= 0 || d->D > kMaxWidth) return GDN_ERR_INVALID_ARG;
  if (d->W < 1 || d->W > kConvMaxW || !dtype_ok(d->dtype)) return GDN_ERR_UNSUPPORTED;
  if (d->ld_x < 0 || (d->ld_x > 0 && d->ld_x < d->D) || d->ld_x > ((int64_t)1 << 31)) return GDN_ERR_INVALID_ARG;
  if (d->flags & ~GDN_CONV_SILU) return GDN_ERR_INVALID_ARG;
  return GDN_OK;
}

Conv conv_of(const gdn_conv_dims* d, const Seqs& s) {
  Conv c{};
  c.seqs = s;
  c.D = d->D;
  c.ld = d->ld_x ? d->ld_x : d->D;
  c.W = (int)d->W;
  c.dtype = d->dtype;
  c.silu = (d->flags & GDN_CONV_SILU) != 0;
  return c;
}

size_t conv_bytes(const gdn_conv_dims* d, bool varlen, int pass) {
  const Seqs s = sequences(d->B, d->T, d->N, some_cu(), varlen, nullptr);
  return kAlign + (pass == 1 ? up256((size_t)conv_bwd_units(s, d->D) * (d->W + 1) * d->D * sizeof(float)) : 0);
}

// ------------------------------------------------------------------------------ scan

int check_ssm(const gdn_ssm_dims* d, bool varlen) {
  if (!d) return GDN_ERR_INVALID_ARG;
  if (int rc = check_sequences(d->B, d->T, d->N, varlen)) return rc;
  if (d->D <= 0 || d->D > kMaxWidth || d->G <= 0 || d->D % d->G || d->S <= 0) return GDN_ERR_INVALID_ARG;
  if (d->S > 64 || !dtype_ok(d->dtype)) return GDN_ERR_UNSUPPORTED;
  const int64_t ls[] = {d->ld_x, d->ld_dt, d->ld_b, d->ld_c}, ws[] = {d->D, d->D, d->G * d->S, d->G * d->S};
  for (int i = 0; i < 4; ++i)
    if (ls[i] < 0 || (ls[i] > 0 && ls[i] < ws[i]) || ls[i] > ((int64_t)1 << 31)) return GDN_ERR_INVALID_ARG;
  const int NP = ssm_padded((int)d->S), CC = 512 / NP;
  if (d->G * ((d->D / d->G + CC - 1) / CC) > kMaxGridY) return GDN_ERR_INVALID_ARG;
  const int64_t n = varlen ? d->N : d->B;
  if ((d->D * NP + 255) / 256 > kMaxGrid / n) return GDN_ERR_INVALID_ARG;
  return GDN_OK;
}

struct SsmPlan {
  SsmSizes z;
  size_t starts, sums, ckpt, part_bc, part_par, fwd, total;
};

SsmPlan ssm_plan(const gdn_ssm_dims* d, bool varlen) {
  SsmPlan p{};
  const Seqs s = sequences(d->B, d->T, d->N, some_cu(), varlen, nullptr);
  p.z = ssm_sizes(s, d->B * d->T, d->D, (int)d->S, (int)d->G);
  size_t o = kAlign;
  auto take = [&](int64_t floats) {
    const size_t at = o;
    o += up256((size_t)floats * sizeof(float));
    return at;
  };
  p.starts = take(p.z.starts);
  p.sums = take(p.z.sums);
  p.fwd = o;
  p.ckpt = take(p.z.ckpt);
  p.part_bc = take(p.z.part_bc);
  p.part_par = take(p.z.part_par);
  p.total = o;
  return p;
}

Ssm ssm_of(const gdn_ssm_dims* d, const Seqs& s, const SsmPlan& p, void* ws, int pass) {
  Ssm c{};
  c.seqs = s;
  c.D = d->D;
  c.N = (int)d->S;
  c.G = (int)d->G;
  c.dtype = d->dtype;
  c.ld_x = d->ld_x ? d->ld_x : d->D;
  c.ld_dt = d->ld_dt ? d->ld_dt : d->D;
  c.ld_b = d->ld_b ? d->ld_b : d->G * d->S;
  c.ld_c = d->ld_c ? d->ld_c : d->G * d->S;
  c.lg = p.z.lg[pass];
  c.cut = p.z.cut[pass];
  char* b = static_cast<char*>(ws);
  auto at = [&](size_t o) { return reinterpret_cast<float*>(b + o); };
  c.starts = at(p.starts);
  c.sums = at(p.sums);
  c.ckpt = at(p.ckpt);
  c.part_bc = at(p.part_bc);
  c.part_par = at(p.part_par);
  return c;
}

// Accesses of x, dt, y (dy, dx, ddt): of 16 (or 4) bytes where rows, their strides and a group's channels are multiples.
int ssm_vec(const Ssm& c) {
  const void* ps[] = {c.x, c.dt, c.y, c.dy, c.dx, c.ddt};
  for (int mode = 2; mode > 0; --mode) {
    const size_t b = mode == 2 ? 16 : 4;
    const int64_t V = (int64_t)(b / esize(c.dtype));
    if ((c.D / c.G) % V == 0 && c.ld_x % V == 0 && c.ld_dt % V == 0 && !any_misaligned(ps, b)) return mode;
  }
  return 0;
}
// and of B and C
int ssm_vec_bc(const Ssm& c) {
  const void* ps[] = {c.Bm, c.Cm};
  for (int mode = 2; mode > 0; --mode) {
    const size_t b = mode == 2 ? 16 : 4;
    const int64_t V = (int64_t)(b / esize(c.dtype));
    if (c.N % V == 0 && c.ld_b % V == 0 && c.ld_c % V == 0 && !any_misaligned(ps, b)) return mode;
  }
  return 0;
}

// ------------------------------------------------------------------------------ norm

int check_norm(const gdn_norm_dims* d) {
  if (!d || d->rows < 0 || d->D <= 0 || d->D > kMaxWidth || d->rows > ((int64_t)1 << 40) / d->D * 4) return GDN_ERR_INVALID_ARG;
  if (!dtype_ok(d->dtype)) return GDN_ERR_UNSUPPORTED;
  if (d->inner_x < 0 || d->inner_gate < 0 || d->ld_x < 0 || d->ld_gate < 0 || (d->flags & ~GDN_NORM_RMS)) return GDN_ERR_INVALID_ARG;
  const int64_t ix = d->inner_x ? d->inner_x : 1, iz = d->inner_gate ? d->inner_gate : 1;
  if (ix > ((int64_t)1 << 40) / d->D || iz > ((int64_t)1 << 40) / d->D) return GDN_ERR_INVALID_ARG;
  if ((d->ld_x && d->ld_x < ix * d->D) || (d->ld_gate && d->ld_gate < iz * d->D)) return GDN_ERR_INVALID_ARG;
  if (d->ld_x > ((int64_t)1 << 40) || d->ld_gate > ((int64_t)1 << 40)) return GDN_ERR_INVALID_ARG;
  if (!(d->eps >= 0.f) || std::isinf(d->eps)) return GDN_ERR_INVALID_ARG;
  return GDN_OK;
}

Norm norm_of(const gdn_norm_dims* d) {
  Norm c{};
  c.rows = d->rows;
  c.D = d->D;
  c.inner_x = d->inner_x ? d->inner_x : 1;
  c.ld_x = d->ld_x ? d->ld_x : c.inner_x * d->D;
  c.inner_z = d->inner_gate ? d->inner_gate : 1;
  c.ld_z = d->ld_gate ? d->ld_gate : c.inner_z * d->D;
  c.dtype = d->dtype;
  c.rms = (d->flags & GDN_NORM_RMS) != 0;
  c.eps = d->eps;
  return c;
}

size_t norm_extent(int64_t rows, int64_t inner, int64_t ld, int64_t D, size_t es) {
  return rows ? (size_t)(((rows - 1) / inner) * ld + inner * D) * es : 0;
}

}  // namespace

extern "C" {

size_t gdn_conv_workspace_bytes(const gdn_conv_dims* d, int varlen, int pass) {
  if (check_conv(d, varlen != 0) != GDN_OK || (pass != 0 && pass != 1)) return 0;
  return conv_bytes(d, varlen != 0, pass);
}

int gdn_conv_fwd(const gdn_conv_dims* d, const void* x, const float* weight, const float* bias,
                 const int64_t* cu_seqlens, const void* initial_state, void* y, void* final_state, void* workspace,
                 size_t workspace_bytes, void* stream) {
  const bool varlen = cu_seqlens != nullptr;
  if (int rc = check_conv(d, varlen)) return rc;
  const int64_t R = d->B * d->T, n = varlen ? d->N : d->B;
  const size_t es = esize(d->dtype), st = (size_t)n * (d->W - 1) * d->D * es;
  if (((!x || !y) && R) || !weight || misaligned(x, es)) return GDN_ERR_INVALID_ARG;
  const void* ps[] = {weight, bias, cu_seqlens, initial_state, y, final_state};
  if (any_misaligned(ps, 16)) return GDN_ERR_INVALID_ARG;
  Conv c = conv_of(d, sequences(d->B, d->T, d->N, cu_seqlens, varlen, workspace));
  const size_t need = conv_bytes(d, varlen, 0), par = (size_t)d->D * sizeof(float);
  const Span outs[] = {{y, (size_t)R * d->D * es}, {final_state, st}, {workspace, need}};
  const Span ins[] = {{x, extent(R, c.ld, d->D, es)}, {weight, par * d->W}, {bias, par}, {cu_seqlens, cu_bytes(n)}, {initial_state, st}};
  if (clash(outs, ins)) return GDN_ERR_INVALID_ARG;
  if (!workspace_ok(workspace, workspace_bytes, need)) return GDN_ERR_WORKSPACE;
  c.x = x;
  c.weight = weight;
  c.bias = bias;
  c.init = initial_state;
  c.y = y;
  c.final = final_state;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (varlen)
    if (cudaError_t e = check_packing(c.seqs, s)) return status_of(e);
  return status_of(conv_forward(c, s));
}

int gdn_conv_bwd(const gdn_conv_dims* d, const void* x, const float* weight, const float* bias,
                 const int64_t* cu_seqlens, const void* initial_state, const void* dy, const void* dfinal_state, void* dx,
                 float* dweight, float* dbias, void* dinitial_state, void* workspace, size_t workspace_bytes,
                 void* stream) {
  const bool varlen = cu_seqlens != nullptr;
  if (int rc = check_conv(d, varlen)) return rc;
  const int64_t R = d->B * d->T, n = varlen ? d->N : d->B;
  const size_t es = esize(d->dtype), st = (size_t)n * (d->W - 1) * d->D * es, rows = (size_t)R * d->D * es;
  if (((!x || !dy || !dx) && R) || !weight || misaligned(x, es)) return GDN_ERR_INVALID_ARG;
  const void* ps[] = {weight, bias, cu_seqlens, initial_state, dy, dfinal_state, dx, dweight, dbias, dinitial_state};
  if (any_misaligned(ps, 16)) return GDN_ERR_INVALID_ARG;
  Conv c = conv_of(d, sequences(d->B, d->T, d->N, cu_seqlens, varlen, workspace));
  const size_t need = conv_bytes(d, varlen, 1), par = (size_t)d->D * sizeof(float);
  const Span outs[] = {{dx, rows}, {dweight, par * d->W}, {dbias, par}, {dinitial_state, st}, {workspace, need}};
  const Span ins[] = {{x, extent(R, c.ld, d->D, es)}, {weight, par * d->W}, {bias, par}, {cu_seqlens, cu_bytes(n)}, {initial_state, st},
                      {dy, rows}, {dfinal_state, st}};
  if (clash(outs, ins)) return GDN_ERR_INVALID_ARG;
  if (!workspace_ok(workspace, workspace_bytes, need)) return GDN_ERR_WORKSPACE;
  c.x = x;
  c.weight = weight;
  c.bias = bias;
  c.init = initial_state;
  c.dy = dy;
  c.dfinal = dfinal_state;
  c.dx = dx;
  c.dweight = dweight;
  c.dbias = dbias;
  c.dinit = dinitial_state;
  c.part = dweight || dbias ? reinterpret_cast<float*>(static_cast<char*>(workspace) + kAlign) : nullptr;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (varlen)
    if (cudaError_t e = check_packing(c.seqs, s)) return status_of(e);
  return status_of(conv_backward(c, s));
}

int gdn_conv_step(const gdn_conv_dims* d, const void* x, const float* weight, const float* bias, const void* state,
                  void* y, void* final_state, void* stream) {
  if (int rc = check_conv(d, false)) return rc;
  if (d->T != 1) return GDN_ERR_INVALID_ARG;
  const size_t es = esize(d->dtype), st = (size_t)d->B * (d->W - 1) * d->D * es;
  const bool states = d->W > 1;
  if (!x || !weight || !y || (states && (!state || !final_state)) || misaligned(x, es)) return GDN_ERR_INVALID_ARG;
  const void* ps[] = {weight, bias, state, y, final_state};
  if (any_misaligned(ps, 16)) return GDN_ERR_INVALID_ARG;
  if (d->B * d->D / 256 >= kMaxGrid) return GDN_ERR_INVALID_ARG;
  Conv c = conv_of(d, sequences(d->B, 1, 0, nullptr, false, nullptr));
  const size_t par = (size_t)d->D * sizeof(float);
  const Span outs[] = {{y, (size_t)d->B * d->D * es}, {final_state, st}};
  const Span ins[] = {{x, extent(d->B, c.ld, d->D, es)}, {weight, par * d->W}, {bias, par}, {state, state == final_state ? 0 : st}};
  if (clash(outs, ins)) return GDN_ERR_INVALID_ARG;
  c.x = x;
  c.weight = weight;
  c.bias = bias;
  c.init = state;
  c.y = y;
  c.final = final_state;
  return status_of(conv_step(c, static_cast<cudaStream_t>(stream)));
}

size_t gdn_ssm_workspace_bytes(const gdn_ssm_dims* d, int varlen, int pass) {
  if (check_ssm(d, varlen != 0) != GDN_OK || (pass != 0 && pass != 1)) return 0;
  const SsmPlan p = ssm_plan(d, varlen != 0);
  return pass ? p.total : p.fwd;
}

int gdn_ssm_fwd(const gdn_ssm_dims* d, const void* x, const void* dt, const float* A_log, const void* Bm, const void* Cm,
                const float* D_skip, const float* dt_bias, const int64_t* cu_seqlens, const float* initial_state, void* y,
                float* final_state, void* workspace, size_t workspace_bytes, void* stream) {
  const bool varlen = cu_seqlens != nullptr;
  if (int rc = check_ssm(d, varlen)) return rc;
  const int64_t R = d->B * d->T, n = varlen ? d->N : d->B;
  const size_t es = esize(d->dtype), st = (size_t)n * d->D * d->S * sizeof(float);
  const void* tok[] = {x, dt, Bm, Cm, y};
  if ((any_null(tok) && R) || !A_log) return GDN_ERR_INVALID_ARG;
  const void* el[] = {x, dt, Bm, Cm};
  const void* ps[] = {A_log, D_skip, dt_bias, cu_seqlens, initial_state, y, final_state};
  if (any_misaligned(el, es) || any_misaligned(ps, 16)) return GDN_ERR_INVALID_ARG;
  const SsmPlan p = ssm_plan(d, varlen);
  if (!workspace_ok(workspace, workspace_bytes, p.fwd)) return GDN_ERR_WORKSPACE;
  Ssm c = ssm_of(d, sequences(d->B, d->T, d->N, cu_seqlens, varlen, workspace), p, workspace, 0);
  const size_t par = (size_t)d->D * sizeof(float);
  const bool keeps = workspace_bytes >= p.total;  // the states for the backward
  const Span outs[] = {{y, (size_t)R * d->D * es}, {final_state, st}, {workspace, keeps ? p.total : p.fwd}};
  const Span ins[] = {{x, extent(R, c.ld_x, d->D, es)}, {dt, extent(R, c.ld_dt, d->D, es)}, {A_log, par * d->S},
                      {Bm, extent(R, c.ld_b, d->G * d->S, es)}, {Cm, extent(R, c.ld_c, d->G * d->S, es)}, {D_skip, par}, {dt_bias, par},
                      {cu_seqlens, cu_bytes(n)}, {initial_state, st}};
  if (clash(outs, ins)) return GDN_ERR_INVALID_ARG;
  c.x = x;
  c.dt = dt;
  c.A_log = A_log;
  c.Bm = Bm;
  c.Cm = Cm;
  c.skip = D_skip;
  c.dt_bias = dt_bias;
  c.init = initial_state;
  c.y = y;
  c.final = final_state;
  if (!keeps) c.ckpt = nullptr;
  c.vec = ssm_vec(c);
  c.vec_bc = ssm_vec_bc(c);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (varlen)
    if (cudaError_t e = check_packing(c.seqs, s)) return status_of(e);
  return status_of(ssm_forward(c, s));
}

int gdn_ssm_bwd(const gdn_ssm_dims* d, const void* x, const void* dt, const float* A_log, const void* Bm, const void* Cm,
                const float* D_skip, const float* dt_bias, const int64_t* cu_seqlens, const void* dy,
                const float* dfinal_state, void* dx, void* ddt, void* dB, void* dC, float* dA_log, float* dD_skip,
                float* ddt_bias, float* dinitial_state, void* workspace, size_t workspace_bytes, void* stream) {
  const bool varlen = cu_seqlens != nullptr;
  if (int rc = check_ssm(d, varlen)) return rc;
  const int64_t R = d->B * d->T, n = varlen ? d->N : d->B;
  const size_t es = esize(d->dtype), st = (size_t)n * d->D * d->S * sizeof(float);
  const void* tok[] = {x, dt, Bm, Cm, dy, dx, ddt, dB, dC};
  if ((any_null(tok) && R) || !A_log) return GDN_ERR_INVALID_ARG;
  const void* el[] = {x, dt, Bm, Cm};
  const void* ps[] = {A_log, D_skip, dt_bias, cu_seqlens, dy, dfinal_state, dx, ddt, dB, dC, dA_log, dD_skip, ddt_bias, dinitial_state};
  if (any_misaligned(el, es) || any_misaligned(ps, 16)) return GDN_ERR_INVALID_ARG;
  const SsmPlan p = ssm_plan(d, varlen);
  if (!workspace_ok(workspace, workspace_bytes, p.total)) return GDN_ERR_WORKSPACE;
  Ssm c = ssm_of(d, sequences(d->B, d->T, d->N, cu_seqlens, varlen, workspace), p, workspace, 1);
  const size_t rows = (size_t)R * d->D * es, mats = (size_t)R * d->G * d->S * es, par = (size_t)d->D * sizeof(float);
  const Span outs[] = {{dx, rows}, {ddt, rows}, {dB, mats}, {dC, mats}, {dA_log, par * d->S}, {dD_skip, par}, {ddt_bias, par},
                       {dinitial_state, st}, {workspace, p.total}};
  const Span ins[] = {{x, extent(R, c.ld_x, d->D, es)}, {dt, extent(R, c.ld_dt, d->D, es)}, {A_log, par * d->S},
                      {Bm, extent(R, c.ld_b, d->G * d->S, es)}, {Cm, extent(R, c.ld_c, d->G * d->S, es)}, {D_skip, par}, {dt_bias, par},
                      {cu_seqlens, cu_bytes(n)}, {dy, rows}, {dfinal_state, st}};
  if (clash(outs, ins)) return GDN_ERR_INVALID_ARG;
  c.x = x;
  c.dt = dt;
  c.A_log = A_log;
  c.Bm = Bm;
  c.Cm = Cm;
  c.skip = D_skip;
  c.dt_bias = dt_bias;
  c.dy = dy;
  c.dfinal = dfinal_state;
  c.dx = dx;
  c.ddt = ddt;
  c.dB = dB;
  c.dC = dC;
  c.dA_log = dA_log;
  c.dskip = dD_skip;
  c.ddt_bias = ddt_bias;
  c.dinit = dinitial_state;
  c.vec = ssm_vec(c);
  c.vec_bc = ssm_vec_bc(c);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (varlen)
    if (cudaError_t e = check_packing(c.seqs, s)) return status_of(e);
  return status_of(ssm_backward(c, s));
}

int gdn_ssm_step(const gdn_ssm_dims* d, const void* x, const void* dt, const float* A_log, const void* Bm, const void* Cm,
                 const float* D_skip, const float* dt_bias, const float* state, void* y, float* final_state,
                 void* stream) {
  if (int rc = check_ssm(d, false)) return rc;
  if (d->T != 1) return GDN_ERR_INVALID_ARG;
  const size_t es = esize(d->dtype), st = (size_t)d->B * d->D * d->S * sizeof(float);
  const void* all[] = {x, dt, A_log, Bm, Cm, state, y, final_state};
  if (any_null(all)) return GDN_ERR_INVALID_ARG;
  const void* el[] = {x, dt, Bm, Cm};
  const void* ps[] = {A_log, D_skip, dt_bias, state, y, final_state};
  if (any_misaligned(el, es) || any_misaligned(ps, 16)) return GDN_ERR_INVALID_ARG;
  Ssm c = ssm_of(d, sequences(d->B, 1, 0, nullptr, false, nullptr), SsmPlan{}, nullptr, 0);
  const size_t par = (size_t)d->D * sizeof(float);
  const Span outs[] = {{y, (size_t)d->B * d->D * es}, {final_state, st}};
  const Span ins[] = {{x, extent(d->B, c.ld_x, d->D, es)}, {dt, extent(d->B, c.ld_dt, d->D, es)}, {A_log, par * d->S},
                      {Bm, extent(d->B, c.ld_b, d->G * d->S, es)}, {Cm, extent(d->B, c.ld_c, d->G * d->S, es)}, {D_skip, par},
                      {dt_bias, par}, {state, state == final_state ? 0 : st}};
  if (clash(outs, ins)) return GDN_ERR_INVALID_ARG;
  c.x = x;
  c.dt = dt;
  c.A_log = A_log;
  c.Bm = Bm;
  c.Cm = Cm;
  c.skip = D_skip;
  c.dt_bias = dt_bias;
  c.init = state;
  c.y = y;
  c.final = final_state;
  // a state's four floats as 16 bytes; four values of B and C as one word
  c.vec = d->S % 4 == 0;
  const size_t w = 4 * es;
  c.vec_bc = d->S % 4 == 0 && c.ld_b % 4 == 0 && c.ld_c % 4 == 0 && !misaligned(Bm, w) && !misaligned(Cm, w);
  return status_of(ssm_step(c, static_cast<cudaStream_t>(stream)));
}

size_t gdn_norm_workspace_bytes(const gdn_norm_dims* d) {
  if (check_norm(d) != GDN_OK) return 0;
  return up256(norm_bwd_part_floats(d->rows, d->D) * sizeof(float)) + kAlign;
}

int gdn_norm_fwd(const gdn_norm_dims* d, const void* x, const float* weight, const float* bias, const void* gate, void* y,
                 float* stats, void* stream) {
  if (int rc = check_norm(d)) return rc;
  const size_t es = esize(d->dtype);
  if ((!x || !y) && d->rows) return GDN_ERR_INVALID_ARG;
  const void* el[] = {x, gate};
  const void* ps[] = {weight, bias, y, stats};
  if (any_misaligned(el, es) || any_misaligned(ps, 16)) return GDN_ERR_INVALID_ARG;
  Norm c = norm_of(d);
  const size_t par = (size_t)d->D * sizeof(float);
  const Span outs[] = {{y, (size_t)d->rows * d->D * es}, {stats, (size_t)d->rows * 2 * sizeof(float)}};
  const Span ins[] = {{x, norm_extent(c.rows, c.inner_x, c.ld_x, c.D, es)}, {gate, norm_extent(c.rows, c.inner_z, c.ld_z, c.D, es)},
                      {weight, par}, {bias, par}};
  if (clash(outs, ins)) return GDN_ERR_INVALID_ARG;
  c.x = x;
  c.weight = weight;
  c.bias = bias;
  c.gate = gate;
  c.y = y;
  c.stats = stats;
  return status_of(norm_forward(c, static_cast<cudaStream_t>(stream)));
}

int gdn_norm_bwd(const gdn_norm_dims* d, const void* x, const float* weight, const float* bias, const void* gate,
                 const float* stats, const void* dy, void* dx, void* dgate, float* dweight, float* dbias, void* workspace,
                 size_t workspace_bytes, void* stream) {
  if (int rc = check_norm(d)) return rc;
  const size_t es = esize(d->dtype);
  if ((!x || !dy || !dx || !stats) && d->rows) return GDN_ERR_INVALID_ARG;
  if (d->rows && (gate != nullptr) != (dgate != nullptr)) return GDN_ERR_INVALID_ARG;
  const void* el[] = {x, gate};
  const void* ps[] = {weight, bias, stats, dy, dx, dgate, dweight, dbias};
  if (any_misaligned(el, es) || any_misaligned(ps, 16)) return GDN_ERR_INVALID_ARG;
  Norm c = norm_of(d);
  const bool sums = dweight || dbias;
  const size_t rows = (size_t)d->rows * d->D * es, par = (size_t)d->D * sizeof(float), need = sums ? gdn_norm_workspace_bytes(d) : 0;
  const Span outs[] = {{dx, rows}, {dgate, rows}, {dweight, par}, {dbias, par}, {workspace, need}};
  const Span ins[] = {{x, norm_extent(c.rows, c.inner_x, c.ld_x, c.D, es)}, {gate, norm_extent(c.rows, c.inner_z, c.ld_z, c.D, es)},
                      {weight, par}, {bias, par}, {stats, (size_t)d->rows * 2 * sizeof(float)}, {dy, rows}};
  if (clash(outs, ins)) return GDN_ERR_INVALID_ARG;
  if (sums && !workspace_ok(workspace, workspace_bytes, need)) return GDN_ERR_WORKSPACE;
  c.x = x;
  c.weight = weight;
  c.bias = bias;
  c.gate = gate;
  c.stats = const_cast<float*>(stats);
  c.dy = dy;
  c.dx = dx;
  c.dgate = dgate;
  c.dweight = dweight;
  c.dbias = dbias;
  c.part = sums ? reinterpret_cast<float*>(static_cast<char*>(workspace) + kAlign) : nullptr;
  return status_of(norm_backward(c, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
