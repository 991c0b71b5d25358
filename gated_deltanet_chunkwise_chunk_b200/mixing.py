"""The operators of a mixing layer around its recurrence: the short causal convolution, the selective
state space scan and the (gated) layer norm.  Argument marshalling over the C entry points of
include/gdn.h, like binding.py: tensors are checked, outputs and workspaces allocated with torch, and the
work queued on the current stream of the tensors' device.

Per-token inputs may be slices of a wider projection: their last axis (for Bm and Cm the last two) is
contiguous and their tokens evenly spaced.  Gradients are computed by the matching ``*_bwd`` calls.
"""
from __future__ import annotations

import ctypes

import torch

from .binding import _TORCH_DT, GDN_OK, GDNError, gdn_conv_dims, gdn_norm_dims, gdn_ssm_dims, lib

GDN_CONV_SILU = 1
GDN_NORM_RMS = 1


def _p(t):
    return None if t is None or t.numel() == 0 else t.data_ptr()


def _call(fn, dev, *args):
    """The entry point on the current stream of `dev` (its raw handle: building a Stream object costs more than a
    small kernel takes)."""
    if dev.type != "cuda":
        raise ValueError(f"{fn}: expected CUDA tensors, got {dev}")
    stream = torch._C._cuda_getCurrentRawStream(dev.index)
    if dev.index == torch._C._cuda_getDevice():
        rc = getattr(lib, fn)(*args, stream)
    else:
        with torch.cuda.device(dev):
            rc = getattr(lib, fn)(*args, stream)
    if rc != GDN_OK:
        raise GDNError(fn, rc)


def _dtype(name, t):
    if t.dtype not in _TORCH_DT:
        raise ValueError(f"{name}: dtype {t.dtype} is not fp32, bf16 or fp16")
    return _TORCH_DT[t.dtype]


def _full(name, t, dtype, shape, dev):
    """A contiguous tensor (or None)."""
    if t is not None and (t.dtype != dtype or t.device != dev or t.shape != shape or not t.is_contiguous()):
        raise ValueError(f"{name}: expected contiguous {dtype} {tuple(shape)} on {dev}, got {t.dtype} {tuple(t.shape)} on "
                         f"{t.device} (contiguous={t.is_contiguous()})")


def _tokens(name, t, dtype, shape, dev, lead):
    """The token stride of a tensor whose first `lead` axes count tokens and whose others are one contiguous row."""
    if t.dtype != dtype or t.device != dev or t.shape != shape:
        raise ValueError(f"{name}: expected {dtype} {tuple(shape)} on {dev}, got {t.dtype} {tuple(t.shape)} on {t.device}")
    width = 1
    if t.numel() == 0:
        return 0
    for size, stride in zip(reversed(t.shape[lead:]), reversed(t.stride()[lead:])):
        if size != 1 and stride != width:
            raise ValueError(f"{name}: the row of a token is not contiguous (strides {t.stride()})")
        width *= size
    ld = None  # 0 is a stride too: that of a broadcast axis
    count = 1
    for size, stride in zip(reversed(t.shape[:lead]), reversed(t.stride()[:lead])):
        if size == 1:
            continue
        if ld is None:
            ld = stride
        elif stride != ld * count:
            raise ValueError(f"{name}: tokens are not evenly spaced (strides {t.stride()})")
        count *= size
    if ld is None:
        return width
    if ld < width:
        raise ValueError(f"{name}: tokens overlap (strides {t.stride()})")
    return ld


def _sequences(x, cu_seqlens):
    """(B, T, number of sequences) of x [B, T, ...]."""
    B, T = x.shape[0], x.shape[1]
    if cu_seqlens is None:
        return B, T, B
    n = cu_seqlens.numel() - 1
    _full("cu_seqlens", cu_seqlens, torch.int64, (n + 1,), x.device)
    if B != 1 or n < 1:
        raise ValueError(f"cu_seqlens: packed sequences need a batch of 1 (got {B}) and at least one sequence (got {n})")
    return B, T, n


def _space(fn, need, workspace, dev):
    if need == 0:
        raise GDNError(fn, 1)
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=dev)
    if workspace.dtype != torch.uint8 or workspace.device != dev or not workspace.is_contiguous() or workspace.numel() < need:
        raise ValueError(f"workspace: expected at least {need} contiguous bytes (uint8) on {dev}")
    return workspace


# ---------------------------------------------------------------------------------- convolution


def _activation(a):
    if a not in (None, "silu"):
        raise ValueError(f"activation: expected None or 'silu', got {a!r}")
    return GDN_CONV_SILU if a == "silu" else 0


def _conv_check(x, weight, bias, activation, lead):
    """Dims (sequences not set yet) of x [..., D] with `lead` token axes."""
    if x.dim() != lead + 1 or weight.dim() != 2:
        raise ValueError(f"x: expected {lead + 1} axes and weight 2, got {x.dim()} and {weight.dim()}")
    D, W = weight.shape
    dt = _dtype("x", x)
    ld = _tokens("x", x, x.dtype, (*x.shape[:-1], D), x.device, lead)
    _full("weight", weight, torch.float32, (D, W), x.device)
    _full("bias", bias, torch.float32, (D,), x.device)
    return gdn_conv_dims(1, 1, D, W, 0, ld, dt, _activation(activation))


def conv_workspace_bytes(dims, varlen, backward=False):
    return int(lib.gdn_conv_workspace_bytes(ctypes.byref(dims), int(varlen), int(backward)))


def causal_conv_fwd(x, weight, bias=None, activation="silu", cu_seqlens=None, initial_state=None,
                    output_final_state=False, out=None, final_state=None, workspace=None):
    """Short causal convolution of each channel along the sequence: x [B, T, D], weight [D, W] and bias [D]
    fp32, activation "silu" or None; states [sequences, W-1, D], the last W-1 inputs.  Returns (y, final
    state or None)."""
    d = _conv_check(x, weight, bias, activation, 2)
    d.B, d.T, d.N = B, T, n = _sequences(x, cu_seqlens)
    dev, st = x.device, (n, d.W - 1, d.D)
    _full("initial_state", initial_state, x.dtype, st, dev)
    _full("out", out, x.dtype, x.shape, dev)
    _full("final_state", final_state, x.dtype, st, dev)
    y = out if out is not None else torch.empty(x.shape, dtype=x.dtype, device=dev)
    if final_state is None and output_final_state:
        final_state = torch.empty(st, dtype=x.dtype, device=dev)
    ws = _space("gdn_conv_workspace_bytes", conv_workspace_bytes(d, cu_seqlens is not None), workspace, dev)
    _call("gdn_conv_fwd", dev, ctypes.byref(d), _p(x), _p(weight), _p(bias), _p(cu_seqlens), _p(initial_state), _p(y),
          _p(final_state), _p(ws), ws.numel())
    return y, final_state


def causal_conv_bwd(x, weight, dy, bias=None, activation="silu", cu_seqlens=None, initial_state=None,
                    dfinal_state=None, want_dinitial=True, workspace=None):
    """Backward of causal_conv_fwd for dy [B, T, D] and (optional) dfinal_state.  Returns a dict with dx,
    dweight, dbias (None without bias) and dinitial_state (None without initial_state, or if not wanted)."""
    d = _conv_check(x, weight, bias, activation, 2)
    d.B, d.T, d.N = B, T, n = _sequences(x, cu_seqlens)
    dev, st = x.device, (n, d.W - 1, d.D)
    _full("initial_state", initial_state, x.dtype, st, dev)
    _full("dy", dy, x.dtype, x.shape, dev)
    _full("dfinal_state", dfinal_state, x.dtype, st, dev)
    new = lambda shape, dtype: torch.empty(shape, dtype=dtype, device=dev)  # noqa: E731
    dx, dw = new(x.shape, x.dtype), new(weight.shape, torch.float32)
    db = new(bias.shape, torch.float32) if bias is not None else None
    di = new(st, x.dtype) if want_dinitial and initial_state is not None else None
    ws = _space("gdn_conv_workspace_bytes", conv_workspace_bytes(d, cu_seqlens is not None, True), workspace, dev)
    _call("gdn_conv_bwd", dev, ctypes.byref(d), _p(x), _p(weight), _p(bias), _p(cu_seqlens), _p(initial_state), _p(dy),
          _p(dfinal_state), _p(dx), _p(dw), _p(db), _p(di), _p(ws), ws.numel())
    return dict(dx=dx, dweight=dw, dbias=db, dinitial_state=di)


def causal_conv_step(x, state, weight, bias=None, activation="silu", out=None, final_state=None):
    """One token for each sequence: x [B, D], state [B, W-1, D].  Returns (y, final state); final_state may be
    `state` itself (updated in place), and a new tensor is made when it is not given."""
    d = _conv_check(x, weight, bias, activation, 1)
    d.B = x.shape[0]
    dev, st = x.device, (d.B, d.W - 1, d.D)
    _full("state", state, x.dtype, st, dev)
    _full("out", out, x.dtype, x.shape, dev)
    _full("final_state", final_state, x.dtype, st, dev)
    y = out if out is not None else torch.empty(x.shape, dtype=x.dtype, device=dev)
    if final_state is None:
        final_state = torch.empty(st, dtype=x.dtype, device=dev)
    if d.B:
        _call("gdn_conv_step", dev, ctypes.byref(d), _p(x), _p(weight), _p(bias), _p(state), _p(y), _p(final_state))
    return y, final_state


# ---------------------------------------------------------------------------------- selective scan


def _ssm_check(x, dt, A_log, Bm, Cm, D, dt_bias, lead):
    if x.dim() != lead + 1 or Bm.dim() != lead + 2 or A_log.dim() != 2:
        raise ValueError(f"x, Bm, A_log: expected {lead + 1}, {lead + 2} and 2 axes, got {x.dim()}, {Bm.dim()} and {A_log.dim()}")
    dev, kind, width, S, G = x.device, x.dtype, x.shape[-1], Bm.shape[-1], Bm.shape[-2]
    code = _dtype("x", x)
    lx = _tokens("x", x, kind, x.shape, dev, lead)
    lt = _tokens("dt", dt, kind, x.shape, dev, lead)
    mat = (*x.shape[:lead], G, S)
    lb, lc = _tokens("Bm", Bm, kind, mat, dev, lead), _tokens("Cm", Cm, kind, mat, dev, lead)
    _full("A_log", A_log, torch.float32, (width, S), dev)
    _full("D", D, torch.float32, (width,), dev)
    _full("dt_bias", dt_bias, torch.float32, (width,), dev)
    if G < 1 or width % G:
        raise ValueError(f"Bm: {G} groups do not divide {width} channels")
    return gdn_ssm_dims(1, 1, width, S, G, 0, lx, lt, lb, lc, code)


def ssm_dims(x, Bm, cu_seqlens=None):
    """The sizes that ssm_workspace_bytes asks for: x [B, T, D], Bm [B, T, G, S]."""
    B, T, n = _sequences(x, cu_seqlens)
    return gdn_ssm_dims(B, T, x.shape[2], Bm.shape[3], Bm.shape[2], n, 0, 0, 0, 0, _dtype("x", x))


def ssm_workspace_bytes(dims, varlen, backward=False):
    return int(lib.gdn_ssm_workspace_bytes(ctypes.byref(dims), int(varlen), int(backward)))


def ssm_scan_fwd(x, dt, A_log, Bm, Cm, D=None, dt_bias=None, cu_seqlens=None, initial_state=None,
                 output_final_state=True, out=None, final_state=None, workspace=None):
    """Selective state space scan over sequences: x, dt [B, T, D], A_log [D, S], Bm, Cm [B, T, G, S], D and
    dt_bias [D] or None, states [sequences, D, S] fp32.  Returns (y, final state or None).  For an
    ssm_scan_bwd afterwards, pass a workspace of ssm_workspace_bytes(dims, varlen, backward=True) bytes: the
    forward then keeps in it what the backward reads."""
    d = _ssm_check(x, dt, A_log, Bm, Cm, D, dt_bias, 2)
    d.B, d.T, d.N = B, T, n = _sequences(x, cu_seqlens)
    dev, st = x.device, (n, d.D, d.S)
    _full("initial_state", initial_state, torch.float32, st, dev)
    _full("out", out, x.dtype, x.shape, dev)
    _full("final_state", final_state, torch.float32, st, dev)
    y = out if out is not None else torch.empty(x.shape, dtype=x.dtype, device=dev)
    if final_state is None and output_final_state:
        final_state = torch.empty(st, dtype=torch.float32, device=dev)
    ws = _space("gdn_ssm_workspace_bytes", ssm_workspace_bytes(d, cu_seqlens is not None), workspace, dev)
    _call("gdn_ssm_fwd", dev, ctypes.byref(d), _p(x), _p(dt), _p(A_log), _p(Bm), _p(Cm), _p(D), _p(dt_bias),
          _p(cu_seqlens), _p(initial_state), _p(y), _p(final_state), _p(ws), ws.numel())
    return y, final_state


def ssm_scan_bwd(x, dt, A_log, Bm, Cm, dy, workspace, D=None, dt_bias=None, cu_seqlens=None, dfinal_state=None,
                 want_dinitial=True):
    """Backward of ssm_scan_fwd; `workspace` is the one in which that call, with the same inputs, kept its
    states.  Returns a dict with dx, ddt, dB, dC, dA_log, dD and ddt_bias (None without D, dt_bias) and
    dinitial_state (None if not wanted)."""
    d = _ssm_check(x, dt, A_log, Bm, Cm, D, dt_bias, 2)
    d.B, d.T, d.N = B, T, n = _sequences(x, cu_seqlens)
    dev, st = x.device, (n, d.D, d.S)
    _full("dy", dy, x.dtype, x.shape, dev)
    _full("dfinal_state", dfinal_state, torch.float32, st, dev)
    if workspace is None:
        raise ValueError("workspace: the backward reads the forward's")
    ws = _space("gdn_ssm_workspace_bytes", ssm_workspace_bytes(d, cu_seqlens is not None, True), workspace, dev)
    new = lambda shape, dtype=torch.float32: torch.empty(shape, dtype=dtype, device=dev)  # noqa: E731
    dx, ddt = new(x.shape, x.dtype), new(x.shape, x.dtype)
    dB, dC = new(Bm.shape, x.dtype), new(Bm.shape, x.dtype)
    dA = new(A_log.shape)
    dD = new(D.shape) if D is not None else None
    db = new(dt_bias.shape) if dt_bias is not None else None
    di = new(st) if want_dinitial else None
    _call("gdn_ssm_bwd", dev, ctypes.byref(d), _p(x), _p(dt), _p(A_log), _p(Bm), _p(Cm), _p(D), _p(dt_bias),
          _p(cu_seqlens), _p(dy), _p(dfinal_state), _p(dx), _p(ddt), _p(dB), _p(dC), _p(dA), _p(dD), _p(db), _p(di),
          _p(ws), ws.numel())
    return dict(dx=dx, ddt=ddt, dB=dB, dC=dC, dA_log=dA, dD=dD, ddt_bias=db, dinitial_state=di)


def ssm_step(x, dt, A_log, Bm, Cm, state, D=None, dt_bias=None, out=None, final_state=None):
    """One token for each sequence: x, dt [B, D], Bm, Cm [B, G, S], state [B, D, S] fp32.  Returns (y, final
    state); final_state may be `state` itself (updated in place), and a new tensor is made when it is not
    given."""
    d = _ssm_check(x, dt, A_log, Bm, Cm, D, dt_bias, 1)
    d.B = x.shape[0]
    dev, st = x.device, (d.B, d.D, d.S)
    _full("state", state, torch.float32, st, dev)
    _full("out", out, x.dtype, x.shape, dev)
    _full("final_state", final_state, torch.float32, st, dev)
    y = out if out is not None else torch.empty(x.shape, dtype=x.dtype, device=dev)
    if final_state is None:
        final_state = torch.empty(st, dtype=torch.float32, device=dev)
    if d.B:
        _call("gdn_ssm_step", dev, ctypes.byref(d), _p(x), _p(dt), _p(A_log), _p(Bm), _p(Cm), _p(D), _p(dt_bias),
              _p(state), _p(y), _p(final_state))
    return y, final_state


# ---------------------------------------------------------------------------------- layer norm


def _rows(name, t, like, dev):
    """(inner, ld) of a tensor of rows: row r starts at (r // inner) * ld + (r % inner) * D."""
    if t.dtype != like.dtype or t.device != dev or t.shape != like.shape:
        raise ValueError(f"{name}: expected {like.dtype} {tuple(like.shape)} on {dev}, got {t.dtype} {tuple(t.shape)} on {t.device}")
    D = t.shape[-1]
    if t.is_contiguous():
        return 1, D
    if D != 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: rows are not contiguous (strides {t.stride()})")
    axes = [(n, s) for n, s in zip(t.shape[:-1], t.stride()[:-1]) if n != 1]
    inner = 1
    while axes and axes[-1][1] == inner * D:
        inner *= axes.pop()[0]
    if not axes:
        return 1, D
    ld, step = axes[-1][1], axes[-1][1]
    if ld < inner * D:
        raise ValueError(f"{name}: rows overlap (strides {t.stride()})")
    for n, s in reversed(axes):
        if s != step:
            raise ValueError(f"{name}: rows are not evenly spaced (strides {t.stride()})")
        step *= n
    return inner, ld


def _norm_check(x, weight, bias, gate, rms, eps):
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("x: expected rows along a last axis that is not empty")
    D, dev, code = x.shape[-1], x.device, _dtype("x", x)
    ix, lx = _rows("x", x, x, dev)
    iz, lz = _rows("gate", gate, x, dev) if gate is not None else (0, 0)
    _full("weight", weight, torch.float32, (D,), dev)
    _full("bias", bias, torch.float32, (D,), dev)
    return gdn_norm_dims(x.numel() // D, D, ix, lx, iz, lz, code, GDN_NORM_RMS if rms else 0, eps)


def norm_workspace_bytes(dims):
    return int(lib.gdn_norm_workspace_bytes(ctypes.byref(dims)))


def layer_norm_fwd(x, weight=None, bias=None, gate=None, eps=1e-5, rms=False, out=None, output_stats=True, stats=None):
    """Layer norm over the last axis of x (rms: the mean is kept), times weight plus bias, and times silu(gate)
    where there is a gate (shaped like x).  Returns (y, stats), y contiguous, stats [rows, 2] fp32 (mean, 1/std)
    as layer_norm_bwd reads them, or None."""
    d = _norm_check(x, weight, bias, gate, rms, eps)
    dev = x.device
    _full("out", out, x.dtype, x.shape, dev)
    _full("stats", stats, torch.float32, (d.rows, 2), dev)
    y = out if out is not None else torch.empty(x.shape, dtype=x.dtype, device=dev)
    if stats is None and output_stats:
        stats = torch.empty((d.rows, 2), dtype=torch.float32, device=dev)
    _call("gdn_norm_fwd", dev, ctypes.byref(d), _p(x), _p(weight), _p(bias), _p(gate), _p(y), _p(stats))
    return y, stats


def layer_norm_bwd(x, dy, stats, weight=None, bias=None, gate=None, rms=False, workspace=None):
    """Backward of layer_norm_fwd for dy (contiguous, shaped like x) and the forward's stats.  Returns a dict
    with dx, dweight, dbias and dgate (None without weight, bias, gate)."""
    d = _norm_check(x, weight, bias, gate, rms, 0.0)
    dev = x.device
    _full("dy", dy, x.dtype, x.shape, dev)
    if stats is None:
        raise ValueError("stats: the backward reads the forward's")
    _full("stats", stats, torch.float32, (d.rows, 2), dev)
    new = lambda shape, dtype=torch.float32: torch.empty(shape, dtype=dtype, device=dev)  # noqa: E731
    dx = new(x.shape, x.dtype)
    dg = new(x.shape, x.dtype) if gate is not None else None
    dw = new((d.D,)) if weight is not None else None
    db = new((d.D,)) if bias is not None else None
    ws = None
    if dw is not None or db is not None:
        ws = _space("gdn_norm_workspace_bytes", norm_workspace_bytes(d), workspace, dev)
    _call("gdn_norm_bwd", dev, ctypes.byref(d), _p(x), _p(weight), _p(bias), _p(gate), _p(stats), _p(dy), _p(dx), _p(dg),
          _p(dw), _p(db), _p(ws), 0 if ws is None else ws.numel())
    return dict(dx=dx, dweight=dw, dbias=db, dgate=dg)
