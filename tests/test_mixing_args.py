"""Refusals of the mixing-layer operators, on the CPU: what the Python calls check before anything is queued, and
what the C entry points return for bad sizes, pointers and buffers that overlap."""
import ctypes

import pytest
import torch

import gated_deltanet_chunkwise_chunk_b200 as gdn
from gated_deltanet_chunkwise_chunk_b200 import binding

lib, P = binding.lib, ctypes.c_void_p
INVALID, UNSUPPORTED, WORKSPACE = binding.GDN_ERR_INVALID_ARG, binding.GDN_ERR_UNSUPPORTED, binding.GDN_ERR_WORKSPACE
MB = 1 << 30


def at(k, off=0):
    """Distinct aligned addresses that nothing reads: every call below is refused before a launch."""
    return P((k + 1) * MB + off)


def conv(**kw):
    return binding.gdn_conv_dims(**{**dict(B=2, T=10, D=64, W=4, N=0, ld_x=0, dtype=1, flags=1), **kw})


def ssm(**kw):
    return binding.gdn_ssm_dims(**{**dict(B=2, T=10, D=64, S=16, G=1, N=0, ld_x=0, ld_dt=0, ld_b=0, ld_c=0, dtype=1), **kw})


def norm(**kw):
    return binding.gdn_norm_dims(**{**dict(rows=10, D=64, inner_x=0, ld_x=0, inner_gate=0, ld_gate=0, dtype=1, flags=0, eps=1e-5), **kw})


def conv_fwd(d, x=at(0), w=at(1), b=None, cu=None, init=None, y=at(3), fin=None, ws=at(5), n=1 << 40):
    return lib.gdn_conv_fwd(ctypes.byref(d), x, w, b, cu, init, y, fin, ws, n, None)


def conv_bwd(d, dx=at(4), dw=at(6), di=None, init=None, dfin=None, n=1 << 40):
    return lib.gdn_conv_bwd(ctypes.byref(d), at(0), at(1), None, None, init, at(3), dfin, dx, dw, None, di, at(5), n, None)


def ssm_fwd(d, x=at(0), dt=at(1), A=at(2), B=at(3), C=at(4), cu=None, init=None, y=at(6), fin=None, ws=at(8), n=1 << 60):
    return lib.gdn_ssm_fwd(ctypes.byref(d), x, dt, A, B, C, None, None, cu, init, y, fin, ws, n, None)


def ssm_bwd(d, dx=at(10), ddt=at(11), dB=at(12), dC=at(13), di=None, dfin=None, n=1 << 60):
    return lib.gdn_ssm_bwd(ctypes.byref(d), at(0), at(1), at(2), at(3), at(4), None, None, None, at(5), dfin, dx, ddt, dB, dC,
                           None, None, None, di, at(20), n, None)


def norm_fwd(d, x=at(0), y=at(1), w=None, z=None, stats=None):
    return lib.gdn_norm_fwd(ctypes.byref(d), x, w, None, z, y, stats, None)


def norm_bwd(d, x=at(0), z=None, stats=at(2), dy=at(3), dx=at(4), dz=None, dw=at(6), ws=at(7), n=1 << 40):
    return lib.gdn_norm_bwd(ctypes.byref(d), x, None, None, z, stats, dy, dx, dz, dw, None, ws, n, None)


def test_convolution_sizes():
    for kw in (dict(B=0), dict(T=-1), dict(D=0), dict(D=(1 << 20) + 1), dict(ld_x=63), dict(flags=2), dict(B=1 << 16, T=1 << 15)):
        assert conv_fwd(conv(**kw)) == INVALID, kw
        assert lib.gdn_conv_workspace_bytes(ctypes.byref(conv(**kw)), 0, 1) == 0
    for kw in (dict(W=0), dict(W=9), dict(dtype=3)):
        assert conv_fwd(conv(**kw)) == UNSUPPORTED, kw
    assert conv_fwd(conv(N=2), cu=at(9)) == INVALID  # packed sequences need a batch of 1
    assert conv_fwd(conv(B=1, N=0), cu=at(9)) == INVALID
    assert lib.gdn_conv_workspace_bytes(ctypes.byref(conv()), 0, 2) == 0
    assert lib.gdn_conv_workspace_bytes(ctypes.byref(conv()), 0, 0) == 256


def test_convolution_buffers():
    assert conv_fwd(conv(), x=None) == INVALID
    assert conv_fwd(conv(), w=None) == INVALID
    assert conv_fwd(conv(), x=at(0, 1)) == INVALID  # not even aligned to an element
    assert conv_fwd(conv(), y=at(3, 2)) == INVALID
    assert conv_fwd(conv(), y=at(0)) == INVALID  # in place: neighbours still read it
    assert conv_fwd(conv(ld_x=128), y=at(0, 128)) == INVALID  # the other half of x's rows
    assert conv_fwd(conv(), init=at(7), fin=at(7)) == INVALID
    assert conv_fwd(conv(), init=at(7), fin=at(7, 512)) == INVALID  # 2 x 3 x 64 x 2 bytes
    assert conv_fwd(conv(), n=255) == WORKSPACE
    assert conv_fwd(conv(), ws=at(5, 128)) == WORKSPACE
    assert conv_bwd(conv(), dx=at(0)) == INVALID
    assert conv_bwd(conv(), dx=at(3)) == INVALID
    assert conv_bwd(conv(), init=at(7), di=at(7)) == INVALID
    assert conv_bwd(conv(), dfin=at(7), di=at(7)) == INVALID
    assert conv_bwd(conv(), n=256) == WORKSPACE
    step = lambda d, x=at(0), st=at(2), y=at(3), fin=at(2): lib.gdn_conv_step(ctypes.byref(d), x, at(1), None, st, y, fin, None)  # noqa: E731
    assert step(conv(T=2)) == INVALID
    assert step(conv(T=1), st=None) == INVALID
    assert step(conv(T=1), fin=at(2, 64)) == INVALID  # neither the state nor apart from it
    assert step(conv(T=1), y=at(0)) == INVALID


def test_scan_sizes():
    for kw in (dict(B=0), dict(T=-1), dict(D=0), dict(G=0), dict(G=3), dict(S=0), dict(ld_x=63), dict(ld_b=15), dict(ld_c=-1),
               dict(B=1 << 16, T=1 << 15), dict(D=1 << 20, S=64, T=1), dict(B=1 << 29, T=1, D=1 << 10)):
        assert ssm_fwd(ssm(**kw)) == INVALID, kw
        assert lib.gdn_ssm_workspace_bytes(ctypes.byref(ssm(**kw)), 0, 1) == 0
    for kw in (dict(S=65), dict(dtype=7)):
        assert ssm_fwd(ssm(**kw)) == UNSUPPORTED, kw
    assert ssm_fwd(ssm(N=2), cu=at(9)) == INVALID
    d = ctypes.byref(ssm())
    assert 0 < lib.gdn_ssm_workspace_bytes(d, 0, 0) < lib.gdn_ssm_workspace_bytes(d, 0, 1)


def test_scan_buffers():
    for k in ("x", "dt", "A", "B", "C", "y"):
        assert ssm_fwd(ssm(), **{k: None}) == INVALID, k
    assert ssm_fwd(ssm(), B=at(3, 1)) == INVALID
    assert ssm_fwd(ssm(), A=at(2, 4)) == INVALID
    for k in (0, 1, 3, 4):
        assert ssm_fwd(ssm(), y=at(k)) == INVALID
    assert ssm_fwd(ssm(), init=at(9), fin=at(9)) == INVALID
    assert ssm_fwd(ssm(), n=255) == WORKSPACE
    for k in (0, 1, 3, 4, 5):
        assert ssm_bwd(ssm(), dx=at(k)) == INVALID
    assert ssm_bwd(ssm(), dC=at(12)) == INVALID  # dB's
    assert ssm_bwd(ssm(), di=at(14), dfin=at(14)) == INVALID
    assert ssm_bwd(ssm(), n=lib.gdn_ssm_workspace_bytes(ctypes.byref(ssm()), 0, 0)) == WORKSPACE  # a forward's alone
    step = lambda d, st=at(5), y=at(6), fin=at(5): lib.gdn_ssm_step(ctypes.byref(d), at(0), at(1), at(2), at(3), at(4), None, None, st, y, fin, None)  # noqa: E731
    assert step(ssm(T=3)) == INVALID
    assert step(ssm(T=1), st=None) == INVALID
    assert step(ssm(T=1), fin=at(5, 16)) == INVALID
    assert step(ssm(T=1), y=at(1)) == INVALID


def test_norm_sizes_and_buffers():
    for kw in (dict(rows=-1), dict(D=0), dict(D=(1 << 20) + 1), dict(rows=1 << 50), dict(ld_x=63), dict(inner_x=2, ld_x=127),
               dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(flags=2), dict(inner_gate=-1)):
        assert norm_fwd(norm(**kw)) == INVALID, kw
        assert lib.gdn_norm_workspace_bytes(ctypes.byref(norm(**kw))) == 0
    assert norm_fwd(norm(dtype=5)) == UNSUPPORTED
    assert norm_fwd(norm(), x=None) == INVALID
    assert norm_fwd(norm(), y=at(1, 2)) == INVALID
    assert norm_fwd(norm(), y=at(0)) == INVALID
    assert norm_fwd(norm(), z=at(1)) == INVALID
    assert norm_bwd(norm(), stats=None) == INVALID
    assert norm_bwd(norm(), z=at(8)) == INVALID  # a gate without dgate
    assert norm_bwd(norm(), dz=at(8)) == INVALID
    assert norm_bwd(norm(), dx=at(3)) == INVALID
    assert norm_bwd(norm(), z=at(8), dz=at(4)) == INVALID
    assert norm_bwd(norm(), ws=None) == WORKSPACE
    assert norm_bwd(norm(), n=64) == WORKSPACE


BF = torch.bfloat16


def _z(*s, dtype=BF):
    return torch.zeros(*s, dtype=dtype)


F = torch.float32


@pytest.mark.parametrize("kw,word", [
    (dict(x=_z(2, 3, 8, dtype=torch.float64)), "dtype"), (dict(x=_z(3, 8)), "axes"), (dict(weight=_z(8, 4)), "weight"),
    (dict(x=_z(2, 3, 16)[..., ::2]), "not contiguous"), (dict(x=_z(3, 2, 8).transpose(0, 1)), "evenly"),
    (dict(x=_z(1, 1, 8).expand(2, 3, 8)), "evenly|overlap"), (dict(bias=_z(7, dtype=F)), "bias"), (dict(activation="gelu"), "activation"),
    (dict(initial_state=_z(2, 4, 8)), "initial_state"), (dict(initial_state=_z(2, 3, 8, dtype=F)), "initial_state"),
    (dict(cu_seqlens=torch.zeros(3, dtype=torch.int64)), "batch of 1"), (dict(cu_seqlens=torch.zeros(3, dtype=torch.int32)), "cu_seqlens"),
    (dict(workspace=torch.zeros(16, dtype=torch.uint8)), "workspace"), (dict(out=_z(2, 3, 9)), "out"), (dict(), "CUDA")])
def test_convolution_tensors(kw, word):
    with pytest.raises(ValueError, match=word):
        gdn.causal_conv_fwd(**{**dict(x=_z(2, 3, 8), weight=_z(8, 4, dtype=F)), **kw})


@pytest.mark.parametrize("kw,word", [
    (dict(dt=_z(2, 3, 8, dtype=F)), "dt"), (dict(Bm=_z(2, 3, 4)), "axes"), (dict(Cm=_z(2, 3, 2, 4)), "Cm"),
    (dict(Bm=_z(2, 3, 3, 4), Cm=_z(2, 3, 3, 4)), "groups"), (dict(A_log=_z(8, 4)), "A_log"), (dict(A_log=_z(8, 5, dtype=F)), "A_log"),
    (dict(Bm=_z(2, 3, 4, 1).transpose(2, 3)[..., ::1].expand(2, 3, 1, 4)[..., [0, 1, 2, 3]].transpose(0, 1)), "Bm"),
    (dict(D=_z(7, dtype=F)), "D:"), (dict(dt_bias=_z(8)), "dt_bias"), (dict(initial_state=_z(2, 8, 5, dtype=F)), "initial_state"),
    (dict(final_state=_z(2, 8, 4)), "final_state"), (dict(workspace=torch.zeros(64, dtype=torch.uint8)), "workspace"), (dict(), "CUDA")])
def test_scan_tensors(kw, word):
    with pytest.raises(ValueError, match=word):
        gdn.ssm_scan_fwd(**{**dict(x=_z(2, 3, 8), dt=_z(2, 3, 8), A_log=_z(8, 4, dtype=F), Bm=_z(2, 3, 1, 4), Cm=_z(2, 3, 1, 4)), **kw})


def test_scan_of_too_many_states():
    with pytest.raises(gdn.GDNError):
        gdn.ssm_scan_fwd(_z(1, 2, 8), _z(1, 2, 8), _z(8, 65, dtype=F), _z(1, 2, 1, 65), _z(1, 2, 1, 65))


def test_backward_tensors():
    x, w = _z(2, 3, 8), _z(8, 4, dtype=F)
    with pytest.raises(ValueError, match="dy"):
        gdn.causal_conv_bwd(x, w, _z(2, 3, 7))
    with pytest.raises(ValueError, match="dfinal_state"):
        gdn.causal_conv_bwd(x, w, x.clone(), dfinal_state=_z(2, 2, 8))
    ins = (x, x.clone(), w, _z(2, 3, 1, 4), _z(2, 3, 1, 4))
    with pytest.raises(ValueError, match="workspace"):
        gdn.ssm_scan_bwd(*ins, x.clone(), None)
    with pytest.raises(ValueError, match="workspace"):
        gdn.ssm_scan_bwd(*ins, x.clone(), torch.zeros(256, dtype=torch.uint8))
    with pytest.raises(ValueError, match="stats"):
        gdn.layer_norm_bwd(x, x.clone(), None)
    with pytest.raises(ValueError, match="dy"):
        gdn.layer_norm_bwd(x, _z(2, 3, 8, dtype=F), _z(6, 2, dtype=F))


@pytest.mark.parametrize("kw,word", [
    (dict(x=_z(3, 0)), "not empty"), (dict(x=_z(3, 8, dtype=torch.int32)), "dtype"), (dict(x=_z(3, 16)[:, ::2]), "not contiguous"),
    (dict(x=_z(4, 3, 2, 8).permute(1, 0, 2, 3)), "evenly"), (dict(x=_z(1, 8).expand(3, 8)), "overlap"), (dict(gate=_z(3, 9)), "gate"),
    (dict(weight=_z(8)), "weight"), (dict(stats=_z(3, 1, dtype=F)), "stats"), (dict(), "CUDA")])
def test_norm_tensors(kw, word):
    with pytest.raises(ValueError, match=word):
        gdn.layer_norm_fwd(**{**dict(x=_z(3, 8)), **kw})


@pytest.mark.parametrize("shape", [(2, 1, 8), (1, 3, 8)])
def test_tokens_that_share_memory(shape):
    """A per-token tensor broadcast along one of its two token axes has too few rows in memory for the kernels."""
    x, w = _z(2, 3, 8), _z(8, 4, dtype=F)
    wide = _z(*shape).expand(2, 3, 8)
    with pytest.raises(ValueError, match="x: tokens"):
        gdn.causal_conv_fwd(wide, w)
    with pytest.raises(ValueError, match="x: tokens"):
        gdn.causal_conv_bwd(wide, w, x)
    mat = _z(2, 3, 1, 4)
    thin = _z(*shape[:2], 1, 4).expand(2, 3, 1, 4)
    for name, bad in (("x", (wide, x, w, mat, mat)), ("dt", (x, wide, w, mat, mat)), ("Bm", (x, x, w, thin, mat)),
                      ("Cm", (x, x, w, mat, thin))):
        with pytest.raises(ValueError, match=f"{name}: tokens"):
            gdn.ssm_scan_fwd(*bad)
    with pytest.raises(ValueError, match="x: rows"):
        gdn.layer_norm_fwd(wide)


def _call(fn, dims, names, given, swap, tail):
    """An entry point on distinct buffers (each far longer than needed), with buffer `swap[0]` at `swap[1]`'s address."""
    place = {n: at(100 + i) for i, n in enumerate(given)}
    place[swap[0]] = place[swap[1]]
    return getattr(lib, fn)(ctypes.byref(dims), *(place.get(n) for n in names), *tail)


OVERLAPS = [  # entry point, sizes, arguments in order, inputs, outputs, what follows
    ("gdn_conv_fwd", conv(B=1, N=2), "x weight bias cu init y final ws", "x weight bias cu init", "y final ws", (1 << 40, None)),
    ("gdn_conv_bwd", conv(B=1, N=2), "x weight bias cu init dy dfinal dx dweight dbias dinit ws", "x weight bias cu init dy dfinal",
     "dx dweight dbias dinit ws", (1 << 40, None)),
    ("gdn_conv_step", conv(T=1), "x weight bias state y final", "x weight bias state", "y final", (None,)),
    ("gdn_ssm_fwd", ssm(B=1, N=2), "x dt A Bm Cm D dt_bias cu init y final ws", "x dt A Bm Cm D dt_bias cu init", "y final ws", (1 << 60, None)),
    ("gdn_ssm_bwd", ssm(B=1, N=2), "x dt A Bm Cm D dt_bias cu dy dfinal dx ddt dB dC dA dD ddt_bias dinit ws",
     "x dt A Bm Cm D dt_bias cu dy dfinal", "dx ddt dB dC dA dD ddt_bias dinit ws", (1 << 60, None)),
    ("gdn_ssm_step", ssm(T=1), "x dt A Bm Cm D dt_bias state y final", "x dt A Bm Cm D dt_bias state", "y final", (None,)),
    ("gdn_norm_fwd", norm(), "x weight bias gate y stats", "x weight bias gate", "y stats", (None,)),
    ("gdn_norm_bwd", norm(), "x weight bias gate stats dy dx dgate dweight dbias ws", "x weight bias gate stats dy",
     "dx dgate dweight dbias ws", (1 << 40, None))]


@pytest.mark.parametrize("fn,dims,names,ins,outs,tail", OVERLAPS, ids=[o[0] for o in OVERLAPS])
def test_no_output_overlaps_another_buffer(fn, dims, names, ins, outs, tail):
    names, ins, outs = names.split(), ins.split(), outs.split()
    for o in outs:
        for other in ins + outs:
            if other == o or (o, other) == ("final", "state"):
                continue
            assert _call(fn, dims, names, ins + outs, (o, other), tail) == INVALID, (o, other)
