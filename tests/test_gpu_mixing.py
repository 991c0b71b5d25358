"""The mixing-layer operators on the GPU against the fp64 references.

Tolerances are bounds, in half steps of fp32 (u = 2^-24) and of the output's type (finfo.eps / 2):
 - convolution: pre is W + 1 fused products, so it is off by (W + 2) u S, S = |bias| + sum |w x|; the silu's
   slope is at most 1.1 and its derivative's at most 0.5; the sigmoid of a 16-bit call is off by
   (16 + 3 |pre|) u relative, that of an fp32 call by less;
 - scan: the running bounds of the oracle (every token's rounding carried along by the recurrence);
 - norm: sums of D terms along chains of at most 64 terms and butterflies (L = 80; rows over 8192 elements:
   D / 1024 more), the mean and the variance to first order, rsqrt of 2 ulp.
Sums over tokens add a chain of at most `chain` terms: the strips or rows of a block, the units of 32 strands.
"""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

from oracle import mixing as om

pytestmark = pytest.mark.gpu

U = om.U
TINY = {torch.float32: 1e-35, torch.bfloat16: 1e-35, torch.float16: 2.0 ** -24}
F32, BF, FP = torch.float32, torch.bfloat16, torch.float16


def _gdn():
    import gated_deltanet_chunkwise_chunk_b200 as gdn
    return gdn


def _np(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _rand(gen, *s, dtype=F32, scale=1.0):
    return (torch.randn(*s, generator=gen, dtype=torch.float32) * scale).to(dtype).cuda()


def _close(name, got, ref, err):
    """|got - ref| <= err (before rounding) + half a step of the output's type, with 2% for second order terms."""
    half = torch.finfo(got.dtype).eps / 2
    bound = 1.02 * (err + half * (np.abs(ref) + err)) + TINY[got.dtype]
    off = np.abs(_np(got) - ref)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    assert not np.isnan(off).any(), name
    assert (off <= bound).all(), f"{name}: {float((off / bound).max()):.3f} times its bound"


def _cu(lengths):
    return [0] + [int(v) for v in np.cumsum(lengths)]


def _shape(lengths, packed):
    return (1, sum(lengths)) if packed else (len(lengths), lengths[0])


# ------------------------------------------------------------------------------- convolution


def _conv_case(seed, lengths, packed, D, W, dtype, state, bias, silu, wide):
    gen = torch.Generator().manual_seed(seed)
    shape = _shape(lengths, packed)
    x = _rand(gen, *shape, D + wide, dtype=dtype)[..., :D]
    c = dict(x=x, weight=_rand(gen, D, W, scale=0.5), bias=_rand(gen, D) if bias else None, activation="silu" if silu else None,
             cu_seqlens=torch.tensor(_cu(lengths), device="cuda") if packed else None,
             initial_state=_rand(gen, len(lengths), W - 1, D, dtype=dtype) if state else None)
    return c, _rand(gen, *shape, D, dtype=dtype), _rand(gen, len(lengths), W - 1, D, dtype=dtype) if state else None


def _conv_check(c, dy, dfin, lengths):
    gdn = _gdn()
    x, D, W = c["x"], c["x"].shape[-1], c["weight"].shape[1]
    cu, silu, R = _cu(lengths), c["activation"] == "silu", sum(lengths)
    y, fin = gdn.causal_conv_fwd(**c, output_final_state=True)
    g = gdn.causal_conv_bwd(c["x"], c["weight"], dy, c["bias"], c["activation"], c["cu_seqlens"], c["initial_state"], dfin)
    torch.cuda.synchronize()
    flat = lambda t: None if t is None else _np(t).reshape(R, D)  # noqa: E731
    xn, w, b, init, dyn = flat(x), _np(c["weight"]), _np(c["bias"]), _np(c["initial_state"]), flat(dy)
    ry, rfin, pre, _ = om.conv_fwd(xn, w, b, cu, init, silu)
    _, _, S, _ = om.conv_fwd(np.abs(xn), np.abs(w), None if b is None else np.abs(b), cu, None if init is None else np.abs(init), False)
    E = (W + 2) * U * S
    _close("y", y, ry.reshape(y.shape), (1.1 * E + np.abs(ry) * (16 + 3 * np.abs(pre)) * U).reshape(y.shape))
    assert np.array_equal(_np(fin), rfin)
    r = om.conv_bwd(xn, w, b, cu, dyn, init, _np(dfin), silu)
    Ed = np.abs(dyn) * (0.5 * E + (1 + np.abs(pre)) * (20 + 3 * np.abs(pre)) * U) if silu else U * np.abs(dyn)
    # the same adjoint, with the errors and magnitudes in the place of the values
    Edp = om.conv_bwd(np.abs(xn), np.abs(w), None, cu, Ed + (W + 2) * U * np.abs(r["dpre"]), None, None, False)
    Edi = om.conv_bwd(np.abs(xn), np.abs(w), None, cu, Ed, None if init is None else np.abs(init), None, False)
    mag = om.conv_bwd(np.abs(xn), np.abs(w), None, cu, np.abs(r["dpre"]), None if init is None else np.abs(init), None, False)
    lanes = 32
    chain = 16 + 256 + R // (32 * 16) + len(lengths) // 32 + 64
    assert lanes == 32
    _close("dx", g["dx"], r["dx"].reshape(y.shape), (Edp["dx"] + 2 * U * np.abs(r["dx"])).reshape(y.shape))
    _close("dweight", g["dweight"], r["dweight"], Edi["dweight"] + chain * U * mag["dweight"])
    if b is None:
        assert g["dbias"] is None
    else:
        _close("dbias", g["dbias"], r["dbias"], Ed.sum(0) + chain * U * np.abs(r["dpre"]).sum(0))
    if init is None:
        assert g["dinitial_state"] is None
    else:
        _close("dinitial_state", g["dinitial_state"], r["dinitial_state"], Edp["dinitial_state"] + 2 * U * np.abs(r["dinitial_state"]))


CONV = [  # lengths, packed, D, W
    ([1], False, 8, 4), ([0, 0], False, 16, 4), ([3, 3], False, 5, 4), ([65], False, 64, 2), ([130, 130], False, 264, 4),
    ([2, 0, 1, 70, 5], True, 48, 4), ([0, 300, 0], True, 257, 3), ([1, 1, 1, 1, 16, 15, 17], True, 8, 8), ([40], True, 2056, 5),
    ([0], True, 8, 1), ([33, 31], True, 12, 1), ([20], False, 1, 6), ([257], False, 20, 7)]


@pytest.mark.parametrize("dtype", [F32, BF, FP])
@pytest.mark.parametrize("lengths,packed,D,W", CONV)
def test_convolution(lengths, packed, D, W, dtype):
    for k, (state, bias, silu, wide) in enumerate([(True, True, True, 0), (False, False, False, 8), (True, False, True, 3)]):
        c, dy, dfin = _conv_case(len(lengths) + D + k, lengths, packed, D, W, dtype, state, bias, silu, wide)
        _conv_check(c, dy, dfin, lengths)


@pytest.mark.parametrize("dtype", [F32, BF, FP])
@pytest.mark.parametrize("B,D,W,in_place", [(1, 8, 4, True), (3, 33, 4, False), (70, 256, 2, True), (2, 40, 1, True), (5, 17, 8, True)])
def test_convolution_step(B, D, W, in_place, dtype):
    """A step is the sequence form's token, and its state the sequence form's."""
    gdn = _gdn()
    gen = torch.Generator().manual_seed(B)
    x, st = _rand(gen, B, 1, D, dtype=dtype), _rand(gen, B, W - 1, D, dtype=dtype)
    w, b = _rand(gen, D, W), _rand(gen, D)
    y, fin = gdn.causal_conv_fwd(x, w, b, initial_state=st, output_final_state=True)
    y1, fin1 = gdn.causal_conv_step(x[:, 0], st, w, b, final_state=st if in_place else None)
    assert fin1 is st or not in_place
    assert torch.equal(y[:, 0], y1) and torch.equal(fin, fin1)


def test_convolution_keeps_what_it_does_not_see_apart():
    """Infinities and NaN before a sequence, in another sequence's tokens, in the rest of x's rows and in unused
    state slots reach no output."""
    gdn = _gdn()
    gen = torch.Generator().manual_seed(5)
    D = 16
    for W in (2, 4):
        buf = _rand(gen, 1, 40, 2 * D, dtype=BF)
        buf[..., D:] = float("nan")
        x = buf[..., :D]
        x[0, :9] = float("inf")
        w = _rand(gen, D, W)
        cu = torch.tensor([0, 9, 9, 40], device="cuda")
        y, fin = gdn.causal_conv_fwd(x, w, cu_seqlens=cu, output_final_state=True)
        g = gdn.causal_conv_bwd(x, w, torch.ones_like(x).contiguous(), cu_seqlens=cu)
        alone, _ = gdn.causal_conv_fwd(x[:, 9:].contiguous(), w)
        assert torch.equal(y[:, 9:], alone) and torch.isfinite(g["dx"][:, 9:].float()).all()
        assert (fin[1] == 0).all()


# ---------------------------------------------------------------------------------- scan


def _scan_case(seed, lengths, packed, D, N, G, dtype, full=True, strided=False):
    gen = torch.Generator().manual_seed(seed)
    shape, n = _shape(lengths, packed), len(lengths)
    x, dt = _rand(gen, *shape, D + 3 * strided, dtype=dtype)[..., :D], _rand(gen, *shape, D + 5 * strided, dtype=dtype)[..., :D]
    bc = _rand(gen, *shape, 2 * G * N, dtype=dtype)
    Bm, Cm = (bc[..., k * G * N:(k + 1) * G * N].unflatten(-1, (G, N)) for k in (0, 1))
    c = dict(x=x, dt=dt, A_log=_rand(gen, D, N, scale=0.7), Bm=Bm, Cm=Cm, D=_rand(gen, D) if full else None,
             dt_bias=_rand(gen, D) - 1 if full else None, cu_seqlens=torch.tensor(_cu(lengths), device="cuda") if packed else None)
    init = _rand(gen, n, D, N) if full else None
    return c, init, _rand(gen, *shape, D, dtype=dtype), _rand(gen, n, D, N) if full else None


def _scan_run(c, init, dy, dfin):
    gdn = _gdn()
    dims = gdn.ssm_dims(c["x"], c["Bm"], c["cu_seqlens"])
    ws = torch.empty(gdn.ssm_workspace_bytes(dims, c["cu_seqlens"] is not None, True), dtype=torch.uint8, device="cuda")
    y, fin = gdn.ssm_scan_fwd(**c, initial_state=init, workspace=ws)
    ins = (c["x"], c["dt"], c["A_log"], c["Bm"], c["Cm"])
    g = gdn.ssm_scan_bwd(*ins, dy, ws, D=c["D"], dt_bias=c["dt_bias"], cu_seqlens=c["cu_seqlens"], dfinal_state=dfin)
    return dict(y=y, state=fin, **g)


def _scan_check(c, init, dy, dfin, lengths):
    got = _scan_run(c, init, dy, dfin)
    y2, fin2 = _gdn().ssm_scan_fwd(**c, initial_state=init)  # a prompt's call, without the backward's states
    assert torch.equal(y2, got["y"]) and torch.equal(fin2, got["state"])
    R, D = sum(lengths), c["x"].shape[-1]
    G, N = c["Bm"].shape[-2:]
    flat = lambda t, *s: _np(t).reshape(R, *s)  # noqa: E731
    # a join's decay: the sum of a segment's deltas is off by a chain of T / 32 + 5, x e^-x <= 0.37
    extra = 0.37 * (max(lengths) / 32 + 6)
    val, err = om.ssm(flat(c["x"], D), flat(c["dt"], D), _np(c["A_log"]), flat(c["Bm"], G, N), flat(c["Cm"], G, N), _np(c["D"]),
                      _np(c["dt_bias"]), _cu(lengths), _np(init), flat(dy, D), _np(dfin), extra)
    for k, v in got.items():
        if v is None:
            assert k in ("dD", "ddt_bias")
            continue
        _close(k, v, val[k].reshape(v.shape), err[k].reshape(v.shape))


SCAN = [  # lengths, packed, D, N, G
    ([1], False, 8, 16, 1), ([0, 0], False, 8, 4, 1), ([3, 3], False, 6, 5, 2), ([33], False, 40, 16, 1), ([64, 64], False, 72, 16, 1),
    ([2, 0, 1, 40, 5], True, 32, 16, 1), ([0, 47, 0], True, 33, 9, 1), ([16, 17, 15, 1], True, 64, 8, 4), ([31], True, 130, 32, 1),
    ([32, 33], True, 24, 64, 2), ([0], True, 16, 16, 1), ([20], False, 7, 1, 7), ([35, 35], False, 48, 24, 3), ([18], False, 9, 64, 1)]


@pytest.mark.parametrize("dtype", [F32, BF, FP])
@pytest.mark.parametrize("lengths,packed,D,N,G", SCAN)
def test_scan(lengths, packed, D, N, G, dtype):
    for full, strided in ((True, False), (False, True)):
        _scan_check(*_scan_case(D + N, lengths, packed, D, N, G, dtype, full, strided), lengths)


@pytest.mark.parametrize("lengths,packed,D,N", [([700], False, 8, 16), ([300, 5, 0, 530], True, 16, 16), ([400, 400], False, 4, 3)])
def test_scan_of_long_sequences(lengths, packed, D, N):
    """Few channels and many tokens: sequences are cut along time where that makes the call faster."""
    _scan_check(*_scan_case(3, lengths, packed, D, N, 1, F32), lengths)


@pytest.mark.parametrize("lengths,packed,D,N,G", [([900], False, 8, 16, 1), ([2000, 3, 0, 1100], True, 16, 16, 2), ([1025, 1025], False, 4, 5, 1),
                                                  ([800], True, 3, 33, 1)])
def test_scan_cut_in_both_directions(lengths, packed, D, N, G):
    """Long enough that the forward is cut along time too, with tails of odd lengths and an empty sequence between."""
    for dtype in (F32, BF):
        _scan_check(*_scan_case(5, lengths, packed, D, N, G, dtype), lengths)


@pytest.mark.parametrize("lengths,packed,D,N,G", [([900], False, 8, 5, 1), ([1025, 1025], False, 6, 24, 2), ([2000, 3, 0, 1100], True, 16, 33, 1),
                                                  ([800], True, 3, 9, 1), ([300, 300], False, 4, 3, 1)])
def test_cut_scan_reads_only_what_it_wrote(lengths, packed, D, N, G):
    """A workspace full of NaN bits changes nothing: sequences cut along time, with states that do not fill a lane's four."""
    gdn = _gdn()
    for dtype in (F32, BF):
        c, init, dy, dfin = _scan_case(6, lengths, packed, D, N, G, dtype)
        ins, rest = (c["x"], c["dt"], c["A_log"], c["Bm"], c["Cm"]), dict(D=c["D"], dt_bias=c["dt_bias"], cu_seqlens=c["cu_seqlens"])
        need = gdn.ssm_workspace_bytes(gdn.ssm_dims(c["x"], c["Bm"], c["cu_seqlens"]), packed, True)
        got = []
        for fill in (0, 255):
            ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
            y, fin = gdn.ssm_scan_fwd(*ins, **rest, initial_state=init, workspace=ws)
            got.append(dict(y=y, state=fin, **gdn.ssm_scan_bwd(*ins, dy, ws, **rest, dfinal_state=dfin)))
        for k in got[0]:
            assert torch.isfinite(got[0][k].float()).all() and torch.equal(got[0][k], got[1][k]), k


@pytest.mark.parametrize("dtype", [F32, BF, FP])
@pytest.mark.parametrize("B,D,N,G,in_place", [(1, 8, 16, 1, True), (3, 33, 16, 1, False), (9, 24, 5, 2, True), (2, 40, 64, 1, True), (70, 16, 32, 4, False),
                                             (301, 2048, 16, 1, True), (130, 4096, 8, 2, False), (90, 4100, 12, 1, True)])
def test_scan_step(B, D, N, G, in_place, dtype):
    gdn = _gdn()
    c, st, _, _ = _scan_case(B + N, [1] * B, False, D, N, G, dtype)
    val, err = om.ssm(_np(c["x"][:, 0]), _np(c["dt"][:, 0]), _np(c["A_log"]), _np(c["Bm"][:, 0]), _np(c["Cm"][:, 0]), _np(c["D"]),
                      _np(c["dt_bias"]), list(range(B + 1)), _np(st))
    ins = (c["x"][:, 0], c["dt"][:, 0], c["A_log"], c["Bm"][:, 0], c["Cm"][:, 0], st)
    y, fin = gdn.ssm_step(*ins, D=c["D"], dt_bias=c["dt_bias"], final_state=st if in_place else None)
    assert fin is st or not in_place
    _close("y", y, val["y"], err["y"])
    _close("state", fin, val["state"], err["state"])


@pytest.mark.parametrize("dtype", [F32, BF, FP])
@pytest.mark.parametrize("B,D,N,G", [(440, 2048, 4, 1), (430, 2050, 8, 2), (101, 4096, 12, 4), (61, 4096, 32, 1), (41, 4100, 64, 2)])
def test_scan_step_of_many_requests(B, D, N, G, dtype):
    """Enough requests for the states to travel through the threads' rings (at least sixteen for each of the grid's rows of
    blocks), for every number of lanes to a channel."""
    across = -(-D * max(2, 2 ** int(np.ceil(np.log2(N))) // 4) // 256)
    assert (B + 3) // 4 >= 4 * max(1, 148 * 3 // across) and N % 4 == 0
    test_scan_step(B, D, N, G, True, dtype)


def test_scan_extremes():
    """Steps above 20, decays of 0 and 1 and sequences beside infinite ones."""
    c, init, dy, dfin = _scan_case(1, [50, 30], True, 16, 16, 1, F32)
    c["dt"][0, 3] = 25.0
    c["dt"][0, 60] = -80.0
    c["A_log"][0] = 6.0
    c["A_log"][1] = -60.0
    _scan_check(c, init, dy, dfin, [50, 30])
    before = _scan_run(c, init, dy, dfin)
    c["x"][0, 49] = float("inf")
    c["dt"][0, 48] = float("nan")
    dy[0, 20] = float("nan")
    after = _scan_run(c, init, dy, dfin)
    for k in ("y", "dx", "ddt", "dB", "dC"):
        assert torch.equal(before[k][0, 50:], after[k][0, 50:]), k
    assert torch.equal(before["y"][0, :48], after["y"][0, :48])
    for k in ("state", "dinitial_state"):
        assert torch.equal(before[k][1], after[k][1]), k
    c["A_log"][2] = 100.0  # exp overflows: the state is the last input alone
    c["x"][0, 49] = 1.0
    c["dt"][0, 48] = 1.0
    y, fin = _gdn().ssm_scan_fwd(**c, initial_state=init)
    assert torch.isfinite(y).all() and torch.isfinite(fin).all()


@pytest.mark.parametrize("dtype", [F32, BF, FP])
@pytest.mark.parametrize("lengths,D", [([50, 30], 16), ([900, 40], 8), ([33, 0], 40)])
def test_scan_of_nan_rates(lengths, D, dtype):
    """A NaN in A_log reaches all that its state enters, in both forms, and nothing else."""
    gdn = _gdn()
    N, ch, st = 16, 3, 5
    c, init, dy, dfin = _scan_case(2, lengths, True, D, N, 1, dtype)
    before = _scan_run(c, init, dy, dfin)
    c["A_log"][ch, st] = float("nan")
    after = _scan_run(c, init, dy, dfin)
    rest = [d for d in range(D) if d != ch]
    for k in ("y", "dx", "ddt"):
        assert torch.equal(before[k][..., rest], after[k][..., rest]), k
    assert after["y"][..., ch].isnan().all()
    for k in ("state", "dinitial_state"):
        wrong = after[k] != before[k]
        assert all(after[k][s, ch, st].isnan() for s, n in enumerate(lengths) if n > 0), k
        wrong[[s for s, n in enumerate(lengths) if n > 0], ch, st] = False
        assert not wrong.any(), k
    assert after["dA_log"][ch, st].isnan() and after["ddt_bias"][ch].isnan()
    B = 3
    c, s0, _, _ = _scan_case(2, [1] * B, False, D, N, 1, dtype)
    ins = (c["x"][:, 0], c["dt"][:, 0], c["A_log"], c["Bm"][:, 0], c["Cm"][:, 0], s0)
    y, fin = gdn.ssm_step(*ins, D=c["D"], dt_bias=c["dt_bias"])
    c["A_log"][ch, st] = float("nan")
    y2, fin2 = gdn.ssm_step(*ins, D=c["D"], dt_bias=c["dt_bias"])
    assert y2[:, ch].isnan().all() and fin2[:, ch, st].isnan().all()
    assert torch.equal(y[:, rest], y2[:, rest]) and torch.equal(fin[:, rest], fin2[:, rest])


@pytest.mark.parametrize("dtype", [F32, BF, FP])
@pytest.mark.parametrize("lengths,D,at", [([30, 50], 16, 40), ([40, 900], 8, 700), ([5, 300], 8, 20)])
def test_scan_backward_of_nan_steps(lengths, D, at, dtype):
    """A NaN step is in every gradient that passes back through it: dx and ddt of its sequence's earlier tokens and the
    initial state's gradient of its channel.  Later tokens' dx, other channels and other sequences do not see it."""
    c, init, dy, dfin = _scan_case(4, lengths, True, D, 16, 1, dtype)
    ch, lo = 2, lengths[0]
    before = _scan_run(c, init, dy, dfin)
    c["dt"][0, at, ch] = float("nan")
    after = _scan_run(c, init, dy, dfin)
    rest = [d for d in range(D) if d != ch]
    for k in ("dx", "ddt"):
        assert after[k][0, lo:at + 1, ch].isnan().all(), k
        assert torch.equal(before[k][..., rest], after[k][..., rest]) and torch.equal(before[k][0, :lo], after[k][0, :lo]), k
    assert torch.equal(before["dx"][0, at + 1:], after["dx"][0, at + 1:])
    g = after["dinitial_state"]
    assert g[1, ch].isnan().all() and torch.equal(g[0], before["dinitial_state"][0]) and torch.equal(g[1, rest], before["dinitial_state"][1, rest])


@pytest.mark.parametrize("dtype", [F32, BF, FP])
@pytest.mark.parametrize("lengths,D", [([50, 30], 16), ([33], 40), ([900], 8)])
def test_scan_of_rates_past_fp32(lengths, D, dtype):
    """exp(A_log) near and beyond the largest fp32: the state is the last input alone, and the gradients are as finite
    as the formulas', behind a sequence's last token (segments do not end on a tile) too."""
    c, init, dy, dfin = _scan_case(8, lengths, True, D, 16, 1, dtype)
    c["A_log"][1] = 100.0
    c["A_log"][2, 3:] = 88.0
    c["A_log"][5, ::2] = 95.0
    c["dt"].clamp_(min=-2.0)  # with the bias: steps of 1e-3 and more, whose decays are 0 at these rates
    c["dt_bias"].clamp_(min=-4.0)
    _scan_check(c, init, dy, 30 * dfin, lengths)


@pytest.mark.parametrize("dtype", [F32, BF, FP])
def test_sums_over_a_long_whole_sequence(dtype):
    """A sequence that is not cut along time (208 blocks): the parameters' gradients over its 6000 tokens are added
    by rows of 256 tokens: a running sum of 128 pairs, a butterfly of the lanes, then 24 rows in 8 strands (160 additions at
    most).  The skip's terms are exact products and all equal, so that one running sum over the sequence would round the
    same way at every token: 674 half ulps."""
    T, D, N = 6000, 208, 2
    c, init, dy, dfin = _scan_case(1, [T], False, D, N, D, dtype)
    c["x"].fill_(1 + 2.0 ** -7)
    dy.fill_(1 + 2.0 ** -7)
    got = _scan_run(c, init, dy, dfin)
    flat = lambda t, *s: _np(t).reshape(T, *s)  # noqa: E731
    val, err = om.ssm(flat(c["x"], D), flat(c["dt"], D), _np(c["A_log"]), flat(c["Bm"], D, N), flat(c["Cm"], D, N), _np(c["D"]),
                      _np(c["dt_bias"]), [0, T], _np(init), flat(dy, D), _np(dfin), chain=160)
    for k in ("dD", "dA_log", "ddt_bias"):
        _close(k, got[k], val[k], err[k])


@pytest.mark.parametrize("dtype", [BF, FP])
def test_decays_of_16_bit_calls_have_little_bias(dtype):
    """States that only decay, in a 16-bit call against the same values in an fp32 call, whose exponential has no bias: a
    token's relative error averaged over decays of 2^-14 to 2^-1 octaves.  The hardware's exponential is low there by
    1.4e-8 on average; the offset of its argument takes 9.7e-9 of that out and has to leave less than it took.  (A
    channel's error is up to 2^-23 at every token, the same each time: over 4096 channels 2e-9 at three deviations; the
    fp32 exponential's own average is below 2e-9.)"""
    gdn = _gdn()
    T, D = 128, 4096
    t = -torch.exp2(torch.linspace(-14, -1, D, dtype=torch.float64)) * np.log(2.0)  # log of the decay
    bias = torch.log(torch.expm1(-t)).float().cuda()  # its softplus is the step
    got = []
    for kind in (dtype, F32):
        z = torch.zeros(1, T, D, dtype=kind, device="cuda")
        mat = torch.zeros(1, T, 1, 1, dtype=kind, device="cuda")
        _, st = gdn.ssm_scan_fwd(z, z, torch.zeros(D, 1, device="cuda"), mat, mat, dt_bias=bias,
                                 initial_state=torch.ones(1, D, 1, device="cuda"))
        got.append(_np(st).ravel())
    live = got[1] > 1e-30
    off = (got[0][live] / got[1][live] - 1) / T
    assert live.sum() > 3500 and np.abs(off).max() <= 2 * 2.0 ** -23
    assert abs(off.mean()) <= 9.7e-9, off.mean()


@pytest.mark.parametrize("dtype", [F32, BF, FP])
@pytest.mark.parametrize("T", [1, 33, 900])
def test_steps_of_zero_keep_the_state(T, dtype):
    """A step that underflows to 0 decays by exactly 1: the state's bits stay, whole or cut along time, and in single tokens."""
    gdn = _gdn()
    D, N = 24, 16
    c, init, _, _ = _scan_case(3, [T], False, D, N, 1, dtype)
    c["dt"].fill_(-1000.0)
    y, fin = gdn.ssm_scan_fwd(**c, initial_state=init)
    assert torch.equal(fin, init)
    ins = (c["x"][:, 0], c["dt"][:, 0], c["A_log"], c["Bm"][:, 0], c["Cm"][:, 0], init)
    assert torch.equal(gdn.ssm_step(*ins, D=c["D"], dt_bias=c["dt_bias"])[1], init)


def _short_memory(T, D, dtype):
    """Inputs whose states forget within a few tokens (delta A <= -3 for every state), so that a call's last tokens
    can be computed from the few before them."""
    gen = torch.Generator().manual_seed(T)
    x = torch.empty(1, T, D, dtype=dtype, device="cuda").uniform_(-1, 1)
    dt = torch.full((1, T, D), 3.0, dtype=dtype, device="cuda")
    Bm, Cm = (torch.empty(1, T, 1, 4, dtype=dtype, device="cuda").uniform_(-1, 1) for _ in range(2))
    return x, dt, torch.zeros(D, 4, device="cuda"), Bm, Cm, _rand(gen, D)


def test_offsets_past_32_bits():
    """Tensors of more than 2^31 elements: the ends of a call's tensors agree with a short call on them."""
    gdn = _gdn()
    D, T = 2048, (1 << 20) + 40
    x, dt, A_log, Bm, Cm, skip = _short_memory(T, D, BF)
    y, st = gdn.ssm_scan_fwd(x, dt, A_log, Bm, Cm, skip)
    tail = [t[:, -64:].contiguous() for t in (x, dt, Bm, Cm)]
    y2, st2 = gdn.ssm_scan_fwd(tail[0], tail[1], A_log, tail[2], tail[3], skip)
    # 32 tokens back a state is e^-96 of itself, far below half a step of its fp32 value
    assert torch.equal(y[:, -32:], y2[:, -32:]) and torch.equal(st, st2)
    del dt, y, Bm, Cm
    gen = torch.Generator().manual_seed(1)
    w, b = _rand(gen, D, 4), _rand(gen, D)
    y, fin = gdn.causal_conv_fwd(x, w, b, output_final_state=True)
    y2, fin2 = gdn.causal_conv_fwd(tail[0], w, b, output_final_state=True)
    assert torch.equal(y[:, -60:], y2[:, -60:]) and torch.equal(fin, fin2)
    g = gdn.causal_conv_bwd(x, w, y, b)
    g2 = gdn.causal_conv_bwd(tail[0], w, y[:, -64:].contiguous(), b)
    assert torch.equal(g["dx"][:, -60:], g2["dx"][:, -60:])
    del g
    n, stats = gdn.layer_norm_fwd(x, w[:, 0].contiguous(), rms=True)
    n2, stats2 = gdn.layer_norm_fwd(tail[0], w[:, 0].contiguous(), rms=True)
    # (a different split of a row over threads: the same to the rounding of its sums)
    half = torch.finfo(BF).eps
    assert (n[:, -64:].float() - n2.float()).abs().max() <= half * n2.float().abs().max()
    g = gdn.layer_norm_bwd(x, y, stats, w[:, 0].contiguous(), rms=True)
    g2 = gdn.layer_norm_bwd(tail[0], y[:, -64:].contiguous(), stats2, w[:, 0].contiguous(), rms=True)
    assert (g["dx"][:, -64:].float() - g2["dx"].float()).abs().max() <= half * g2["dx"].float().abs().max()


# ---------------------------------------------------------------------------------- norm


def _norm_check(x, w, b, z, dy, eps, rms):
    gdn = _gdn()
    y, stats = gdn.layer_norm_fwd(x, w, b, gate=z, eps=eps, rms=rms)
    g = gdn.layer_norm_bwd(x, dy, stats, w, b, gate=z, rms=rms)
    torch.cuda.synchronize()
    D = x.shape[-1]
    rows = x.numel() // D
    r2 = lambda t: None if t is None else _np(t).reshape(rows, D)  # noqa: E731
    xn, zn, dyn, wn, bn = r2(x), r2(z), r2(dy), _np(w), _np(b)
    ry, mu, rstd, n = om.norm_fwd(xn, wn, bn, zn, eps, rms)
    rg = om.norm_bwd(xn, dyn, wn, bn, zn, eps, rms)
    L = 80 + D // 1024
    mean = lambda v: v.mean(-1, keepdims=True)  # noqa: E731
    d = np.abs(xn - mu)
    Em = 0 * mu if rms else (L + 2) * U * mean(np.abs(xn))
    Er = rstd ** 2 * ((L + 4) * U * mean(d * d) + 2 * mean(d) * Em) / 2 + 6 * U  # relative, of rstd
    xh = (xn - mu) * rstd
    Eh = rstd * (Em + U * d) + np.abs(xh) * (Er + U)
    wa = 1 if wn is None else np.abs(wn)
    En = wa * Eh + 2 * U * (np.abs(n) + (0 if bn is None else np.abs(bn)))
    Esg = 0 if zn is None else (16 + 3 * np.abs(zn)) * U
    sl = 1 if zn is None else zn * om.sigmoid(zn)
    _close("y", y, ry.reshape(x.shape), (np.abs(sl) * En + np.abs(ry) * (Esg + 2 * U)).reshape(x.shape))
    _close("mean", stats[:, :1], mu, Em)
    _close("rstd", stats[:, 1:], rstd, rstd * Er)
    dn = dyn * sl
    Edn = np.abs(dn) * (Esg + 2 * U)
    if zn is not None:
        s = om.sigmoid(zn)
        q = s * (1 + zn * (1 - s))
        Edz = np.abs(dyn) * (np.abs(q) * En + np.abs(n) * s * (1 + np.abs(zn)) * (20 + 3 * np.abs(zn)) * U)
        _close("dgate", g["dgate"], rg["dgate"].reshape(x.shape), (Edz + 4 * U * np.abs(rg["dgate"])).reshape(x.shape))
    u = dn * (1 if wn is None else wn)
    Eu = Edn * wa + U * np.abs(u)
    Ea0 = 0 if rms else mean(Eu) + (L + 2) * U * mean(np.abs(u))
    a1 = mean(u * xh)
    Ea1 = mean(Eu * np.abs(xh) + np.abs(u) * Eh) + (L + 2) * U * mean(np.abs(u * xh))
    inner = Eu + Ea0 + np.abs(xh) * Ea1 + np.abs(a1) * Eh + 3 * U * (np.abs(u) + (0 if rms else np.abs(mean(u))) + np.abs(xh * a1))
    _close("dx", g["dx"], rg["dx"].reshape(x.shape), (rstd * inner + np.abs(rg["dx"]) * (Er + U)).reshape(x.shape))
    chain = rows // 128 + 256 + 32 + 16
    if w is not None:
        _close("dweight", g["dweight"], rg["dweight"], (Edn * np.abs(xh) + np.abs(dn) * Eh).sum(0) + chain * U * np.abs(dn * xh).sum(0))
    if b is not None:
        _close("dbias", g["dbias"], rg["dbias"], Edn.sum(0) + chain * U * np.abs(dn).sum(0))


NORM = [(1, 1), (5, 7), (3, 64), (64, 128), (1000, 128), (17, 256), (9, 333), (33, 512), (6, 520), (5, 1000), (7, 1999), (40, 2048),
        (3, 4096), (2, 5001), (4, 8192), (2, 8200), (2, 12288), (1, 16400), (700, 96)]


@pytest.mark.parametrize("dtype", [F32, BF, FP])
@pytest.mark.parametrize("rows,D", NORM)
def test_norm(rows, D, dtype):
    for k, (rms, gated, wb) in enumerate([(False, False, 3), (True, True, 1), (False, True, 3), (True, False, 2), (False, False, 0)]):
        gen = torch.Generator().manual_seed(rows + D + k)
        x = _rand(gen, rows, D, dtype=dtype) * 1.5 + 0.5
        w, b = (_rand(gen, D) if wb & 1 else None), (_rand(gen, D) if wb & 2 else None)
        z = _rand(gen, rows, 2 * D, dtype=dtype)[:, D:] if gated else None
        _norm_check(x, w, b, z, _rand(gen, rows, D, dtype=dtype), 1e-5, rms)


def test_norm_of_strided_heads():
    """x and the gate as slices of a projection, head by head; rows of equal values; a large mean."""
    gen = torch.Generator().manual_seed(0)
    for D, heads in ((64, 4), (12, 3), (1, 5)):
        buf = _rand(gen, 6, 2 * heads * D + 4, dtype=BF)
        x, z = buf[:, :heads * D].unflatten(1, (heads, D)), buf[:, heads * D:2 * heads * D].unflatten(1, (heads, D))
        _norm_check(x, _rand(gen, D), None, z, _rand(gen, 6, heads, D, dtype=BF), 1e-6, True)
    x = torch.full((4, 256), 3.0, device="cuda")
    _norm_check(x, None, None, None, _rand(gen, 4, 256), 1e-5, False)
    x = _rand(gen, 4, 1024) + 1000.0
    _norm_check(x, _rand(gen, 1024), _rand(gen, 1024), None, _rand(gen, 4, 1024), 1e-5, False)


def test_norm_of_no_rows():
    gdn = _gdn()
    x = torch.empty(0, 64, device="cuda", dtype=BF)
    w = torch.ones(64, device="cuda")
    y, stats = gdn.layer_norm_fwd(x, w, w)
    g = gdn.layer_norm_bwd(x, x, stats, w, w)
    assert y.shape == x.shape and (g["dweight"] == 0).all() and (g["dbias"] == 0).all()


def test_norm_rows_stay_apart():
    gdn = _gdn()
    gen = torch.Generator().manual_seed(2)
    for D in (64, 1024):
        x, w = _rand(gen, 40, D, dtype=BF), _rand(gen, D)
        y, _ = gdn.layer_norm_fwd(x, w)
        x[7] = float("inf")
        x[20, 0] = float("nan")
        y2, _ = gdn.layer_norm_fwd(x, w)
        keep = [i for i in range(40) if i not in (7, 20)]
        assert torch.equal(y[keep], y2[keep]) and torch.isnan(y2[20].float()).all()


# ------------------------------------------------------------------------- all of them, as used


def test_bad_packing_writes_nothing():
    gdn = _gdn()
    gen = torch.Generator().manual_seed(0)
    x = _rand(gen, 1, 20, 16, dtype=BF)
    w = _rand(gen, 16, 4)
    for cu in ([0, 9, 21], [0, 12, 9, 20], [1, 20], [0, 19], [-4, 20]):
        bad = torch.tensor(cu, device="cuda")
        ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
        y = torch.full_like(x, 7.0)
        gdn.causal_conv_fwd(x, w, cu_seqlens=bad, out=y, workspace=ws)
        assert gdn.gdn_device_status(ws) == 1 and (y == 7).all(), cu
        c, _, _, _ = _scan_case(0, [20], True, 16, 16, 1, BF)
        c["cu_seqlens"] = bad
        y.fill_(7.0)
        gdn.ssm_scan_fwd(**c, out=y, workspace=ws)
        assert gdn.gdn_device_status(ws) == 1 and (y == 7).all(), cu
    c["cu_seqlens"] = torch.tensor([0, 20], device="cuda")
    gdn.ssm_scan_fwd(**c, out=y, workspace=ws)
    assert gdn.gdn_device_status(ws) == 0
    gdn.causal_conv_fwd(x, w, workspace=ws.fill_(255))
    assert gdn.gdn_device_status(ws) == 0


def test_bad_packing_leaves_gradients_alone():
    """The C entry points of the backward passes with an invalid packing: the status word is set and no output changes."""
    from gated_deltanet_chunkwise_chunk_b200 import binding
    gdn, lib = _gdn(), binding.lib
    gen = torch.Generator().manual_seed(0)
    T, D, W, N = 20, 16, 4, 16
    x, dy, w, b = _rand(gen, 1, T, D, dtype=BF), _rand(gen, 1, T, D, dtype=BF), _rand(gen, D, W), _rand(gen, D)
    A_log, Bm, Cm = _rand(gen, D, N), _rand(gen, 1, T, 1, N, dtype=BF), _rand(gen, 1, T, 1, N, dtype=BF)
    ptr = lambda t: t.data_ptr()  # noqa: E731
    stream = torch.cuda.current_stream().cuda_stream
    for cu in ([0, 9, 21], [0, 12, 9, 20], [1, 20], [0, 19], [-4, 20]):
        bad, n = torch.tensor(cu, device="cuda"), len(cu) - 1
        d = binding.gdn_conv_dims(1, T, D, W, n, 0, 1, 1)
        ws = torch.full((gdn.conv_workspace_bytes(d, True, True),), 255, dtype=torch.uint8, device="cuda")
        outs = [torch.full(s, 7.0, dtype=t, device="cuda") for s, t in (((1, T, D), BF), ((D, W), F32), ((D,), F32), ((n, W - 1, D), BF))]
        assert lib.gdn_conv_bwd(ctypes.byref(d), ptr(x), ptr(w), ptr(b), ptr(bad), None, ptr(dy), None, *map(ptr, outs), ptr(ws), ws.numel(),
                                stream) == 0
        assert gdn.gdn_device_status(ws) == 1 and all((o == 7).all() for o in outs), cu
        d = binding.gdn_ssm_dims(1, T, D, N, 1, n, 0, 0, 0, 0, 1)
        ws = torch.full((gdn.ssm_workspace_bytes(d, True, True),), 255, dtype=torch.uint8, device="cuda")
        outs = [torch.full(s, 7.0, dtype=t, device="cuda") for s, t in (
            ((1, T, D), BF), ((1, T, D), BF), ((1, T, 1, N), BF), ((1, T, 1, N), BF), ((D, N), F32), ((D,), F32), ((D,), F32), ((n, D, N), F32))]
        assert lib.gdn_ssm_bwd(ctypes.byref(d), ptr(x), ptr(x), ptr(A_log), ptr(Bm), ptr(Cm), None, None, ptr(bad), ptr(dy), None,
                               *map(ptr, outs), ptr(ws), ws.numel(), stream) == 0
        assert gdn.gdn_device_status(ws) == 1 and all((o == 7).all() for o in outs), cu


def test_sums_read_only_what_their_passes_wrote():
    """Workspaces full of NaN bits change no gradient of the convolution and of the norm, with idle units and blocks too."""
    gdn = _gdn()
    spaces = [torch.full((1 << 24,), fill, dtype=torch.uint8, device="cuda") for fill in (0, 255)]
    for lengths, packed, D, W in (([2, 0, 1, 300, 5], True, 48, 4), ([33, 0, 257], True, 257, 3), ([130, 130], False, 8, 8)):
        c, dy, dfin = _conv_case(1, lengths, packed, D, W, BF, True, True, True, 0)
        got = [gdn.causal_conv_bwd(c["x"], c["weight"], dy, c["bias"], "silu", c["cu_seqlens"], c["initial_state"], dfin, workspace=ws.clone())
               for ws in spaces]
        assert all(torch.equal(got[0][k], got[1][k]) for k in got[0])
    gen = torch.Generator().manual_seed(1)
    for rows, D in ((1, 64), (700, 96), (3, 4096), (2, 16400), (40, 333)):
        x, dy, w, b = _rand(gen, rows, D), _rand(gen, rows, D), _rand(gen, D), _rand(gen, D)
        _, stats = gdn.layer_norm_fwd(x, w, b)
        got = [gdn.layer_norm_bwd(x, dy, stats, w, b, workspace=ws.clone()) for ws in spaces]
        assert all(torch.equal(got[0][k], got[1][k]) for k in ("dx", "dweight", "dbias"))


class Layer:
    """[x | z] -> convolution -> dt, B, C -> scan -> norm gated by z."""

    def __init__(self, D, N, W, gen, dtype):
        self.D, self.N = D, N
        self.conv = dict(weight=_rand(gen, D, W, scale=0.5), bias=_rand(gen, D))
        self.proj = _rand(gen, D, D + 2 * N, dtype=dtype, scale=0.2)
        self.A_log, self.skip, self.dt_bias = _rand(gen, D, N, scale=0.3), _rand(gen, D), _rand(gen, D) - 2
        self.norm = _rand(gen, D)

    def split(self, u):
        p = u @ self.proj
        D, N = self.D, self.N
        return p[..., :D], p[..., None, D:D + N], p[..., None, D + N:]

    def prompt(self, xz, cu=None, conv_state=None, state=None, ws=None):
        gdn, D = _gdn(), self.D
        u, cs = gdn.causal_conv_fwd(xz[..., :D], **self.conv, cu_seqlens=cu, initial_state=conv_state, output_final_state=True)
        dt, Bm, Cm = self.split(u)
        h, st = gdn.ssm_scan_fwd(u, dt, self.A_log, Bm, Cm, self.skip, self.dt_bias, cu, state, workspace=ws)
        y, stats = gdn.layer_norm_fwd(h, self.norm, gate=xz[..., D:], rms=True)
        return y, cs, st, (u, dt, Bm, Cm, h, stats)

    def step(self, xz, conv_state, state):
        gdn, D = _gdn(), self.D
        u, _ = gdn.causal_conv_step(xz[:, :D], conv_state, **self.conv, final_state=conv_state)
        dt, Bm, Cm = self.split(u)
        h, _ = gdn.ssm_step(u, dt, self.A_log, Bm, Cm, state, self.skip, self.dt_bias, final_state=state)
        return gdn.layer_norm_fwd(h, self.norm, gate=xz[:, D:], rms=True, output_stats=False)[0]


def test_layer_prompt_then_single_tokens():
    """A prompt and then tokens one by one give what the whole sequence gives at once.  Between the two forms
    only the convolution's sums and its rounding are the same; the projections (a matrix product per form) may
    round differently, so outputs are compared at the accuracy of a product of D fp32 terms: relative to the
    largest output, (D + 64) half steps carried through the norm and the scan with a factor of 64."""
    gen = torch.Generator().manual_seed(0)
    D, N, T, P = 48, 16, 40, 29
    layer = Layer(D, N, 4, gen, F32)
    xz = _rand(gen, 2, T, 2 * D)
    whole, cs, st, _ = layer.prompt(xz)
    y, c1, s1, _ = layer.prompt(xz[:, :P].contiguous())
    outs = [y] + [layer.step(xz[:, t], c1, s1)[:, None] for t in range(P, T)]
    tol = 64 * (D + 64) * U
    assert (torch.cat(outs, 1) - whole).abs().max() <= tol * whole.abs().max()
    assert torch.equal(cs, c1) and (st - s1).abs().max() <= tol * st.abs().max()


def test_layer_gradients():
    """The layer's gradient through the operators' backward calls, against differences of the fp64 references
    along random directions (the projection is differentiated by hand).  The operators run in fp32: each stage's
    relative error is below 2e-5 at these sizes (the bounds above), five stages of condition below 10."""
    gdn = _gdn()
    gen = torch.Generator().manual_seed(4)
    D, N, T = 12, 5, 23
    layer = Layer(D, N, 3, gen, F32)
    cu = [0, 9, 9, 23]
    cut = torch.tensor(cu, device="cuda")
    xz, dy = _rand(gen, 1, T, 2 * D), _rand(gen, 1, T, D)
    ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    y, _, _, (u, dt, Bm, Cm, h, stats) = layer.prompt(xz, cut, ws=ws)
    gn = gdn.layer_norm_bwd(h, dy, stats, layer.norm, gate=xz[..., D:], rms=True)
    gs = gdn.ssm_scan_bwd(u, dt, layer.A_log, Bm, Cm, gn["dx"], ws, layer.skip, layer.dt_bias, cut)
    dp = torch.cat([gs["ddt"], gs["dB"][..., 0, :], gs["dC"][..., 0, :]], -1)
    du = gs["dx"] + dp @ layer.proj.t()
    gc = gdn.causal_conv_bwd(xz[..., :D], layer.conv["weight"], du, layer.conv["bias"], cu_seqlens=cut)
    grads = dict(xz=torch.cat([gc["dx"], gn["dgate"]], -1), weight=gc["dweight"], bias=gc["dbias"], A_log=gs["dA_log"], skip=gs["dD"],
                 dt_bias=gs["ddt_bias"], norm=gn["dweight"])
    base = dict(xz=xz, weight=layer.conv["weight"], bias=layer.conv["bias"], A_log=layer.A_log, skip=layer.skip, dt_bias=layer.dt_bias,
                norm=layer.norm)
    base = {k: _np(v) for k, v in base.items()}
    proj = _np(layer.proj)

    def loss(v):
        a = v["xz"][0]
        c, _, _, _ = om.conv_fwd(a[:, :D], v["weight"], v["bias"], cu)
        p = c @ proj
        s, _ = om.ssm(c, p[:, :D], v["A_log"], p[:, None, D:D + N], p[:, None, D + N:], v["skip"], v["dt_bias"], cu)
        o, _, _, _ = om.norm_fwd(s["y"], v["norm"], None, a[:, D:], 1e-5, True)
        return (o * _np(dy)[0]).sum()

    r = np.random.default_rng(0)
    for k, g in grads.items():
        way = r.normal(size=base[k].shape)
        eps = 1e-6
        want = (loss({**base, k: base[k] + eps * way}) - loss({**base, k: base[k] - eps * way})) / (2 * eps)
        got = float((_np(g) * way).sum())
        assert abs(got - want) <= 1e-3 * np.abs(_np(g) * way).sum() + 1e-6, (k, got, want)


def test_streams_graphs_and_repeats():
    """On a stream of its own and replayed from a graph the calls give the same bits, and so do repeats."""
    gdn = _gdn()
    lengths = [50, 0, 30, 3]
    c, init, dy, dfin = _scan_case(9, lengths, True, 40, 16, 1, BF)
    conv, cdy, cfin = _conv_case(9, lengths, True, 40, 4, BF, True, True, True, 8)
    w = torch.ones(40, device="cuda")

    def all_of():
        o = _scan_run(c, init, dy, dfin)
        y, fin = gdn.causal_conv_fwd(**conv, output_final_state=True)
        g = gdn.causal_conv_bwd(conv["x"], conv["weight"], cdy, conv["bias"], "silu", conv["cu_seqlens"], conv["initial_state"], cfin)
        n, stats = gdn.layer_norm_fwd(o["y"], w, w, gate=y)
        b = gdn.layer_norm_bwd(o["y"], cdy, stats, w, w, gate=y)
        return [*o.values(), y, fin, *g.values(), n, stats, *b.values()]

    first = all_of()
    assert all(torch.equal(a, b) for a, b in zip(first, all_of()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = all_of()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(first, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = all_of()
    for t in held:
        t.fill_(0)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, held))


def test_two_streams_at_once():
    """Calls on two streams, each with its own workspace, do not disturb each other."""
    cases = [_scan_case(k, [200, 200], False, 64, 16, 1, BF) for k in (1, 2)]
    want = [_scan_run(*c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = []
    for s, c in zip(streams, cases):
        with torch.cuda.stream(s):
            got.append([_scan_run(*c) for _ in range(3)])
    torch.cuda.synchronize()
    for w, runs in zip(want, got):
        for g in runs:
            assert all(torch.equal(w[k], g[k]) for k in w)
