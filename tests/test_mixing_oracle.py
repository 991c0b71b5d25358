"""The fp64 references of the mixing-layer operators against differences, closed forms and each other."""
import numpy as np
import pytest

from oracle import mixing as om

CU = [0, 5, 5, 6, 13]


def _numeric(f, a, eps=1e-6):
    g = np.zeros_like(a)
    flat, out = a.reshape(-1), g.reshape(-1)
    for i in range(flat.size):
        keep = flat[i]
        flat[i] = keep + eps
        hi = f()
        flat[i] = keep - eps
        lo = f()
        flat[i] = keep
        out[i] = (hi - lo) / (2 * eps)
    return g


def _near(a, b):
    # central differences of step 1e-6: truncation ~1e-12, cancellation ~1e-16 |f| / 1e-6 with |f| < 100
    assert np.abs(a - b).max(initial=0) <= 1e-7 * (1 + np.abs(b).max(initial=0))


@pytest.mark.parametrize("W", [1, 2, 4, 7])
@pytest.mark.parametrize("silu", [True, False])
def test_convolution_gradients(W, silu):
    r = np.random.default_rng(W)
    D, n = 3, len(CU) - 1
    x, w, b, init = r.normal(size=(CU[-1], D)), r.normal(size=(D, W)), r.normal(size=D), r.normal(size=(n, W - 1, D))
    dy, dfin = r.normal(size=x.shape), r.normal(size=init.shape)

    def loss():
        y, fin, _, _ = om.conv_fwd(x, w, b, CU, init, silu)
        return (y * dy).sum() + (fin * dfin).sum()

    g = om.conv_bwd(x, w, b, CU, dy, init, dfin, silu)
    for name, a in (("dx", x), ("dweight", w), ("dbias", b), ("dinitial_state", init)):
        _near(g[name], _numeric(loss, a))


def test_scan_gradients():
    r = np.random.default_rng(0)
    D, N, G, R, n = 4, 3, 2, CU[-1], len(CU) - 1
    x, dt = r.normal(size=(R, D)), r.normal(size=(R, D))
    dt[2, 1] = 21.0  # the pass-through branch
    A_log, Bm, Cm = r.normal(size=(D, N)), r.normal(size=(R, G, N)), r.normal(size=(R, G, N))
    skip, bias, init = r.normal(size=D), r.normal(size=D), r.normal(size=(n, D, N))
    dy, dfin = r.normal(size=x.shape), r.normal(size=init.shape)
    bias[1] = 0.5

    def loss():
        v, _ = om.ssm(x, dt, A_log, Bm, Cm, skip, bias, CU, init)
        return (v["y"] * dy).sum() + (v["state"] * dfin).sum()

    v, e = om.ssm(x, dt, A_log, Bm, Cm, skip, bias, CU, init, dy, dfin)
    for name, a in (("dx", x), ("ddt", dt), ("dA_log", A_log), ("dB", Bm), ("dC", Cm), ("dD", skip), ("ddt_bias", bias),
                    ("dinitial_state", init)):
        _near(v[name], _numeric(loss, a))
        assert (e[name] >= 0).all()


def test_scan_against_the_closed_form():
    """h[T] = sum_s exp(A (S_T - S_s)) delta_s x_s B_s + exp(A S_T) h0, S the running sum of delta."""
    r = np.random.default_rng(1)
    T, D, N = 9, 2, 3
    x, dt, A_log = r.normal(size=(T, D)), r.normal(size=(T, D)), r.normal(size=(D, N))
    Bm, Cm, h0 = r.normal(size=(T, 1, N)), r.normal(size=(T, 1, N)), r.normal(size=(1, D, N))
    v, _ = om.ssm(x, dt, A_log, Bm, Cm, cu=[0, T], init=h0)
    d = np.log1p(np.exp(dt))
    S, A = np.cumsum(d, 0), -np.exp(A_log)
    h = np.exp(A * S[-1][:, None]) * h0[0]
    for s in range(T):
        h = h + np.exp(A * (S[-1] - S[s])[:, None]) * (d[s] * x[s])[:, None] * Bm[s]
    assert np.abs(h - v["state"][0]).max() < 1e-13
    assert np.abs((h * Cm[-1]).sum(-1) - v["y"][-1]).max() < 1e-13


@pytest.mark.parametrize("rms", [True, False])
@pytest.mark.parametrize("gated", [True, False])
def test_norm_gradients(rms, gated):
    r = np.random.default_rng(2)
    x, w, b, dy = r.normal(size=(4, 6)), r.normal(size=6), r.normal(size=6), r.normal(size=(4, 6))
    z = r.normal(size=(4, 6)) if gated else None
    loss = lambda: (om.norm_fwd(x, w, b, z, 1e-5, rms)[0] * dy).sum()  # noqa: E731
    g = om.norm_bwd(x, dy, w, b, z, 1e-5, rms)
    for name, a in (("dx", x), ("dweight", w), ("dbias", b)) + ((("dgate", z),) if gated else ()):
        _near(g[name], _numeric(loss, a))
