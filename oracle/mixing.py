"""fp64 references of the mixing-layer operators, token by token in numpy, and first-order running bounds of
the rounding error of an fp32 evaluation of the same formulas.  Test infrastructure: shares nothing with the
CUDA path.

Sequences are given as boundaries cu (list of n + 1 ints) over flattened tokens.
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24  # half a step of fp32, relative


def sigmoid(v):
    return 1.0 / (1.0 + np.exp(-np.minimum(np.maximum(v, -700.0), 700.0)))


def softplus20(v):
    return np.where(v > 20, v, np.log1p(np.exp(np.minimum(v, 20.0))))


# ------------------------------------------------------------------------------- convolution


def conv_fwd(x, weight, bias, cu, init=None, silu=True):
    """x [R, D]; returns y, final [n, W-1, D], pre, lines (each sequence's inputs with the state before)."""
    D, W = weight.shape
    n = len(cu) - 1
    pre, final, lines = np.zeros_like(x), np.zeros((n, W - 1, D)), []
    for k in range(n):
        lo, hi = cu[k], cu[k + 1]
        line = np.concatenate([np.zeros((W - 1, D)) if init is None else init[k], x[lo:hi]])
        lines.append(line)
        for t in range(hi - lo):
            pre[lo + t] = (weight.T * line[t:t + W]).sum(0) + (0 if bias is None else bias)
        final[k] = line[len(line) - (W - 1):]
    return (pre * sigmoid(pre) if silu else pre), final, pre, lines


def conv_slope(pre, silu):
    s = sigmoid(pre)
    return s * (1 + pre * (1 - s)) if silu else np.ones_like(pre)


def conv_bwd(x, weight, bias, cu, dy, init=None, dfinal=None, silu=True):
    D, W = weight.shape
    n = len(cu) - 1
    _, _, pre, lines = conv_fwd(x, weight, bias, cu, init, silu)
    dpre = dy * conv_slope(pre, silu)
    dx, dw, dinit = np.zeros_like(x), np.zeros_like(weight), np.zeros((n, W - 1, D))
    for k in range(n):
        lo, hi = cu[k], cu[k + 1]
        dl = np.zeros_like(lines[k])
        for t in range(hi - lo):
            dl[t:t + W] += weight.T * dpre[lo + t]
            dw += (lines[k][t:t + W] * dpre[lo + t]).T
        if dfinal is not None:
            dl[len(dl) - (W - 1):] += dfinal[k]
        dinit[k], dx[lo:hi] = dl[:W - 1], dl[W - 1:]
    return dict(dx=dx, dweight=dw, dbias=dpre.sum(0), dinitial_state=dinit, dpre=dpre)


# ---------------------------------------------------------------------------------- scan


def ssm(x, dt, A_log, Bm, Cm, D=None, dt_bias=None, cu=None, init=None, dy=None, dfinal=None, extra=0.0, chain=None):
    """Forward, and with dy the backward.  x, dt [R, D]; Bm, Cm [R, G, N]; states [n, D, N].  Returns (values,
    bounds): dicts of the outputs and of bounds on the error that fp32 arithmetic (fused products, an exponential
    of 2 ulp, a softplus of (|v| + 20) half ulps) makes before an output is rounded to its type.  `extra`
    (in half ulps of the state or gradient, at every 64th token): what a join of segments adds.  `chain`: additions
    that a term of a sum over all tokens goes through, one for each token where it is not given."""
    R, W = x.shape
    G, N = Bm.shape[1:]
    n = len(cu) - 1
    A = -np.exp(A_log)
    v = dt + (0 if dt_bias is None else dt_bias)
    delta = softplus20(v)
    ed = (np.abs(v) + 20) * U  # relative error of delta
    group = np.arange(W) // (W // G)
    skip = np.zeros(W) if D is None else D
    h = np.zeros((n, W, N)) if init is None else init.copy()
    Eh = np.zeros_like(h)
    y, Ey = np.zeros_like(x), np.zeros_like(x)
    hs, Es, prev, Eprev, decay, Ea = ([None] * R for _ in range(6))
    for k in range(n):
        for t in range(cu[k], cu[k + 1]):
            b, c = Bm[t][group], Cm[t][group]
            d = delta[t][:, None]
            a = np.exp(d * A)
            ea = np.abs(d * A) * (ed[t][:, None] + 7 * U) + 4 * U  # relative error of a
            prev[t], Eprev[t], decay[t], Ea[t] = h[k].copy(), Eh[k].copy(), a, ea
            inp = d * x[t][:, None] * b
            new = a * h[k] + inp
            E = a * Eh[k] + a * np.abs(h[k]) * ea + np.abs(inp) * (ed[t][:, None] + 2 * U) + U * np.abs(new)
            if (t - cu[k]) % 64 == 0:
                E = E + extra * U * np.abs(new)
            hs[t], Es[t] = new, E
            h[k], Eh[k] = new, E
            y[t] = (c * new).sum(-1) + skip * x[t]
            Ey[t] = (np.abs(c) * E).sum(-1) + (N + 2) * U * (np.abs(c * new).sum(-1) + np.abs(skip * x[t]))
    val, err = dict(y=y, state=h), dict(y=Ey, state=Eh)
    if dy is None:
        return val, err
    ga = np.zeros((n, W, N)) if dfinal is None else dfinal.copy()
    Ega = np.zeros_like(ga)
    dx, ddt = np.zeros_like(x), np.zeros_like(x)
    Edx, Eddt = np.zeros_like(x), np.zeros_like(x)
    dB, dC, EdB, EdC = (np.zeros_like(Bm) for _ in range(4))
    dA, EdA, SdA = (np.zeros_like(A) for _ in range(3))
    slope = np.where(v > 20, 1.0, sigmoid(v))
    L = 16 + 4 + W // G  # terms added one after another: butterflies, warps, channel tiles
    for k in range(n):
        for t in range(cu[k + 1] - 1, cu[k] - 1, -1):
            b, c = Bm[t][group], Cm[t][group]
            d, xx, gy = delta[t][:, None], x[t][:, None], dy[t][:, None]
            g = c * gy + ga[k]
            Eg = Ega[k] + U * np.abs(g)
            if (cu[k + 1] - 1 - t) % 64 == 0:
                Eg = Eg + extra * U * np.abs(g)
            gb, Egb = (g * b).sum(-1), (np.abs(b) * Eg).sum(-1) + (N + 1) * U * np.abs(g * b).sum(-1)
            a = decay[t]
            new = a * g
            Enew = a * Eg + np.abs(new) * (Ea[t] + U)
            q = new * prev[t]
            Eq = np.abs(new) * Eprev[t] + np.abs(prev[t]) * Enew + U * np.abs(q)
            dx[t] = delta[t] * gb + skip * dy[t]
            Edx[t] = delta[t] * (Egb + np.abs(gb) * ed[t]) + 3 * U * (np.abs(delta[t] * gb) + np.abs(skip * dy[t]))
            dd = x[t] * gb + (A * q).sum(-1)
            Edd = np.abs(x[t]) * Egb + (np.abs(A) * Eq).sum(-1) + (N + 10) * U * (np.abs(x[t] * gb) + np.abs(A * q).sum(-1))
            ddt[t] = dd * slope[t]
            Eddt[t] = Edd * slope[t] + np.abs(ddt[t]) * (16 + np.abs(v[t])) * U
            ub, hb = g * d * xx, gy * hs[t]
            Eub = np.abs(d * xx) * Eg + np.abs(ub) * (ed[t][:, None] + 3 * U)
            Ehb = np.abs(gy) * Es[t] + U * np.abs(hb)
            over = lambda v: v.reshape(G, W // G, N).sum(1)  # noqa: E731  (a group's channels are neighbours)
            dB[t], dC[t] = over(ub), over(hb)
            EdB[t] = over(Eub) + L * U * over(np.abs(ub))
            EdC[t] = over(Ehb) + L * U * over(np.abs(hb))
            dA += d * q
            SdA += np.abs(d * q)
            EdA += d * Eq + np.abs(d * q) * (ed[t][:, None] + 2 * U)
            ga[k], Ega[k] = new, Enew
    if chain is None:
        chain = R + 64  # tokens one after another, then units and strands
    val.update(dx=dx, ddt=ddt, dB=dB, dC=dC, dA_log=dA * A, dD=(dy * x).sum(0), ddt_bias=ddt.sum(0), dinitial_state=ga)
    err.update(dx=Edx, ddt=Eddt, dB=EdB, dC=EdC, dA_log=np.abs(A) * (EdA + chain * U * SdA) + 6 * U * np.abs(dA * A),
               dD=chain * U * np.abs(dy * x).sum(0), ddt_bias=Eddt.sum(0) + chain * U * np.abs(ddt).sum(0),
               dinitial_state=Ega)
    return val, err


# ---------------------------------------------------------------------------------- norm


def norm_fwd(x, weight=None, bias=None, gate=None, eps=1e-5, rms=False):
    mu = np.zeros(x.shape[:-1] + (1,)) if rms else x.mean(-1, keepdims=True)
    rstd = 1 / np.sqrt(((x - mu) ** 2).mean(-1, keepdims=True) + eps)
    n = (x - mu) * rstd * (1 if weight is None else weight) + (0 if bias is None else bias)
    return (n if gate is None else n * gate * sigmoid(gate)), mu, rstd, n


def norm_bwd(x, dy, weight=None, bias=None, gate=None, eps=1e-5, rms=False):
    _, mu, rstd, n = norm_fwd(x, weight, bias, gate, eps, rms)
    xh = (x - mu) * rstd
    out, dn = {}, dy
    if gate is not None:
        s = sigmoid(gate)
        out["dgate"] = dy * n * s * (1 + gate * (1 - s))
        dn = dy * gate * s
    u = dn * (1 if weight is None else weight)
    out["dx"] = rstd * (u - (0 if rms else u.mean(-1, keepdims=True)) - xh * (u * xh).mean(-1, keepdims=True))
    lead = tuple(range(x.ndim - 1))
    out["dweight"], out["dbias"] = (dn * xh).sum(lead), dn.sum(lead)
    return out
