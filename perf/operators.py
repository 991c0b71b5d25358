"""Cases of the mixing-layer operators around the recurrences: the short causal convolution, the
selective state space scan and the layer norm (plain, or as the gated norm of a head's output).

A layer projects its input to [x | z], convolves x along the sequence, projects dt, B and C, scans,
and normalises the result (gated by z).  A case names one operator, one direction ("fwd": a prompt,
"train": forward and backward, "step": one token for each of a batch of sequences), the sizes and
the type.  Sequences are "dense" (B of length T) or "ragged" (B sequences packed into T tokens
in all, some of length 0 and 1).
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one layer's convolution in a training step: two sequences of 8k tokens, inner width 4096
        dict(name="conv_train", op="conv", go="train", dtype="bf16", B=2, T=8192, D=4096, W=4, layout="dense"),
        # prompts of 32 requests packed into one batch, with the states that serving goes on from
        dict(name="conv_prompts", op="conv", go="fwd", dtype="fp16", B=32, T=33333, D=2048, W=4, layout="ragged"),
        # one token for each of 256 requests
        dict(name="conv_step", op="conv", go="step", dtype="bf16", B=256, T=1, D=4096, W=4, layout="dense"),
        # one long prompt
        dict(name="scan_prompt", op="scan", go="fwd", dtype="bf16", B=1, T=32768, D=4096, N=16, G=1, layout="dense"),
        # packed prompts of many lengths
        dict(name="scan_prompts", op="scan", go="fwd", dtype="fp16", B=32, T=20011, D=2048, N=16, G=1, layout="ragged"),
        # a training step of one layer
        dict(name="scan_train", op="scan", go="train", dtype="bf16", B=2, T=4096, D=2048, N=16, G=1, layout="dense"),
        # the same in fp32, packed, with two groups, an odd width and an odd state size
        dict(name="scan_train_fp32", op="scan", go="train", dtype="fp32", B=5, T=1531, D=522, N=9, G=2, layout="ragged"),
        # one token for each of 256 requests: the state's traffic
        dict(name="scan_step", op="scan", go="step", dtype="bf16", B=256, T=1, D=4096, N=16, G=1, layout="dense"),
        # the norm of a recurrence's output, head by head, gated: 8k tokens, 32 value heads of 128
        dict(name="norm_heads_train", op="norm", go="train", dtype="bf16", B=8192, T=32, D=128, rms=True, gate=True),
        # a block's layer norm with weight and bias
        dict(name="norm_block_train", op="norm", go="train", dtype="bf16", B=8192, T=1, D=4096, rms=False, gate=False),
        # an odd width in fp32
        dict(name="norm_fp32", op="norm", go="fwd", dtype="fp32", B=2047, T=1, D=1999, rms=False, gate=True),
        # one token for each of 16 requests: the smallest call
        dict(name="norm_step", op="norm", go="fwd", dtype="bf16", B=16, T=1, D=2048, rms=True, gate=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    d = _log(rng, lo, hi)
    return d if rng.random() < 0.4 else max(8, d // 8 * 8)


def draw(rng):
    op = rng.choice(["conv", "scan", "scan", "norm"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op == "norm":
        c = dict(op="norm", go=rng.choice(["fwd", "train"]), dtype=dtype, B=_log(rng, 1, 8192), T=rng.choice([1, 1, 4, 16]),
                 D=_width(rng, 16, 8192), rms=rng.random() < 0.5, gate=rng.random() < 0.5)
        while c["B"] * c["T"] * c["D"] > 1 << 25:
            c["B"] = max(1, c["B"] // 2)
        return c
    go = rng.choice(["fwd", "train", "step"])
    D = _width(rng, 32, 4096)
    if go == "step":
        c = dict(op=op, go=go, dtype=dtype, B=_log(rng, 1, 256), T=1, D=D, layout="dense")
    elif rng.random() < 0.5:
        c = dict(op=op, go=go, dtype=dtype, B=rng.choice([1, 1, 2, 3, 8]), T=_log(rng, 1, 8192), D=D, layout="dense")
    else:
        c = dict(op=op, go=go, dtype=dtype, B=rng.randint(1, 40), T=_log(rng, 64, 16384), D=D, layout="ragged")
    if op == "conv":
        c["W"] = rng.choice([2, 3, 4, 4, 4, 5, 8])
        most = 1 << 25
    else:
        c["N"] = rng.choice([4, 8, 16, 16, 16, 16, 24, 32, 64])
        c["G"] = rng.choice([1, 1, 1, 2, 4])
        c["D"] = max(c["G"], c["D"] // c["G"] * c["G"])
        most = (1 << 27) // c["N"]
    rows = lambda: c["B"] * c["T"] if c["layout"] == "dense" else c["T"]  # noqa: E731
    while rows() * c["D"] > most:
        c["T" if c["T"] > 1 else "B"] //= 2
    return c


def _rows(c):
    return c["T"] if c.get("layout") == "ragged" else c["B"] * c["T"]


def _cu(c, seed):
    """Boundaries of the packed sequences, from the seed: random lengths, the second empty, the third a single token."""
    if c["layout"] == "dense":
        return [i * c["T"] for i in range(c["B"] + 1)]
    r, T, n = random.Random(seed), c["T"], c["B"]
    cut = sorted(r.randint(0, T) for _ in range(n - 1))
    if n >= 4 and T >= 2:
        cut[1] = cut[0]
        cut[2] = max(cut[2], min(T, cut[1] + 1)) if n < 6 else min(T, cut[1] + 1)
        cut = sorted(cut)
    return [0] + cut + [T]


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt_ = DT[c["dtype"]]
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    unif = lambda *s: torch.rand(*s, generator=gen, device="cuda")  # noqa: E731
    D = c["D"]
    s = {"c": c, "go": c["go"], "op": c["op"]}
    if c["op"] == "norm":
        shape = (c["B"], c["T"], D)
        s["x"] = (rand(*shape) * 1.5 + 0.25).to(dt_)
        s["weight"] = 1 + 0.2 * rand(D)
        s["bias"] = None if c["rms"] else 0.1 * rand(D)
        # z is the second half of the projection [x | z]
        s["gate"] = rand(c["B"], 2, c["T"], D).to(dt_)[:, 1] if c["gate"] else None
        s["dy"] = rand(*shape).to(dt_)
        s["rms"], s["eps"] = c["rms"], 1e-5
        return s
    R = _rows(c)
    cu = _cu(c, seed)
    s["cu_host"] = cu
    n = len(cu) - 1
    ragged = c["layout"] == "ragged"
    s["cu"] = torch.tensor(cu, device="cuda")
    s["cu_seqlens"] = s["cu"] if ragged else None
    shape = (1, R) if ragged else (c["B"], c["T"])
    s["shape"] = shape
    if c["op"] == "conv":
        W = c["W"]
        # x is the first half of the projection [x | z]
        s["x"] = rand(*shape, 2 * D).to(dt_)[..., :D]
        s["weight"] = (unif(D, W) * 2 - 1) / math.sqrt(W)
        s["bias"] = (unif(D) * 2 - 1) / math.sqrt(W)
        s["state"] = rand(n, W - 1, D).to(dt_)
        s["next"] = torch.empty_like(s["state"])
        s["dy"] = rand(*shape, D).to(dt_)
        s["dfinal"] = rand(n, W - 1, D).to(dt_)
    else:
        N, G = c["N"], c["G"]
        s["x"] = torch.nn.functional.silu(rand(*shape, D)).to(dt_)
        s["dt"] = (0.5 * rand(*shape, D)).to(dt_)
        # B and C are two slices of one projection
        bc = rand(*shape, 2 * G * N).to(dt_)
        s["Bm"], s["Cm"] = (bc[..., k * G * N:(k + 1) * G * N].unflatten(-1, (G, N)) for k in (0, 1))
        # the usual start: A = -(1..N) in every channel, softplus(dt_bias) log-uniform in [1e-3, 1e-1]
        s["A_log"] = torch.log(torch.arange(1, N + 1, device="cuda", dtype=torch.float32)).repeat(D, 1) + 0.05 * rand(D, N)
        d0 = torch.exp(unif(D) * math.log(100.0) + math.log(1e-3))
        s["dt_bias"] = d0 + torch.log(-torch.expm1(-d0))
        s["D"] = 1 + 0.1 * rand(D)
        s["state"] = 0.1 * rand(n, D, N)
        s["next"] = torch.empty_like(s["state"])
        s["dy"] = rand(*shape, D).to(dt_)
        s["dfinal"] = 0.1 * rand(n, D, N)
    return s


# ---------------------------------------------------------------------------------- plain forms


def _where(s):
    """For each token its sequence and its place in it."""
    cu = s["cu"]
    t = torch.arange(int(s["cu_host"][-1]), device=cu.device)
    seq = torch.searchsorted(cu, t, right=True) - 1
    return t, seq, t - cu[seq]


def _sigmoid(v):
    return 1 / (1 + torch.exp(-v))


def _conv_inputs(s, x, t, seq, pos, W):
    """The W inputs that each token sees, oldest first: [R, W, D]."""
    back = torch.arange(W - 1, -1, -1, device=t.device)
    at = pos[:, None] - back
    here = x[(t[:, None] - back).clamp(min=0)]
    if W == 1:
        return here
    before = s["state"].float()[seq[:, None], (at + W - 1).clamp(0, W - 2)]
    return torch.where((at >= 0)[..., None], here, before)


def _conv_final(s, x, W):
    """The last W-1 inputs of each sequence, the state before it where it is shorter."""
    cu = s["cu"]
    i = torch.arange(W - 1, device=cu.device)
    at = (cu[1:] - cu[:-1])[:, None] - (W - 1) + i
    if x.shape[0] == 0 or W == 1:
        return s["state"].clone()
    here = x[(cu[:-1, None] + at).clamp(0, x.shape[0] - 1)]
    before = torch.gather(s["state"], 1, (at + W - 1).clamp(0, W - 2)[..., None].expand_as(s["state"]))
    return torch.where((at >= 0)[..., None], here, before)


def _plain_conv(s):
    c, W = s["c"], s["c"]["W"]
    x = s["x"].reshape(-1, c["D"])
    t, seq, pos = _where(s)
    seen = _conv_inputs(s, x.float(), t, seq, pos, W)
    pre = s["bias"] + (seen * s["weight"].t()).sum(1)
    sig = _sigmoid(pre)
    out = {"y": (pre * sig).to(x.dtype).view(*s["shape"], -1), "state": _conv_final(s, x, W)}
    if s["go"] != "train":
        return out
    dpre = s["dy"].reshape(-1, c["D"]).float() * sig * (1 + pre * (1 - sig))
    cu, R, n = s["cu"], x.shape[0], len(s["cu_host"]) - 1
    ahead = torch.arange(W - 1, -1, -1, device=t.device)  # token t + ahead[j] reads token t by tap j
    left = (cu[1:] - cu[:-1])[seq] - pos
    used = (ahead < left[:, None])[..., None]
    dx = (torch.where(used, dpre[(t[:, None] + ahead).clamp(max=R - 1)], 0.0) * s["weight"].t()).sum(1)
    dstate = torch.zeros(n, max(W - 1, 0), c["D"], device=x.device)
    if W > 1:
        slot = W - 1 - left  # a token's place in the final state
        kept = slot >= 0
        dx[kept] += s["dfinal"].float()[seq[kept], slot[kept]]
        i = torch.arange(W - 1, device=x.device)
        j = torch.arange(W, device=x.device)
        p = i[:, None] - j  # slot i of the state before is read by tap j of token i - j
        lens = cu[1:] - cu[:-1]
        read = (p >= 0) & (p < lens[:, None, None])
        at = (cu[:-1, None, None] + p).clamp(0, R - 1)
        dstate = (torch.where(read[..., None], dpre[at], 0.0) * s["weight"].t()).sum(2)
        to = i - lens[:, None]  # and kept at this place of the final state
        keep = (to >= 0)[..., None]
        dstate = dstate + torch.where(keep, torch.gather(s["dfinal"].float(), 1, to.clamp(0)[..., None].expand_as(dstate)), 0.0)
    out["dx"] = dx.to(x.dtype).view(*s["shape"], -1)
    out["dweight"] = (seen * dpre[:, None]).sum(0).t().contiguous()
    out["dbias"] = dpre.sum(0)
    out["dstate"] = dstate.to(x.dtype)
    return out


def _doubling(a, b):
    """h[t] = a[t] h[t-1] + b[t] along dim 0, from zero; overwrites both."""
    k = 1
    while k < a.shape[0]:
        b[k:] = b[k:] + a[k:] * b[:-k]
        a[k:] = a[k:] * a[:-k]
        k *= 2
    return b


def _plain_scan(s):
    c = s["c"]
    D, N, G = c["D"], c["N"], c["G"]
    R, kind = s["x"].shape[0] * s["x"].shape[1], s["x"].dtype
    cu = s["cu"]
    some = cu[1:] > cu[:-1]
    first, last = cu[:-1][some], cu[1:][some] - 1
    x = s["x"].reshape(R, D).float()
    pre = s["dt"].reshape(R, D).float() + s["dt_bias"]
    delta = torch.where(pre > 20, pre, torch.log1p(torch.exp(pre.clamp(max=20))))
    A = -torch.exp(s["A_log"])
    group = torch.arange(D, device=cu.device) // (D // G)
    Bm, Cm = (s[k].reshape(R, G, N).float()[:, group] for k in ("Bm", "Cm"))
    a = torch.exp(delta[..., None] * A)
    b = (delta * x)[..., None] * Bm
    b[first] += a[first] * s["state"][some]
    keep = a.clone() if s["go"] == "train" else None
    a[first] = 0
    h = _doubling(a, b)
    y = (h * Cm).sum(-1) + s["D"] * x
    final = s["state"].clone()
    final[some] = h[last]
    out = {"y": y.to(kind).view(*s["shape"], D), "state": final}
    if s["go"] != "train":
        return out
    a = keep
    dy = s["dy"].reshape(R, D).float()
    g = dy[..., None] * Cm
    g[last] += s["dfinal"][some]
    ahead = torch.zeros_like(a)
    ahead[:-1] = a[1:]
    ahead[last] = 0
    g = _doubling(ahead.flip(0), g.flip(0)).flip(0)
    del ahead
    before = torch.empty_like(h)
    before[1:] = h[:-1]
    before[first] = s["state"][some]
    q = before.mul_(a).mul_(g)
    gB = (g * Bm).sum(-1)
    slope = torch.where(pre > 20, 1.0, _sigmoid(pre))
    ddt = ((q * A).sum(-1) + x * gB) * slope
    dh0 = s["dfinal"].clone()
    dh0[some] = a[first] * g[first]
    out["dx"] = (delta * gB + s["D"] * dy).to(kind).view(*s["shape"], D)
    out["ddt"] = ddt.to(kind).view(*s["shape"], D)
    shape = (*s["shape"], G, N)
    out["dA_log"] = (q.mul_(delta[..., None])).double().sum(0).float() * A
    del q, before
    out["dB"] = (g.mul_((delta * x)[..., None])).view(R, G, D // G, N).sum(2).to(kind).view(shape)
    out["dC"] = (h.mul_(dy[..., None])).view(R, G, D // G, N).sum(2).to(kind).view(shape)
    out["dD"] = (dy * x).double().sum(0).float()
    out["ddt_bias"] = ddt.double().sum(0).float()
    out["dstate"] = dh0
    return out


def _plain_norm(s):
    x = s["x"].float()
    mean = 0.0 if s["rms"] else x.mean(-1, keepdim=True)
    rstd = torch.rsqrt((x - mean).square().mean(-1, keepdim=True) + s["eps"])
    xh = (x - mean) * rstd
    n = xh * s["weight"] + (0.0 if s["bias"] is None else s["bias"])
    y = n
    if s["gate"] is not None:
        z = s["gate"].float()
        sig = _sigmoid(z)
        y = n * (z * sig)
    out = {"y": y.to(s["x"].dtype)}
    if s["go"] != "train":
        return out
    dn = s["dy"].float()
    if s["gate"] is not None:
        out["dgate"] = (dn * n * sig * (1 + z * (1 - sig))).to(x_type(s))
        dn = dn * (z * sig)
    u = dn * s["weight"]
    dx = u - xh * (u * xh).mean(-1, keepdim=True)
    if not s["rms"]:
        dx = dx - u.mean(-1, keepdim=True)
        out["dbias"] = dn.double().sum((0, 1)).float()
    out["dx"] = (dx * rstd).to(x_type(s))
    out["dweight"] = (dn * xh).double().sum((0, 1)).float()
    return out


def x_type(s):
    return s["x"].dtype


# ------------------------------------------------------------------------- the framework's calls


def _own_conv(s, gdn):
    if s["go"] == "step":
        y, st = gdn.causal_conv_step(s["x"][:, 0], s["state"], s["weight"], s["bias"], activation="silu", final_state=s["next"])
        return {"y": y[:, None], "state": st}
    y, st = gdn.causal_conv_fwd(s["x"], s["weight"], s["bias"], activation="silu", cu_seqlens=s["cu_seqlens"],
                                initial_state=s["state"], output_final_state=True)
    out = {"y": y, "state": st}
    if s["go"] == "train":
        g = gdn.causal_conv_bwd(s["x"], s["weight"], s["dy"], s["bias"], activation="silu", cu_seqlens=s["cu_seqlens"],
                                initial_state=s["state"], dfinal_state=s["dfinal"])
        out.update(dx=g["dx"], dweight=g["dweight"], dbias=g["dbias"], dstate=g["dinitial_state"])
    return out


def _own_scan(s, gdn):
    par = dict(D=s["D"], dt_bias=s["dt_bias"])
    if s["go"] == "step":
        y, st = gdn.ssm_step(s["x"][:, 0], s["dt"][:, 0], s["A_log"], s["Bm"][:, 0], s["Cm"][:, 0], s["state"],
                             final_state=s["next"], **par)
        return {"y": y[:, None], "state": st}
    ins = (s["x"], s["dt"], s["A_log"], s["Bm"], s["Cm"])
    ws = None
    if s["go"] == "train":  # what the forward leaves in it, the backward reads
        dims = gdn.ssm_dims(s["x"], s["Bm"], s["cu_seqlens"])
        ws = torch.empty(gdn.ssm_workspace_bytes(dims, s["cu_seqlens"] is not None, True), dtype=torch.uint8, device="cuda")
    y, st = gdn.ssm_scan_fwd(*ins, cu_seqlens=s["cu_seqlens"], initial_state=s["state"], workspace=ws, **par)
    out = {"y": y, "state": st}
    if s["go"] == "train":
        g = gdn.ssm_scan_bwd(*ins, s["dy"], ws, cu_seqlens=s["cu_seqlens"], dfinal_state=s["dfinal"], **par)
        out.update(dstate=g.pop("dinitial_state"), **g)
    return out


def _own_norm(s, gdn):
    y, stats = gdn.layer_norm_fwd(s["x"], s["weight"], s["bias"], gate=s["gate"], eps=s["eps"], rms=s["rms"])
    out = {"y": y}
    if s["go"] == "train":
        g = gdn.layer_norm_bwd(s["x"], s["dy"], stats, s["weight"], s["bias"], gate=s["gate"], rms=s["rms"])
        out.update({k: v for k, v in g.items() if v is not None})
    return out


def run(state):
    op = state["op"]
    if own:
        import gated_deltanet_chunkwise_chunk_b200 as gdn
        return {"conv": _own_conv, "scan": _own_scan, "norm": _own_norm}[op](state, gdn)
    return {"conv": _plain_conv, "scan": _plain_scan, "norm": _plain_norm}[op](state)


def work(case):
    c = case
    es = 4 if c["dtype"] == "fp32" else 2
    train = c["go"] == "train"
    if c["op"] == "norm":
        rows, D = c["B"] * c["T"], c["D"]
        b = rows * D * es * ((4 if train else 2) + (2 if train and c["gate"] else 1 if c["gate"] else 0))
        return {"bytes": b + 4 * D * (1 if c["rms"] else 2) * (2 if train else 1),
                "flops": rows * D * ((8 + 5 * c["gate"]) + train * (12 + 8 * c["gate"]))}
    R, D, n = _rows(c), c["D"], c["B"]
    if c["op"] == "conv":
        W = c["W"]
        return {"bytes": R * D * es * (4 if train else 2) + n * (W - 1) * D * es * (4 if train else 2) + 4 * D * (W + 1) * (2 if train else 1),
                "flops": R * D * (2 * W + 6 + train * (6 * W + 10))}
    N, G = c["N"], c["G"]
    b = R * D * es * (6 if train else 3) + R * G * N * es * (4 if train else 2)
    b += n * D * N * 4 * (4 if train else 2) + 4 * D * (N + 2) * (2 if train else 1)
    # per state: product in the exponent, exponential, decay and input, output; backward about twice as much again
    return {"bytes": b, "flops": R * D * (N * (7 + train * 14) + 16)}


# ------------------------------------------------------------------------------- in 64 bits


def _steps(cu):
    """For each step the tokens at that place of the sequences that reach it, and those sequences."""
    lens = [b - a for a, b in zip(cu, cu[1:])]
    order = sorted(range(len(lens)), key=lambda k: -lens[k])
    where = torch.tensor([cu[k] for k in order], device="cuda")
    order_t = torch.tensor(order, device="cuda")
    live = len(order)
    for i in range(max(lens, default=0)):
        while lens[order[live - 1]] <= i:
            live -= 1
        yield where[:live] + i, order_t[:live]


def _exact_scan(s):
    c = s["c"]
    D, N, G = c["D"], c["N"], c["G"]
    R, train = s["x"].shape[0] * s["x"].shape[1], s["go"] == "train"
    f = lambda k: s[k].double()  # noqa: E731
    x, raw = f("x").reshape(R, D), f("dt").reshape(R, D) + f("dt_bias")
    delta = torch.where(raw > 20, raw, torch.nn.functional.softplus(raw, threshold=1e9))
    A = -f("A_log").exp()
    Bm, Cm, skip = f("Bm").reshape(R, G, 1, N), f("Cm").reshape(R, G, 1, N), f("D")
    state = f("state")
    y, seen = torch.zeros_like(x), []
    for tok, seq in _steps(s["cu_host"]):
        old = state[seq]
        d = delta[tok][..., None]
        k = len(tok)
        u = (d * x[tok][..., None]).view(k, G, -1, 1) * Bm[tok]
        new = torch.exp(d * A) * old + u.view(k, D, N)
        state[seq] = new
        y[tok] = (new.view(k, G, -1, N) * Cm[tok]).sum(-1).view(k, D)
        if train:
            seen.append((tok, seq, old, new))
    y += skip * x
    out = {"y": y.view(*s["shape"], D), "state": state}
    if not train:
        return out
    dy = f("dy").reshape(R, D)
    carry = f("dfinal")  # gradient of the state behind a token
    dx, ddelta = skip * dy, torch.zeros_like(x)
    dB, dC = torch.zeros(R, G, N, device="cuda").double(), torch.zeros(R, G, N, device="cuda").double()
    dA = torch.zeros_like(A)
    for tok, seq, old, new in reversed(seen):
        k = len(tok)
        d = delta[tok][..., None]
        dC[tok] = (dy[tok].view(k, G, -1, 1) * new.view(k, G, -1, N)).sum(2)
        gr = carry[seq] + (dy[tok].view(k, G, -1, 1) * Cm[tok]).view(k, D, N)
        du = (gr.view(k, G, -1, N) * Bm[tok]).sum(-1).view(k, D)
        dB[tok] = (gr.view(k, G, -1, N) * (d * x[tok][..., None]).view(k, G, -1, 1)).sum(2)
        decay = torch.exp(d * A)
        dlog = gr * old * decay
        dx[tok] += du * d[..., 0]
        ddelta[tok] = du * x[tok] + (dlog * A).sum(-1)
        dA += (dlog * d).sum(0)
        carry[seq] = gr * decay
    ddt = ddelta * torch.where(raw > 20, 1.0, torch.sigmoid(raw))
    sh = s["shape"]
    out.update(dx=dx.view(*sh, D), ddt=ddt.view(*sh, D), dA_log=dA * A, dB=dB.view(*sh, G, N), dC=dC.view(*sh, G, N),
               dD=(dy * x).sum(0), ddt_bias=ddt.sum(0), dstate=carry)
    return out


def _exact_conv(s):
    c, W = s["c"], s["c"]["W"]
    D = c["D"]
    leaves = [s[k].double().clone().requires_grad_(s["go"] == "train") for k in ("x", "state", "weight", "bias")]
    x, state, w, b = leaves
    flat, ys, ends = x.reshape(-1, D), [], []
    for k, (lo, hi) in enumerate(zip(s["cu_host"], s["cu_host"][1:])):
        line = torch.cat([state[k], flat[lo:hi]])
        ends.append(line[line.shape[0] - (W - 1):])
        if hi > lo:
            ys.append(sum(line[j:j + hi - lo] * w[:, j] for j in range(W)) + b)
    pre = torch.cat(ys).view(x.shape)
    y, end = pre * torch.sigmoid(pre), torch.stack(ends)
    out = {"y": y.detach(), "state": end.detach()}
    if s["go"] == "train":
        loss = (y * s["dy"].double()).sum() + (end * s["dfinal"].double()).sum()
        g = torch.autograd.grad(loss, leaves, allow_unused=True)
        out.update(dx=g[0], dstate=torch.zeros_like(state) if g[1] is None else g[1], dweight=g[2], dbias=g[3])
    return out


def _exact_norm(s):
    train = s["go"] == "train"
    keys = [k for k in ("x", "weight", "bias", "gate") if s[k] is not None]
    v = {k: s[k].double().clone().requires_grad_(train) for k in keys}
    x = v["x"]
    if not s["rms"]:
        x = x - x.mean(-1, keepdim=True)
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * v["weight"]
    if "bias" in v:
        y = y + v["bias"]
    if "gate" in v:
        y = y * torch.nn.functional.silu(v["gate"])
    out = {"y": y.detach()}
    if train:
        g = torch.autograd.grad((y * s["dy"].double()).sum(), [v[k] for k in keys])
        out.update({"d" + k: t for k, t in zip(keys, g)})
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"conv": _exact_conv, "scan": _exact_scan, "norm": _exact_norm}[s["op"]](s)
