"""The parts of a selective state space layer: cases to measure.

Selective scan.  Per batch row, channel c (of C) and state n (of N), with g = c // (C/G) the
channel's group:

    d_t = softplus(dt_t + dt_bias)      (or dt_t + dt_bias itself)
    h_t[n] = exp(d_t A[n]) h_{t-1}[n] + d_t u_t B_t[g,n]
    y_t = (sum_n C_t[g,n] h_t[n] + D u_t) * silu(z_t)      (no gate without z)

u, dt, z, y (B,T,C), B, C (B,T,G,N) of one type (bfloat16 or float32); A (C,N), D, dt_bias (C)
and the states (B,C,N) in float32.  ``lengths`` (B,) int32 makes tokens at or beyond a row's
length absent: they leave the state alone, their outputs and gradients are zero.

Short convolution, causal, one filter of K taps a channel, before such a scan:

    y_t = act(bias + sum_k weight[k] x_{t-K+1+k})

x, y (B,T,C) and the state (B,K-1,C), the inputs before the first token, of one type; weight
(C,K), bias (C) in float32.

Root-mean-square norm behind the residual's addition:

    s = x + r,   y = s / sqrt(mean(s^2) + eps) * weight

x, y (N,C) of one type, r and s (N,C) of that type or float32, weight (C) in float32; the norm is
that of s as stored.

The plain forms below take all tokens at once, in float32; ``exact`` walks the tokens one by one
in float64.
"""

from __future__ import annotations

import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases -----------------------------------------------------------------------------

def _scan(name, op, dt, B, T, C, N, G=1, z=True, softplus=True, state=False, ragged=False):
    return {"name": name, "op": op, "dtype": dt, "B": B, "T": T, "C": C, "N": N, "G": G, "z": z,
            "softplus": softplus, "state": state, "ragged": ragged}


def _conv(name, op, dt, B, T, C, K, state=False, ragged=False, act="silu"):
    return {"name": name, "op": op, "dtype": dt, "B": B, "T": T, "C": C, "K": K, "state": state, "ragged": ragged,
            "act": act}


def _norm(name, op, dt, rdt, N, C, residual=True):
    return {"name": name, "op": op, "dtype": dt, "rdtype": rdt, "N": N, "C": C, "residual": residual}


def listed():
    return [
        # A short prompt of one user, an odd length; latency counts.
        _scan("scan_short", "scan_forward", "bf16", 1, 77, 1536, 16),
        # B=8 T=1024, a layer of twice 768 channels.
        _scan("scan_B8_T1024", "scan_forward", "bf16", 8, 1024, 1536, 16),
        # One long document in pieces: the state is carried in and out.
        _scan("scan_long", "scan_forward", "bf16", 1, 32768, 2048, 16, state=True),
        # A serving batch of prompts of unlike lengths (an empty one and one of a single token
        # among them) in single precision: two groups, a channel count that no tile divides, no
        # gate, steps given as they are.
        _scan("scan_ragged_f32", "scan_forward", "f32", 16, 2000, 1000, 8, G=2, z=False, softplus=False, state=True,
              ragged=True),
        # A training step (forward and all gradients) at B=8 T=4096 C=2560.
        _scan("scan_train_B8_T4096", "scan_train", "bf16", 8, 4096, 2560, 16),
        # Training in single precision: two groups, a state of 24, ragged rows, carried states.
        _scan("scan_train_f32", "scan_train", "f32", 4, 500, 200, 24, G=2, state=True, ragged=True),
        # One token for each of 64 users.
        _scan("scan_step_B64", "scan_step", "bf16", 64, 1, 5120, 16, state=True),
        # The convolution over a serving batch of ragged prompts that go on from earlier inputs.
        _conv("conv_ragged", "conv_forward", "bf16", 16, 2000, 2560, 4, state=True, ragged=True),
        # The convolution of a training step at B=8 T=4096 C=2560.
        _conv("conv_train", "conv_train", "bf16", 8, 4096, 2560, 4),
        # One token of the convolution for each of 64 users.
        _conv("conv_step_B64", "conv_step", "bf16", 64, 1, 5120, 4, state=True),
        # The norm of a decode step for 64 users, its residual stream in float32.
        _norm("norm_step", "norm_forward", "bf16", "f32", 64, 2560),
        # The norm of a training step at B=8 T=4096 C=2560: forward and all gradients.
        _norm("norm_train", "norm_train", "bf16", "bf16", 32768, 2560),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["scan_forward", "scan_forward", "scan_train", "scan_train", "scan_step", "conv_forward",
                     "conv_train", "conv_step", "norm_forward", "norm_train"])
    dt = rng.choice(["bf16", "bf16", "f32"])
    most = 8 * 4096 * 2560 // (1 if dt == "bf16" else 2)
    if op.startswith("norm"):
        while True:
            N, C = _logint(rng, 1, 32768), _logint(rng, 16, 8192)
            if N * C <= most:
                break
        c = _norm("", op, dt, rng.choice([dt, "f32"]), N, C, rng.random() < 0.8)
    else:
        while True:
            B, T, C = _logint(rng, 1, 64), _logint(rng, 1, 32768), _logint(rng, 16, 5120)
            if op.endswith("step"):
                T = 1
            if op == "scan_train":
                T = min(T, 4096)
            N = rng.choice([16, 16, 8, _logint(rng, 1, 64)])
            if op.startswith("conv") and B * T * C <= most or op.startswith("scan") and B * T * C * N <= most * 16:
                break
        state, ragged = rng.random() < 0.5 or T == 1, rng.random() < 0.4 and not op.endswith("step")
        if op.startswith("conv"):
            c = _conv("", op, dt, B, T, C, rng.choice([4, 4, 3, 2, _logint(rng, 1, 8)]), state, ragged,
                      rng.choice(["silu", "silu", "none"]))
        else:
            G = rng.choice([1, 1, 1, 2, 4])
            c = _scan("", op, dt, B, T, G * max(1, C // G), N, G, rng.random() < 0.7, rng.random() < 0.8, state, ragged)
    del c["name"]
    return c


def _lengths(case):
    """Row lengths of a ragged batch: spread over [0, T], with 0, 1 and T among them where
    the batch has room for them."""
    B, T = case["B"], case["T"]
    out = [max(0, T - (T * 7 * i) // (8 * B) - (i % 3)) for i in range(B)]
    if B > 1:
        out[1] = 0
    if B > 2:
        out[2] = min(1, T)
    out[0] = T
    return out


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"].startswith("norm"):
        n, C, r = case["N"] * case["C"], case["C"], 2 if case["rdtype"] == "bf16" else 4
        res = case["residual"]
        fwd = {"bytes": n * (2 * e + (2 * r if res else 0)) + 4 * C, "flops": n * 5}
        if case["op"] == "norm_forward":
            return fwd
        # A step: the forward, and a backward that reads s and both upstream gradients and
        # writes the sum's gradient (and x's, where that is of another type).
        other = e if res and r != e else 0
        return {"bytes": fwd["bytes"] + n * (e + (3 * r if res else 3 * e) + other) + 8 * C, "flops": n * 17}
    B, C = case["B"], case["C"]
    tokens = sum(_lengths(case)) if case["ragged"] else B * case["T"]
    n = tokens * C
    if case["op"].startswith("conv"):
        K, st = case["K"], B * (case["K"] - 1) * C * e
        states = st * (2 if case["state"] else 1)
        par = 4 * C * (K + 1)
        fwd = {"bytes": 2 * n * e + states + par, "flops": n * (2 * K + 5)}
        if case["op"] != "conv_train":
            return fwd
        return {"bytes": fwd["bytes"] + 3 * n * e + (states + st if case["state"] else 0) + 2 * par,
                "flops": n * (8 * K + 20)}
    N, gates = case["N"], 1 if case["z"] else 0
    st = 4 * B * C * N
    bc = 2 * tokens * case["G"] * N * e
    par = 4 * C * (N + 2)
    fwd = {"bytes": n * e * (3 + gates) + bc + st * (2 if case["state"] else 1) + par,
           "flops": n * (7 * N + 10 + 5 * gates)}
    if case["op"] != "scan_train":
        return fwd
    # A step: the forward, and a backward that reads u, dt, z, B, C and the upstream gradients and
    # writes all gradients.
    return {"bytes": fwd["bytes"] + n * e * (5 + 2 * gates) + 2 * bc + (3 * st if case["state"] else 0) + 2 * par,
            "flops": fwd["flops"] + n * (25 * N + 20 + 10 * gates)}


# ---- inputs ----------------------------------------------------------------------------

def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32)

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device=dev, dtype=torch.float32)

    dt = _DT[case["dtype"]]
    op = case["op"]
    st = {"case": dict(case)}
    if op.startswith("norm"):
        N, C, rdt = case["N"], case["C"], _DT[case["rdtype"]]
        st["x"] = normal(N, C).to(dt)
        st["residual"] = (2.0 * normal(N, C) + 0.5 * normal(C)).to(rdt) if case["residual"] else None
        st["weight"] = 1.0 + 0.2 * normal(C)
        st["eps"] = 1e-5
        if op == "norm_train":
            st["gy"] = normal(N, C).to(dt)
            st["gsum"] = normal(N, C).to(rdt) if case["residual"] else None
        return st
    B, T, C = case["B"], case["T"], case["C"]
    lead = (B,) if op.endswith("step") else (B, T)
    st["lengths"] = torch.tensor(_lengths(case), dtype=torch.int32, device=dev) if case["ragged"] else None
    if op.startswith("conv"):
        K = case["K"]
        st["x"] = normal(*lead, C).to(dt)
        st["weight"] = K ** -0.5 * (2.0 * uniform(C, K) - 1.0)
        st["bias"] = 0.1 * normal(C)
        st["state"] = normal(B, K - 1, C).to(dt) if case["state"] else None
        if op == "conv_train":
            st["gy"] = normal(B, T, C).to(dt)
            st["gstate"] = normal(B, K - 1, C).to(dt) if case["state"] else None
        if op == "conv_step":
            st["state_out"] = torch.empty_like(st["state"])
        return st
    N, G = case["N"], case["G"]
    x = normal(*lead, C)
    st["u"] = (x / (1.0 + torch.exp(-x))).to(dt)
    # Decays A from -1 to -N over the states; steps from 1e-3 to 1e-1 over the channels.
    st["A"] = -torch.arange(1, N + 1, device=dev, dtype=torch.float32) * torch.exp(0.1 * normal(C, N))
    step = torch.exp(math.log(1e-3) + uniform(C) * math.log(1e2))
    if case["softplus"]:
        st["dt"] = (0.5 * normal(*lead, C)).to(dt)
        st["dt_bias"] = step + torch.log(-torch.expm1(-step))
    else:
        st["dt"] = (step * torch.exp(0.5 * normal(*lead, C))).to(dt)
        st["dt_bias"] = None
    st["B"], st["C"] = normal(*lead, G, N).to(dt), normal(*lead, G, N).to(dt)
    st["D"] = 1.0 + 0.1 * normal(C)
    st["z"] = normal(*lead, C).to(dt) if case["z"] else None
    st["state"] = 0.3 * normal(B, C, N) if case["state"] else None
    if op == "scan_train":
        st["gy"] = normal(B, T, C).to(dt)
        st["gstate"] = 0.3 * normal(B, C, N) if case["state"] else None
    if op == "scan_step":
        st["state_out"] = torch.empty_like(st["state"])
    return st


# ---- the calls -------------------------------------------------------------------------

def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if not own:
        return _PLAIN[op](s, case)
    import linear_recurrence_rnn_amd as L

    if op.startswith("norm"):
        y, total = L.rms_norm_add(s["x"], s["weight"], residual=s["residual"], eps=s["eps"])
        if op == "norm_forward":
            return [y] + ([total] if case["residual"] else [])
        gx, gtotal, gw = L.rms_norm_add_backward(total, s["weight"], s["gy"], gsum=s["gsum"], eps=s["eps"])
        return [y, total, gx, gtotal, gw] if case["residual"] else [y, gx, gw]
    if op.startswith("conv"):
        if op == "conv_step":
            y = L.short_conv_decode_step(s["x"], s["weight"], s["state"], bias=s["bias"], act=case["act"],
                                         state_out=s["state_out"])
            return [y, s["state_out"]]
        keep = {"bias": s["bias"], "act": case["act"], "state": s["state"], "lengths": s["lengths"]}
        y, state_out = L.short_conv_act(s["x"], s["weight"], **keep)
        if op == "conv_forward":
            return [y, state_out]
        grads = L.short_conv_act_backward(s["x"], s["weight"], s["gy"], gstate=s["gstate"], **keep)
        return [y, state_out] + [g for g in grads if g is not None]
    args = [s[n] for n in ("u", "dt", "A", "B", "C")]
    keep = {"D": s["D"], "z": s["z"], "dt_bias": s["dt_bias"], "softplus": case["softplus"]}
    if op == "scan_step":
        y = L.scan_selective_decode_step(*args, s["state"], state_out=s["state_out"], **keep)
        return [y, s["state_out"]]
    keep.update(state=s["state"], lengths=s["lengths"])
    if op == "scan_forward":
        return list(L.scan_selective(*args, **keep))
    y, state_out, ckpt = L.scan_selective_ckpt(*args, **keep)
    grads = L.scan_selective_backward(*args, s["gy"], gstate=s["gstate"], ckpt=ckpt, **keep)
    return [y, state_out] + [g for g in grads if g is not None]


# ---- plain forms -----------------------------------------------------------------------

def _sigmoid(x):
    return 1.0 / (1.0 + torch.exp(-x))


def _softplus(x):
    return torch.clamp(x, min=0.0) + torch.log1p(torch.exp(-torch.abs(x)))


def _silu_both(x):
    """silu(x) and its derivative."""
    sg = _sigmoid(x)
    return x * sg, sg * (1.0 + x * (1.0 - sg))


def _live(s, case):
    """(B,T,1) truth values of the tokens that are there, or None where all are."""
    if s["lengths"] is None:
        return None
    t = torch.arange(case["T"], device=s["lengths"].device)
    return (t[None, :] < s["lengths"][:, None])[:, :, None]


def _affine_scan(a, b):
    """h_t = a_t h_{t-1} + b_t over axis 1 from h_{-1} = 0, by doubling strides."""
    d, T = 1, a.shape[1]
    while d < T:
        b = torch.cat([b[:, :d], b[:, d:] + a[:, d:] * b[:, :-d]], dim=1)
        a = torch.cat([a[:, :d], a[:, d:] * a[:, :-d]], dim=1)
        d *= 2
    return b


def _per_channel(x, C):
    """(..., G, N) -> (..., C, N)."""
    return x.float().repeat_interleave(C // x.shape[-2], dim=-2)


def _plain_scan_step(s, case):
    u, A = s["u"].float(), s["A"]
    raw = s["dt"].float() + (s["dt_bias"] if s["dt_bias"] is not None else 0.0)
    d = _softplus(raw) if case["softplus"] else raw
    B, C = _per_channel(s["B"], case["C"]), _per_channel(s["C"], case["C"])
    h = torch.exp(d[..., None] * A) * s["state"] + (d * u)[..., None] * B
    y = torch.sum(C * h, dim=-1) + s["D"] * u
    if s["z"] is not None:
        z = s["z"].float()
        y = y * z * _sigmoid(z)
    return [y.to(s["u"].dtype), h]


def _plain_scan(s, case, grads):
    Bn, T, Cn, N, G = (case[n] for n in ("B", "T", "C", "N", "G"))
    dt, live, A, D = s["u"].dtype, _live(s, case), s["A"], s["D"]
    u = s["u"].float()
    raw = s["dt"].float() + (s["dt_bias"] if s["dt_bias"] is not None else 0.0)
    d = _softplus(raw) if case["softplus"] else raw
    if live is not None:
        d = torch.where(live, d, torch.zeros_like(d))
    B, C = _per_channel(s["B"], Cn), _per_channel(s["C"], Cn)
    a = torch.exp(d[..., None] * A)
    b = (d * u)[..., None] * B
    if s["state"] is not None:
        b[:, 0] += a[:, 0] * s["state"]
    h = _affine_scan(a, b)
    del b
    core = torch.sum(C * h, dim=-1) + D * u
    gate = dgate = None
    y = core
    if s["z"] is not None:
        gate, dgate = _silu_both(s["z"].float())
        y = core * gate
    if live is not None:
        y = torch.where(live, y, torch.zeros_like(y))
    res = [y.to(dt), h[:, -1].clone()]
    if not grads:
        return res
    gy = s["gy"].float()
    if live is not None:
        gy = torch.where(live, gy, torch.zeros_like(gy))
    gz = None
    if gate is not None:
        gz = gy * core * dgate
        gy = gy * gate
    # gh_t = C_t gy_t + a_{t+1} gh_{t+1}: the same scan over the tokens in reverse.
    e = C * gy[..., None]
    if s["gstate"] is not None:
        e[:, -1] += s["gstate"]
    ar = torch.cat([torch.ones_like(a[:, :1]), torch.flip(a, [1])[:, :-1]], dim=1)
    gh = torch.flip(_affine_scan(ar, torch.flip(e, [1])), [1])
    del e, ar
    if live is not None:  # what passes an absent token is the final state's gradient alone
        ghl = torch.where(live[..., None], gh, torch.zeros_like(gh))
    else:
        ghl = gh
    gC = torch.sum((gy[..., None] * h).view(Bn, T, G, Cn // G, N), dim=3)
    gB = torch.sum((ghl * (d * u)[..., None]).view(Bn, T, G, Cn // G, N), dim=3)
    gBu = torch.sum(ghl * B, dim=-1)
    first = s["state"][:, None] if s["state"] is not None else torch.zeros_like(h[:, :1])
    m = ghl * a * torch.cat([first, h[:, :-1]], dim=1)
    gstate = a[:, 0] * gh[:, 0] if s["state"] is not None else None
    del gh, ghl, h, a
    gd = torch.sum(m * A, dim=-1) + u * gBu
    gA = torch.sum(m * d[..., None], dim=(0, 1))
    graw = gd * _sigmoid(raw) if case["softplus"] else gd
    gu = D * gy + d * gBu
    gD = torch.sum(gy * u, dim=(0, 1))
    res += [gu.to(dt), graw.to(dt), gA, gB.to(dt), gC.to(dt), gD]
    if gz is not None:
        res.append(gz.to(dt))
    if s["dt_bias"] is not None:
        res.append(torch.sum(graw, dim=(0, 1)))
    return res + ([gstate] if gstate is not None else [])


def _act(x, act):
    return _silu_both(x) if act == "silu" else (x, torch.ones_like(x))


def _plain_conv(s, case, grads):
    Bn, C, K = case["B"], case["C"], case["K"]
    dt, w = s["x"].dtype, s["weight"]
    step = case["op"] == "conv_step"
    x = s["x"].float()[:, None] if step else s["x"].float()
    T = x.shape[1]
    first = s["state"].float() if s["state"] is not None else x.new_zeros(Bn, K - 1, C)
    xp = torch.cat([first, x], dim=1)
    win = xp.unfold(1, K, 1)  # (B,T,C,K)
    pre = torch.sum(win * w, dim=-1) + s["bias"]
    y, dact = _act(pre, case["act"])
    live = None if step else _live(s, case)
    if live is not None:
        y = torch.where(live, y, torch.zeros_like(y))
        last = s["lengths"].long()[:, None] + torch.arange(K - 1, device=x.device)
        keep = torch.gather(xp, 1, last[..., None].expand(Bn, K - 1, C))
    else:
        keep = xp[:, T:]
    res = [(y[:, 0] if step else y).to(dt), keep.to(dt)]
    if not grads:
        return res
    g = s["gy"].float() * dact
    if live is not None:
        g = torch.where(live, g, torch.zeros_like(g))
    pad = x.new_zeros(Bn, K - 1, C)
    gxp = torch.sum(torch.cat([pad, g, pad], dim=1).unfold(1, K, 1) * torch.flip(w, [1]), dim=-1)
    if s["gstate"] is not None:
        if live is not None:
            gxp.scatter_add_(1, last[..., None].expand(Bn, K - 1, C), s["gstate"].float())
        else:
            gxp[:, T:] += s["gstate"].float()
    if live is not None:
        win = torch.where(live[..., None], win, torch.zeros_like(win))
    res += [gxp[:, K - 1:].to(dt), torch.sum(win * g[..., None], dim=(0, 1)), torch.sum(g, dim=(0, 1))]
    return res + ([gxp[:, :K - 1].to(dt)] if s["state"] is not None else [])


def _plain_norm(s, case, grads):
    dt, rdt = s["x"].dtype, _DT[case["rdtype"]]
    w = s["weight"]
    total = s["x"]
    if case["residual"]:
        total = (s["x"].float() + s["residual"].float()).to(rdt)
    x = total.float()
    r = torch.rsqrt(torch.mean(x * x, dim=-1, keepdim=True) + s["eps"])
    n = x * r
    y = (n * w).to(dt)
    res = [y, total] if case["residual"] else [y]
    if not grads:
        return res
    gy = s["gy"].float()
    dn = gy * w
    gs = r * (dn - n * torch.mean(dn * n, dim=-1, keepdim=True))
    gw = torch.sum(gy * n, dim=0)
    if case["residual"]:
        gs = gs + s["gsum"].float()
        return res + [gs.to(dt), gs.to(rdt), gw]
    return res + [gs.to(dt), gw]


_PLAIN = {
    "scan_forward": lambda s, c: _plain_scan(s, c, False),
    "scan_train": lambda s, c: _plain_scan(s, c, True),
    "scan_step": _plain_scan_step,
    "conv_forward": lambda s, c: _plain_conv(s, c, False),
    "conv_train": lambda s, c: _plain_conv(s, c, True),
    "conv_step": lambda s, c: _plain_conv(s, c, False),
    "norm_forward": lambda s, c: _plain_norm(s, c, False),
    "norm_train": lambda s, c: _plain_norm(s, c, True),
}


# ---- the definition in float64, one token after the other ------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    f = {n: v.double() for n, v in s.items() if isinstance(v, torch.Tensor) and n != "lengths"}
    if case["op"].startswith("norm"):
        return _exact_norm(f, s, case)
    if case["op"].startswith("conv"):
        return _exact_conv(f, s, case)
    return _exact_scan(f, s, case)


def _exact_scan(f, s, case):
    B, T, C, N, G = (case[n] for n in ("B", "T", "C", "N", "G"))
    train = case["op"] == "scan_train"
    if B * T * C * N * 8 > 60e9:
        return None  # the states of all tokens would not fit beside the rest
    one = case["op"] == "scan_step"
    tok = (lambda name, t: f[name]) if one else (lambda name, t: f[name][:, t])
    rows = torch.tensor(_lengths(case) if case["ragged"] else [T] * B, device=f["u"].device)
    pos = f["A"].new_zeros(B, C, N)
    h = f["state"].clone() if "state" in f else pos.clone()
    kept, ys, cores = [h], [], []

    def raw_of(t):
        return tok("dt", t) + (f["dt_bias"] if "dt_bias" in f else 0.0)

    def step_of(t):
        r = raw_of(t)
        return torch.logaddexp(r, torch.zeros_like(r)) if case["softplus"] else r

    def spread(x):  # (B,G,N) -> (B,C,N)
        return x[:, :, None, :].expand(B, G, C // G, N).reshape(B, C, N)

    for t in range(T):
        on = (t < rows)[:, None]
        d, u = step_of(t), tok("u", t)
        new = torch.exp(d[:, :, None] * f["A"]) * h + (d * u)[:, :, None] * spread(tok("B", t))
        h = torch.where(on[:, :, None], new, h)
        core = (spread(tok("C", t)) * h).sum(-1) + f["D"] * u
        y = core
        if "z" in f:
            z = tok("z", t)
            y = core * (z * torch.special.expit(z))
        ys.append(torch.where(on, y, torch.zeros_like(y)))
        if train:
            kept.append(h)
            cores.append(core)
    if one:
        return [ys[0], h]
    y = torch.stack(ys, dim=1)
    if not train:
        return [y, h]
    gh = f["gstate"].clone() if "gstate" in f else pos.clone()
    gA, gD, gbias = torch.zeros_like(f["A"]), torch.zeros_like(f["D"]), torch.zeros_like(f["D"])
    gu, gdt, gz = (torch.zeros_like(f["u"]) for _ in range(3))
    gB, gC = torch.zeros_like(f["B"]), torch.zeros_like(f["C"])
    for t in reversed(range(T)):
        on = (t < rows)[:, None]
        d, u, g = step_of(t), tok("u", t), f["gy"][:, t]
        g = torch.where(on, g, torch.zeros_like(g))
        if "z" in f:
            z = tok("z", t)
            sg = torch.special.expit(z)
            gz[:, t] = g * cores[t] * (sg + z * sg * (1.0 - sg))
            g = g * z * sg
        Bt, Ct = spread(tok("B", t)), spread(tok("C", t))
        full = gh + Ct * g[:, :, None]
        ga = full * torch.exp(d[:, :, None] * f["A"])
        full = torch.where(on[:, :, None], full, pos)
        m = torch.where(on[:, :, None], ga * kept[t], pos)
        gC[:, t] = (g[:, :, None] * kept[t + 1]).view(B, G, C // G, N).sum(2)
        gB[:, t] = (full * (d * u)[:, :, None]).view(B, G, C // G, N).sum(2)
        into = (full * Bt).sum(-1)
        gd = (m * f["A"]).sum(-1) + u * into
        gA += (m * d[:, :, None]).sum(0)
        if case["softplus"]:
            gd = gd * torch.special.expit(raw_of(t))
        gdt[:, t] = gd
        gbias += gd.sum(0)
        gu[:, t] = f["D"] * g + d * into
        gD += (g * u).sum(0)
        gh = torch.where(on[:, :, None], ga, gh)
    res = [y, h, gu, gdt, gA, gB, gC, gD]
    if "z" in f:
        res.append(gz)
    if "dt_bias" in f:
        res.append(gbias)
    return res + ([gh] if "state" in f else [])


def _exact_conv(f, s, case):
    B, T, C, K = (case[n] for n in ("B", "T", "C", "K"))
    x = f["x"].view(B, T, C)
    w = f["weight"]
    line = x.new_zeros(B, T + K - 1, C)
    line[:, K - 1:] = x
    if "state" in f:
        line[:, :K - 1] = f["state"]
    pre = f["bias"].expand(B, T, C).clone()
    for k in range(K):
        pre += w[:, k] * line[:, k:k + T]
    sg = torch.special.expit(pre) if case["act"] == "silu" else torch.ones_like(pre)
    y = pre * sg
    rows = _lengths(case) if case["ragged"] else [T] * B
    keep = torch.stack([line[b, n:n + K - 1] for b, n in enumerate(rows)])
    for b, n in enumerate(rows):
        y[b, n:] = 0.0
    if case["op"] == "conv_step":
        return [y[:, 0], keep]
    if case["op"] == "conv_forward":
        return [y, keep]
    g = f["gy"] * (sg + pre * sg * (1.0 - sg) if case["act"] == "silu" else 1.0)
    for b, n in enumerate(rows):
        g[b, n:] = 0.0
    gline, gw = torch.zeros_like(line), torch.zeros_like(w)
    for k in range(K):
        gline[:, k:k + T] += w[:, k] * g
        gw[:, k] = (g * line[:, k:k + T]).sum((0, 1))
    if "gstate" in f:
        for b, n in enumerate(rows):
            gline[b, n:n + K - 1] += f["gstate"][b]
    res = [y, keep, gline[:, K - 1:], gw, g.sum((0, 1))]
    return res + ([gline[:, :K - 1]] if "state" in f else [])


def _exact_norm(f, s, case):
    x = f["x"]
    total = x
    if case["residual"]:
        # s is what the sum is stored as; the norm and its gradients are those of that value.
        total = x + f["residual"]
        x = total.to(_DT[case["rdtype"]]).double()
    var = (x ** 2).mean(-1, keepdim=True) + s["eps"]
    y = x / var.sqrt() * f["weight"]
    res = [y, total] if case["residual"] else [y]
    if case["op"] == "norm_forward":
        return res
    v = f["gy"] * f["weight"]
    gs = v / var.sqrt() - x * (v * x).mean(-1, keepdim=True) / var ** 1.5
    gw = (f["gy"] * x / var.sqrt()).sum(0)
    if case["residual"]:
        gs = gs + f["gsum"]
        return res + [gs, gs, gw]
    return res + [gs, gw]
