"""The gated delta rule and the per-token group norm that follows it: cases to measure.

Two operators of a time-mix layer whose state is a matrix per head.

Gated delta rule.  Per batch row and value head, with S (Dk, Dv) the state, a_t = e^{g_t}:

    x_t = v_t - (a_t S_{t-1})^T k_t
    S_t = a_t S_{t-1} + beta_t k_t x_t^T
    o_t = scale * S_t^T q_t

q, k (B,T,Hk,Dk), v (B,T,Hv,Dv), g, beta (B,T,Hv), all of one type (bfloat16 or float32), states
(B,Hv,Dk,Dv) in float32.  Value head h reads key head h // (Hv / Hk).  ``lengths`` (B,) int32 makes tokens at or beyond a
row's length absent: they leave the state alone, their outputs and gradients are zero.

Group norm with an activation, channels last.  Each token's C channels are normalised in G
groups of C/G (biased variance), y = n * weight + bias, and the output is act(y), or
y * act(gate) where a gate is given.

The plain forms below are chunked torch products in float32; ``exact`` walks the tokens one
by one in float64.
"""

from __future__ import annotations

import math

import torch

own = False

CHUNK = 64

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases -----------------------------------------------------------------------------

def _fwd(name, dt, B, T, Hk, Hv, Dk, Dv, state=False, ragged=False):
    return {"name": name, "op": "delta_forward", "dtype": dt, "B": B, "T": T, "Hk": Hk, "Hv": Hv, "Dk": Dk,
            "Dv": Dv, "state": state, "ragged": ragged}


def _train(name, dt, B, T, Hk, Hv, Dk, Dv, state=False, ragged=False):
    return dict(_fwd(name, dt, B, T, Hk, Hv, Dk, Dv, state, ragged), op="delta_train")


def _step(name, dt, B, Hk, Hv, Dk, Dv):
    return {"name": name, "op": "delta_step", "dtype": dt, "B": B, "Hk": Hk, "Hv": Hv, "Dk": Dk, "Dv": Dv}


def _norm(name, op, dt, N, C, G, gate):
    return {"name": name, "op": op, "dtype": dt, "N": N, "C": C, "G": G, "gate": gate, "act": "silu"}


def listed():
    return [
        # A short prompt of one user: 12 heads of 64 (C=768), an odd length; latency counts.
        _fwd("prefill_short", "bf16", 1, 77, 12, 12, 64, 64),
        # The forward headline's shape, B=8 T=1024 C=768, as heads of 64.
        _fwd("forward_B8_T1024", "bf16", 8, 1024, 12, 12, 64, 64),
        # A serving batch of prompts of unlike lengths (an empty one and one of a single token
        # among them) that go on from earlier states; two value heads to a key head.
        _fwd("prefill_ragged", "bf16", 16, 2000, 4, 8, 128, 128, True, True),
        # One long document: few heads, a long chain.
        _fwd("prefill_long", "bf16", 1, 32768, 8, 16, 128, 128),
        # Single precision, odd length and head sizes that are no power of two.
        _fwd("forward_f32", "f32", 2, 999, 4, 4, 96, 80, True),
        # A training step (forward and all gradients) at the backward workload's size, B=8
        # T=4096 C=2560, as 20 heads of 128.
        _train("train_B8_T4096", "bf16", 8, 4096, 20, 20, 128, 128),
        # Training in single precision: three value heads share a key head, odd sizes, ragged rows.
        _train("train_f32", "f32", 4, 500, 2, 6, 48, 100, True, True),
        # One token for one user.
        _step("step_B1", "bf16", 1, 12, 12, 64, 64),
        # One token for each of 64 users: 20 heads of 128.
        _step("step_B64", "bf16", 64, 20, 20, 128, 128),
        # The norm behind such a decode step: 64 tokens, C=2560, gated.
        _norm("norm_step", "norm_forward", "bf16", 64, 2560, 20, True),
        # The norm of a training step at B=8 T=4096 C=2560: forward and all gradients, gated.
        _norm("norm_train", "norm_train", "bf16", 32768, 2560, 20, True),
        # Single precision, groups of 125 channels, the activation on the norm itself.
        _norm("norm_train_f32", "norm_train", "f32", 2997, 1000, 8, False),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["delta_forward", "delta_forward", "delta_train", "delta_train", "delta_step", "norm_forward",
                     "norm_train"])
    dt = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("norm"):
        while True:
            N, G, D = _logint(rng, 1, 32768), _logint(rng, 1, 40), _logint(rng, 16, 512)
            if N * G * D <= (32768 * 2560) // (1 if dt == "bf16" else 2) and G * D <= 8192:
                break
        c = _norm("", op, dt, N, G * D, G, rng.random() < 0.6)
        c["act"] = rng.choice(["silu", "silu", "none"])
    else:
        while True:
            Hk, r = _logint(rng, 1, 20), rng.choice([1, 1, 2, 3])
            Dk = rng.choice([64, 128, _logint(rng, 16, 128)])
            Dv = rng.choice([64, 128, Dk, _logint(rng, 16, 128)])
            if op == "delta_step":
                B, T = _logint(rng, 1, 64), 1
            else:
                B, T = _logint(rng, 1, 16), _logint(rng, 2, 32768 if op == "delta_forward" else 4096)
            cap = 8 * 4096 * 20 * 128 if op == "delta_train" else 32768 * 16 * 128
            if dt == "f32":
                cap //= 4
            if op == "delta_step":
                cap = 64 * 20 * 128
            if B * T * Hk * r * max(Dk, Dv) <= cap:
                break
        if op == "delta_step":
            c = _step("", dt, B, Hk, Hk * r, Dk, Dv)
        else:
            c = _fwd("", dt, B, T, Hk, Hk * r, Dk, Dv, rng.random() < 0.5, rng.random() < 0.4)
            c["op"] = op
    del c["name"]
    return c


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"].startswith("norm"):
        n, C = case["N"] * case["C"], case["C"]
        g = 1 if case["gate"] else 0
        fwd = {"bytes": n * e * (2 + g) + 8 * C, "flops": n * (12 + 4 * g)}
        if case["op"] == "norm_forward":
            return fwd
        # A step: forward, and a backward that reads x, gate and the upstream gradient.
        return {"bytes": fwd["bytes"] + n * e * (3 + 2 * g) + 16 * C, "flops": fwd["flops"] + n * (24 + 8 * g)}
    B, Hk, Hv, Dk, Dv = (case[k] for k in ("B", "Hk", "Hv", "Dk", "Dv"))
    st = 4 * B * Hv * Dk * Dv
    if case["op"] == "delta_step":
        return {"bytes": 2 * st + B * e * (2 * Hk * Dk + 2 * Hv * Dv + 2 * Hv), "flops": 9 * B * Hv * Dk * Dv}
    T = sum(_lengths(case)) / B if case["ragged"] else case["T"]
    qk, v, gb, C = B * T * Hk * Dk * e, B * T * Hv * Dv * e, B * T * Hv * e, CHUNK
    states = st * (2 if case["state"] else 1)
    fwd_b = 2 * qk + 2 * v + 2 * gb + states
    # Per token and head, in chunks of C: three products with the state, and the lower
    # triangles of the products within the chunk.
    fwd_f = B * T * Hv * (6 * Dk * Dv + C * (2 * Dk + 2 * Dv))
    if case["op"] == "delta_forward":
        return {"bytes": int(fwd_b), "flops": int(fwd_f)}
    bwd_b = 4 * qk + 3 * v + 4 * gb + st * (3 if case["state"] else 1)
    bwd_f = fwd_f + B * T * Hv * (12 * Dk * Dv + C * (4 * Dk + 4 * Dv))
    return {"bytes": int(fwd_b + bwd_b), "flops": int(fwd_f + bwd_f)}


def _lengths(case):
    """Row lengths of a ragged batch: spread over [0, T], with 0, 1 and T among them where
    the batch has room for them."""
    B, T = case["B"], case["T"]
    out = [T - (T * 7 * i) // (8 * B) - (i % 3) for i in range(B)]
    out = [max(0, x) for x in out]
    if B > 1:
        out[1] = 0
    if B > 2:
        out[2] = min(1, T)
    out[0] = T
    return out


# ---- inputs ----------------------------------------------------------------------------

def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32)

    dt = _DT[case["dtype"]]
    st = {"case": dict(case)}
    if case["op"].startswith("norm"):
        N, C = case["N"], case["C"]
        st["x"] = (normal(N, C) * 0.3 + 0.1 * normal(C)).to(dt)
        st["gate"] = normal(N, C).to(dt) if case["gate"] else None
        st["weight"] = 1.0 + 0.2 * normal(C)
        st["bias"] = 0.1 * normal(C)
        if case["op"] == "norm_train":
            st["go"] = normal(N, C).to(dt)
        st["eps"] = 1e-5
        return st
    B, Hk, Hv, Dk, Dv = (case[k] for k in ("B", "Hk", "Hv", "Dk", "Dv"))
    T = case.get("T", 1)
    lead = (B,) if case["op"] == "delta_step" else (B, T)

    def unit(*shape):
        x = normal(*shape)
        return (x / torch.sqrt(torch.sum(x * x, dim=-1, keepdim=True) + 1e-6)).to(dt)

    st["q"], st["k"] = unit(*lead, Hk, Dk), unit(*lead, Hk, Dk)
    st["v"] = normal(*lead, Hv, Dv).to(dt)
    # Decays from nearly none to strong over the heads: e^g has a half life of a few hundred
    # tokens on the first head, of about one on the last.
    rate = torch.exp(torch.linspace(math.log(2e-3), 0.0, Hv, device=dev))
    st["g"] = (-rate * torch.log1p(torch.exp(normal(*lead, Hv)))).to(dt)
    st["beta"] = (1.0 / (1.0 + torch.exp(-normal(*lead, Hv)))).to(dt)
    st["scale"] = Dk ** -0.5
    with_state = case["op"] == "delta_step" or case["state"]
    st["state"] = 0.3 * normal(B, Hv, Dk, Dv) if with_state else None
    ragged = case.get("ragged", False)
    st["lengths"] = torch.tensor(_lengths(case), dtype=torch.int32, device=dev) if ragged else None
    if case["op"] == "delta_train":
        st["go"] = normal(B, T, Hv, Dv).to(dt)
        st["gstate"] = 0.3 * normal(B, Hv, Dk, Dv) if case["state"] else None
    if case["op"] == "delta_step":
        st["state_out"] = torch.empty_like(st["state"])
    return st


# ---- the calls -------------------------------------------------------------------------

def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if not own:
        return _PLAIN[op](s, case)
    import linear_recurrence_rnn_amd as L

    if op == "norm_forward":
        return L.group_norm_act(s["x"], case["G"], s["weight"], s["bias"], gate=s["gate"], act=case["act"],
                                eps=s["eps"])
    if op == "norm_train":
        y = L.group_norm_act(s["x"], case["G"], s["weight"], s["bias"], gate=s["gate"], act=case["act"],
                             eps=s["eps"])
        gx, gw, gb, gg = L.group_norm_act_backward(s["x"], case["G"], s["weight"], s["bias"], s["go"], gate=s["gate"],
                                                   act=case["act"], eps=s["eps"])
        return [y, gx, gw, gb] + ([gg] if gg is not None else [])
    if op == "delta_step":
        o = L.gated_delta_decode_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], scale=s["scale"],
                                      state_out=s["state_out"])
        return [o, s["state_out"]]
    args = [s[n] for n in ("q", "k", "v", "g", "beta")]
    keep = {n: s[n] for n in ("state", "lengths", "scale")}
    if op == "delta_forward":
        return list(L.gated_delta_forward(*args, **keep))
    o, state_out, ckpt = L.gated_delta_forward_ckpt(*args, **keep)
    grads = L.gated_delta_backward(*args, s["go"], gstate=s["gstate"], ckpt=ckpt, **keep)
    return [o, state_out] + [x for x in grads if x is not None]


# ---- plain forms -----------------------------------------------------------------------

def _sigmoid(x):
    return 1.0 / (1.0 + torch.exp(-x))


def _plain_norm(s, case, grads):
    N, C, G = case["N"], case["C"], case["G"]
    dt = s["x"].dtype
    x = s["x"].float().view(N, G, C // G)
    w, b = s["weight"].view(1, G, -1), s["bias"].view(1, G, -1)
    c = x - x.mean(dim=-1, keepdim=True)
    r = torch.rsqrt((c * c).mean(dim=-1, keepdim=True) + s["eps"])
    n = c * r
    y = n * w + b
    z = s["gate"].float().view(N, G, C // G) if s["gate"] is not None else None
    t = y if z is None else z
    if case["act"] == "silu":
        sg = _sigmoid(t)
        act, dact = t * sg, sg * (1.0 + t * (1.0 - sg))
    else:
        act, dact = t, torch.ones_like(t)
    out = (act if z is None else y * act).view(N, C).to(dt)
    if not grads:
        return out
    go = s["go"].float().view(N, G, C // G)
    dz = None
    if z is None:
        dy = go * dact
    else:
        dy, dz = go * act, go * y * dact
    gw, gb = (dy * n).sum(dim=0).view(C), dy.sum(dim=0).view(C)
    dn = dy * w
    dx = r * (dn - dn.mean(dim=-1, keepdim=True) - n * (dn * n).mean(dim=-1, keepdim=True))
    res = [out, dx.view(N, C).to(dt), gw, gb]
    return res if dz is None else res + [dz.view(N, C).to(dt)]


def _plain_step(s, case):
    r = case["Hv"] // case["Hk"]
    dt = s["q"].dtype
    q, k = (s[n].float().repeat_interleave(r, dim=1) for n in ("q", "k"))
    v = s["v"].float()
    g, beta = s["g"].float(), s["beta"].float()
    S = torch.exp(g)[..., None, None] * s["state"]
    x = v - torch.sum(S * k[..., None], dim=-2)
    S = S + k[..., None] * (beta[..., None] * x)[..., None, :]
    o = s["scale"] * torch.sum(S * q[..., None], dim=-2)
    return [o.to(dt), S]


def _chunks(x, n):
    """(B, T, H, D) float32, padded with zeros to n chunks -> (n, B*H, CHUNK, D)."""
    B, T, H, D = x.shape
    out = x.new_zeros(B, n * CHUNK, H, D)
    out[:, :T] = x
    return out.view(B, n, CHUNK, H, D).permute(1, 0, 3, 2, 4).reshape(n, B * H, CHUNK, D).contiguous()


def _unchunk(x, B, T):
    n, BH, _, D = x.shape
    H = BH // B
    return x.view(n, B, H, CHUNK, D).permute(1, 0, 3, 2, 4).reshape(B, n * CHUNK, H, D)[:, :T].contiguous()


def _plain_delta(s, case, grads):
    B, T, Hk, Hv, Dk, Dv = (case[n] for n in ("B", "T", "Hk", "Hv", "Dk", "Dv"))
    rep, dt, scale = Hv // Hk, s["q"].dtype, s["scale"]
    n = (T + CHUNK - 1) // CHUNK
    dev = s["q"].device
    live = None
    if s["lengths"] is not None:
        live = torch.arange(T, device=dev)[None, :] < s["lengths"][:, None]

    def take(x):
        x = x.float()
        if x.dim() == 3:
            x = x[..., None]
        elif x.shape[2] != Hv:
            x = x.repeat_interleave(rep, dim=2)
        if live is not None:
            x = torch.where(live[:, :, None, None], x, torch.zeros_like(x))
        return _chunks(x, n)

    q, k, v, g, beta = (take(s[m]) for m in ("q", "k", "v", "g", "beta"))
    q = q * scale
    gam = torch.cumsum(g[..., 0], dim=-1)
    i = torch.arange(CHUNK, device=dev)
    low, strict = i[:, None] >= i[None, :], i[:, None] > i[None, :]
    dec = torch.exp(torch.where(low, gam[..., :, None] - gam[..., None, :], torch.full_like(gam[..., None], -1e30)))
    bt = beta[..., 0]
    Gm = torch.where(strict, torch.matmul(k, k.transpose(-1, -2).contiguous()) * dec, torch.zeros_like(dec))
    P = torch.matmul(q, k.transpose(-1, -2).contiguous()) * dec
    A = Gm * bt[..., None, :]
    inv = torch.eye(CHUNK, device=dev).expand_as(A).contiguous()
    for j in range(1, CHUNK):
        inv[..., j:j + 1, :j] = -torch.matmul(A[..., j:j + 1, :j], inv[..., :j, :j])
    eg = torch.exp(gam)[..., None]
    end = eg[..., -1:, :]
    kw = k * torch.exp(gam[..., -1:] - gam)[..., None]
    kr, qr = k * eg, q * eg
    S = s["state"].view(B * Hv, Dk, Dv).clone() if s["state"] is not None else torch.zeros(B * Hv, Dk, Dv, device=dev)
    o, X, S0 = torch.empty_like(v), torch.empty_like(v), []
    for c in range(n):
        if grads:
            S0.append(S)
        X[c] = torch.matmul(inv[c], v[c] - torch.matmul(kr[c], S))
        U = X[c] * beta[c]
        o[c] = torch.matmul(qr[c], S) + torch.matmul(P[c], U)
        S = end[c] * S + torch.matmul(kw[c].transpose(-1, -2), U)
    out = [_unchunk(o, B, T).to(dt), S.view(B, Hv, Dk, Dv)]
    if not grads:
        return out
    do = take(s["go"])
    dS = s["gstate"].view(B * Hv, Dk, Dv) if s["gstate"] is not None else torch.zeros_like(S)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dg, db = torch.empty_like(gam), torch.empty_like(gam)
    for c in range(n - 1, -1, -1):
        U = X[c] * beta[c]
        dU = torch.matmul(P[c].transpose(-1, -2), do[c]) + torch.matmul(kw[c], dS)
        dZ = torch.matmul(inv[c].transpose(-1, -2), beta[c] * dU)
        dv[c] = dZ
        H = torch.matmul(do[c], X[c].transpose(-1, -2)) * dec[c]
        E = torch.matmul(dZ, X[c].transpose(-1, -2)) * torch.where(strict, dec[c], torch.zeros_like(dec[c]))
        qk = torch.matmul(q[c], k[c].transpose(-1, -2))
        kk = torch.matmul(k[c], k[c].transpose(-1, -2))
        M = qk * H - kk * E
        S0T = S0[c].transpose(-1, -2)
        rq = eg[c] * torch.matmul(do[c], S0T)
        rk = -eg[c] * torch.matmul(dZ, S0T)
        wk = torch.matmul(X[c], dS.transpose(-1, -2)) * (kw[c] * 0 + torch.exp(gam[c][:, -1:] - gam[c])[..., None])
        Hb, Eb = H * bt[c][:, None, :], E * bt[c][:, None, :]
        dq[c] = scale * (rq + torch.matmul(Hb, k[c]))
        dk[c] = (beta[c] * wk + torch.matmul(Hb.transpose(-1, -2), q[c]) - torch.matmul(Eb.transpose(-1, -2), k[c])
                 + rk - torch.matmul(Eb, k[c]))
        wr = torch.sum(k[c] * wk, dim=-1)
        db[c] = M.sum(dim=-2) + wr
        Mb = M * bt[c][:, None, :]
        a = torch.sum(q[c] * rq + k[c] * rk, dim=-1)
        bw = bt[c] * wr
        # e^{g_t} carries what is written before t to what is read at or after t.
        D = torch.cumsum(Mb.sum(dim=-2) - Mb.sum(dim=-1), dim=-1)
        cross = torch.cat([torch.zeros_like(D[:, :1]), D[:, :-1]], dim=-1)
        after = torch.flip(torch.cumsum(torch.flip(a, [-1]), dim=-1), [-1])
        before = torch.cumsum(bw, dim=-1) - bw
        through = end[c][:, 0] * torch.sum(S0[c] * dS, dim=(-1, -2))[:, None]
        dg[c] = after + before + through + cross
        dS = end[c] * dS + torch.matmul(qr[c].transpose(-1, -2), do[c]) - torch.matmul(kr[c].transpose(-1, -2), dZ)

    def give(x, dtype, heads):
        x = _unchunk(x, B, T)
        if live is not None:
            x = torch.where(live[:, :, None, None], x, torch.zeros_like(x))
        if heads != Hv:
            x = x.view(B, T, heads, rep, -1).sum(dim=3)
        return x.to(dtype)

    out += [give(dq, dt, Hk), give(dk, dt, Hk), give(dv, dt, Hv), give(dg[..., None], dt, Hv)[..., 0],
            give(db[..., None], dt, Hv)[..., 0]]
    return out if s["state"] is None else out + [dS.view(B, Hv, Dk, Dv)]


_PLAIN = {
    "norm_forward": lambda s, c: _plain_norm(s, c, False),
    "norm_train": lambda s, c: _plain_norm(s, c, True),
    "delta_step": _plain_step,
    "delta_forward": lambda s, c: _plain_delta(s, c, False),
    "delta_train": lambda s, c: _plain_delta(s, c, True),
}


# ---- float64 from the definitions ------------------------------------------------------

def _exact_norm(s, case):
    N, C, G = case["N"], case["C"], case["G"]
    train = case["op"] == "norm_train"
    x = s["x"].double().requires_grad_(train)
    w = s["weight"].double().requires_grad_(train)
    b = s["bias"].double().requires_grad_(train)
    z = s["gate"].double().requires_grad_(train) if s["gate"] is not None else None
    xs = x.view(N, G, C // G)
    mean = xs.mean(-1, keepdim=True)
    var = ((xs - mean) ** 2).mean(-1, keepdim=True)
    y = ((xs - mean) / torch.sqrt(var + s["eps"])).reshape(N, C) * w + b

    def act(t):
        return t / (1.0 + torch.exp(-t)) if case["act"] == "silu" else t

    out = act(y) if z is None else y * act(z)
    if not train:
        return out
    ins = [x, w, b] + ([z] if z is not None else [])
    gs = torch.autograd.grad(out, ins, s["go"].double())
    return [out.detach()] + list(gs)


def _exact_delta(s, case):
    """Token by token, and the adjoint of each token's step in reverse order; the states of a
    stretch of tokens are formed again from the one kept at its start."""
    B, Hk, Hv, Dk, Dv = (case[n] for n in ("B", "Hk", "Hv", "Dk", "Dv"))
    T, rep = case.get("T", 1), Hv // Hk
    dev = s["q"].device
    seq = case["op"] != "delta_step"

    def tokens(x, heads=False):
        x = x.double()
        if not seq:
            x = x[:, None]
        if heads:
            x = x.repeat_interleave(rep, dim=2)
        return x.transpose(0, 1).contiguous()  # (T, B, H, ...)

    q, k, v, g, beta = tokens(s["q"], True), tokens(s["k"], True), tokens(s["v"]), tokens(s["g"]), tokens(s["beta"])
    live = None
    if s.get("lengths") is not None:
        live = (torch.arange(T, device=dev)[:, None] < s["lengths"][None, :]).view(T, B, 1)
        q, k, v = (torch.where(live[..., None], x, torch.zeros_like(x)) for x in (q, k, v))
        g, beta = (torch.where(live, x, torch.zeros_like(x)) for x in (g, beta))
    a = torch.exp(g)
    S = s["state"].double().clone() if s["state"] is not None else torch.zeros(B, Hv, Dk, Dv, dtype=torch.float64,
                                                                              device=dev)

    def step(t, S):
        Sd = a[t][..., None, None] * S
        x = v[t] - (k[t].unsqueeze(-2) @ Sd).squeeze(-2)
        return Sd, x, Sd + k[t].unsqueeze(-1) * (beta[t][..., None] * x).unsqueeze(-2)

    train = case["op"] == "delta_train"
    o = torch.empty(T, B, Hv, Dv, dtype=torch.float64, device=dev)
    span, kept = 32, []
    for t in range(T):
        if train and t % span == 0:
            kept.append(S)
        S = step(t, S)[2]
        o[t] = s["scale"] * (q[t].unsqueeze(-2) @ S).squeeze(-2)
    out = o.transpose(0, 1)
    out = [out if seq else out[:, 0], S]
    if not train:
        return out
    go = tokens(s["go"])
    if live is not None:
        go = torch.where(live[..., None], go, torch.zeros_like(go))
    dS = s["gstate"].double().clone() if s["gstate"] is not None else torch.zeros_like(S)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dg, db = torch.empty_like(g), torch.empty_like(beta)
    for c in range(len(kept) - 1, -1, -1):
        t0, t1 = c * span, min(T, (c + 1) * span)
        prev, mid, xs, cur = [], [], [], kept[c]
        for t in range(t0, t1):
            prev.append(cur)
            Sd, x, cur = step(t, cur)
            mid.append(Sd)
            xs.append(x)
        for t in range(t1 - 1, t0 - 1, -1):
            nxt = prev[t + 1 - t0] if t + 1 < t1 else cur
            dS = dS + s["scale"] * q[t].unsqueeze(-1) * go[t].unsqueeze(-2)
            dq[t] = s["scale"] * (nxt @ go[t].unsqueeze(-1)).squeeze(-1)
            du = (k[t].unsqueeze(-2) @ dS).squeeze(-2)
            db[t] = (du * xs[t - t0]).sum(-1)
            dx = beta[t][..., None] * du
            dv[t] = dx
            dk[t] = (dS @ (beta[t][..., None] * xs[t - t0]).unsqueeze(-1)).squeeze(-1) - (
                mid[t - t0] @ dx.unsqueeze(-1)).squeeze(-1)
            dS = dS - k[t].unsqueeze(-1) * dx.unsqueeze(-2)
            dg[t] = (dS * mid[t - t0]).sum((-1, -2))
            dS = a[t][..., None, None] * dS

    def give(x, heads):
        if live is not None:
            x = torch.where(live if x.dim() == 3 else live[..., None], x, torch.zeros_like(x))
        x = x.transpose(0, 1)
        return x if heads == Hv else x.reshape(B, T, heads, rep, -1).sum(3)

    out += [give(dq, Hk), give(dk, Hk), give(dv, Hv), give(dg, Hv), give(db, Hv)]
    return out if s["state"] is None else out + [dS]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("norm"):
        return _exact_norm(s, case)
    return _exact_delta(s, case)
