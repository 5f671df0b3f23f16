"""Float64 oracle of the gated delta rule and of the per-token group norm -- TEST
INFRASTRUCTURE ONLY, in plain numpy and independent of the kernels: the recurrence is walked
token by token (no chunks), its gradient by the adjoint of each token's step.

    x_t = v_t - (a_t S_{t-1})^T k_t,  S_t = a_t S_{t-1} + beta_t k_t x_t^T,
    o_t = scale S_t^T q_t,            a_t = e^{g_t}
"""

from __future__ import annotations

import numpy as np


def _expand(x, Hv):
    """(B,T,Hk,D) -> (B,T,Hv,D): value head h reads key head h // (Hv // Hk)."""
    return np.repeat(x.astype(np.float64), Hv // x.shape[2], axis=2)


def _masked(x, live):
    return np.where(live.reshape(live.shape + (1,) * (x.ndim - 2)), x, 0.0)


def _inputs(q, k, v, g, beta, s_in, lengths, scale):
    B, T, Hv, Dv = v.shape
    Dk = q.shape[-1]
    live = np.ones((B, T), bool) if lengths is None else np.arange(T)[None] < np.asarray(lengths)[:, None]
    q, k = _masked(_expand(q, Hv), live), _masked(_expand(k, Hv), live)
    v, g, beta = (_masked(np.asarray(x, np.float64), live) for x in (v, g, beta))
    S = np.zeros((B, Hv, Dk, Dv)) if s_in is None else s_in.astype(np.float64)
    return q, k, v, np.exp(g), beta, S, live, Dk ** -0.5 if scale is None else scale


def gated_delta_forward(q, k, v, g, beta, s_in=None, lengths=None, scale=None):
    """(o, s_out), float64."""
    q, k, v, a, beta, S, _, scale = _inputs(q, k, v, g, beta, s_in, lengths, scale)
    o = np.empty_like(v)
    for t in range(v.shape[1]):
        Sd = a[:, t, :, None, None] * S
        x = v[:, t] - np.einsum("bhkv,bhk->bhv", Sd, k[:, t])
        S = Sd + np.einsum("bhk,bhv->bhkv", k[:, t], beta[:, t, :, None] * x)
        o[:, t] = scale * np.einsum("bhkv,bhk->bhv", S, q[:, t])
    return o, S


def gated_delta_backward(q, k, v, g, beta, go, s_in=None, gs_out=None, lengths=None, scale=None):
    """(gq, gk, gv, gg, gbeta, gs_in), float64, for the upstream gradients go of o and gs_out
    (or None) of the final state."""
    Hk = q.shape[2]
    q, k, v, a, beta, S, live, scale = _inputs(q, k, v, g, beta, s_in, lengths, scale)
    go = _masked(np.asarray(go, np.float64), live)
    B, T, Hv, Dv = v.shape
    dec, xs, after = [], [], []
    for t in range(T):
        Sd = a[:, t, :, None, None] * S
        x = v[:, t] - np.einsum("bhkv,bhk->bhv", Sd, k[:, t])
        S = Sd + np.einsum("bhk,bhv->bhkv", k[:, t], beta[:, t, :, None] * x)
        dec.append(Sd), xs.append(x), after.append(S)
    dS = np.zeros_like(S) if gs_out is None else gs_out.astype(np.float64)
    gq, gk, gv, gg, gb = (np.empty_like(x) for x in (q, k, v, a, beta))
    for t in range(T - 1, -1, -1):
        b = beta[:, t, :, None]
        dS = dS + scale * np.einsum("bhk,bhv->bhkv", q[:, t], go[:, t])
        gq[:, t] = scale * np.einsum("bhkv,bhv->bhk", after[t], go[:, t])
        du = np.einsum("bhkv,bhk->bhv", dS, k[:, t])
        gb[:, t] = np.sum(du * xs[t], axis=-1)
        gv[:, t] = b * du
        gk[:, t] = np.einsum("bhkv,bhv->bhk", dS, b * xs[t]) - np.einsum("bhkv,bhv->bhk", dec[t], gv[:, t])
        dS = dS - np.einsum("bhk,bhv->bhkv", k[:, t], gv[:, t])
        gg[:, t] = np.sum(dS * dec[t], axis=(-1, -2))
        dS = a[:, t, :, None, None] * dS
    gq, gk, gv, gg, gb = (_masked(x, live) for x in (gq, gk, gv, gg, gb))

    def shared(x):  # the heads that read one key head
        return x.reshape(B, T, Hk, Hv // Hk, x.shape[-1]).sum(axis=3)

    return shared(gq), shared(gk), gv, gg, gb, dS


def _act(t, act):
    t = np.asarray(t, np.float64)
    if act == "none":
        return t, np.ones_like(t)
    s = 1.0 / (1.0 + np.exp(-t))
    return t * s, s * (1.0 + t * (1.0 - s))


def _norm(x, groups, eps):
    N, C = x.shape
    x = x.astype(np.float64).reshape(N, groups, C // groups)
    c = x - x.mean(axis=-1, keepdims=True)
    r = 1.0 / np.sqrt((c * c).mean(axis=-1, keepdims=True) + eps)
    return c * r, r


def group_norm_act(x, groups, weight, bias, gate=None, act="silu", eps=1e-5):
    """act(y) or y act(gate), y = n * weight + bias, x (N,C), float64."""
    n, _ = _norm(x, groups, eps)
    y = n.reshape(x.shape) * weight + bias
    return _act(y, act)[0] if gate is None else y * _act(gate, act)[0]


def group_norm_act_backward(x, groups, weight, bias, gout, gate=None, act="silu", eps=1e-5):
    """(gx, gweight, gbias, ggate), float64."""
    n, r = _norm(x, groups, eps)
    go = gout.astype(np.float64)
    flat = n.reshape(x.shape)
    y = flat * weight + bias
    gg = None
    if gate is None:
        dy = go * _act(y, act)[1]
    else:
        a, da = _act(gate, act)
        dy, gg = go * a, go * y * da
    dn = (dy * weight).reshape(n.shape)
    gx = r * (dn - dn.mean(axis=-1, keepdims=True) - n * (dn * n).mean(axis=-1, keepdims=True))
    return gx.reshape(x.shape), (dy * flat).sum(axis=0), dy.sum(axis=0), gg
