"""Float64 oracle of the selective state space scan, the short causal convolution and the
root-mean-square norm -- TEST INFRASTRUCTURE ONLY, in plain numpy and independent of the kernels: the
recurrence is walked token by token, its gradient by the adjoint of each token's step.

    d_t = softplus(dt_t + bias),  h_t = e^{d_t A} h_{t-1} + d_t u_t B_t,
    y_t = (sum_n C_t h_t + D u_t) silu(z_t)
"""

from __future__ import annotations

import numpy as np


def _f(x):
    return None if x is None else np.asarray(x, np.float64)


def _live(B, T, lengths):
    return np.ones((B, T), bool) if lengths is None else np.arange(T)[None] < np.asarray(lengths)[:, None]


def _masked(x, live):
    return None if x is None else np.where(live.reshape(live.shape + (1,) * (x.ndim - 2)), x, 0.0)


def _logistic(x):
    return np.where(x >= 0, 1 / (1 + np.exp(-np.abs(x))), np.exp(-np.abs(x)) / (1 + np.exp(-np.abs(x))))


def _steps(dt, dt_bias, softplus, live):
    """d (0 for absent tokens) and its derivative by dt."""
    raw = _masked(_f(dt), live) + (0.0 if dt_bias is None else _f(dt_bias))
    d = np.logaddexp(raw, 0.0) if softplus else raw
    return _masked(d, live), _masked(_logistic(raw) if softplus else np.ones_like(raw), live)


def scan_selective(u, dt, A, B, C, D=None, z=None, dt_bias=None, softplus=True, s_in=None, lengths=None, trace=None):
    """(y, s_out), float64.  trace: a list that gets (h before the token, h after it, core)."""
    Bn, T, Ch = u.shape
    N, r = A.shape[1], Ch // B.shape[2]
    live = _live(Bn, T, lengths)
    u, B, C, z = (_masked(_f(x), live) for x in (u, B, C, z))
    A = _f(A)
    d, _ = _steps(dt, dt_bias, softplus, live)
    h = np.zeros((Bn, Ch, N)) if s_in is None else _f(s_in)
    y = np.zeros((Bn, T, Ch))
    for t in range(T):
        Bt, Ct = np.repeat(B[:, t], r, axis=1), np.repeat(C[:, t], r, axis=1)
        on = live[:, t, None, None]
        new = np.where(on, np.exp(np.where(on, d[:, t, :, None] * A, 0.0)) * h + (d[:, t] * u[:, t])[:, :, None] * Bt, h)
        core = (Ct * new).sum(-1) + (0.0 if D is None else _f(D) * u[:, t])
        if trace is not None:
            trace.append((h, new, core))
        h = new
        y[:, t] = core if z is None else core * z[:, t] * _logistic(z[:, t])
    return _masked(y, live), h


def scan_selective_backward(u, dt, A, B, C, gy, D=None, z=None, dt_bias=None, softplus=True, s_in=None, gs_out=None,
                            lengths=None):
    """(gu, gdt, gA, gB, gC, gD, gz, gdt_bias, gs_in), float64; None for inputs that are None (gs_in:
    always given)."""
    trace = []
    scan_selective(u, dt, A, B, C, D, z, dt_bias, softplus, s_in, lengths, trace)
    Bn, T, Ch = u.shape
    G, N = B.shape[2:]
    r = Ch // G
    live = _live(Bn, T, lengths)
    u, B, C, z, gy = (_masked(_f(x), live) for x in (u, B, C, z, gy))
    A = _f(A)
    d, slope = _steps(dt, dt_bias, softplus, live)
    g = np.zeros((Bn, Ch, N)) if gs_out is None else _f(gs_out)
    gu, gdt, gz = (np.zeros((Bn, T, Ch)) for _ in range(3))
    gB, gC = np.zeros_like(B), np.zeros_like(C)
    gA, gD = np.zeros_like(A), np.zeros(Ch)
    for t in range(T - 1, -1, -1):
        before, after, core = trace[t]
        on = live[:, t, None, None]
        p = gy[:, t]
        if z is not None:
            sg = _logistic(z[:, t])
            gz[:, t] = p * core * sg * (1 + z[:, t] * (1 - sg))
            p = p * z[:, t] * sg
        Bt, Ct = np.repeat(B[:, t], r, axis=1), np.repeat(C[:, t], r, axis=1)
        gC[:, t] = np.where(on, p[:, :, None] * after, 0.0).reshape(Bn, G, r, N).sum(2)
        gh = g + Ct * p[:, :, None]
        x = d[:, t] * u[:, t]
        gB[:, t] = np.where(on, gh * x[:, :, None], 0.0).reshape(Bn, G, r, N).sum(2)
        into = np.where(on, gh * Bt, 0.0).sum(-1)
        a = np.exp(np.where(on, d[:, t, :, None] * A, 0.0))
        m = np.where(on, gh * a * before, 0.0)
        gA += (m * d[:, t, :, None]).sum(0)
        gdt[:, t] = ((m * A).sum(-1) + into * u[:, t]) * slope[:, t]
        gu[:, t] = into * d[:, t] + (0.0 if D is None else _f(D) * p)
        gD += (p * u[:, t]).sum(0)
        g = np.where(on, gh * a, g)
    return (_masked(gu, live), _masked(gdt, live), gA, gB, gC, None if D is None else gD,
            None if z is None else _masked(gz, live), None if dt_bias is None else _masked(gdt, live).sum((0, 1)), g)


def _act(x, act):
    if act == "none":
        return x, np.ones_like(x)
    s = _logistic(x)
    return x * s, s * (1 + x * (1 - s))


def _line(x, s_in, K, live):
    """(B, T+K-1, C): the carried inputs, then the tokens'."""
    B, T, C = x.shape
    first = np.zeros((B, K - 1, C)) if s_in is None else _f(s_in)
    return np.concatenate([first, _masked(_f(x), live)], axis=1)


def short_conv_act(x, weight, bias=None, act="silu", s_in=None, lengths=None):
    """(y, s_out), float64."""
    B, T, C = x.shape
    K = weight.shape[1]
    live = _live(B, T, lengths)
    line = _line(x, s_in, K, live)
    pre = np.zeros((B, T, C)) + (0.0 if bias is None else _f(bias))
    for k in range(K):
        pre += _f(weight)[:, k] * line[:, k:k + T]
    n = live.sum(1)
    return _masked(_act(pre, act)[0], live), np.stack([line[b, n[b]:n[b] + K - 1] for b in range(B)])


def short_conv_act_backward(x, weight, gy, bias=None, act="silu", s_in=None, gs_out=None, lengths=None):
    """(gx, gweight, gbias, gs_in), float64."""
    B, T, C = x.shape
    K = weight.shape[1]
    live = _live(B, T, lengths)
    line = _line(x, s_in, K, live)
    w = _f(weight)
    pre = np.zeros((B, T, C)) + (0.0 if bias is None else _f(bias))
    for k in range(K):
        pre += w[:, k] * line[:, k:k + T]
    q = _masked(_f(gy), live) * _act(pre, act)[1]
    q = _masked(q, live)
    gline, gw = np.zeros_like(line), np.zeros_like(w)
    for k in range(K):
        gline[:, k:k + T] += w[:, k] * q
        gw[:, k] = (q * line[:, k:k + T]).sum((0, 1))
    if gs_out is not None:
        for b, n in enumerate(live.sum(1)):
            gline[b, n:n + K - 1] += _f(gs_out)[b]
    return gline[:, K - 1:], gw, q.sum((0, 1)), gline[:, :K - 1]


def rms_norm_add(x, weight, residual=None, eps=1e-5, stored=None):
    """(y, s), float64; ``stored`` rounds s to the type it is kept in."""
    s = _f(x) if residual is None else _f(x) + _f(residual)
    k = s if stored is None else _f(stored(s))
    return k / np.sqrt((k * k).mean(-1, keepdims=True) + eps) * _f(weight), s


def rms_norm_add_backward(s, weight, gy, gsum=None, eps=1e-5):
    """(gs, gweight), float64."""
    s, w, gy = _f(s), _f(weight), _f(gy)
    r = 1 / np.sqrt((s * s).mean(-1, keepdims=True) + eps)
    v = gy * w
    gs = r * v - s * r ** 3 * (v * s).mean(-1, keepdims=True)
    if gsum is not None:
        gs = gs + _f(gsum)
    return gs, (gy * s * r).reshape(-1, s.shape[-1]).sum(0)
