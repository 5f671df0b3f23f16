"""The gated delta rule and the group norm on tensors of more than 2^32 bytes: offsets past 32 bits over
batch rows, over tokens and over the norm's rows, forward and backward, against the float64 oracle on
sampled parts.  Inputs are drawn on the GPU (unit-norm q and k; v, go ~ N(0,1)).

A long row is compared in windows: the state is cleared (g = -inf) before a window and before the
token after it, so that what lies outside has no part in its outputs and gradients (the clearing
token after it aside, whose own gradients are not compared).  Tolerances as for the other shapes."""

import sys

import numpy as np
import pytest

from oracle import delta
from delta_cases import TOL_BF16, TOL_F32, rms_err

pytestmark = pytest.mark.gpu

INS = ("q", "k", "v", "g", "beta")
# As for the other shapes' bfloat16 gradients: largest error of an element and 2-norm.
BF16_MAX, BF16_FRO = 2.0 ** -4, 2.0 ** -7


def announce(*what):
    sys.__stderr__.write("[gpu case] beyond 4 GiB %s\n" % (what,))
    sys.__stderr__.flush()


@pytest.fixture(autouse=True)
def release():
    import torch
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def inputs(B, T, Hk, Hv, Dk, Dv, seed):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.bfloat16)

    def unit(*shape):
        return torch.nn.functional.normalize(normal(*shape).float(), dim=-1).bfloat16()

    d = {"q": unit(B, T, Hk, Dk), "k": unit(B, T, Hk, Dk), "v": normal(B, T, Hv, Dv),
         "g": -0.02 * torch.nn.functional.softplus(normal(B, T, Hv)), "beta": torch.sigmoid(normal(B, T, Hv))}
    return d, normal(B, T, Hv, Dv)


def far(x, *at):
    """x[at] on the host, float32."""
    return x[at].float().cpu().numpy()


def check_gradients(got, ref):
    for name, x, y in zip(INS, got, ref):
        e = float(np.linalg.norm(x - y) / np.linalg.norm(y))
        assert rms_err(x, y) <= BF16_MAX and e <= BF16_FRO, (name, e)


def test_many_rows():
    import torch
    import linear_recurrence_rnn_amd as L
    B, T, Hk, Hv, Dk, Dv = 4200, 64, 1, 64, 32, 128
    announce("rows", B, T, Hk, Hv, Dk, Dv)
    d, go = inputs(B, T, Hk, Hv, Dk, Dv, 1)
    assert d["v"].numel() * 2 > 1 << 32 and B * Hv * Dk * Dv * 4 > 1 << 32
    args = [d[n] for n in INS]
    o, s, ck = L.gated_delta_forward_ckpt(*args)
    o2, s2 = L.gated_delta_forward(*args)
    assert torch.equal(o, o2) and torch.equal(s, s2)
    got = L.gated_delta_backward(*args, go, gstate=s, ckpt=ck)[:5]
    del ck, o2, s2
    for b in (0, 2047, 2048, 4199):
        r = slice(b, b + 1)
        ins = [far(x, r) for x in args]
        ro, rs = delta.gated_delta_forward(*ins)
        assert rms_err(far(o, r), ro) <= TOL_BF16 and rms_err(far(s, r), rs) <= TOL_F32
        ref = delta.gated_delta_backward(*ins, far(go, r), gs_out=far(s, r))
        check_gradients([far(x, r) for x in got], ref)


def test_a_long_row():
    import torch
    import linear_recurrence_rnn_amd as L
    T, Hk, Hv, Dk, Dv, W = 540001, 4, 32, 64, 128, 150
    announce("tokens", T, Hk, Hv, Dk, Dv)
    d, go = inputs(1, T, Hk, Hv, Dk, Dv, 2)
    assert d["v"].numel() * 2 > 1 << 32
    starts = (1000, T // 2, T - 20000, T - W)  # windows of W tokens, at the end the row's last ones
    for t in starts:
        d["g"][:, t] = -float("inf")
        if t + W < T:
            d["g"][:, t + W] = -float("inf")
    args = [d[n] for n in INS]
    o, s, ck = L.gated_delta_forward_ckpt(*args)
    got = L.gated_delta_backward(*args, go, ckpt=ck)[:5]
    o2, s2 = L.gated_delta_forward(*args)
    assert torch.equal(o, o2) and torch.equal(s, s2)
    for t in starts:
        r = (slice(0, 1), slice(t, t + W))
        ins = [far(x, *r) for x in args]
        ro, rs = delta.gated_delta_forward(*ins)
        assert rms_err(far(o, *r), ro) <= TOL_BF16
        if t + W == T:
            assert rms_err(far(s), rs) <= TOL_F32
        check_gradients([far(x, *r) for x in got], delta.gated_delta_backward(*ins, far(go, *r)))


def test_group_norm():
    import torch
    import linear_recurrence_rnn_amd as L
    N, C, G = 1100003, 1000, 8
    announce("norm", N, C, G)
    gen = torch.Generator(device="cuda").manual_seed(3)
    x, go = (torch.randn(N, C, generator=gen, device="cuda") for _ in range(2))
    w, b = 1 + 0.3 * torch.randn(C, generator=gen, device="cuda"), 0.3 * torch.randn(C, generator=gen, device="cuda")
    assert x.numel() * 4 > 1 << 32
    y = L.group_norm_act(x, G, w, b)
    gx, gw, gb, _ = L.group_norm_act_backward(x, G, w, b, go)
    par = [t.cpu().numpy() for t in (w, b)]
    for n in (0, N // 2, N - 7):
        r = slice(n, n + 7)
        xs, gs = far(x, r), far(go, r)
        assert rms_err(far(y, r), delta.group_norm_act(xs, G, *par)) <= TOL_F32
        assert rms_err(far(gx, r), delta.group_norm_act_backward(xs, G, *par, gs)[0]) <= TOL_F32
    rw, rb = torch.zeros(C, dtype=torch.float64, device="cuda"), torch.zeros(C, dtype=torch.float64, device="cuda")
    for n in range(0, N, 50000):
        p = x[n:n + 50000].double().view(-1, G, C // G)
        p = p - p.mean(-1, keepdim=True)
        p = (p / torch.sqrt((p * p).mean(-1, keepdim=True) + 1e-5)).view(-1, C)
        t = p * w.double() + b.double()
        sg = torch.sigmoid(t)
        dy = go[n:n + 50000].double() * sg * (1 + t * (1 - sg))
        rw += (dy * p).sum(0)
        rb += dy.sum(0)
    assert rms_err(gw.cpu().numpy(), rw.cpu().numpy()) <= TOL_F32
    assert rms_err(gb.cpu().numpy(), rb.cpu().numpy()) <= TOL_F32
