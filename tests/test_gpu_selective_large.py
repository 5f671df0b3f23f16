"""The selective scan, the short convolution and the norm where they are large: rows of many segments, many
rows, tensors of more than 2^31 elements; and gradients against differences of the calls themselves."""

import sys

import numpy as np
import pytest

from selective_cases import TOL_BF16, TOL_F32, make_conv, make_rms, make_scan
from test_gpu_scan_selective import F32S, GRADS, INS, L, check, to_gpu  # noqa: F401

pytestmark = pytest.mark.gpu


def announce(msg):
    sys.__stderr__.write("[gpu case] %s\n" % (msg,))
    sys.__stderr__.flush()


# A state forgets over 1 / (d |A|) tokens, 100 for the median step and the slowest state and 1400 at the most, so that
# rounding adds up over as many tokens and not over the row: the tolerances for 400 tokens hold.
@pytest.mark.parametrize("shape,dtype,lengths", [
    ((1, 2500, 40, 1, 16), "f32", None),           # segments of four tiles
    ((2, 2047, 70, 2, 8), "bf16", [2047, 1025]),   # segments of two, some without tokens
    ((1, 1300, 130, 1, 40), "f32", [1201]),
    ((3, 1100, 64, 1, 100), "bf16", None),
    ((700, 20, 64, 1, 16), "f32", None),           # too many rows for eight waves each
    ((90, 130, 300, 3, 5), "bf16", None),
    # so many workgroups that a backward's take 128 and 256 tokens
    ((320, 300, 5, 5, 16), "f32", [300, 129, 128, 127, 0] * 64),
    ((480, 310, 5, 5, 3), "f32", [310, 257, 256, 255, 64, 1] * 80),
    ((480, 310, 5, 5, 17), "bf16", [310, 300, 288, 0, 65, 200] * 80),
    ((260, 260, 70, 1, 16), "f32", [260] * 130 + [0] * 65 + [1] * 65),
], ids=lambda x: str(x)[:24])
def test_many_segments_and_rows(L, shape, dtype, lengths):  # noqa: F811
    check(L, shape, dtype, lengths=lengths, seed=31)


def difference(call, inputs, names, eps, seed):
    """(central difference, sum of the gradients' products) of ``call`` along random directions of ``names``:
    call(inputs) gives a float64 number and, asked to, gradients by name."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    grads = call(inputs, True)
    got = []
    for name in names:
        x = inputs[name]
        v = torch.randn(x.shape, generator=gen, device="cuda")
        hi, lo = dict(inputs), dict(inputs)
        hi[name], lo[name] = x + eps * v, x - eps * v
        # the steps as rounded
        moved = (hi[name].double() - lo[name].double())
        got.append((name, call(hi, False) - call(lo, False), (moved * grads[name].double()).sum().item(),
                    (moved * grads[name].double()).norm().item()))
    return got


# Central differences at 3e-3 of values of order 1: the third derivatives' part is (3e-3)^2 of the first's, 1e-5 (the
# exponential's own, times d |A| < 10), and rounding 2^-24 of the outputs' sums, spread over sqrt(n) terms, against
# steps of 3e-3: below 1e-4 of the norm of the terms that are summed.
def close(rows):
    for name, diff, want, size in rows:
        assert abs(diff - want) <= 5e-3 * max(abs(want), size), (name, diff, want, size)


def test_scan_differences(L):  # noqa: F811
    g = to_gpu(make_scan(2, 130, 70, 2, 16, 41), "f32")
    names = ("u", "dt", "A", "B", "C", "D", "z", "dt_bias", "s_in")

    def call(x, grads):
        kw = dict(D=x["D"], z=x["z"], dt_bias=x["dt_bias"], state=x["s_in"])
        y, s, ck = L.scan_selective_ckpt(*(x[n] for n in INS), **kw)
        if not grads:
            return (y.double() * g["gy"].double()).sum().item() + (s.double() * g["gs_out"].double()).sum().item()
        r = L.scan_selective_backward(*(x[n] for n in INS), g["gy"], gstate=g["gs_out"], ckpt=ck, **kw)
        return dict(zip((n[1:] if n != "gdt_bias" else "dt_bias" for n in GRADS[:8]), r[:8]), s_in=r[8])

    close(difference(call, g, names, 3e-3, 1))


def test_conv_differences(L):  # noqa: F811
    import torch
    g = {n: torch.from_numpy(x).cuda() for n, x in make_conv(3, 60, 70, 4, 42).items()}

    def call(x, grads):
        y, s = L.short_conv_act(x["x"], x["weight"], bias=x["bias"], state=x["s_in"])
        if not grads:
            return (y.double() * g["gy"].double()).sum().item() + (s.double() * g["gs_out"].double()).sum().item()
        r = L.short_conv_act_backward(x["x"], x["weight"], g["gy"], bias=x["bias"], state=x["s_in"], gstate=g["gs_out"])
        return dict(zip(("x", "weight", "bias", "s_in"), r))

    close(difference(call, g, ("x", "weight", "bias", "s_in"), 3e-3, 2))


def test_norm_differences(L):  # noqa: F811
    import torch
    g = {n: torch.from_numpy(x).cuda() for n, x in make_rms(50, 300, 43).items()}

    def call(x, grads):
        y, s = L.rms_norm_add(x["x"], x["weight"], residual=x["residual"])
        if not grads:
            return (y.double() * g["gy"].double()).sum().item() + (s.double() * g["gsum"].double()).sum().item()
        gx, gs, gw = L.rms_norm_add_backward(s, x["weight"], g["gy"], gsum=g["gsum"])
        return {"x": gx, "residual": gs, "weight": gw}

    close(difference(call, g, ("x", "residual", "weight"), 3e-3, 3))


# ---- more than 2^31 elements: what lies behind them, against calls on that part alone ------------

T, C = 1050000, 2056  # 2.16e9 elements
CUT = T // 64 // 2 * 64


def off(a, b):
    """The largest difference of two tensors, relative to the larger of an element and the RMS, a part at a time."""
    worst = 0.0
    for x, y in zip(a.flatten(0, -2).split(1 << 17), b.flatten(0, -2).split(1 << 17)):
        x, y = x.float(), y.float()
        worst = max(worst, ((x - y).abs() / y.abs().clamp_min(y.square().mean().sqrt())).max().item())
    return worst


def large(seed, T=T, C=C):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.empty(1, T, C, dtype=torch.bfloat16, device="cuda")
    for part in x.split(1 << 17, dim=1):
        part.copy_(torch.randn(part.shape, generator=gen, device="cuda"))
    return x


# (the second: more blocks than the sums over states of more than 16 have workgroups)
@pytest.mark.parametrize("T,C,N", [(T, C, 4), (640000, 70, 17)])
def test_scan_of_more_than_2_31_elements(L, T, C, N):  # noqa: F811
    import torch
    announce("scan (1, %d, %d), %d states" % (T, C, N))
    u, dt = large(1, T, C), large(2, T, C)
    d = to_gpu(make_scan(1, 1, C, 1, N, 44), "bf16")
    B, Cm = (large_rows(T, N, s) for s in (3, 4))
    CUT = T // 64 // 2 * 64
    kw = dict(D=d["D"], z=dt, dt_bias=d["dt_bias"])
    y, s, ck = L.scan_selective_ckpt(u, dt, d["A"], B, Cm, **kw)
    g = L.scan_selective_backward(u, dt, d["A"], B, Cm, u, gstate=d["gs_out"], ckpt=ck, **kw)
    del ck
    tail = [x[:, CUT:].contiguous() for x in (u, dt, B, Cm)]
    head = [x[:, :CUT].contiguous() for x in (u, dt, B, Cm)]
    kw["z"] = head[1]
    mid = L.scan_selective(head[0], head[1], d["A"], head[2], head[3], **kw)[1]
    kw["z"], kw["state"] = tail[1], mid
    del head
    y2, s2 = L.scan_selective(tail[0], tail[1], d["A"], tail[2], tail[3], **kw)
    # Two float32 values that are TOL_F32 apart, each rounded to bfloat16 by up to 2^-8 of itself: where they lie on
    # either side of the middle between two neighbours they end up a whole step apart, 2 * 2^-8.
    assert off(y[:, CUT:], y2) <= 2 * TOL_BF16 and off(s, s2) <= TOL_F32
    del y, y2
    g2 = L.scan_selective_backward(tail[0], tail[1], d["A"], tail[2], tail[3], tail[0], gstate=d["gs_out"], **kw)
    for i in (0, 1, 3, 4, 6):
        assert off(g[i][:, CUT:], g2[i]) <= 2 * TOL_BF16, GRADS[i]
    torch.cuda.synchronize()


def large_rows(T, N, seed):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(1, T, 1, N, generator=gen, device="cuda").bfloat16()


def test_conv_of_more_than_2_31_elements(L):  # noqa: F811
    import torch
    announce("conv (1, %d, %d)" % (T, C))
    x = large(5)
    w = torch.randn(C, 4, device="cuda")
    y, s = L.short_conv_act(x, w)
    gx, gw, _, _ = L.short_conv_act_backward(x, w, y)
    tail, before = x[:, CUT:].contiguous(), x[:, CUT - 3:CUT].contiguous()
    y2, s2 = L.short_conv_act(tail, w, state=before)
    assert torch.equal(y[:, CUT:], y2) and torch.equal(s, s2)
    gx2 = L.short_conv_act_backward(tail, w, y2, state=before)[0]
    assert torch.equal(gx[:, CUT:], gx2)


def test_norm_of_more_than_2_31_elements(L):  # noqa: F811
    import torch
    announce("norm (%d, %d)" % (T, C))
    x = large(6)[0]
    w = torch.randn(C, device="cuda")
    y, s = L.rms_norm_add(x, w, residual=x)
    gx, gs, gw = L.rms_norm_add_backward(s, w, y, gsum=x)
    y2, s2 = L.rms_norm_add(x[CUT:].contiguous(), w, residual=x[CUT:].contiguous())
    assert torch.equal(y[CUT:], y2) and torch.equal(s[CUT:], s2)
    gx2, gs2, _ = L.rms_norm_add_backward(s2, w, y2, gsum=x[CUT:].contiguous())
    assert torch.equal(gx[CUT:], gx2) and torch.equal(gs[CUT:], gs2)
