"""Sums over all tokens, of calls with more than 2^31 elements, against the sums of the row's two halves; and the
gradients against differences to what those are good for."""

import pytest

import test_gpu_selective_large as large
from selective_cases import TOL_F32, make_scan
from test_gpu_scan_selective import L, to_gpu  # noqa: F401

pytestmark = pytest.mark.gpu

# A sum over a million tokens is formed from some ten thousand partial sums of 64 to 2500 tokens, sixteen strips of
# them at once: at most 2500 additions in a row, each off by 2^-24 of what has come together, of either sign: sqrt(2500)
# * 2^-24 = 3e-6 of the sum in each of the three calls, five times that for the largest of ten thousand: below 1e-4.


def near(whole, *parts):
    want = sum(p.double() for p in parts)
    floor = want.square().mean().sqrt()
    assert ((whole.double() - want).abs() / want.abs().clamp_min(floor)).max().item() <= TOL_F32


@pytest.mark.parametrize("T,C,N", [(large.T, large.C, 4), (640000, 70, 17)])
def test_scan(L, T, C, N):  # noqa: F811
    large.announce("sums of the scan (1, %d, %d), %d states" % (T, C, N))
    u, dt = large.large(1, T, C), large.large(2, T, C)
    d = to_gpu(make_scan(1, 1, C, 1, N, 44), "bf16")
    B, Cm = (large.large_rows(T, N, s) for s in (3, 4))
    cut = T // 64 // 2 * 64
    same = dict(D=d["D"], dt_bias=d["dt_bias"])

    def half(at, gstate, state=None):
        x = [t[:, at].contiguous() for t in (u, dt, B, Cm)]
        return L.scan_selective_backward(x[0], x[1], d["A"], x[2], x[3], x[0], z=x[1], gstate=gstate, state=state, **same)

    whole = half(slice(None), d["gs_out"])
    head = [t[:, :cut].contiguous() for t in (u, dt, B, Cm)]
    mid = L.scan_selective(head[0], head[1], d["A"], head[2], head[3], z=head[1], **same)[1]
    del head
    tail = half(slice(cut, None), d["gs_out"], mid)
    head = half(slice(0, cut), tail[8])
    for i in (2, 5, 7):  # of A, D and dt_bias
        near(whole[i], head[i], tail[i])


def test_conv(L):  # noqa: F811
    import torch
    large.announce("sums of the convolution")
    x, cut = large.large(5), large.CUT
    w, bias = torch.randn(large.C, 4, device="cuda"), torch.randn(large.C, device="cuda")
    y, _ = L.short_conv_act(x, w, bias=bias)
    gw, gb = L.short_conv_act_backward(x, w, y, bias=bias)[1:3]
    a = L.short_conv_act_backward(x[:, :cut].contiguous(), w, y[:, :cut].contiguous(), bias=bias)
    b = L.short_conv_act_backward(x[:, cut:].contiguous(), w, y[:, cut:].contiguous(), bias=bias,
                                  state=x[:, cut - 3:cut].contiguous())
    near(gw, a[1], b[1])
    near(gb, a[2], b[2])


def test_norm(L):  # noqa: F811
    import torch
    large.announce("sums of the norm")
    x, cut = large.large(6)[0], large.CUT
    w = torch.randn(large.C, device="cuda")
    gy = x.flip(0)
    near(*(L.rms_norm_add_backward(t.contiguous(), w, g.contiguous())[2]
           for t, g in ((x, gy), (x[:cut], gy[:cut]), (x[cut:], gy[cut:]))))


# The differences of test_gpu_selective_large to the bound that their steps give: rounding, ten steps of 2^-24 of an output,
# over the n outputs of a call on either side, sqrt(2 n) * 6e-7, against products of norm 2 * 3e-3 * sqrt(n): 1.4e-4; and
# the third derivatives' 1e-5.  1e-3 holds seven times that.
def close(rows):
    for name, diff, want, size in rows:
        print(name, abs(diff - want) / max(abs(want), size))
        assert abs(diff - want) <= 1e-3 * max(abs(want), size), (name, diff, want, size)


@pytest.mark.parametrize("which", ["scan", "conv", "norm"])
def test_differences(L, which, monkeypatch):  # noqa: F811
    monkeypatch.setattr(large, "close", close)
    getattr(large, "test_%s_differences" % which)(L)
