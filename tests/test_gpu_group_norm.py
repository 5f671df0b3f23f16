"""GPU parity of the per-token group norm with an activation or a gate, forward and backward,
against the float64 oracle; group widths on both sides of every lane layout, widths and
pointers that rule out 16-byte accesses, and degenerate groups."""

import sys

import numpy as np
import pytest

from oracle import delta
from delta_cases import TOL_BF16, TOL_F32, host, make_norm, rms_err, to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    import linear_recurrence_rnn_amd as L
    from linear_recurrence_rnn_amd import binding
    binding.load()
    return L


def check(L, N, C, G, dtype, gated, act, d, eps=1e-5):
    sys.__stderr__.write("[gpu case] group_norm %s\n" % ((N, C, G, dtype, gated, act),))
    sys.__stderr__.flush()
    tol = TOL_BF16 if dtype == "bf16" else TOL_F32
    gate = d["gate"] if gated else None
    x, go, z = to_dev(d["x"], dtype), to_dev(d["gout"], dtype), to_dev(gate, dtype)
    w, b = to_dev(d["weight"]), to_dev(d["bias"])
    y = L.group_norm_act(x, G, w, b, gate=z, act=act, eps=eps)
    gx, gw, gb, gg = L.group_norm_act_backward(x, G, w, b, go, gate=z, act=act, eps=eps)
    assert y.dtype == x.dtype and gw.dtype == w.dtype
    assert rms_err(host(y), delta.group_norm_act(d["x"], G, d["weight"], d["bias"], gate, act, eps)) <= tol
    rx, rw, rb, rg = delta.group_norm_act_backward(d["x"], G, d["weight"], d["bias"], d["gout"], gate, act, eps)
    assert rms_err(host(gx), rx) <= tol
    assert rms_err(host(gw), rw) <= TOL_F32
    assert rms_err(host(gb), rb) <= TOL_F32
    assert (gg is None) == (rg is None)
    if gated:
        assert rms_err(host(gg), rg) <= tol


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("gated,act", [(True, "silu"), (False, "silu"), (True, "none"), (False, "none")])
@pytest.mark.parametrize("N,C,G", [(1, 24, 1), (7, 96, 3), (130, 640, 5), (33, 1000, 8), (5, 75, 3)], ids=str)
def test_small(L, N, C, G, gated, act, dtype):
    check(L, N, C, G, dtype, gated, act, make_norm(N, C, 11, dtype))


# One group width on each side of every lane layout (32, 64, 128, 256, 512, 1024, 2048, 8192).
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [2, 32, 33, 64, 72, 128, 136, 256, 264, 512, 520, 1024, 1032, 2048, 2056, 2047, 8192, 8191])
def test_group_widths(L, D, dtype):
    G = 3 if D <= 1024 else 1
    check(L, 9, D * G, G, dtype, True, "silu", make_norm(9, D * G, D, dtype))


def test_many_tokens(L):
    check(L, 40000, 128, 2, "bf16", True, "silu", make_norm(40000, 128, 3, "bf16"))
    check(L, 3000, 2560, 20, "f32", False, "silu", make_norm(3000, 2560, 4))


def test_a_large_mean_costs_no_digits(L):
    # The relative step of the inputs at 1000 is 2^-24 * 1000 = 6e-5 of their unit spread; the
    # oracle sees the same rounded inputs, so the tolerance stays that of float32.
    check(L, 50, 256, 2, "f32", False, "none", make_norm(50, 256, 5, mean=1000.0))


def test_constant_and_single_channel_groups(L):
    d = make_norm(6, 16, 8)
    d["x"][:, :8] = 3.25  # variance 0: n = 0, y = bias
    check(L, 6, 16, 2, "f32", False, "silu", d)
    check(L, 6, 16, 16, "f32", True, "silu", d)


def test_pointers_off_16_bytes(L):
    import torch
    d = make_norm(12, 128, 9)
    ref = delta.group_norm_act(d["x"], 2, d["weight"], d["bias"], d["gate"], "silu")
    for dtype, off in ((torch.float32, 1), (torch.bfloat16, 3)):
        def shifted(x):
            t = torch.empty(x.size + off, dtype=dtype, device="cuda")[off:]
            return t.copy_(torch.from_numpy(x).flatten()).view(12, 128)
        y = L.group_norm_act(shifted(d["x"]), 2, to_dev(d["weight"]), to_dev(d["bias"]), gate=shifted(d["gate"]))
        e = rms_err(host(y), ref)
        # bfloat16 rounds the inputs too (2^-9 each of x and gate), which the oracle does not see.
        assert e <= (TOL_F32 if dtype == torch.float32 else TOL_BF16 * 2)


def test_empty(L):
    import torch
    x = torch.empty(0, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    assert L.group_norm_act(x, 4, w, w).shape == (0, 64)
    gx, gw, gb, gg = L.group_norm_act_backward(x, 4, w, w, x)
    assert gx.shape == (0, 64) and gg is None
    assert not host(gw).any() and not host(gb).any()


def test_a_nan_stays_in_its_group(L):
    d = make_norm(5, 96, 10)
    d["x"][2, 40] = np.nan
    y = host(L.group_norm_act(to_dev(d["x"]), 3, to_dev(d["weight"]), to_dev(d["bias"])))
    bad = np.isnan(y)
    assert bad[2, 32:64].all() and bad.sum() == 32


def test_same_bits_again(L):
    d = make_norm(3001, 640, 12, "bf16")
    a = [to_dev(d[n], "bf16") for n in ("x", "gout", "gate")]
    w, b = to_dev(d["weight"]), to_dev(d["bias"])
    one = [host(t) for t in L.group_norm_act_backward(a[0], 5, w, b, a[1], gate=a[2])]
    two = [host(t) for t in L.group_norm_act_backward(a[0], 5, w, b, a[1], gate=a[2])]
    assert all(np.array_equal(p, q) for p, q in zip(one, two))


def test_another_stream(L):
    import torch
    d = make_norm(257, 256, 13)
    ref = delta.group_norm_act(d["x"], 4, d["weight"], d["bias"])
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        y = L.group_norm_act(to_dev(d["x"]), 4, to_dev(d["weight"]), to_dev(d["bias"]))
    s.synchronize()
    assert rms_err(host(y), ref) <= TOL_F32


def test_refusals(L):
    import torch
    x, w = torch.zeros(4, 64, device="cuda"), torch.ones(64, device="cuda")
    with pytest.raises(L.LinrecError, match="does not divide"):
        L.group_norm_act(x, 5, w, w)
    with pytest.raises(ValueError):
        L.group_norm_act(x, 4, w, w, act="gelu")
    with pytest.raises(TypeError):
        L.group_norm_act(x.half(), 4, w, w)
    with pytest.raises(TypeError):
        L.group_norm_act(x, 4, w.bfloat16(), w)
    with pytest.raises(ValueError):
        L.group_norm_act(x.t(), 2, w[:4].contiguous(), w[:4].contiguous())
    with pytest.raises(ValueError):
        L.group_norm_act(x, 4, w, w, gate=x[:2])
    with pytest.raises(L.LinrecError, match="eps"):
        L.group_norm_act(x, 4, w, w, eps=-1.0)
    with pytest.raises(ValueError, match="expected a ROCm device"):
        L.group_norm_act(x.cpu(), 4, w.cpu(), w.cpu())
    big = torch.zeros(1, 8193, device="cuda")
    with pytest.raises(L.LinrecError, match="8193 channels"):
        L.group_norm_act(big, 1, big[0], big[0])
