"""GPU parity of the root-mean-square norm behind a residual's addition against the float64 oracle:
every size class, odd channel counts, each pair of types, unaligned pointers, captured calls, refusals."""

import sys

import numpy as np
import pytest

from oracle import selective as S
from selective_cases import check_one, dev, host, make_rms, rounder

pytestmark = pytest.mark.gpu

TYPES = [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")]


@pytest.fixture(scope="module")
def L():
    import linear_recurrence_rnn_amd as L
    from linear_recurrence_rnn_amd import binding
    binding.load()
    return L


def announce(msg):
    sys.__stderr__.write("[gpu case] %s\n" % (msg,))
    sys.__stderr__.flush()


def check(L, N, C, dtype, rtype, residual=True, gsum=True, seed=0, eps=1e-5, d=None):
    announce("rms_norm_add %s" % ((N, C, dtype, rtype, residual, gsum),))
    if not residual:
        rtype = dtype
    d = make_rms(N, C, seed, dtype, rtype) if d is None else d
    x, w, gy = dev(d["x"], dtype), dev(d["weight"], None), dev(d["gy"], dtype)
    res = dev(d["residual"], rtype) if residual else None
    gs_in = dev(d["gsum"], rtype) if gsum else None
    bf16, rbf = dtype == "bf16", rtype == "bf16"
    y, s = L.rms_norm_add(x, w, residual=res, eps=eps)
    ry, rs = S.rms_norm_add(d["x"], d["weight"], d["residual"] if residual else None, eps, rounder(rtype))
    check_one("y", host(y), ry, bf16)
    if residual:
        # One float32 addition and, in bfloat16, its rounding.
        assert np.array_equal(host(s), rounder(rtype)((d["x"] + d["residual"]).astype(np.float32)))
    else:
        assert s is x
    gx, gs, gw = L.rms_norm_add_backward(s, w, gy, gsum=gs_in, eps=eps)
    rg, rw = S.rms_norm_add_backward(host(s), d["weight"], d["gy"], d["gsum"] if gsum else None, eps)
    assert gx.dtype == gy.dtype and gs.dtype == s.dtype
    # gs is a difference, v rstd - n rstd mean(v n), of which little is left where v is along n (with
    # one channel, eps / (s^2 + eps) of it).
    hs = host(s).astype(np.float64)
    v = d["gy"] * d["weight"] / np.sqrt((hs * hs).mean(-1, keepdims=True) + eps)
    check_one("gs", host(gs), rg, rbf, terms=v)
    check_one("gx", host(gx), rg, bf16, terms=v)
    check_one("gweight", host(gw), rw, False)


@pytest.mark.parametrize("types", TYPES, ids=str)
@pytest.mark.parametrize("C", [1, 2, 7, 8, 64, 100, 128, 129, 512, 513, 768, 1000, 1024, 1032, 2048, 2056, 2560, 4096, 5000,
                               8192])
def test_channels(L, C, types):
    check(L, 5, C, *types, seed=C)
    check(L, 3, C, *types, residual=False, gsum=False, seed=C)


@pytest.mark.parametrize("types", TYPES, ids=str)
@pytest.mark.parametrize("N", [1, 2, 3, 17, 300, 20000])
def test_tokens(L, N, types):
    check(L, N, 96, *types, seed=N)
    check(L, min(N, 5000), 1040, *types, gsum=False, seed=N)


def test_large_and_small_rows(L):
    # Zero rows give zeros (eps holds them), rows of 1e15 and of 1e-12 are normalised or not by eps.
    d = make_rms(4, 256, 3)
    d["x"][0] = d["residual"][0] = 0
    d["x"][1] *= 1e15
    d["residual"][2] *= 1e-12
    d["x"][2] *= 1e-12
    x, w, r = dev(d["x"], None), dev(d["weight"], None), dev(d["residual"], None)
    y, s = L.rms_norm_add(x, w, residual=r)
    ry, _ = S.rms_norm_add(d["x"], d["weight"], d["residual"], stored=rounder("f32"))
    for i in range(4):
        check_one("row %d" % i, host(y)[i], ry[i], False)


def test_leading_axes_in_place_and_none(L):
    import torch
    d = make_rms(12, 40, 4)
    x, w, r = (dev(d[n], None) for n in ("x", "weight", "residual"))
    y, s = L.rms_norm_add(x, w, residual=r)
    y3, s3 = L.rms_norm_add(x.view(3, 4, 40), w, residual=r.view(3, 4, 40))
    assert y3.shape == (3, 4, 40) and host(y3).tobytes() == host(y).tobytes() and host(s3).tobytes() == host(s).tobytes()
    stream, out = r.clone(), torch.empty_like(x)
    L.rms_norm_add(x, w, residual=stream, out=(out, stream))  # the residual stream updated in place
    assert host(out).tobytes() == host(y).tobytes() and host(stream).tobytes() == host(s).tobytes()
    gy, gsum = dev(d["gy"], None), dev(d["gsum"], None)
    gx, gs, gw = L.rms_norm_add_backward(s, w, gy, gsum=gsum)
    own = gsum.clone()
    L.rms_norm_add_backward(s, w, gy, gsum=own, out=(None, own, gw))
    assert host(own).tobytes() == host(gs).tobytes()
    none = x[:0]
    y, s = L.rms_norm_add(none, w, residual=none)
    assert y.shape == (0, 40)
    assert not host(L.rms_norm_add_backward(s, w, y)[2]).any()


@pytest.mark.parametrize("types", TYPES, ids=str)
@pytest.mark.parametrize("C", [64, 768, 2560])
def test_unaligned(L, C, types):
    import torch
    d = make_rms(6, C, 5, *types)
    g = {n: dev(v, types[1] if n in ("residual", "gsum") else None if n == "weight" else types[0]) for n, v in d.items()}

    def shift(t):
        flat = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
        flat[1:] = t.reshape(-1)
        return flat[1:].view(t.shape)

    odd = {n: shift(x) for n, x in g.items()}
    a = L.rms_norm_add(g["x"], g["weight"], residual=g["residual"])
    b = L.rms_norm_add(odd["x"], odd["weight"], residual=odd["residual"])
    a += L.rms_norm_add_backward(a[1], g["weight"], g["gy"], gsum=g["gsum"])
    b += L.rms_norm_add_backward(shift(b[1]), odd["weight"], odd["gy"], gsum=odd["gsum"])
    for x, y in zip(a, b):
        assert host(x).tobytes() == host(y).tobytes()


def test_captured_and_guards(L):
    import torch
    d = make_rms(300, 768, 6, "bf16", "bf16")
    g = {n: dev(v, None if n == "weight" else "bf16") for n, v in d.items()}
    n = L.rms_norm_add_workspace_size(300, 768)
    raw = torch.full((n + 512,), 0xA5, dtype=torch.uint8, device="cuda")

    def step():
        y, s = L.rms_norm_add(g["x"], g["weight"], residual=g["residual"])
        return (y, s) + L.rms_norm_add_backward(s, g["weight"], g["gy"], gsum=g["gsum"], workspace=raw[256:256 + n])

    want = [host(x).tobytes() for x in step()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(3):
        for x in out:
            x.zero_()
        graph.replay()
        assert [host(x).tobytes() for x in out] == want
        assert [host(x).tobytes() for x in step()] == want
    assert bool((raw[:256] == 0xA5).all()) and bool((raw[256 + n:] == 0xA5).all())


def test_refusals(L):
    import torch
    from linear_recurrence_rnn_amd import LinrecError
    x = torch.zeros(4, 16, device="cuda")
    w = torch.ones(16, device="cuda")
    for kind, f in ((TypeError, lambda: L.rms_norm_add(x.half(), w)),
                    (ValueError, lambda: L.rms_norm_add(x.cpu(), w)),
                    (TypeError, lambda: L.rms_norm_add(x, w.bfloat16())),
                    (TypeError, lambda: L.rms_norm_add(x, w, residual=x.bfloat16())),
                    (ValueError, lambda: L.rms_norm_add(x, w, residual=x[:2])),
                    (ValueError, lambda: L.rms_norm_add(x[:, ::2], w[:8])),
                    (ValueError, lambda: L.rms_norm_add_backward(x, w, x, gsum=x[:2])),
                    (LinrecError, lambda: L.rms_norm_add(x, w, eps=-1.0)),
                    (LinrecError, lambda: L.rms_norm_add(torch.zeros(1, 8200, device="cuda"),
                                                         torch.ones(8200, device="cuda")))):
        with pytest.raises(kind):
            f()
