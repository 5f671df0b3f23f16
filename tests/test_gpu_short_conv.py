"""GPU parity of the short causal convolution (forward, gradients, one token) against the float64
oracle: lengths from none, every tap count, odd channel counts, carried inputs, ragged rows with rubbish
in absent tokens, unaligned pointers, captured calls, refusals."""

import sys

import numpy as np
import pytest

from oracle import selective as S
from selective_cases import check_one, dev, host, lens, make_conv

pytestmark = pytest.mark.gpu

F32S = ("weight", "bias")


@pytest.fixture(scope="module")
def L():
    import linear_recurrence_rnn_amd as L
    from linear_recurrence_rnn_amd import binding
    binding.load()
    return L


def announce(msg):
    sys.__stderr__.write("[gpu case] %s\n" % (msg,))
    sys.__stderr__.flush()


def to_gpu(d, dtype):
    return {n: dev(x, None if n in F32S else dtype) for n, x in d.items()}


def check(L, B, T, C, K, dtype="f32", act="silu", bias=True, state=True, lengths=None, seed=0, d=None):
    announce("short_conv_act %s" % ((B, T, C, K, dtype, act, bias, state, lengths),))
    d = make_conv(B, T, C, K, seed, dtype) if d is None else d
    g = to_gpu(d, dtype)
    bf16 = dtype == "bf16"
    o = dict(bias=d["bias"] if bias else None, act=act, s_in=d["s_in"] if state else None, lengths=lengths)
    k = dict(bias=g["bias"] if bias else None, act=act, state=g["s_in"] if state else None, lengths=lens(lengths))
    y, s = L.short_conv_act(g["x"], g["weight"], **k)
    ry, rs = S.short_conv_act(d["x"], d["weight"], **o)
    check_one("y", host(y), ry, bf16)
    assert np.array_equal(host(s), rs.astype(np.float32))  # copies of inputs
    grads = L.short_conv_act_backward(g["x"], g["weight"], g["gy"], gstate=g["gs_out"], **k)
    ref = S.short_conv_act_backward(d["x"], d["weight"], d["gy"], gs_out=d["gs_out"], **o)
    for name, a, r in zip(("gx", "gweight", "gbias", "gs_in"), grads, ref):
        if a is not None and r.size:
            check_one(name, host(a), r, bf16 and name in ("gx", "gs_in"))
    assert (grads[2] is None) == (not bias) and (grads[3] is None) == (not state)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 2, 3, 4, 15, 16, 17, 31, 32, 33, 64, 65, 200])
def test_lengths(L, T, dtype):
    check(L, 2, T, 64, 4, dtype, state=T % 2 == 1, seed=T)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K", range(1, 9))
@pytest.mark.parametrize("T", [1, 5, 50])
def test_taps(L, K, T, dtype):
    check(L, 3, T, 40, K, dtype, seed=K)
    check(L, 3, T, 13, K, dtype, act="none", bias=False, seed=K)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("C", [1, 7, 8, 63, 64, 65, 255, 512, 520, 1000])
def test_channels(L, C, dtype):
    check(L, 2, 37, C, 4, dtype, seed=C)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lengths", [[0, 1, 50], [2, 3, 4], [16, 17, 18], [50, 48, 47], [0, 0, 0]], ids=str)
@pytest.mark.parametrize("K", [2, 4, 8])
@pytest.mark.parametrize("state", [False, True])
def test_ragged_rows(L, lengths, K, state, dtype):
    d = make_conv(3, 50, 24, K, 8, dtype)
    for b, n in enumerate(lengths):
        d["x"][b, n:] = (np.nan, np.inf, -np.inf)[b]
        d["gy"][b, n:] = np.nan
    check(L, 3, 50, 24, K, dtype, lengths=lengths, state=state, d=d)


def test_many_rows(L):
    # More runs than walkers, so that a walker takes several.
    check(L, 300, 70, 72, 4, "bf16", lengths=[(7 * i) % 71 for i in range(300)], seed=2)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K", [1, 2, 4, 8])
def test_decode_step(L, K, dtype):
    """Tokens one by one are the row; the state is shifted in place."""
    d = make_conv(3, 12, 40, K, 9, dtype)
    g = to_gpu(d, dtype)
    ry, rs = S.short_conv_act(d["x"], d["weight"], d["bias"], s_in=d["s_in"])
    state = g["s_in"].clone()
    ys = []
    for t in range(12):
        before = state.clone()
        other = state.clone()
        y2 = L.short_conv_decode_step(g["x"][:, t].contiguous(), g["weight"], state, bias=g["bias"], state_out=other)
        assert host(state).tobytes() == host(before).tobytes()
        y = L.short_conv_decode_step(g["x"][:, t].contiguous(), g["weight"], state, bias=g["bias"])
        assert host(y).tobytes() == host(y2).tobytes() and host(state).tobytes() == host(other).tobytes()
        ys.append(host(y))
    check_one("y", np.stack(ys, 1), ry, dtype == "bf16")
    assert np.array_equal(host(state), rs.astype(np.float32))


def test_state_in_place_and_no_tokens(L):
    d = make_conv(2, 20, 24, 4, 10)
    g = to_gpu(d, "f32")
    want = L.short_conv_act(g["x"], g["weight"], state=g["s_in"])
    s, y = g["s_in"].clone(), g["x"].clone()
    L.short_conv_act(g["x"], g["weight"], state=s, out=(y, s))
    assert host(y).tobytes() == host(want[0]).tobytes() and host(s).tobytes() == host(want[1]).tobytes()
    none = g["x"][:, :0].contiguous()
    y, s = L.short_conv_act(none, g["weight"], state=g["s_in"])
    assert y.shape == (2, 0, 24) and host(s).tobytes() == d["s_in"].tobytes()
    gx, gw, gb, gs = L.short_conv_act_backward(none, g["weight"], none, bias=g["bias"], state=g["s_in"], gstate=g["gs_out"])
    assert not host(gw).any() and not host(gb).any() and host(gs).tobytes() == d["gs_out"].tobytes()
    empty = g["x"][:0].contiguous()
    gx, gw, gb, gs = L.short_conv_act_backward(empty, g["weight"], empty, bias=g["bias"])
    assert not host(gw).any() and not host(gb).any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_unaligned(L, dtype):
    import torch
    d = make_conv(2, 37, 64, 4, 11, dtype)
    g = to_gpu(d, dtype)

    def shift(t):
        flat = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
        flat[1:] = t.reshape(-1)
        return flat[1:].view(t.shape)

    odd = {n: shift(x) for n, x in g.items()}
    a = L.short_conv_act(g["x"], g["weight"], bias=g["bias"], state=g["s_in"])
    b = L.short_conv_act(odd["x"], odd["weight"], bias=odd["bias"], state=odd["s_in"])
    a += L.short_conv_act_backward(g["x"], g["weight"], g["gy"], bias=g["bias"], state=g["s_in"], gstate=g["gs_out"])
    b += L.short_conv_act_backward(odd["x"], odd["weight"], odd["gy"], bias=odd["bias"], state=odd["s_in"],
                                   gstate=odd["gs_out"])
    for name, x, y in zip(("y", "s", "gx", "gw", "gb", "gs"), a, b):
        check_one(name, host(y), host(x), dtype == "bf16")


def test_captured_and_guards(L):
    import torch
    d = make_conv(3, 70, 72, 4, 12, "bf16")
    g = to_gpu(d, "bf16")
    k = dict(bias=g["bias"], state=g["s_in"])
    ws_bytes = L.short_conv_act_workspace_size(3, 70, 72, 4, torch.bfloat16)
    raw = torch.full((ws_bytes + 512,), 0xA5, dtype=torch.uint8, device="cuda")

    def step():
        return L.short_conv_act(g["x"], g["weight"], **k) + L.short_conv_act_backward(
            g["x"], g["weight"], g["gy"], gstate=g["gs_out"], workspace=raw[256:256 + ws_bytes], **k)

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
    assert bool((raw[:256] == 0xA5).all()) and bool((raw[256 + ws_bytes:] == 0xA5).all())


def test_refusals(L):
    import torch
    from linear_recurrence_rnn_amd import LinrecError
    d = make_conv(2, 8, 6, 4, 13)
    g = to_gpu(d, "f32")
    for kind, f in ((TypeError, lambda: L.short_conv_act(g["x"].half(), g["weight"])),
                    (ValueError, lambda: L.short_conv_act(g["x"].cpu(), g["weight"])),
                    (ValueError, lambda: L.short_conv_act(g["x"], g["weight"][:5].contiguous())),
                    (ValueError, lambda: L.short_conv_act(g["x"], g["weight"], act="relu")),
                    (ValueError, lambda: L.short_conv_act(g["x"], g["weight"], state=g["s_in"][:, :2].contiguous())),
                    (ValueError, lambda: L.short_conv_act(g["x"][:, ::2], g["weight"])),
                    (LinrecError, lambda: L.short_conv_act(g["x"], torch.zeros(6, 9, device="cuda"))),
                    (LinrecError, lambda: L.short_conv_act_backward(
                        g["x"], g["weight"], g["gy"], state=g["s_in"], gstate=g["gs_out"],
                        out=(torch.empty_like(g["x"]), torch.empty_like(g["weight"]), None, g["gs_out"])))):
        with pytest.raises(kind):
            f()
