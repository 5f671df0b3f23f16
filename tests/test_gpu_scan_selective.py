"""GPU parity of the selective state space scan (forward, gradients, one token) against the float64
oracle: lengths from one token, odd channel and state counts, groups, optional inputs, carried
states, ragged rows with rubbish in absent tokens, extreme decays, unaligned pointers, captured
calls, refusals."""

import sys

import numpy as np
import pytest

from oracle import selective as S
from selective_cases import check_one, dev, host, lens, make_scan, to_dev

pytestmark = pytest.mark.gpu

INS = ("u", "dt", "A", "B", "C")
F32S = ("A", "D", "dt_bias", "s_in", "gs_out")
GRADS = ("gu", "gdt", "gA", "gB", "gC", "gD", "gz", "gdt_bias", "gs_in")


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


def options(d, g, drop, softplus, state, lengths):
    """Keyword arguments of the oracle's and of the library's calls."""
    o = {n: None if n in drop else d[n] for n in ("D", "z", "dt_bias")}
    k = {n: None if n in drop else g[n] for n in ("D", "z", "dt_bias")}
    o.update(softplus=softplus, s_in=d["s_in"] if state else None, lengths=lengths)
    k.update(softplus=softplus, state=g["s_in"] if state else None, lengths=lens(lengths))
    return o, k


def check(L, shape, dtype="f32", softplus=True, state=True, lengths=None, drop=(), seed=0, rate=1.0, grads=True, d=None,
          gstate=True):
    announce("scan_selective %s" % ((shape, dtype, softplus, state, lengths, drop, rate),))
    d = make_scan(*shape, seed, dtype, softplus, rate) if d is None else d
    g = to_gpu(d, dtype)
    o, k = options(d, g, drop, softplus, state, lengths)
    ref = S.scan_selective(*(d[n] for n in INS), **o)
    bf16 = dtype == "bf16"
    if not grads:
        y, s = L.scan_selective(*(g[n] for n in INS), **k)
    else:
        y, s, ckpt = L.scan_selective_ckpt(*(g[n] for n in INS), **k)
    assert y.dtype == g["u"].dtype
    check_one("y", host(y), ref[0], bf16)
    check_one("s_out", host(s), ref[1], False)
    if not grads:
        return
    rg = S.scan_selective_backward(*(d[n] for n in INS), d["gy"], gs_out=d["gs_out"] if gstate else None, **o)
    kept = L.scan_selective_backward(*(g[n] for n in INS), g["gy"], gstate=g["gs_out"] if gstate else None, ckpt=ckpt, **k)
    again = L.scan_selective_backward(*(g[n] for n in INS), g["gy"], gstate=g["gs_out"] if gstate else None, **k)
    for name, a, b, r in zip(GRADS, kept, again, rg):
        if a is None:
            assert b is None and (r is None or name == "gs_in")
            continue
        assert host(a).tobytes() == host(b).tobytes(), name
        check_one(name, host(a), r, bf16 and name in ("gu", "gdt", "gB", "gC", "gz"))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200, 321])
def test_lengths(L, T, dtype):
    check(L, (2, T, 40, 1, 16), dtype, state=T % 2 == 1, seed=T)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N", [1, 2, 3, 4, 5, 8, 9, 15, 16, 17, 24, 32, 33, 64, 65, 100, 128])
def test_states(L, N, dtype):
    check(L, (2, 70, 33, 1, N), dtype, seed=N)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("C,G", [(1, 1), (7, 7), (64, 1), (65, 1), (128, 2), (130, 2), (200, 4), (150, 3), (513, 1)])
def test_channels_and_groups(L, C, G, dtype):
    check(L, (2, 50, C, G, 16), dtype, seed=C)


@pytest.mark.parametrize("drop", [("D",), ("z",), ("dt_bias",), ("D", "z", "dt_bias")], ids=str)
@pytest.mark.parametrize("softplus", [True, False])
def test_optional_inputs(L, drop, softplus):
    check(L, (2, 90, 48, 2, 16), "f32", softplus, drop=drop, seed=3)
    check(L, (1, 90, 48, 2, 20), "bf16", softplus, state=False, drop=drop, seed=4, gstate=False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lengths", [[0, 1, 150], [64, 65, 63], [150, 150, 0], [1, 128, 149], [16, 17, 15]], ids=str)
@pytest.mark.parametrize("state", [False, True])
@pytest.mark.parametrize("N", [16, 24])
def test_ragged_rows(L, lengths, state, dtype, N):
    # What lies in absent tokens is not used, whatever it is.
    d = make_scan(3, 150, 70, 2, N, 21, dtype)
    for b, n in enumerate(lengths):
        for name in ("u", "dt", "B", "C", "z", "gy"):
            d[name][b, n:] = (np.nan, np.inf, -np.inf)[b]
    check(L, (3, 150, 70, 2, N), dtype, state=state, lengths=lengths, d=d)


def test_lengths_are_clamped(L):
    d = make_scan(2, 70, 16, 1, 8, 5)
    g = to_gpu(d, "f32")
    y, s = L.scan_selective(*(g[n] for n in INS), state=g["s_in"], lengths=lens([-3, 1000]))
    ref = S.scan_selective(*(d[n] for n in INS), s_in=d["s_in"], lengths=[0, 70])
    check_one("y", host(y), ref[0], False)
    check_one("s_out", host(s), ref[1], False)


@pytest.mark.parametrize("rate", [0.0, 1e-3, 30.0, 3e3])
def test_decays(L, rate):
    # No decay at all, and decays that underflow at once.
    check(L, (1, 300, 64, 1, 16), "f32", rate=rate, seed=9)
    check(L, (1, 300, 64, 1, 16), "bf16", rate=rate, seed=9)


def test_growing_states(L):
    check(L, (2, 100, 20, 1, 4), "f32", rate=-0.2, seed=10)


def test_extreme_steps(L):
    # Steps of nothing (softplus(-200), softplus(-inf) = 0) and large ones (softplus(50) = 50).
    d = make_scan(2, 80, 30, 1, 16, 11)
    d["dt"][:, ::7] = -200.0
    d["dt"][:, 3] = -np.inf
    d["dt"][:, 5::11] = 50.0
    check(L, None, d=d)


@pytest.mark.parametrize("x", [-20.0, -12.0, -8.0, -3.0, -0.5, 0.0, 0.5, 5.0, 30.0])
def test_softplus(L, x):
    # One token, one state: y = softplus(x) u B C, to a few roundings, however small it is.
    import torch
    n = 4096
    r = np.random.default_rng(0)
    raw = (x + 0.4 * r.standard_normal(n)).astype(np.float32)
    one = torch.ones(1, 1, 1, 1, device="cuda")
    y, _ = L.scan_selective(torch.ones(1, 1, n, device="cuda"), to_dev(raw).view(1, 1, n), torch.zeros(n, 1, device="cuda"),
                            one, one)
    ref = np.logaddexp(raw.astype(np.float64), 0.0)
    # The exponential (1.5 steps), the logarithm (1.5), two sums and two products: under 8 steps.
    assert np.max(np.abs(host(y).ravel() - ref) / ref) <= 8 * 2.0 ** -24


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_pieces_of_a_row(L, dtype):
    """A row in three calls, the state carried, is the row in one."""
    d = make_scan(2, 150, 70, 2, 16, 12, dtype)
    g = to_gpu(d, dtype)
    kw = {n: g[n] for n in ("D", "dt_bias")}
    s, ys = g["s_in"], []
    for a, b in ((0, 31), (31, 100), (100, 150)):
        cut = [g[n][:, a:b].contiguous() if n not in F32S else g[n] for n in INS]
        y, s = L.scan_selective(*cut, z=g["z"][:, a:b].contiguous(), state=s, **kw)
        ys.append(host(y))
    ref = S.scan_selective(*(d[n] for n in INS), D=d["D"], z=d["z"], dt_bias=d["dt_bias"], s_in=d["s_in"])
    check_one("y", np.concatenate(ys, 1), ref[0], dtype == "bf16")
    check_one("s_out", host(s), ref[1], False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N", [1, 3, 4, 16, 20, 64, 100, 128])
@pytest.mark.parametrize("C,G", [(1, 1), (66, 2)])
def test_decode_step(L, N, C, G, dtype):
    announce("decode step %s" % ((N, C, G, dtype),))
    d = make_scan(3, 1, C, G, N, N, dtype)
    g = to_gpu(d, dtype)
    args = [g[n] if n in F32S else g[n][:, 0].contiguous() for n in INS]
    kw = {n: g[n] for n in ("D", "dt_bias")}
    ref = S.scan_selective(*(d[n] for n in INS), D=d["D"], z=d["z"], dt_bias=d["dt_bias"], s_in=d["s_in"])
    state, out = g["s_in"].clone(), g["s_in"].clone()
    y = L.scan_selective_decode_step(*args, g["s_in"], z=g["z"][:, 0].contiguous(), state_out=out, **kw)
    assert host(g["s_in"]).tobytes() == d["s_in"].tobytes()
    check_one("y", host(y), ref[0][:, 0], dtype == "bf16")
    check_one("s", host(out), ref[1], False)
    y2 = L.scan_selective_decode_step(*args, state, z=g["z"][:, 0].contiguous(), **kw)  # in place
    assert host(y2).tobytes() == host(y).tobytes() and host(state).tobytes() == host(out).tobytes()
    bare = L.scan_selective_decode_step(*args, g["s_in"], softplus=False, state_out=out)
    # The raw steps, some below 0: e^(d A) is up to e^(2 * 1.4 N), beyond float32 (3.4e38 = e^88.7) from N =
    # 32 on, where no float32 result can be right; a decay of e^88 has 1.5 * 88 * 2^-24 = 8e-6.
    ref = S.scan_selective(*(d[n] for n in INS), softplus=False, s_in=d["s_in"])
    factor = (d["dt"][:, 0, :, None].astype(np.float64) * d["A"]).max(-1)  # alone it has to be a float32 too
    fits = (np.abs(ref[1]).max(-1) < 1e38) & (factor < 87)
    check_one("bare y", host(bare)[fits], ref[0][:, 0][fits], dtype == "bf16")


def test_state_in_place(L):
    d = make_scan(2, 150, 70, 1, 16, 13)
    g = to_gpu(d, "f32")
    want = L.scan_selective(*(g[n] for n in INS), state=g["s_in"])
    s = g["s_in"].clone()
    y = g["u"].clone()
    L.scan_selective(*(g[n] for n in INS), state=s, out=(y, s))
    assert host(y).tobytes() == host(want[0]).tobytes() and host(s).tobytes() == host(want[1]).tobytes()
    gs = g["gs_out"].clone()
    grads = L.scan_selective_backward(*(g[n] for n in INS), g["gy"], state=g["s_in"], gstate=g["gs_out"])
    bufs = [None if x is None else x.clone() for x in grads[:8]] + [gs]
    L.scan_selective_backward(*(g[n] for n in INS), g["gy"], state=g["s_in"], gstate=gs, out=bufs)
    for a, b in zip(grads, bufs):
        assert a is None or host(a).tobytes() == host(b).tobytes()


def test_no_tokens(L):
    import torch
    d = make_scan(2, 1, 6, 1, 3, 14)
    g = to_gpu(d, "f32")
    none = {n: g[n][:, :0].contiguous() if n not in F32S else g[n] for n in INS + ("gy",)}
    y, s = L.scan_selective(*(none[n] for n in INS), state=g["s_in"])
    assert y.shape == (2, 0, 6) and host(s).tobytes() == d["s_in"].tobytes()
    grads = L.scan_selective_backward(*(none[n] for n in INS), none["gy"], D=g["D"], dt_bias=g["dt_bias"], state=g["s_in"],
                                      gstate=g["gs_out"])
    assert host(grads[8]).tobytes() == d["gs_out"].tobytes()
    assert all(not host(grads[i]).any() for i in (2, 5, 7))
    empty = {n: g[n][:0].contiguous() if n not in ("A",) else g[n] for n in INS + ("gy",)}
    assert L.scan_selective(*(empty[n] for n in INS))[0].shape == (0, 1, 6)
    assert not host(L.scan_selective_backward(*(empty[n] for n in INS), empty["gy"])[2]).any()
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_unaligned(L, dtype):
    """Tensors that start one element past an aligned address."""
    import torch
    d = make_scan(2, 70, 66, 2, 16, 15, dtype)
    g = to_gpu(d, dtype)

    def shift(t):
        flat = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
        flat[1:] = t.reshape(-1)
        return flat[1:].view(t.shape)

    kw = {n: g[n] for n in ("D", "z", "dt_bias")}
    odd = {n: shift(x) for n, x in g.items()}
    okw = {n: odd[n] for n in ("D", "z", "dt_bias")}
    a = L.scan_selective(*(g[n] for n in INS), state=g["s_in"], **kw)
    b = L.scan_selective(*(odd[n] for n in INS), state=odd["s_in"], **okw)
    ga = L.scan_selective_backward(*(g[n] for n in INS), g["gy"], state=g["s_in"], gstate=g["gs_out"], **kw)
    gb = L.scan_selective_backward(*(odd[n] for n in INS), odd["gy"], state=odd["s_in"], gstate=odd["gs_out"], **okw)
    for x, y in zip(a + ga, b + gb):
        assert host(x).tobytes() == host(y).tobytes()
    one = [x if n in F32S else x[:, 0].contiguous() for n, x in ((n, g[n]) for n in INS)]
    s1, s2 = g["s_in"].clone(), shift(g["s_in"])
    y1 = L.scan_selective_decode_step(*one, s1, D=g["D"])
    y2 = L.scan_selective_decode_step(*(shift(x) for x in one), s2, D=odd["D"])
    check_one("y", host(y2), host(y1), dtype == "bf16")
    check_one("s", host(s2), host(s1), False)


def test_workspace_is_enough_and_bounds_hold(L):
    """Workspace, checkpoint and outputs of exactly the stated sizes, with guards around them."""
    import torch
    for shape, dtype in (((3, 77, 50, 2, 5), "f32"), ((2, 333, 70, 1, 24), "bf16"), ((1, 700, 64, 1, 16), "bf16")):
        announce("guards %s" % ((shape, dtype),))
        B, T, C, G, N = shape
        d = make_scan(*shape, 16, dtype)
        g = to_gpu(d, dtype)
        ty = g["u"].dtype
        kw = {n: g[n] for n in ("D", "z", "dt_bias")}
        kw["state"] = g["s_in"]
        want = L.scan_selective_ckpt(*(g[n] for n in INS), **kw)
        wgr = L.scan_selective_backward(*(g[n] for n in INS), g["gy"], gstate=g["gs_out"], ckpt=want[2], **kw)
        pool = []

        def guarded(t=None, nbytes=0):
            n = nbytes if t is None else t.numel() * t.element_size()
            raw = torch.full((n + 512,), 0xA5, dtype=torch.uint8, device="cuda")
            pool.append((raw, n))
            body = raw[256:256 + n]
            return body if t is None else body.view(t.dtype).view(t.shape)

        outs = [guarded(t) for t in want]
        ws = guarded(nbytes=L.scan_selective_workspace_size(B, T, C, G, N, ty))
        L.scan_selective_ckpt(*(g[n] for n in INS), out=outs, workspace=ws, **kw)
        gouts = [guarded(t) for t in wgr]
        ws = guarded(nbytes=L.scan_selective_workspace_size(B, T, C, G, N, ty, backward=True))
        L.scan_selective_backward(*(g[n] for n in INS), g["gy"], gstate=g["gs_out"], ckpt=outs[2], out=gouts, workspace=ws,
                                  **kw)
        gouts2 = [guarded(t) for t in wgr]
        ws = guarded(nbytes=L.scan_selective_workspace_size(B, T, C, G, N, ty, backward=True, ckpt=False))
        L.scan_selective_backward(*(g[n] for n in INS), g["gy"], gstate=g["gs_out"], out=gouts2, workspace=ws, **kw)
        for a, b, c in zip(wgr, gouts, gouts2):
            assert host(a).tobytes() == host(b).tobytes() == host(c).tobytes()
        for a, b in zip(want[:2], outs):
            assert host(a).tobytes() == host(b).tobytes()
        for raw, n in pool:
            assert bool((raw[:256] == 0xA5).all()) and bool((raw[256 + n:] == 0xA5).all())


def test_captured_and_two_at_once(L):
    """A training step captured and replayed, with other work between; two streams at once."""
    import torch
    d = make_scan(2, 200, 96, 1, 16, 17, "bf16")
    g = to_gpu(d, "bf16")
    kw = {n: g[n] for n in ("D", "z", "dt_bias")}
    kw["state"] = g["s_in"]

    def step():
        y, s, ck = L.scan_selective_ckpt(*(g[n] for n in INS), **kw)
        return (y, s) + L.scan_selective_backward(*(g[n] for n in INS), g["gy"], gstate=g["gs_out"], ckpt=ck, **kw)

    want = [host(x).tobytes() for x in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    also = step()
    torch.cuda.synchronize()
    for x in (got, also):
        assert [host(t).tobytes() for t in x] == want
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(3):
        for x in out:
            x.zero_()
        graph.replay()
        assert [host(t).tobytes() for t in out] == want
        assert [host(t).tobytes() for t in step()] == want


def test_refusals(L):
    import torch
    from linear_recurrence_rnn_amd import LinrecError
    d = make_scan(2, 8, 6, 2, 3, 18)
    g = to_gpu(d, "f32")
    args = [g[n] for n in INS]

    def refused(kind, f):
        with pytest.raises(kind):
            f()

    refused(TypeError, lambda: L.scan_selective(args[0].half(), *args[1:]))
    refused(TypeError, lambda: L.scan_selective(args[0], args[1].bfloat16(), *args[2:]))
    refused(ValueError, lambda: L.scan_selective(args[0].cpu(), *args[1:]))
    refused(ValueError, lambda: L.scan_selective(args[0], args[1].cpu(), *args[2:]))
    refused(ValueError, lambda: L.scan_selective(*args[:2], g["A"][:, :2].contiguous(), *args[3:]))
    refused(ValueError, lambda: L.scan_selective(args[0].transpose(0, 1), *args[1:]))
    refused(ValueError, lambda: L.scan_selective(*args, lengths=lens([1, 2, 3])))
    refused(ValueError, lambda: L.scan_selective(*args, state=g["s_in"][:1]))
    refused(ValueError, lambda: L.scan_selective(*args, workspace=torch.empty(8, dtype=torch.uint8, device="cuda")))
    refused(LinrecError, lambda: L.scan_selective(torch.zeros(1, 2, 5, device="cuda"), torch.zeros(1, 2, 5, device="cuda"),
                                                  torch.zeros(5, 3, device="cuda"), *(args[3][:1, :2].contiguous(),) * 2))
    refused(LinrecError, lambda: L.scan_selective(*args[:2], torch.zeros(6, 129, device="cuda"),
                                                  *(torch.zeros(2, 8, 1, 129, device="cuda"),) * 2))
    y, s, ck = L.scan_selective_ckpt(*args)
    refused(ValueError, lambda: L.scan_selective_backward(*args, g["gy"], ckpt=ck[:-1]))
    bufs = [torch.empty_like(g["u"])] * 9
    refused(ValueError, lambda: L.scan_selective_backward(*args, g["gy"], out=bufs))
