"""GPU parity of the gated delta rule (chunked forward, one-token decode step) against the
float64 oracle: lengths from one token, odd head widths, shared key heads, carried states,
ragged rows, extreme decays, unaligned pointers, refusals."""

import sys

import numpy as np
import pytest

from oracle import delta
from delta_cases import TOL_BF16, TOL_F32, host, make_delta, rms_err, to_dev

pytestmark = pytest.mark.gpu

INS = ("q", "k", "v", "g", "beta")


@pytest.fixture(scope="module")
def L():
    import linear_recurrence_rnn_amd as L
    from linear_recurrence_rnn_amd import binding
    binding.load()
    return L


def announce(msg):
    sys.__stderr__.write("[gpu case] %s\n" % (msg,))
    sys.__stderr__.flush()


def forward(L, d, dtype, state=True, lengths=None, **kw):
    args = [to_dev(d[n], dtype) for n in INS]
    o, s = L.gated_delta_forward(*args, state=to_dev(d["s_in"]) if state else None,
                                 lengths=None if lengths is None else to_dev(np.asarray(lengths, np.int32)), **kw)
    assert o.dtype == args[0].dtype
    return host(o), host(s)


def check(L, shape, dtype, state=True, lengths=None, seed=0, decay=0.1, d=None):
    announce("gated_delta_forward %s" % ((shape, dtype, state, lengths, decay),))
    d = make_delta(*shape, seed, dtype, decay) if d is None else d
    o, s = forward(L, d, dtype, state, lengths)
    ro, rs = delta.gated_delta_forward(*(d[n] for n in INS), s_in=d["s_in"] if state else None, lengths=lengths)
    assert rms_err(o, ro) <= (TOL_BF16 if dtype == "bf16" else TOL_F32)
    assert rms_err(s, rs) <= TOL_F32


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 31, 63, 64, 65, 127, 128, 129, 200])
def test_lengths(L, T, dtype):
    check(L, (2, T, 2, 2, 64, 64), dtype, state=T % 2 == 1, seed=T)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Dk,Dv", [(1, 1), (7, 5), (16, 16), (24, 40), (33, 65), (64, 128), (96, 80), (128, 64),
                                   (128, 128), (127, 255), (128, 256), (48, 100)])
def test_head_widths(L, Dk, Dv, dtype):
    check(L, (1, 150, 1, 2, Dk, Dv), dtype, seed=Dk)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Hk,Hv", [(1, 1), (1, 3), (2, 4), (3, 9), (5, 5)])
def test_shared_key_heads(L, Hk, Hv, dtype):
    check(L, (2, 70, Hk, Hv, 32, 48), dtype, seed=Hk)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lengths", [[0, 1, 150], [64, 65, 63], [150, 150, 0], [1, 128, 149]], ids=str)
@pytest.mark.parametrize("state", [False, True])
def test_ragged_rows(L, lengths, state, dtype):
    # What lies in absent tokens is not used, whatever it is.
    d = make_delta(3, 150, 2, 4, 64, 32, 21, dtype)
    for b, n in enumerate(lengths):
        for name in INS:
            d[name][b, n:] = np.nan if b % 2 else np.inf
    check(L, (3, 150, 2, 4, 64, 32), dtype, state, lengths, d=d)


def test_lengths_are_clamped(L):
    d = make_delta(2, 70, 1, 1, 16, 16, 5)
    o, s = forward(L, d, "f32", lengths=[-3, 1000])
    ro, rs = delta.gated_delta_forward(*(d[n] for n in INS), s_in=d["s_in"], lengths=[0, 70])
    assert rms_err(o, ro) <= TOL_F32 and rms_err(s, rs) <= TOL_F32


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("decay", [0.0, 1e-3, 3.0, 40.0])
def test_decays(L, decay, dtype):
    # No decay over 300 tokens, and decays that underflow within a chunk.
    check(L, (1, 300, 2, 2, 64, 64), dtype, decay=decay, seed=9)


def test_cleared_states(L):
    d = make_delta(2, 200, 1, 2, 32, 32, 12)
    for t in (0, 5, 63, 64, 130):
        d["g"][:, t] = -np.inf
    check(L, None, "f32", d=d)


def test_repeated_keys_and_full_writes(L):
    # beta = 1 with one key over and over: the chunk's triangular system at its stiffest.
    d = make_delta(1, 190, 1, 1, 32, 32, 13)
    d["k"][:] = d["k"][:, :1]
    d["beta"][:] = 1.0
    check(L, None, "f32", d=d)
    d["beta"][:] = 0.0  # nothing is written
    check(L, None, "f32", d=d)


def test_long_row(L):
    check(L, (1, 3000, 1, 1, 64, 64), "bf16", decay=0.01)
    check(L, (1, 3000, 1, 1, 64, 64), "f32", decay=0.01)


# Few heads and many chunks: the row is walked in segments that are joined (six or more of at
# least eight chunks each), also where rows end in different segments.
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape,lengths", [((1, 3200, 1, 1, 64, 64), None), ((1, 3137, 1, 2, 128, 128), None),
                                           ((2, 4000, 1, 1, 24, 40), [4000, 777]), ((3, 3500, 1, 2, 64, 160), [0, 1, 3499])],
                         ids=str)
def test_segments(L, shape, lengths, dtype):
    check(L, shape, dtype, state=True, lengths=lengths, decay=0.01, seed=shape[1])
    d = make_delta(*shape, 5, dtype, 0.01)
    args = [to_dev(d[n], dtype) for n in INS]
    s = to_dev(d["s_in"])
    ln = None if lengths is None else to_dev(np.asarray(lengths, np.int32))
    o, ref = L.gated_delta_forward(*args, state=s, lengths=ln)
    o2, s2, _ = L.gated_delta_forward_ckpt(*args, state=s, lengths=ln)
    L.gated_delta_forward(*args, state=s, lengths=ln, out=(o2, s))  # in place
    assert np.array_equal(host(o), host(o2)) and np.array_equal(host(s), host(ref)) and np.array_equal(host(s2), host(ref))


def test_in_place_state_and_no_state(L):
    import torch
    d = make_delta(2, 100, 1, 2, 64, 64, 14)
    args = [to_dev(d[n]) for n in INS]
    s = to_dev(d["s_in"])
    o = torch.empty(2, 100, 2, 64, device="cuda")
    L.gated_delta_forward(*args, state=s, out=(o, s))
    ro, rs = delta.gated_delta_forward(*(d[n] for n in INS), s_in=d["s_in"])
    assert rms_err(host(o), ro) <= TOL_F32 and rms_err(host(s), rs) <= TOL_F32
    o2, none = L.gated_delta_forward(*args, want_state=False, scale=2.0)
    assert none is None
    assert rms_err(host(o2), delta.gated_delta_forward(*(d[n] for n in INS), scale=2.0)[0]) <= TOL_F32


def test_pieces_equal_the_whole(L):
    d = make_delta(2, 230, 2, 2, 64, 64, 15)
    o, s = forward(L, d, "f32")
    cut = {n: d[n][:, :101] for n in INS}
    o1, s1 = forward(L, dict(cut, s_in=d["s_in"]), "f32")
    o2, s2 = forward(L, dict({n: d[n][:, 101:] for n in INS}, s_in=s1), "f32")
    assert rms_err(np.concatenate([o1, o2], 1), o) <= TOL_F32 and rms_err(s2, s) <= TOL_F32


def test_no_tokens(L):
    import torch
    d = make_delta(2, 0, 1, 2, 8, 8, 16)
    o, s = forward(L, d, "f32")
    assert o.shape == (2, 0, 2, 8) and np.array_equal(s, d["s_in"])
    _, s = forward(L, d, "f32", state=False)
    assert not s.any()
    e = torch.empty(0, 5, 1, 8, device="cuda")
    o, s = L.gated_delta_forward(e, e, e, e[..., 0].contiguous(), e[..., 0].contiguous())
    assert o.shape == (0, 5, 1, 8) and s.shape == (0, 1, 8, 8)


def test_unaligned_pointers(L):
    import torch
    d = make_delta(2, 100, 1, 1, 64, 64, 17, "bf16")
    for dtype, off in ((torch.float32, 1), (torch.bfloat16, 1)):
        def shifted(x, dt=dtype):
            t = torch.empty(x.size + off, dtype=dt, device="cuda")[off:]
            return t.copy_(torch.from_numpy(x).flatten()).view(x.shape)
        o, s = L.gated_delta_forward(*(shifted(d[n]) for n in INS), state=shifted(d["s_in"], torch.float32))
        ro, rs = delta.gated_delta_forward(*(d[n] for n in INS), s_in=d["s_in"])
        assert rms_err(host(o), ro) <= (TOL_F32 if dtype == torch.float32 else TOL_BF16)
        assert rms_err(host(s), rs) <= TOL_F32


def test_same_bits_again_and_on_another_stream(L):
    import torch
    d = make_delta(3, 400, 2, 4, 128, 128, 18, "bf16")
    a = forward(L, d, "bf16")
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        b = forward(L, d, "bf16")
    st.synchronize()
    assert all(np.array_equal(x, y) for x, y in zip(a, b))


def test_graph_replays(L):
    import torch
    d = make_delta(2, 300, 2, 2, 64, 64, 19, "bf16")
    args = [to_dev(d[n], "bf16") for n in INS]
    s0 = to_dev(d["s_in"])
    ws = torch.empty(max(1, L.gated_delta_workspace_size(2, 300, 2, 2, 64, 64, torch.bfloat16)), dtype=torch.uint8,
                     device="cuda")
    out = (torch.empty_like(args[2]), torch.empty_like(s0))
    L.gated_delta_forward(*args, state=s0, out=out, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        L.gated_delta_forward(*args, state=s0, out=out, workspace=ws)
    for i in range(3):
        args[2].mul_(1.5)
        ref = L.gated_delta_forward(*args, state=s0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], ref[0]) and torch.equal(out[1], ref[1]), i


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,Hk,Hv,Dk,Dv", [(1, 2, 2, 64, 64), (3, 2, 6, 128, 128), (2, 1, 1, 33, 70), (70, 4, 4, 16, 256),
                                           (2, 1, 2, 1, 3), (64, 20, 20, 128, 128)])
def test_decode_step(L, B, Hk, Hv, Dk, Dv, dtype):
    announce("gated_delta_decode_step %s" % ((B, Hk, Hv, Dk, Dv, dtype),))
    d = make_delta(B, 1, Hk, Hv, Dk, Dv, 30, dtype)
    args = [to_dev(d[n][:, 0], dtype) for n in INS]
    s = to_dev(d["s_in"])
    other = s.clone().zero_()
    o2 = L.gated_delta_decode_step(*args, s, state_out=other)
    assert np.array_equal(host(s), d["s_in"])
    o = L.gated_delta_decode_step(*args, s)
    ro, rs = delta.gated_delta_forward(*(d[n] for n in INS), s_in=d["s_in"])
    tol = TOL_BF16 if dtype == "bf16" else TOL_F32
    assert rms_err(host(o), ro[:, 0]) <= tol and rms_err(host(s), rs) <= TOL_F32
    assert np.array_equal(host(o2), host(o)) and np.array_equal(host(other), host(s))


def test_decoding_follows_the_prefill(L):
    d = make_delta(2, 90, 1, 2, 64, 64, 31)
    ro, rs = delta.gated_delta_forward(*(d[n] for n in INS), s_in=d["s_in"])
    _, s = L.gated_delta_forward(*(to_dev(d[n][:, :70]) for n in INS), state=to_dev(d["s_in"]))
    for t in range(70, 90):
        o = L.gated_delta_decode_step(*(to_dev(d[n][:, t]) for n in INS), s)
        assert rms_err(host(o), ro[:, t]) <= TOL_F32
    assert rms_err(host(s), rs) <= TOL_F32


def test_refusals(L):
    import torch
    d = make_delta(2, 8, 2, 2, 16, 16, 40)
    a = {n: to_dev(d[n]) for n in INS}
    s = to_dev(d["s_in"])

    def call(**kw):
        b = dict(a, **kw)
        return L.gated_delta_forward(*(b[n] for n in INS), state=b.get("state"), lengths=b.get("lengths"))

    with pytest.raises(TypeError):
        call(q=a["q"].half())
    with pytest.raises(TypeError):
        call(beta=a["beta"].bfloat16())
    with pytest.raises(ValueError):
        call(k=a["k"][:, :4])
    with pytest.raises(ValueError):
        call(v=a["v"].transpose(1, 2))
    with pytest.raises(ValueError):
        call(q=a["q"][0])
    with pytest.raises(ValueError):
        call(state=s[:1])
    with pytest.raises(TypeError):
        call(state=s.bfloat16())
    with pytest.raises(TypeError):
        call(lengths=torch.tensor([1, 2], device="cuda"))
    with pytest.raises(ValueError):
        call(g=a["g"].cpu())
    with pytest.raises(L.LinrecError, match="multiple"):
        call(v=torch.cat([a["v"], a["v"][:, :, :1]], 2), g=torch.cat([a["g"], a["g"][..., :1]], 2),
             beta=torch.cat([a["beta"], a["beta"][..., :1]], 2))
    with pytest.raises(ValueError, match="expected a ROCm device"):
        L.gated_delta_forward(*(a[n].cpu() for n in INS))
    wide = torch.zeros(1, 4, 1, 129, device="cuda")
    one = torch.zeros(1, 4, 1, device="cuda")
    with pytest.raises(L.LinrecError, match="widths"):
        L.gated_delta_forward(wide, wide, wide, one, one)
