"""GPU parity of the gated delta rule's backward (with a checkpoint and without) against the
float64 oracle: every gradient, over lengths, head widths, shared key heads, carried states,
ragged rows and extreme decays.

Tolerances.  float32 calls and state gradients: the library's 1e-4.  bfloat16 gradients: a
gradient sums up to four products whose operands (x, dv, the kept states, the weights) were
rounded to bfloat16 about three times in a chain, 2^-9 at most each, 2^-9/sqrt(3) in the RMS:
sqrt(12) 2^-9 / sqrt(3) = 2^-8 of the RMS, within 2^-7 in the Frobenius norm with the result's own
rounding.  An element of a token whose row is three times the RMS may be five deviations off:
15 * 2^-8 < 2^-4 of the RMS.
"""

import sys

import numpy as np
import pytest

from oracle import delta
from delta_cases import TOL_F32, host, make_delta, rms_err, to_dev

pytestmark = pytest.mark.gpu

INS = ("q", "k", "v", "g", "beta")
BF16_MAX, BF16_FRO = 2.0 ** -4, 2.0 ** -7


@pytest.fixture(scope="module")
def L():
    import linear_recurrence_rnn_amd as L
    from linear_recurrence_rnn_amd import binding
    binding.load()
    return L


def fro(out, ref):
    return float(np.linalg.norm(out - ref) / max(np.linalg.norm(ref), 1e-30))


def gradients(L, d, dtype, state, lengths, ckpt):
    args = [to_dev(d[n], dtype) for n in INS]
    kw = {"state": to_dev(d["s_in"]) if state else None,
          "lengths": None if lengths is None else to_dev(np.asarray(lengths, np.int32))}
    if ckpt:
        kw["ckpt"] = L.gated_delta_forward_ckpt(*args, **kw)[2]
    gs = L.gated_delta_backward(*args, to_dev(d["go"], dtype), gstate=to_dev(d["gs_out"]) if state else None, **kw)
    assert all(g.dtype == args[0].dtype for g in gs[:5]) and (gs[5] is None) == (not state)
    return [host(g) for g in gs]


def check(L, shape, dtype, state=True, lengths=None, seed=0, decay=0.1, d=None, ckpt=True):
    sys.__stderr__.write("[gpu case] gated_delta_backward %s\n" % ((shape, dtype, state, lengths, decay, ckpt),))
    sys.__stderr__.flush()
    d = make_delta(*shape, seed, dtype, decay, grads=True) if d is None else d
    got = gradients(L, d, dtype, state, lengths, ckpt)
    ref = delta.gated_delta_backward(*(d[n] for n in INS), d["go"], d["s_in"] if state else None,
                                     d["gs_out"] if state else None, lengths)
    for name, x, y in zip(INS + ("state",), got, ref):
        if x is None:
            continue
        if dtype == "f32" or name == "state":
            assert rms_err(x, y) <= TOL_F32, name
        else:
            assert rms_err(x, y) <= BF16_MAX, name
            assert fro(x, y) <= BF16_FRO, name


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 2, 16, 17, 63, 64, 65, 128, 129, 200])
def test_lengths(L, T, dtype):
    check(L, (2, T, 2, 2, 64, 64), dtype, state=T % 2 == 1, seed=T)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Dk,Dv", [(1, 1), (7, 5), (16, 16), (24, 40), (33, 65), (64, 128), (96, 80), (128, 64),
                                   (128, 128), (127, 255), (128, 256), (48, 100)])
def test_head_widths(L, Dk, Dv, dtype):
    check(L, (1, 150, 1, 2, Dk, Dv), dtype, seed=Dk, ckpt=Dk % 2 == 0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Hk,Hv", [(1, 3), (2, 4), (3, 9), (5, 5)])
def test_shared_key_heads(L, Hk, Hv, dtype):
    check(L, (2, 70, Hk, Hv, 32, 48), dtype, seed=Hk, state=False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lengths", [[0, 1, 150], [64, 65, 63], [150, 150, 0], [1, 128, 149]], ids=str)
@pytest.mark.parametrize("state", [False, True])
def test_ragged_rows(L, lengths, state, dtype):
    d = make_delta(3, 150, 2, 4, 64, 32, 21, dtype, grads=True)
    for b, n in enumerate(lengths):
        for name in INS + ("go",):
            d[name][b, n:] = np.nan if b % 2 else np.inf
    check(L, None, dtype, state, lengths, d=d, ckpt=state)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("decay", [0.0, 1e-3, 3.0, 40.0])
def test_decays(L, decay, dtype):
    check(L, (1, 300, 2, 2, 64, 64), dtype, decay=decay, seed=9)


def test_cleared_states(L):
    d = make_delta(2, 200, 1, 2, 32, 32, 12, grads=True)
    for t in (0, 5, 63, 64, 130):
        d["g"][:, t] = -np.inf
    check(L, None, "f32", d=d)


def test_repeated_keys_and_writes_of_nothing(L):
    d = make_delta(1, 190, 1, 1, 32, 32, 13, grads=True)
    d["k"][:] = d["k"][:, :1]
    d["beta"][:] = 1.0
    check(L, None, "f32", d=d)
    d["beta"][:] = 0.0  # dbeta still says what a write would do
    check(L, None, "f32", d=d)


def test_long_row(L):
    check(L, (1, 2000, 1, 1, 64, 64), "bf16", decay=0.01)
    check(L, (1, 2000, 1, 1, 64, 64), "f32", decay=0.01)


def test_segments(L):
    check(L, (1, 3300, 1, 1, 64, 48), "bf16", decay=0.01)
    check(L, (2, 3137, 1, 2, 32, 64), "f32", decay=0.01, lengths=[3137, 900], ckpt=False)


def test_against_differences_of_the_forward(L):
    # <grad, direction> against the forward's own difference quotient along it, in float32: the
    # quotient's truncation is of order eps^2 = 1e-4 relative, its rounding about 1e-6/eps = 1e-4.
    d = make_delta(1, 100, 1, 2, 32, 32, 14, grads=True)
    g = gradients(L, d, "f32", True, None, True)
    rng = np.random.default_rng(0)
    eps = 1e-2

    def loss(x):
        o, s = L.gated_delta_forward(*(to_dev(x[n]) for n in INS), state=to_dev(x["s_in"]))
        return float(np.sum(host(o).astype(np.float64) * d["go"]) + np.sum(host(s).astype(np.float64) * d["gs_out"]))

    for i, name in enumerate(INS + ("s_in",)):
        v = rng.standard_normal(d[name].shape).astype(np.float32)
        v /= np.linalg.norm(v)
        up, dn = dict(d), dict(d)
        up[name], dn[name] = d[name] + eps * v, d[name] - eps * v
        want = (loss(up) - loss(dn)) / (2 * eps)
        scale = np.linalg.norm(g[i])
        assert abs(np.sum(g[i].astype(np.float64) * v) - want) <= 2e-3 * scale, name


def test_checkpoint_changes_nothing_and_bits_repeat(L):
    d = make_delta(2, 300, 2, 4, 128, 128, 15, "bf16", grads=True)
    a = gradients(L, d, "bf16", True, None, True)
    b = gradients(L, d, "bf16", True, None, False)
    c = gradients(L, d, "bf16", True, None, True)
    assert all(np.array_equal(x, y) and np.array_equal(x, z) for x, y, z in zip(a, b, c))


def test_checkpointing_forward_is_the_forward(L):
    d = make_delta(2, 300, 2, 4, 64, 64, 16, "bf16")
    args = [to_dev(d[n], "bf16") for n in INS]
    o, s = L.gated_delta_forward(*args, state=to_dev(d["s_in"]))
    o2, s2, _ = L.gated_delta_forward_ckpt(*args, state=to_dev(d["s_in"]))
    assert np.array_equal(host(o), host(o2)) and np.array_equal(host(s), host(s2))


def test_no_tokens(L):
    import torch
    d = make_delta(2, 0, 1, 2, 8, 8, 17, grads=True)
    g = gradients(L, d, "f32", True, None, True)
    assert np.array_equal(g[5], d["gs_out"]) and g[0].shape == (2, 0, 1, 8)
    s = torch.ones(2, 2, 8, 8, device="cuda")
    e = [to_dev(d[n]) for n in INS]
    assert not host(L.gated_delta_backward(*e, to_dev(d["go"]), state=s)[5]).any()


def test_unaligned_pointers(L):
    import torch
    d = make_delta(1, 100, 1, 1, 64, 64, 18, "bf16", grads=True)

    def shifted(x):
        t = torch.empty(x.size + 1, dtype=torch.bfloat16, device="cuda")[1:]
        return t.copy_(torch.from_numpy(x).flatten()).view(x.shape)

    got = L.gated_delta_backward(*(shifted(d[n]) for n in INS), shifted(d["go"]))
    ref = delta.gated_delta_backward(*(d[n] for n in INS), d["go"])
    for x, y in zip(got[:5], ref):
        assert fro(host(x), y) <= BF16_FRO


def test_graph_replays(L):
    import torch
    d = make_delta(2, 150, 1, 2, 64, 64, 19, "bf16", grads=True)
    args = [to_dev(d[n], "bf16") for n in INS]
    go = to_dev(d["go"], "bf16")
    out = [torch.empty_like(t) for t in args] + [None]
    ws = torch.empty(L.gated_delta_workspace_size(2, 150, 1, 2, 64, 64, torch.bfloat16, True), dtype=torch.uint8,
                     device="cuda")
    L.gated_delta_backward(*args, go, out=out, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        L.gated_delta_backward(*args, go, out=out, workspace=ws)
    for i in range(3):
        go.mul_(1.5)
        ref = L.gated_delta_backward(*args, go)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(out[:5], ref[:5])), i


def test_refusals(L):
    import torch
    d = make_delta(2, 70, 1, 1, 16, 16, 20, grads=True)
    a = [to_dev(d[n]) for n in INS]
    go = to_dev(d["go"])
    with pytest.raises(ValueError):
        L.gated_delta_backward(*a, go[:, :3])
    with pytest.raises(TypeError):
        L.gated_delta_backward(*a, go.bfloat16())
    with pytest.raises(ValueError):
        L.gated_delta_backward(*a, go, gstate=to_dev(d["gs_out"])[:1])
    with pytest.raises(ValueError):
        L.gated_delta_backward(*a, go, ckpt=torch.empty(10, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        L.gated_delta_backward(*a, go, workspace=torch.empty(10, dtype=torch.uint8, device="cuda"))
