"""The gated delta rule's and the group norm's entry points on seeded random sizes, optional arguments on
and off, against the float64 oracle; and six runs of each on larger ones, every other beside a
concurrent kernel, bit for bit.  Tolerances as for the fixed shapes."""

import sys

import numpy as np
import pytest

from oracle import delta
from delta_cases import TOL_BF16, TOL_F32, host, make_delta, make_norm, rms_err, to_dev

pytestmark = pytest.mark.gpu

INS = ("q", "k", "v", "g", "beta")
# As for the fixed shapes' bfloat16 gradients: largest error of an element and 2-norm.
BF16_MAX, BF16_FRO = 2.0 ** -4, 2.0 ** -7
RUNS = 6


def announce(*what):
    sys.__stderr__.write("[gpu case] random %s\n" % (what,))
    sys.__stderr__.flush()


def fro(out, ref):
    return float(np.linalg.norm(out - ref) / max(np.linalg.norm(ref), 1e-30))


@pytest.mark.parametrize("seed", range(24))
def test_gated_delta(seed):
    import linear_recurrence_rnn_amd as L
    rng = np.random.default_rng(1000 + seed)
    dtype = ("f32", "bf16")[seed % 2]
    B, T, Hk = int(rng.integers(1, 5)), int(np.exp(rng.uniform(0, np.log(400)))), int(rng.integers(1, 4))
    Hv, Dk, Dv = Hk * int(rng.integers(1, 4)), int(rng.integers(1, 129)), int(rng.integers(1, 257))
    state, gstate, ragged = (bool(x) for x in rng.integers(0, 2, 3))
    lengths = [int(x) for x in rng.integers(0, T + 1, B)] if ragged else None
    announce(B, T, Hk, Hv, Dk, Dv, dtype, state, gstate, lengths)
    # Rows of 16 of these decays remember about 60 tokens.
    d = make_delta(B, T, Hk, Hv, Dk, Dv, seed, dtype, decay=0.02, grads=True)
    args = [to_dev(d[n], dtype) for n in INS]
    s, gs = to_dev(d["s_in"]) if state else None, to_dev(d["gs_out"]) if gstate else None
    ln = None if lengths is None else to_dev(np.asarray(lengths, np.int32))
    o, s_out, ck = L.gated_delta_forward_ckpt(*args, state=s, lengths=ln)
    got = L.gated_delta_backward(*args, to_dev(d["go"], dtype), state=s, gstate=gs, lengths=ln, ckpt=ck)
    o1, s1 = L.gated_delta_forward(*args, state=s, lengths=ln)
    s0, g0 = d["s_in"] if state else None, d["gs_out"] if gstate else None
    ro, rs = delta.gated_delta_forward(*(d[n] for n in INS), s_in=s0, lengths=lengths)
    tol = TOL_BF16 if dtype == "bf16" else TOL_F32
    for p, q in ((o, s_out), (o1, s1)):
        assert rms_err(host(p), ro) <= tol and rms_err(host(q), rs) <= TOL_F32
    ref = delta.gated_delta_backward(*(d[n] for n in INS), d["go"], s0, g0, lengths)
    for name, x, y in zip(INS + ("state",), got, ref):
        if x is None:
            assert not state
        elif not np.any(y):
            assert not host(x).any(), name
        elif name == "g" and T == 1:
            continue  # one number a head, a sum that may cancel
        elif dtype == "f32" or name == "state":
            assert rms_err(host(x), y) <= TOL_F32, name
        else:
            assert rms_err(host(x), y) <= BF16_MAX and fro(host(x), y) <= BF16_FRO, name


@pytest.mark.parametrize("seed", range(16))
def test_group_norm(seed):
    import linear_recurrence_rnn_amd as L
    rng = np.random.default_rng(2000 + seed)
    dtype, act = ("f32", "bf16")[seed % 2], ("silu", "none")[int(rng.integers(0, 2))]
    N, G, D = int(rng.integers(1, 300)), int(rng.integers(1, 12)), int(np.exp(rng.uniform(np.log(2), np.log(1500))))
    gated = bool(rng.integers(0, 2))
    announce(N, G, D, dtype, act, gated)
    d = make_norm(N, G * D, seed, dtype)
    gate = d["gate"] if gated else None
    x, go, z, w, b = to_dev(d["x"], dtype), to_dev(d["gout"], dtype), to_dev(gate, dtype), to_dev(d["weight"]), to_dev(d["bias"])
    tol = TOL_BF16 if dtype == "bf16" else TOL_F32
    y = L.group_norm_act(x, G, w, b, gate=z, act=act)
    assert rms_err(host(y), delta.group_norm_act(d["x"], G, d["weight"], d["bias"], gate, act)) <= tol
    got = L.group_norm_act_backward(x, G, w, b, go, gate=z, act=act)
    ref = delta.group_norm_act_backward(d["x"], G, d["weight"], d["bias"], d["gout"], gate, act)
    for name, p, q in zip(("x", "weight", "bias", "gate"), got, ref):
        if q is not None:
            assert rms_err(host(p), q) <= (TOL_F32 if name in ("weight", "bias") else tol), name


def repeat(fn):
    """fn()'s outputs on the host for RUNS runs, odd runs beside a kernel on another stream."""
    import torch
    noise_in = torch.ones(1 << 28, device="cuda")
    noise_out = torch.empty_like(noise_in)
    side = torch.cuda.Stream()
    runs = []
    for i in range(RUNS):
        torch.cuda.synchronize()
        if i % 2:
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                torch.mul(noise_in, 1.5, out=noise_out)
        runs.append([host(t) for t in fn() if t is not None])
    return runs


@pytest.mark.parametrize("shape,dtype", [((2, 500, 2, 4, 128, 128), "bf16"), ((8, 200, 18, 18, 64, 100), "bf16"),
                                         ((1, 5300, 1, 1, 64, 64), "bf16"), ((2, 300, 1, 3, 48, 80), "f32"),
                                         ((1, 3500, 1, 2, 32, 48), "f32")], ids=str)
def test_gated_delta_runs_agree(shape, dtype):
    import linear_recurrence_rnn_amd as L
    announce("runs", shape, dtype)
    d = make_delta(*shape, 7, dtype, decay=0.02, grads=True)
    args, s, gs = [to_dev(d[n], dtype) for n in INS], to_dev(d["s_in"]), to_dev(d["gs_out"])
    go = to_dev(d["go"], dtype)

    def call():
        o, s_out = L.gated_delta_forward(*args, state=s)
        o2, s2, ck = L.gated_delta_forward_ckpt(*args, state=s)
        return (o, s_out, o2, s2) + tuple(L.gated_delta_backward(*args, go, state=s, gstate=gs, ckpt=ck))

    runs = repeat(call)
    assert all(np.array_equal(a, b) for r in runs[1:] for a, b in zip(runs[0], r))


def test_group_norm_runs_agree():
    import linear_recurrence_rnn_amd as L
    d = make_norm(5001, 1000, 8)
    x, go, z, w, b = (to_dev(d[n]) for n in ("x", "gout", "gate", "weight", "bias"))
    runs = repeat(lambda: (L.group_norm_act(x, 8, w, b, gate=z),) + tuple(L.group_norm_act_backward(x, 8, w, b, go, gate=z)))
    assert all(np.array_equal(a, b) for r in runs[1:] for a, b in zip(runs[0], r))
