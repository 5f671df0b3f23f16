"""GPU parity of the gated delta rule where heads fill the chip: bfloat16 calls of more than 64 value
channels and 144 or more heads (times segments) run eight waves a workgroup.  Against the float64
oracle on some of the rows: forward, states, every gradient; tolerances as for the other shapes."""

import sys

import numpy as np
import pytest

from oracle import delta
from delta_cases import TOL_BF16, TOL_F32, host, make_delta, rms_err, to_dev

pytestmark = pytest.mark.gpu

INS = ("q", "k", "v", "g", "beta")
# As for the other shapes' bfloat16 gradients: largest error of an element and 2-norm.
BF16_MAX, BF16_FRO = 2.0 ** -4, 2.0 ** -7


def fro(out, ref):
    return float(np.linalg.norm(out - ref) / max(np.linalg.norm(ref), 1e-30))


def announce(*what):
    sys.__stderr__.write("[gpu case] eight waves %s\n" % (what,))
    sys.__stderr__.flush()


@pytest.mark.parametrize("state", [False, True])
@pytest.mark.parametrize("Dk,Dv", [(32, 65), (64, 100), (128, 128), (24, 200), (96, 256), (128, 72)])
def test_many_heads(Dk, Dv, state):
    import linear_recurrence_rnn_amd as L
    B, T, Hk, Hv = 8, 130, 9, 18
    announce(Dk, Dv, state)
    d = make_delta(B, T, Hk, Hv, Dk, Dv, 70, "bf16", grads=True)
    lengths = [130, 0, 65, 129, 1, 64, 130, 100] if state else None
    for b, n in enumerate(lengths or []):
        for x in INS + ("go",):
            d[x][b, n:] = np.nan
    args, go = [to_dev(d[x], "bf16") for x in INS], to_dev(d["go"], "bf16")
    s = to_dev(d["s_in"]) if state else None
    ln = to_dev(np.asarray(lengths, np.int32)) if state else None
    o, s_out = L.gated_delta_forward(*args, state=s, lengths=ln)
    o2, s2, ck = L.gated_delta_forward_ckpt(*args, state=s, lengths=ln)
    assert np.array_equal(host(o), host(o2)) and np.array_equal(host(s_out), host(s2))
    gs = to_dev(d["gs_out"]) if state else None
    got = [host(g) for g in L.gated_delta_backward(*args, go, state=s, gstate=gs, lengths=ln, ckpt=ck)]
    again = [host(g) for g in L.gated_delta_backward(*args, go, state=s, gstate=gs, lengths=ln)]
    assert all(x is y is None or np.array_equal(x, y) for x, y in zip(got, again))
    o, s_out = host(o), host(s_out)
    for b in (0, 3, 5):
        r = slice(b, b + 1)
        ins = [d[x][r] for x in INS]
        s0 = d["s_in"][r] if state else None
        ln = lengths[r] if state else None
        ro, rs = delta.gated_delta_forward(*ins, s_in=s0, lengths=ln)
        assert rms_err(o[r], ro) <= TOL_BF16 and rms_err(s_out[r], rs) <= TOL_F32
        ref = delta.gated_delta_backward(*ins, d["go"][r], s0, d["gs_out"][r] if state else None, ln)
        for name, x, y in zip(INS + ("state",), got, ref):
            if x is None:
                continue
            if name == "state":
                assert rms_err(x[r], y) <= TOL_F32
            else:
                assert rms_err(x[r], y) <= BF16_MAX and fro(x[r], y) <= BF16_FRO, name


@pytest.mark.parametrize("Dk,Dv", [(128, 128), (40, 200)])
def test_segments_of_many_heads(Dk, Dv):
    # 24 heads in six or more segments: 144 and more workgroups of eight waves.
    import linear_recurrence_rnn_amd as L
    B, T, H = 1, 3300, 24 if Dv <= 128 else 18
    announce("segments", Dk, Dv)
    d = make_delta(B, T, H, H, Dk, Dv, 71, "bf16", decay=0.01)
    args, s = [to_dev(d[x], "bf16") for x in INS], to_dev(d["s_in"])
    o, s_out = (host(t) for t in L.gated_delta_forward(*args, state=s))
    for h in (0, H - 1):
        r = slice(h, h + 1)
        ro, rs = delta.gated_delta_forward(*(d[x][:, :, r] for x in INS), s_in=d["s_in"][:, r])
        assert rms_err(o[:, :, r], ro) <= TOL_BF16 and rms_err(s_out[:, r], rs) <= TOL_F32
