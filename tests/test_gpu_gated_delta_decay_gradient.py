"""The gradient of strong decays: with every token's g at -20 or -50, dg is of the order of e^g, far below
the gradients of what the token writes itself, and keeps its float32 digits at every place in a chunk."""

import numpy as np
import pytest

from oracle import delta
from delta_cases import TOL_F32, host, make_delta, rms_err, to_dev

pytestmark = pytest.mark.gpu

INS = ("q", "k", "v", "g", "beta")


@pytest.mark.parametrize("g", [-5.0, -20.0, -50.0])
@pytest.mark.parametrize("T", [64, 150])
def test_uniform_decays(g, T):
    import linear_recurrence_rnn_amd as L
    d = make_delta(1, T, 1, 2, 32, 48, 95, grads=True)
    d["g"][:] = g
    args = [to_dev(d[n]) for n in INS]
    got = L.gated_delta_backward(*args, to_dev(d["go"]), state=to_dev(d["s_in"]), gstate=to_dev(d["gs_out"]))
    ref = delta.gated_delta_backward(*(d[n] for n in INS), d["go"], d["s_in"], d["gs_out"])
    assert rms_err(host(got[3]), ref[3]) <= TOL_F32
