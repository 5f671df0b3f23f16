"""The group norm of channels whose mean is large beside their spread, forward and backward, against
the float64 oracle on the same float32 inputs.  What the inputs' own rounding costs is in the inputs
already, so the tolerance is the library's float32 one."""

import sys

import numpy as np
import pytest

from oracle import delta
from delta_cases import TOL_F32, host, make_norm, rms_err, to_dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("mean", [1e3, 1e4, -3e4])
@pytest.mark.parametrize("D", [3, 24, 125, 128, 500, 1000, 2048, 8192])
@pytest.mark.parametrize("gated", [False, True])
def test_large_means(D, mean, gated):
    import linear_recurrence_rnn_amd as L
    sys.__stderr__.write("[gpu case] group_norm large mean %s\n" % ((D, mean, gated),))
    sys.__stderr__.flush()
    G = 1 if D > 1000 else 3
    d = make_norm(40, D * G, D, mean=mean)
    gate = d["gate"] if gated else None
    x, go, z, w, b = (to_dev(t) for t in (d["x"], d["gout"], gate, d["weight"], d["bias"]))
    y = L.group_norm_act(x, G, w, b, gate=z)
    got = L.group_norm_act_backward(x, G, w, b, go, gate=z)
    assert rms_err(host(y), delta.group_norm_act(d["x"], G, d["weight"], d["bias"], gate)) <= TOL_F32
    ref = delta.group_norm_act_backward(d["x"], G, d["weight"], d["bias"], d["gout"], gate)
    for name, p, q in zip(("x", "weight", "bias", "gate"), got, ref):
        if q is not None:
            assert rms_err(host(p), q) <= TOL_F32, name


def test_constant_groups_are_zero():
    # x = mean in every channel: n = 0 exactly, whatever D does to the mean's rounding.
    import linear_recurrence_rnn_amd as L
    for D in (3, 125, 1000, 8191):
        x = np.full((5, D), 12345.678, np.float32)
        w, b = np.ones(D, np.float32), np.full(D, 0.5, np.float32)
        y = host(L.group_norm_act(to_dev(x), 1, to_dev(w), to_dev(b), act="none"))
        assert np.max(np.abs(y - 0.5)) <= TOL_F32, D
