"""The float64 oracle of the selective scan, the short convolution and the root-mean-square norm: its
gradients against difference quotients of its forward, and small cases by hand (CPU)."""

import numpy as np
import pytest

from oracle import selective as S
from selective_cases import make_conv, make_rms, make_scan

# Central differences in float64 of step h: truncation h^2 f'''/6, rounding 2^-53 f / h: for h = 1e-5
# and values of order 1 to 100, 1e-9.
H, TOL = 1e-5, 1e-6


def differences(f, d, name, grad, rng, count=6):
    """The gradient along random directions of one input."""
    for _ in range(count):
        v = rng.standard_normal(np.shape(d[name]))
        hi, lo = dict(d), dict(d)
        hi[name], lo[name] = np.asarray(d[name], np.float64) + H * v, np.asarray(d[name], np.float64) - H * v
        got, want = (f(hi) - f(lo)) / (2 * H), float((grad * v).sum())
        assert abs(got - want) <= TOL * (1 + abs(want) + np.linalg.norm(grad)), (name, got, want)


@pytest.mark.parametrize("softplus", [True, False])
@pytest.mark.parametrize("lengths", [None, [0, 9, 5]], ids=str)
@pytest.mark.parametrize("gate", [True, False])
def test_scan_gradients(softplus, lengths, gate):
    d = make_scan(3, 9, 4, 2, 3, 1, softplus=softplus)
    rng = np.random.default_rng(2)

    def parts(d):
        ins = [d[n] for n in ("u", "dt", "A", "B", "C")]
        return ins, dict(D=d["D"], z=d["z"] if gate else None, dt_bias=d["dt_bias"], softplus=softplus, s_in=d["s_in"],
                         lengths=lengths)

    def loss(d):
        ins, kw = parts(d)
        y, s = S.scan_selective(*ins, **kw)
        return float((y * d["gy"]).sum() + (s * d["gs_out"]).sum())

    ins, kw = parts(d)
    g = S.scan_selective_backward(*ins, d["gy"], gs_out=d["gs_out"], **kw)
    for name, x in zip(("u", "dt", "A", "B", "C", "D", "z", "dt_bias", "s_in"), g):
        if x is not None:
            differences(loss, d, name, x, rng)


def test_scan_by_hand():
    # One channel, one state, no decay: h is a running sum.
    u = np.array([1.0, 2.0, 3.0]).reshape(1, 3, 1)
    one = np.ones((1, 3, 1, 1))
    y, s = S.scan_selective(u, np.ones((1, 3, 1)), np.zeros((1, 1)), one, 2 * one, softplus=False)
    assert np.allclose(y.ravel(), [2, 6, 12]) and s.ravel() == [6]
    # A decay of ln 2 halves it; D and the gate.
    y, s = S.scan_selective(u, np.ones((1, 3, 1)), -np.log(2) * np.ones((1, 1)), one, one, D=np.ones(1),
                            z=np.zeros((1, 3, 1)), softplus=False)
    assert np.allclose(y, 0) and np.allclose(s, 3 + 2 / 2 + 1 / 4)


@pytest.mark.parametrize("act", ["silu", "none"])
@pytest.mark.parametrize("K", [1, 2, 4])
@pytest.mark.parametrize("lengths", [None, [0, 6, 2]], ids=str)
def test_conv_gradients(act, K, lengths):
    d = make_conv(3, 6, 4, K, 3)
    rng = np.random.default_rng(4)

    def loss(d):
        y, s = S.short_conv_act(d["x"], d["weight"], d["bias"], act, d["s_in"], lengths)
        return float((y * d["gy"]).sum() + (s * d["gs_out"]).sum())

    g = S.short_conv_act_backward(d["x"], d["weight"], d["gy"], d["bias"], act, d["s_in"], d["gs_out"], lengths)
    for name, x in zip(("x", "weight", "bias", "s_in"), g):
        if x.size:
            differences(loss, d, name, x, rng)


def test_conv_by_hand():
    x = np.array([1.0, 2.0, 3.0]).reshape(1, 3, 1)
    w = np.array([[10.0, 1.0]])
    y, s = S.short_conv_act(x, w, act="none", s_in=np.full((1, 1, 1), 5.0))
    assert np.allclose(y.ravel(), [51, 12, 23]) and s.ravel() == [3]
    y, s = S.short_conv_act(x, w, act="none", s_in=np.full((1, 1, 1), 5.0), lengths=[0])
    assert np.all(y == 0) and s.ravel() == [5]


def test_rms_gradients():
    d = make_rms(5, 7, 5)
    rng = np.random.default_rng(6)

    def loss(d):
        y, s = S.rms_norm_add(d["x"], d["weight"], d["residual"])
        return float((y * d["gy"]).sum() + (s * d["gsum"]).sum())

    s = S.rms_norm_add(d["x"], d["weight"], d["residual"])[1]
    gs, gw = S.rms_norm_add_backward(s, d["weight"], d["gy"], d["gsum"])
    for name, x in (("x", gs), ("residual", gs), ("weight", gw)):
        differences(loss, d, name, x, rng)
