"""Gradients of the gated delta rule and of the group norm against difference quotients of their own
forward in float32, along the gradient and along its parts on random halves of the elements: the
derivative along a part v = m g / |m g| is |m g|, so a term that is missing or counted twice shows
in full.

Tolerance: 1e-3 of the derivative.  The quotient's truncation is of order eps^2 (1e-4 at eps = 1e-2,
v of norm 1 on inputs of norm 10 and more); its rounding is that of two sums of some 10^4 float32
products, 6e-8 * 100 * the RMS of a product (below 1) over 2 eps = 3e-4 against derivatives above 1.
"""

import numpy as np
import pytest

from delta_cases import host, make_delta, make_norm, to_dev

pytestmark = pytest.mark.gpu

INS = ("q", "k", "v", "g", "beta")


def check(loss, d, grads, eps=1e-2, seed=0):
    rng = np.random.default_rng(seed)
    for name, g in grads.items():
        g = g.astype(np.float64)
        for part in range(3):
            m = np.ones(g.shape) if part == 0 else rng.integers(0, 2, g.shape)
            v = m * g
            v /= np.linalg.norm(v)
            up, dn = dict(d), dict(d)
            up[name] = (d[name] + eps * v).astype(np.float32)
            dn[name] = (d[name] - eps * v).astype(np.float32)
            # The step as the float32 inputs took it.
            took = up[name].astype(np.float64) - dn[name]
            got, want = np.sum(g * took), loss(up) - loss(dn)
            assert abs(got - want) <= 1e-3 * abs(got), (name, part, got, want)


@pytest.mark.parametrize("Hk,lengths", [(2, None), (1, [100, 37])], ids=str)
def test_gated_delta(Hk, lengths):
    import linear_recurrence_rnn_amd as L
    d = make_delta(2, 100, Hk, 2, 32, 32, 80, grads=True)
    ln = None if lengths is None else to_dev(np.asarray(lengths, np.int32))
    live = np.arange(100)[None] < np.asarray(lengths or [100, 100])[:, None]

    def loss(x):
        o, s = L.gated_delta_forward(*(to_dev(x[n]) for n in INS), state=to_dev(x["s_in"]), lengths=ln)
        return (np.sum(host(o).astype(np.float64) * d["go"] * live[:, :, None, None]) +
                np.sum(host(s).astype(np.float64) * d["gs_out"]))

    g = L.gated_delta_backward(*(to_dev(d[n]) for n in INS), to_dev(d["go"]), state=to_dev(d["s_in"]),
                               gstate=to_dev(d["gs_out"]), lengths=ln)
    check(loss, d, dict(zip(INS + ("s_in",), (host(t) for t in g))))


@pytest.mark.parametrize("gated", [False, True])
def test_group_norm(gated):
    import linear_recurrence_rnn_amd as L
    d = make_norm(20, 250, 81)

    def call(f, x, *more):
        return f(to_dev(x["x"]), 2, to_dev(x["weight"]), to_dev(x["bias"]), *more,
                 gate=to_dev(x["gate"]) if gated else None)

    g = call(L.group_norm_act_backward, d, to_dev(d["gout"]))
    names = ("x", "weight", "bias") + (("gate",) if gated else ())
    check(lambda x: np.sum(host(call(L.group_norm_act, x)).astype(np.float64) * d["gout"]), d,
          dict(zip(names, (host(t) for t in g))))
