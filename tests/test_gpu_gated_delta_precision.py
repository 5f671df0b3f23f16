"""bfloat16 training on the gated delta rule loses nothing but each result's final rounding: the
gradients against the float64 oracle, measured in units of the error that rounding the oracle's own
result to bfloat16 makes.  With a carried state, without one, and with a final-state gradient of a
row that starts from nothing (the first piece of a sequence trained in pieces).

Tolerance.  The final rounding alone is 1.  What is kept between the passes and what enters a product
carries 16 bits or more (2^-16 relative); four such factors in a chain of products and sums that
cancel to 2^-3 of their terms leave 2^-16 * 4 * 8 = 2^-11 = 4.9e-4 of the result, against the
rounding's 2^-9 / sqrt(3) * 3/2 = 1.7e-3 in the 2-norm: sqrt(1 + 0.29^2) = 1.04, and 1.25 leaves room
for sums that cancel further.
"""

import sys

import numpy as np
import pytest

from oracle import delta
from delta_cases import bf16_round, host, make_delta, to_dev

pytestmark = pytest.mark.gpu

INS = ("q", "k", "v", "g", "beta")


def distance(x, y):
    return float(np.linalg.norm(np.asarray(x, np.float64) - y))


# (s_in given, gs_out given)
@pytest.mark.parametrize("state,gstate", [(False, False), (False, True), (True, True)])
@pytest.mark.parametrize("shape", [(1, 200, 2, 2, 64, 64), (2, 300, 2, 4, 128, 128), (1, 150, 1, 2, 33, 65),
                                   (3, 40, 1, 3, 24, 48)], ids=str)
@pytest.mark.parametrize("decay,ckpt", [(0.1, False), (0.01, True), (0.002, False)])
def test_gradients_are_rounded_once(shape, decay, state, gstate, ckpt):
    import linear_recurrence_rnn_amd as L
    sys.__stderr__.write("[gpu case] gradients_are_rounded_once %s\n" % ((shape, decay, state, gstate, ckpt),))
    sys.__stderr__.flush()
    d = make_delta(*shape, 50, "bf16", decay, grads=True)
    args = [to_dev(d[n], "bf16") for n in INS]
    s = to_dev(d["s_in"]) if state else None
    ck = L.gated_delta_forward_ckpt(*args, state=s)[2] if ckpt else None
    got = L.gated_delta_backward(*args, to_dev(d["go"], "bf16"), state=s,
                                 gstate=to_dev(d["gs_out"]) if gstate else None, ckpt=ck)
    ref = delta.gated_delta_backward(*(d[n] for n in INS), d["go"], d["s_in"] if state else None,
                                     d["gs_out"] if gstate else None)
    ratio = {n: distance(host(x), y) / distance(bf16_round(y), y) for n, x, y in zip(INS, got, ref)}
    assert max(ratio.values()) <= 1.25, ratio
