"""bfloat16 outputs of the gated delta rule lose nothing but their final rounding: against the float64
oracle, in units of the error that rounding the oracle's own outputs makes.  Chunks, segments, token
by token and the decode step; states of the outputs' size and far above it.

Tolerance.  The final rounding alone is 1.  The outputs' products take states and what is written as
two bfloat16 terms, 2^-17 of each: behind sums whose terms cancel to 1/30 of their size that is 2.3e-4
against the rounding's 1.7e-3 in the 2-norm, sqrt(1 + 0.14^2) = 1.01; 1.1 leaves room."""

import sys

import numpy as np
import pytest

from oracle import delta
from delta_cases import bf16_round, host, make_delta, to_dev

pytestmark = pytest.mark.gpu

INS = ("q", "k", "v", "g", "beta")


def ratio(o, ref):
    return float(np.linalg.norm(host(o) - ref) / np.linalg.norm(bf16_round(ref) - ref))


@pytest.mark.parametrize("shape", [(2, 9, 1, 2, 64, 64), (2, 200, 2, 4, 64, 64), (1, 300, 1, 2, 128, 128),
                                   (2, 150, 1, 3, 33, 65), (1, 3200, 1, 1, 64, 80)], ids=str)
@pytest.mark.parametrize("decay", [0.1, 0.002])
@pytest.mark.parametrize("size", [0.0, 1.0, 30.0])
def test_outputs_are_rounded_once(shape, decay, size):
    import linear_recurrence_rnn_amd as L
    sys.__stderr__.write("[gpu case] outputs_are_rounded_once %s\n" % ((shape, decay, size),))
    sys.__stderr__.flush()
    d = make_delta(*shape, 55, "bf16", decay)
    d["s_in"] = d["s_in"] * np.float32(size)
    args, s = [to_dev(d[n], "bf16") for n in INS], to_dev(d["s_in"])
    o, _ = L.gated_delta_forward(*args, state=s)
    ref, _ = delta.gated_delta_forward(*(d[n] for n in INS), s_in=d["s_in"])
    assert ratio(o, ref) <= 1.1
    first = L.gated_delta_decode_step(*(a[:, 0].contiguous() for a in args), s)
    assert ratio(first, ref[:, 0]) <= 1.1
