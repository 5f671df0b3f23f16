"""The final state of rows walked in segments, at chunk counts that their first number of segments
does not divide (81 chunks in ten would leave one of them empty): the same bits over calls, with a
checkpoint and in place, and the float64 oracle's values."""

import sys

import numpy as np
import pytest

from oracle import delta
from delta_cases import TOL_BF16, TOL_F32, host, make_delta, rms_err, to_dev

pytestmark = pytest.mark.gpu

INS = ("q", "k", "v", "g", "beta")


@pytest.mark.parametrize("shape,lengths,dtype", [((1, 5184, 1, 1, 64, 64), None, "bf16"),
                                                 ((1, 5121, 1, 2, 32, 48), None, "f32"),
                                                 ((2, 5130, 1, 1, 64, 128), [5130, 4700], "bf16"),
                                                 ((1, 8256, 2, 16, 32, 32), None, "bf16"),
                                                 ((1, 16448, 1, 1, 64, 64), None, "bf16")], ids=str)
def test_final_states(shape, lengths, dtype):
    import linear_recurrence_rnn_amd as L
    sys.__stderr__.write("[gpu case] segments %s\n" % ((shape, lengths, dtype),))
    sys.__stderr__.flush()
    d = make_delta(*shape, 90, dtype, 0.01)
    args, s = [to_dev(d[n], dtype) for n in INS], to_dev(d["s_in"])
    ln = None if lengths is None else to_dev(np.asarray(lengths, np.int32))
    o, ref = (host(t) for t in L.gated_delta_forward(*args, state=s, lengths=ln))
    for _ in range(5):
        assert np.array_equal(host(L.gated_delta_forward(*args, state=s, lengths=ln)[1]), ref)
    o2, s2, _ = L.gated_delta_forward_ckpt(*args, state=s, lengths=ln)
    assert np.array_equal(host(o2), o) and np.array_equal(host(s2), ref)
    L.gated_delta_forward(*args, state=s, lengths=ln, out=(o2, s))
    assert np.array_equal(host(s), ref)
    ro, rs = delta.gated_delta_forward(*(d[n] for n in INS), s_in=d["s_in"], lengths=lengths)
    assert rms_err(o, ro) <= (TOL_BF16 if dtype == "bf16" else TOL_F32) and rms_err(ref, rs) <= TOL_F32
