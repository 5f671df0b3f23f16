"""Absent tokens of the gated delta rule stay zero whatever the row's own tokens hold: an infinity or
a NaN in a present token reaches the rest of its chunk, but not the outputs and gradients of the
tokens past the row's end, nor the other rows."""

import numpy as np
import pytest

from delta_cases import host, make_delta, to_dev

pytestmark = pytest.mark.gpu

INS = ("q", "k", "v", "g", "beta")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("where", ["q", "k", "v", "g", "beta", "go", "s_in", "gs_out"])
@pytest.mark.parametrize("value", [np.nan, np.inf])
def test_absent_tokens_stay_zero(where, value, dtype):
    import linear_recurrence_rnn_amd as L
    n = 70  # the row ends inside its second chunk
    clean = make_delta(2, 130, 1, 2, 48, 40, 60, dtype, grads=True)
    lengths = to_dev(np.asarray([n, 130], np.int32))

    def run(d):
        args = [to_dev(d[x], dtype) for x in INS]
        s = to_dev(d["s_in"])
        o, _, ck = L.gated_delta_forward_ckpt(*args, state=s, lengths=lengths)
        g = L.gated_delta_backward(*args, to_dev(d["go"], dtype), state=s, gstate=to_dev(d["gs_out"]), lengths=lengths,
                                   ckpt=ck)
        return [host(t) for t in (o,) + tuple(g[:5])]

    d = {x: y.copy() for x, y in clean.items()}
    if where in ("s_in", "gs_out"):
        d[where][0, 1, 3, 5] = value
    else:
        d[where][0, 66] = value
    got, ref = run(d), run(clean)
    for name, x, y in zip(("o",) + INS, got, ref):
        assert not x[0, n:].any(), name  # a NaN counts as something
        assert np.array_equal(x[1], y[1]), name
