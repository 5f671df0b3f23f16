"""The scan and its gradients on whole numbers without decay, where every sum is exact in float32 whatever its
order: a sum that took a value of another token, state or lane shows, however little it would change."""

import sys

import numpy as np
import pytest

from oracle import selective as S
from selective_cases import dev, host, lens
from test_gpu_scan_selective import GRADS, INS, L  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N", [1, 3, 4, 7, 8, 12, 16, 24, 40])
@pytest.mark.parametrize("shape,lengths", [((2, 70, 130, 2), [70, 33]), ((1, 48, 64, 1), None), ((3, 17, 5, 1), [1, 17, 0])],
                         ids=str)
def test_whole_numbers(L, shape, lengths, N):  # noqa: F811
    sys.__stderr__.write("[gpu case] whole numbers %s\n" % ((shape, N, lengths),))
    sys.__stderr__.flush()
    B, T, C, G = shape
    rng = np.random.default_rng(N)

    def whole(*s):
        return rng.integers(-3, 4, s).astype(np.float32)

    # States and what enters them from the right stay below 70 * 9 + 3, sums over 65 channels of a product with 3 or 9
    # of those and over 40 states of 3 times 3 of them below 4e5: all of 24 bits.
    d = {"u": whole(B, T, C), "dt": np.ones((B, T, C), np.float32), "A": np.zeros((C, N), np.float32),
         "B": whole(B, T, G, N), "C": whole(B, T, G, N), "D": whole(C), "s_in": whole(B, C, N), "gy": whole(B, T, C),
         "gs_out": whole(B, C, N)}
    g = {n: dev(x, None) for n, x in d.items()}
    y, s, ck = L.scan_selective_ckpt(*(g[n] for n in INS), D=g["D"], softplus=False, state=g["s_in"], lengths=lens(lengths))
    o = dict(D=d["D"], softplus=False, s_in=d["s_in"], lengths=lengths)
    ry, rs = S.scan_selective(*(d[n] for n in INS), **o)
    assert np.array_equal(host(y), ry) and np.array_equal(host(s), rs)
    grads = L.scan_selective_backward(*(g[n] for n in INS), g["gy"], D=g["D"], softplus=False, state=g["s_in"],
                                      gstate=g["gs_out"], lengths=lens(lengths), ckpt=ck)
    ref = S.scan_selective_backward(*(d[n] for n in INS), d["gy"], gs_out=d["gs_out"], **o)
    for name, a, r in zip(GRADS, grads, ref):
        if name not in ("gA", "gz", "gdt_bias"):  # A's gradient: products of two states, of more than 24 bits
            assert np.array_equal(host(a), r), name
