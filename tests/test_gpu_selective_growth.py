"""States that grow: over a segment or a block of tokens by more than a float32 holds, while they themselves, from
nothing or from little, are ordinary numbers."""

import sys

import numpy as np
import pytest

from oracle import selective as S
from selective_cases import TOL_F32, check_one, dev, host, rms_err
from test_gpu_scan_selective import GRADS, INS, L  # noqa: F401

pytestmark = pytest.mark.gpu

SHAPES = [(1, 300, 64, 1, 16), (1, 700, 40, 1, 4), (2, 300, 70, 2, 24), (1, 500, 33, 1, 64), (1, 1500, 64, 1, 16)]


def inputs(shape, growing):
    """Steps of 1/8 and decays e^-1/8 a token; A is above zero, or the steps are below."""
    B, T, C, G, N = shape
    rng = np.random.default_rng(1)
    sign = -1.0 if growing == "A" else 1.0
    d = {x: rng.standard_normal((B, T) + e).astype(np.float32) for x, e in
         (("u", (C,)), ("B", (G, N)), ("C", (G, N)), ("gy", (C,)))}
    d["A"] = np.full((C, N), -sign, np.float32)
    d["dt"] = np.full((B, T, C), sign / 8, np.float32)
    d["s_in"] = rng.standard_normal((B, C, N)).astype(np.float32)
    d["gs_out"] = rng.standard_normal((B, C, N)).astype(np.float32)
    return d, sign


def announce(*what):
    sys.__stderr__.write("[gpu case] growth %s\n" % (what,))
    sys.__stderr__.flush()


@pytest.mark.parametrize("growing", ["A", "dt"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_growth_of_nothing(L, shape, growing):  # noqa: F811
    # Tokens 60 to 159 take the state times e^6 each, 2^138 over 16 of them, and ten on either side times e^-200: what
    # comes to them from the left, and as a gradient from the right, is zero, and nothing enters between.
    announce(shape, growing)
    d, sign = inputs(shape, growing)
    d["dt"][:, 50:170] = 200 * sign
    d["dt"][:, 60:160] = -6 * sign
    d["u"][:, 50:170] = d["gy"][:, 50:170] = 0
    g = {x: dev(v, None) for x, v in d.items()}
    y, s, ck = L.scan_selective_ckpt(*(g[x] for x in INS), softplus=False, state=g["s_in"])
    ry, rs = S.scan_selective(*(d[x] for x in INS), softplus=False, s_in=d["s_in"])
    check_one("y", host(y), ry, False)
    check_one("s", host(s), rs, False)
    ref = S.scan_selective_backward(*(d[x] for x in INS), d["gy"], softplus=False, s_in=d["s_in"], gs_out=d["gs_out"])
    for keep in (ck, None):
        grads = L.scan_selective_backward(*(g[x] for x in INS), g["gy"], softplus=False, state=g["s_in"], gstate=g["gs_out"],
                                          ckpt=keep)
        for name, a, r in zip(GRADS, grads, ref):
            if a is not None:
                check_one(name, host(a), r, False)


@pytest.mark.parametrize("growing", ["A", "dt"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_growth_of_little(L, shape, growing):  # noqa: F811
    # A state of 1e-37 times e^6 for each of 20 tokens, with nothing entering: 1.3e15.
    announce(shape, growing)
    d, sign = inputs(shape, growing)
    d["s_in"] *= np.float32(1e-37)
    d["dt"][:, :20] = -6 * sign
    d["u"][:, :20] = 0
    g = {x: dev(v, None) for x, v in d.items()}
    y, s = L.scan_selective(*(g[x] for x in INS), softplus=False, state=g["s_in"])
    ry, rs = S.scan_selective(*(d[x] for x in INS), softplus=False, s_in=d["s_in"])
    # The exponent over a segment, up to 174 in base 2, is a product rounded once with a rounded log2(e): 174 * 2^-24 *
    # (1 + 1/4) * ln 2 = 9e-6 of the result, below the float32 tolerance.
    assert rms_err(host(y), ry) <= TOL_F32 and rms_err(host(s), rs) <= TOL_F32
