"""The scan's step, softplus(dt + dt_bias), and its slope are float32 results whatever the tensors' type: the
bias is float32, and so are the states and sums that take them."""

import sys

import numpy as np
import pytest

from selective_cases import bf16_round, dev, host
from test_gpu_scan_selective import L  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N", [1, 4, 16, 17])
@pytest.mark.parametrize("spread", [0.0, 0.5])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("bias", [-20.0, -12.0, -8.0, -7.0, -3.0, -0.5, 0.0, 5.0, 30.0])
def test_steps_and_slopes(L, bias, dtype, spread, N):  # noqa: F811
    # One token, u = B = C = 1 for one of the states and A = 0: that state is the step, its gradient by the step 1,
    # and dt_bias's gradient the slope.
    import torch
    sys.__stderr__.write("[gpu case] steps %s\n" % ((bias, dtype, spread, N),))
    sys.__stderr__.flush()
    n, rng = 2048, np.random.default_rng(7)
    b = (bias + 0.4 * rng.standard_normal(n)).astype(np.float32)
    dt = bf16_round(spread * rng.standard_normal(n).astype(np.float32))
    raw = (dt + b).astype(np.float64)  # the float32 sum is the formula's argument here
    d_dt, d_b = dev(dt.reshape(1, 1, n), dtype), dev(b, None)
    u = torch.ones_like(d_dt)
    A = torch.zeros(n, N, device="cuda")
    one = torch.zeros(1, 1, 1, N, dtype=u.dtype, device="cuda")
    one[..., N - 1] = 1
    step, slope = np.logaddexp(raw, 0.0), 1 / (1 + np.exp(-raw))
    # In steps of 2^-24: the exponential (3), 1 + e (1), the logarithm (2) or the reciprocal (2), a product (1), sums (1).
    tol = 8 * 2.0 ** -24

    def off(t, ref):
        return np.max(np.abs(host(t).ravel() - ref) / ref)

    y, s, ck = L.scan_selective_ckpt(u, d_dt, A, one, one, dt_bias=d_b)
    assert off(s[..., N - 1], step) <= tol
    state = torch.zeros(1, n, N, device="cuda")
    L.scan_selective_decode_step(u[:, 0], d_dt[:, 0], A, one[:, 0], one[:, 0], state, dt_bias=d_b)
    assert off(state[..., N - 1], step) <= tol
    gs = torch.zeros(1, n, N, device="cuda")
    gs[..., N - 1] = 1
    g = L.scan_selective_backward(u, d_dt, A, one, one, torch.zeros_like(u), dt_bias=d_b, gstate=gs, ckpt=ck)
    assert off(g[7], slope) <= tol
