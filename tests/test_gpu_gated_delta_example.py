"""The example's layer (token shift, gated delta rule, gated head norm) as it is used: its
gradients through autograd against a float64 evaluation of the same layer, training lowers the
loss, and a ragged prefill followed by single tokens gives what whole rows give."""

import os
import sys

import pytest

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def layer64(mix, x):
    """The layer in float64 torch, token by token, over detached copies of its parameters."""
    import torch
    import torch.nn.functional as F
    p = {n: t.detach().double().requires_grad_() for n, t in mix.named_parameters()}
    B, T, C = x.shape
    prev = torch.cat([torch.zeros_like(x[:, :1]), x[:, :-1]], 1)
    m = [p["mu"][i] * x + (1 - p["mu"][i]) * prev for i in range(3)]
    q, k, v = ((m[i] @ p[n + ".weight"].T).view(B, T, mix.H, mix.D) for i, n in enumerate("qkv"))
    z, a, b = (m[2] @ p["gates.weight"].T + p["gates.bias"]).split([C, mix.H, mix.H], dim=-1)
    q, k = (F.normalize(F.silu(t), dim=-1) for t in (q, k))
    dec, beta = torch.exp(-torch.exp(p["rate"]) * F.softplus(a)), torch.sigmoid(b)
    S = x.new_zeros(B, mix.H, mix.D, mix.D)
    out = []
    for t in range(T):
        S = dec[:, t, :, None, None] * S
        u = v[:, t] - (S * k[:, t, :, :, None]).sum(2)
        S = S + k[:, t, :, :, None] * (beta[:, t, :, None] * u)[:, :, None]
        out.append((S * q[:, t, :, :, None]).sum(2) * mix.D ** -0.5)
    o = torch.stack(out, 1)
    n = F.layer_norm(o, (mix.D,)).reshape(B, T, C) * p["weight"] + p["bias"]
    return (n * F.silu(z)) @ p["out.weight"].T, p


def test_layer_gradients():
    import torch
    from gated_delta_mix import GatedDeltaMix
    torch.manual_seed(0)
    mix = GatedDeltaMix(64, 2, torch.float32).cuda()
    x = torch.randn(2, 90, 64, device="cuda")
    w = torch.randn(2, 90, 64, device="cuda")
    y, _ = mix(x)
    (y * w).sum().backward()
    y64, p = layer64(mix, x.double())
    (y64 * w.double()).sum().backward()
    # float32 throughout, its projections (inner sums of 64) and the norm of small outputs among
    # it: a few 1e-6 of each tensor's norm.
    assert ((y.double() - y64).norm() / y64.norm()).item() <= 1e-4
    for name, t in mix.named_parameters():
        g = p[name].grad
        assert ((t.grad.double() - g).norm() / g.norm()).item() <= 1e-4, name


def test_training_and_serving():
    import torch
    from gated_delta_mix import serve, train
    losses, model = train(steps=60)
    assert sum(losses[-10:]) < 0.8 * sum(losses[:10])
    # The outputs pass through bfloat16 (2^-9) at the recurrence and at the norm, whose division by
    # a small deviation can magnify the first by an order of magnitude.
    assert serve(model.mix) <= 0.1
    losses, model = train(steps=3, dtype=torch.float32)
    assert serve(model.mix) <= 1e-3
