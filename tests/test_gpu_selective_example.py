"""The example's layers (norm with the residual, short convolution, selective scan) as they are used
together: their gradients through autograd against a float64 evaluation of the same layers, training
runs, and a ragged prefill followed by single tokens gives what whole rows give."""

import os
import sys

import pytest

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def model64(model, tokens):
    """The model in float64 torch, token by token, over detached copies of its parameters."""
    import torch
    import torch.nn.functional as F
    p = {n: t.detach().double().requires_grad_() for n, t in model.named_parameters()}

    def norm(s, w):
        return s / torch.sqrt(s.square().mean(-1, keepdim=True) + 1e-5) * w

    residual = p["embed.weight"][tokens]
    x = torch.zeros_like(residual)
    for i, layer in enumerate(model.layers):
        q = {n.split(".", 2)[2]: t for n, t in p.items() if n.startswith("layers.%d." % i)}
        residual = x + residual
        n = norm(residual, q["norm"])
        pre = n @ q["into.weight"].T
        line = torch.cat([torch.zeros_like(pre[:, :layer.K - 1]), pre], 1)
        T = pre.shape[1]
        u = F.silu(sum(q["conv"][:, k] * line[:, k:k + T] for k in range(layer.K)) + q["conv_bias"])
        low, B, C = (u @ q["maps.weight"].T).split([layer.rank, layer.N, layer.N], dim=-1)
        d = F.softplus(low @ q["step_out.weight"].T + q["dt_bias"])
        A = -torch.exp(q["logA"])
        h = u.new_zeros(u.shape[0], layer.E, layer.N)
        ys = []
        for t in range(T):
            h = torch.exp(d[:, t, :, None] * A) * h + (d[:, t] * u[:, t])[:, :, None] * B[:, t, None]
            ys.append((h * C[:, t, None]).sum(-1) + q["D"] * u[:, t])
        y = torch.stack(ys, 1) * F.silu(n @ q["gate.weight"].T)
        x = y @ q["out.weight"].T
    return norm(x + residual, p["norm"]) @ p["head.weight"].T + p["head.bias"], p


def test_gradients():
    import torch
    from selective_mix import CopyModel
    torch.manual_seed(0)
    model = CopyModel(11, C=48, dtype=torch.float32).cuda()
    tokens = torch.randint(11, (3, 90), device="cuda")
    w = torch.randn(3, 90, 11, device="cuda")
    logits = model(tokens)[0]
    (logits * w).sum().backward()
    ref, p = model64(model, tokens)
    (ref * w.double()).sum().backward()
    # float32 throughout, projections with inner sums of up to 96 among it: a few 1e-6 of each tensor's norm.
    assert ((logits.double() - ref).norm() / ref.norm()).item() <= 1e-4
    for name, t in model.named_parameters():
        g = p[name].grad
        assert ((t.grad.double() - g).norm() / g.norm()).item() <= 1e-4, name


def test_gradients_twice_are_refused():
    import torch
    from selective_mix import CopyModel
    model = CopyModel(5, C=16, layers=1, dtype=torch.float32).cuda()
    loss = model(torch.zeros(1, 4, dtype=torch.long, device="cuda"))[0].sum()
    with pytest.raises(RuntimeError, match="second derivative"):
        torch.autograd.grad(loss, model.head.weight, create_graph=True)[0]
        torch.autograd.grad(loss, model.layers[0].conv, create_graph=True)


def test_training_and_serving():
    import math
    import torch
    from selective_mix import serve, train
    losses, model = train(steps=20)
    assert all(math.isfinite(x) for x in losses)
    # The operators' outputs pass through bfloat16 (2^-8 each, four a layer, two layers and the last norm), of
    # either sign over sums of 64 and 128 terms; a row's logits are small against the largest now and then.
    assert serve(model) <= 0.1
    losses, model = train(steps=3, dtype=torch.float32)
    assert all(math.isfinite(x) for x in losses)
    assert serve(model) <= 1e-3


def test_a_captured_step_beside_eager_ones():
    """A layer's forward and backward calls captured without autograd, replayed with eager passes of the
    same parameters between."""
    import torch
    import linear_recurrence_rnn_amd as L
    from selective_mix import SelectiveMix
    torch.manual_seed(1)
    mix = SelectiveMix(64, dtype=torch.bfloat16).cuda()
    x = torch.randn(2, 70, 64, device="cuda").bfloat16()
    r = torch.randn(2, 70, 64, device="cuda")

    def calls():
        with torch.no_grad():
            n, s = L.rms_norm_add(x, mix.norm, residual=r)
            u0 = torch.cat([n, n], -1)
            u, _ = L.short_conv_act(u0, mix.conv, bias=mix.conv_bias)
            B = n[..., :16].unsqueeze(-2).contiguous()
            A = -torch.exp(mix.logA)
            args = (u, u0, A, B, B)
            kw = dict(D=mix.D, z=u0, dt_bias=mix.dt_bias)
            y, st, ck = L.scan_selective_ckpt(*args, **kw)
            g = L.scan_selective_backward(*args, y, ckpt=ck, **kw)
            c = L.short_conv_act_backward(u0, mix.conv, g[0], bias=mix.conv_bias)
            return [y, st] + [t for t in g if t is not None] + [t for t in c if t is not None]

    want = [t.clone() for t in calls()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = calls()
    for _ in range(3):
        y, res, _ = mix(x, r)
        (y.float().sum() + res.sum()).backward()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b)
