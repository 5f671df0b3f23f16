"""The example's functions have no second derivative: asking for one raises, instead of taking the
first derivative as a constant."""

import os
import sys

import pytest

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def refused(make, x):
    import torch
    (g,) = torch.autograd.grad(make(x).sum(), x)
    assert not g.requires_grad
    for loss in (lambda y: y.sum(), lambda y: y.square().sum()):
        with pytest.raises(RuntimeError, match="no second derivative"):
            torch.autograd.grad(loss(make(x)), x, create_graph=True)


def test_second_derivatives_are_refused():
    import torch
    from gated_delta_mix import GatedDelta, HeadNorm, TokenShift
    torch.manual_seed(0)

    def rand(*shape):
        return torch.randn(*shape, device="cuda")

    v = rand(1, 20, 1, 16).requires_grad_()
    q, k, g, b = 0.3 * rand(1, 20, 1, 16), 0.3 * rand(1, 20, 1, 16), -rand(1, 20, 1).abs(), torch.sigmoid(rand(1, 20, 1))
    refused(lambda x: GatedDelta.apply(q, k, x, g, b, None, None)[0], v)
    x, w, z = rand(4, 32).requires_grad_(), torch.ones(32, device="cuda"), rand(4, 32)
    refused(lambda x: HeadNorm.apply(x, 2, w, w, z), x)
    x, mu = rand(1, 6, 32).requires_grad_(), torch.rand(3, 32, device="cuda")
    refused(lambda x: TokenShift.apply(x, mu, None), x)
