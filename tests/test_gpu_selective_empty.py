"""The scan's gradients where there are no channels: those of B and C have elements all the same, and are zero."""

import pytest

from test_gpu_scan_selective import L  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("given", [False, True])
def test_no_channels(L, dtype, given):  # noqa: F811
    import torch
    ty = torch.bfloat16 if dtype == "bf16" else torch.float32
    u, A = torch.empty(2, 5, 0, dtype=ty, device="cuda"), torch.empty(0, 3, device="cuda")
    B = torch.ones(2, 5, 2, 3, dtype=ty, device="cuda")
    y, s = L.scan_selective(u, u, A, B, B)
    assert y.shape == (2, 5, 0) and s.shape == (2, 0, 3)
    out = None
    if given:
        out = (torch.empty_like(u), torch.empty_like(u), torch.empty_like(A), torch.ones_like(B), torch.ones_like(B)) + (
            None,) * 4
    else:  # memory that was something else's
        torch.full((2, 2, 5, 2, 3), 7, dtype=ty, device="cuda")
    g = L.scan_selective_backward(u, u, A, B, B, u, out=out)
    for i in (3, 4):
        assert g[i].shape == B.shape and not g[i].any().item()
