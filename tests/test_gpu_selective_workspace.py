"""The scan with a workspace and a checkpoint that start on 16 bytes and on no more, the least that the calls
accept: the same bits as anywhere else."""

import pytest

from selective_cases import host, make_scan
from test_gpu_scan_selective import INS, L, to_gpu  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shift", [16, 48])
@pytest.mark.parametrize("shape,dtype", [((2, 333, 70, 1, 16), "bf16"), ((2, 77, 50, 2, 2), "f32"), ((1, 100, 64, 1, 1), "f32"),
                                         ((2, 90, 40, 1, 8), "bf16"), ((1, 140, 64, 1, 100), "f32"), ((1, 70, 30, 1, 24), "bf16")],
                         ids=str)
def test_sixteen_bytes(L, shape, dtype, shift):  # noqa: F811
    import torch
    B, T, C, G, N = shape
    g = to_gpu(make_scan(*shape, 19, dtype), dtype)
    ty = g["u"].dtype
    kw = {n: g[n] for n in ("D", "z", "dt_bias")}
    kw["state"] = g["s_in"]
    args = [g[n] for n in INS]

    def at(nbytes):
        return torch.empty(nbytes + shift, dtype=torch.uint8, device="cuda")[shift:]

    def step(space):
        size = L.scan_selective_workspace_size
        ck = space(L.scan_selective_checkpoint_size(B, T, C, G, N, ty))
        y, s, ck = L.scan_selective_ckpt(*args, workspace=space(size(B, T, C, G, N, ty)), out=(
            torch.empty_like(g["u"]), torch.empty_like(g["s_in"]), ck), **kw)
        a = L.scan_selective_backward(*args, g["gy"], gstate=g["gs_out"], ckpt=ck,
                                      workspace=space(size(B, T, C, G, N, ty, backward=True)), **kw)
        b = L.scan_selective_backward(*args, g["gy"], gstate=g["gs_out"],
                                      workspace=space(size(B, T, C, G, N, ty, backward=True, ckpt=False)), **kw)
        return [host(t).tobytes() for t in (y, s, *a, *b)]

    assert at(64).data_ptr() % 64 == shift
    assert step(at) == step(lambda n: torch.empty(n, dtype=torch.uint8, device="cuda"))
