"""A caller's workspace is refused unless it is a dense tensor on the call's device, large enough: the
kernels would write to host memory, or between the elements of a view."""

import pytest
import torch

from linear_recurrence_rnn_amd import binding

GPU, META = torch.device("cuda", 0), torch.device("meta")


def space(n, device=META):
    return torch.empty(n, dtype=torch.uint8, device=device)


@pytest.mark.parametrize("call", [binding._workspace, lambda n, d, w: binding._scratch(n, d, w)], ids=["pair", "tensor"])
def test_workspace(call):
    with pytest.raises(ValueError, match="expected cuda:0"):
        call(64, GPU, space(64, "cpu"))
    with pytest.raises(ValueError, match="expected cuda:0"):
        call(64, GPU, space(64))
    with pytest.raises(ValueError, match="contiguous"):
        call(64, META, space(128)[::2])
    with pytest.raises(ValueError, match="contiguous"):
        call(64, META, space(1).expand(64))
    with pytest.raises(ValueError, match="too small"):
        call(64, META, space(63))
    with pytest.raises(TypeError, match="torch.Tensor"):
        call(64, META, 0x100000)
    for ws in (space(64), space(16).view(torch.float32).new_empty(16)):
        got = call(64, META, ws)
        assert got is ws or (got[0] is ws and got[1] == 64)
