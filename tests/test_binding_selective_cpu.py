"""The Python calls of the selective scan, the short convolution and the root-mean-square norm on host
tensors, without a GPU: every one is refused by name, its first input given by position or by keyword."""

import inspect

import pytest
import torch

import linear_recurrence_rnn_amd as L


def inputs():
    B, T, C, G, N, K = 2, 5, 6, 2, 3, 4
    seq, one = torch.zeros(B, T, C), torch.zeros(B, C)
    scan = {"u": seq, "dt": seq, "A": torch.zeros(C, N), "B": torch.zeros(B, T, G, N), "C": torch.zeros(B, T, G, N)}
    return {
        "scan_selective": scan,
        "scan_selective_ckpt": scan,
        "scan_selective_backward": dict(scan, gy=seq),
        "scan_selective_decode_step": {"u": one, "dt": one, "A": scan["A"], "B": torch.zeros(B, G, N),
                                       "C": torch.zeros(B, G, N), "state": torch.zeros(B, C, N)},
        "short_conv_act": {"x": seq, "weight": torch.zeros(C, K)},
        "short_conv_act_backward": {"x": seq, "weight": torch.zeros(C, K), "gy": seq},
        "short_conv_decode_step": {"x": one, "weight": torch.zeros(C, K), "state": torch.zeros(B, K - 1, C)},
        "rms_norm_add": {"x": one, "weight": torch.zeros(C)},
        "rms_norm_add_backward": {"s": one, "weight": torch.zeros(C), "gy": one},
    }


@pytest.mark.parametrize("name", sorted(inputs()))
def test_host_tensors_are_refused_by_name(name):
    call, kw = getattr(L, name), inputs()[name]
    assert list(inspect.signature(call).parameters)[:len(kw)] == list(kw)  # as documented
    for args, named in ((tuple(kw.values()), {}), (tuple(kw.values())[:1], dict(list(kw.items())[1:])), ((), kw)):
        with pytest.raises(ValueError, match="expected a ROCm device"):
            call(*args, **named)
    with pytest.raises(TypeError, match="missing"):
        call()
    with pytest.raises(TypeError, match="must be a torch.Tensor"):
        call(**{n: None for n in kw})
