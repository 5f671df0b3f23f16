"""Sizes at the gated delta rule's limits, on the host: products of sizes that pass 64 bits are refused
like those that do not, and a backward whose gradients' grid would pass 2^32 lanes is refused."""

import ctypes
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "linear_recurrence_rnn_amd", "liblinrec.so")

OK, INVALID, WORKSPACE, UNSUPPORTED = 0, 1, 2, 3
P = ctypes.c_void_p(0x100000)  # aligned, never dereferenced


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(LIB):
        pytest.fail("liblinrec.so is not built (run python -m linear_recurrence_rnn_amd.build)")
    from linear_recurrence_rnn_amd import binding
    return binding.load()


@pytest.mark.parametrize("heads", [(1 << 22) + 1, 1 << 60, 1 << 62])
@pytest.mark.parametrize("width", [(1, 1), (4, 8), (16, 16), (128, 128)], ids=str)
def test_many_heads_are_refused_whatever_their_product(lib, heads, width):
    for Hk in (1, heads):
        assert lib.gated_delta_forward(0, 4, Hk, heads, *width, 0, P, P, P, P, P, None, None, 1.0, P, None, P, 1 << 40,
                                       None) == UNSUPPORTED


def test_backward_grid(lib):
    def backward(B, T, H, ws):
        return lib.gated_delta_backward(B, T, H, H, 16, 16, 0, P, P, P, P, P, None, None, 1.0, None, 0, P, None, P, P, P,
                                        P, P, None, P, ws, None)
    assert backward(1 << 13, 64 << 10, 1, 0) == UNSUPPORTED
    assert backward((1 << 13) - 1, 64 << 10, 1, 0) == WORKSPACE
    assert lib.gated_delta_workspace_size(1 << 13, 64 << 10, 1, 1, 16, 16, 0, 0, 1) == 0
    assert lib.gated_delta_workspace_size((1 << 13) - 1, 64 << 10, 1, 1, 16, 16, 0, 0, 1) > 0
    assert lib.gated_delta_workspace_size(1 << 13, 64 << 10, 1, 1, 16, 16, 0, 0, 0) > 0
