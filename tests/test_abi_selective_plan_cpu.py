"""Which rows the selective scan cuts into segments, seen in the workspace that they need: sizes at which one side
was measured at least a sixth faster than the other."""

import pytest

WHOLE = [(8, 128, 1536, 16), (12, 128, 1536, 16), (8, 256, 1536, 16), (12, 256, 1536, 16), (12, 1024, 2560, 16),
         (16, 64, 1536, 4), (32, 128, 1536, 8), (32, 256, 1536, 8), (42, 512, 2560, 4), (8, 128, 1536, 32),
         (8, 256, 1536, 32), (4, 128, 1536, 64), (4, 128, 1536, 128), (12, 4096, 2560, 16), (12, 4096, 2560, 32)]
CUT = [(1, 256, 1536, 16), (2, 256, 1536, 16), (4, 512, 1536, 16), (12, 1024, 1536, 16), (8, 4096, 2560, 16),
       (7, 4096, 2560, 16), (1, 128, 1536, 4), (24, 4096, 2560, 4), (8, 512, 1536, 8), (20, 4096, 2560, 8),
       (1, 128, 1536, 32), (8, 1024, 1536, 32), (7, 4096, 2560, 32), (1, 128, 1536, 64), (2, 1024, 1536, 128)]


def segments_need(B, T, C, N):
    """Bytes of the workspace beyond B and C in float32, which are padded to the states of a workgroup."""
    from linear_recurrence_rnn_amd import binding
    states = N if N <= 2 else 4 if N <= 4 else 8 if N <= 8 else 16 if N <= 16 else 32 if N <= 32 else 64 if N <= 64 else 128
    rows = -(-T // 16) * 16 * B
    return binding.load().linrec_scan_selective_workspace_size(B, T, C, 1, N, 1, 0) - rows * 2 * states * 4


@pytest.mark.parametrize("shape", WHOLE, ids=str)
def test_whole(shape):
    assert 0 <= segments_need(*shape) < 256


@pytest.mark.parametrize("shape", CUT, ids=str)
def test_cut(shape):
    B, T, C, N = shape
    assert segments_need(*shape) >= 4 * B * C * N * 4
