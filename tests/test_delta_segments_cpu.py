"""Segments of a long row's chunks: the sizes that the workspace query reports say how many there are,
and none may be empty (the last segment's workgroups write the final state, and no others)."""

import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "linear_recurrence_rnn_amd", "liblinrec.so")

F32, BF16 = 0, 1


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(LIB):
        pytest.fail("liblinrec.so is not built (run python -m linear_recurrence_rnn_amd.build)")
    from linear_recurrence_rnn_amd import binding
    return binding.load()


def up(n):
    return (n + 255) // 256 * 256


def segments(lib, T, H, Dk, Dv, dtype):
    """The number of segments, from the bytes beyond what every chunk needs: (segments - 1) maps and
    as many states as segments, float32, a head."""
    n = H * ((T + 63) // 64)
    terms = 3 if dtype == F32 else 2
    rest = lib.gated_delta_workspace_size(1, T, H, H, Dk, Dv, dtype, 0, 0)
    rest -= up(n * 3 * 8192) + up(n * terms * 8192) + up(n * 512) + up(n * 768)
    if rest == 0:
        return 1
    dkp = 32 if Dk <= 32 else 64 if Dk <= 64 else 128
    cols = (Dv + 127) // 128 * 128 + dkp
    fits = [s for s in range(2, 257) if up(H * (s - 1) * dkp * cols * 4) + up(H * s * Dk * Dv * 4) == rest]
    assert len(fits) == 1, (T, H, rest)
    return fits[0]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("H", [1, 2, 5, 16, 25])
def test_no_segment_is_empty(lib, H, dtype):
    most = 1
    for nc in list(range(1, 700)) + [1025, 2049, 4097]:
        s = segments(lib, 64 * nc - nc % 64, H, 40, 64, dtype)
        most = max(most, s)
        assert (s - 1) * -(-nc // s) < nc, (nc, s)
    assert most >= 6


def test_segments_are_taken_where_heads_are_few(lib):
    assert segments(lib, 64 * 47, 1, 64, 64, BF16) == 1
    assert segments(lib, 64 * 48, 1, 64, 64, BF16) == 6
    assert segments(lib, 32768, 16, 128, 128, BF16) == 16
    assert segments(lib, 5184, 1, 64, 64, BF16) == 9
    assert segments(lib, 32768, 64, 128, 128, BF16) == 1
