"""The short convolution of very many short rows: a wave of the backward takes several, and the workspace stays
below what the chip's waves need whatever the rows."""

import pytest

import test_gpu_short_conv as conv
from test_gpu_short_conv import L  # noqa: F401


@pytest.mark.parametrize("B", [1 << 18, 1 << 16, 5000, 1])
@pytest.mark.parametrize("C", [1, 250, 256, 2561, 16384])
def test_workspace_does_not_grow_with_rows(B, C):
    import linear_recurrence_rnn_amd as L
    if B * C > 1 << 26:
        pytest.skip("beyond the sizes that a call takes")
    # 4096 waves of 64 lanes with up to four channels, four waves a workgroup, 5 rows of sums each, columns rounded up.
    assert 0 < L.short_conv_act_workspace_size(B, 4, C, 4) <= 5 * 4 * (4096 // 4 * 256 + 256 + C)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
# More rows than 4096 waves over the columns of channels: ten columns of 256, and 17, 41 and 1 of 64.
@pytest.mark.parametrize("B,T,C,K,ragged", [(430, 6, 2560, 4, True), (300, 5, 1027, 8, True), (450, 1, 2561, 2, False),
                                            (4200, 2, 7, 3, True)], ids=str)
def test_many_rows(L, B, T, C, K, ragged, dtype):  # noqa: F811
    conv.check(L, B, T, C, K, dtype, lengths=[(5 * i) % (T + 1) for i in range(B)] if ragged else None, seed=4)
