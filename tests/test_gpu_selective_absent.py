"""Rows that end early with more than 16 states, where the gradients of a token are formed by a kernel of their own:
whole runs of absent tokens, of which nothing is read, and ends inside a run."""

import numpy as np
import pytest

from selective_cases import make_scan
from test_gpu_scan_selective import L, check  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("drop", [(), ("z",)], ids=str)
@pytest.mark.parametrize("lengths", [[0, 1, 200, 64], [3, 4, 5, 0], [61, 63, 65, 127], [128, 129, 199, 2]], ids=str)
def test_rows_that_end(L, lengths, drop, dtype):  # noqa: F811
    d = make_scan(4, 200, 70, 2, 20, 23, dtype)
    for b, n in enumerate(lengths):
        for name in ("u", "dt", "B", "C", "z", "gy"):
            d[name][b, n:] = (np.nan, np.inf, -np.inf, np.nan)[b]
    check(L, (4, 200, 70, 2, 20), dtype, lengths=lengths, drop=drop, d=d)
