"""The example serves a batch in which a prompt is empty: its first token has none before it."""

import os
import sys

import pytest

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_empty_prompt():
    import torch
    from gated_delta_mix import GatedDeltaMix, serve
    torch.manual_seed(0)
    # float32 throughout: the two ways differ by rounding alone, as for other prompts.
    assert serve(GatedDeltaMix(64, 2, torch.float32).cuda(), lengths=(9, 0, 3)) <= 1e-3
