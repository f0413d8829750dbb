"""Calls of include/moe_kv8.h's Python objects and binding that are refused before
anything is launched (no GPU is touched)."""
import pytest
import torch

from moe_expert_layer_warp_gb300 import api, batch


def test_rotated_results_without_their_rows():
    """q_out is where q goes: given without q it would stay as it was."""
    rotary = batch.Rotary.__new__(batch.Rotary)
    x, positions = torch.zeros(3, 2, 64), torch.zeros(3, dtype=torch.int32)
    for args in ((None, x, positions, x, None), (x, None, positions, None, x),
                 (None, x, positions, x, x)):
        with pytest.raises(ValueError, match="q_out and k_out"):
            rotary.rotate(*args)
    desc = api.RotaryDesc(64, 64, 0, 0, 1.0, 1 << 20)
    with pytest.raises(ValueError, match="q_out without q"):
        api.moe_rotary(desc, None, x, positions, q_out=x)
    with pytest.raises(ValueError, match="k_out without k"):
        api.moe_rotary(desc, x, None, positions, k_out=x)
