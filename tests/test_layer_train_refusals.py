"""Training calls that MoELayer refuses before it touches anything (no GPU needed)."""
from __future__ import annotations

import pytest
import torch

import moe_expert_ffn_router_amd as moe


def test_shared_expert_of_a_layer_without_one():
    layer = object.__new__(moe.MoELayer)       # no buffers: the refusal comes first
    layer.T_max, layer.H, layer.shared_I = 8, 128, 0
    with pytest.raises(ValueError, match="shared expert"):
        layer.forward_train(torch.zeros(4, 8), torch.zeros(4, 128), None, Ws=moe.Experts())
