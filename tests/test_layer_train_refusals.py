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


def _layer(E=8, H=128, I=256):
    layer = object.__new__(moe.MoELayer)
    layer.T_max, layer.E, layer.H, layer.I, layer.shared_I, layer.kept = 8, E, H, I, 0, (4, False)
    return layer


@pytest.mark.parametrize("W", [(4, 128, 256), (9, 128, 256), (8, 256, 256), (8, 128, 128)])
def test_weights_of_another_layer(W):
    """Fewer experts would leave the rows of the missing ones as the last batch left them."""
    x, logits = torch.zeros(4, 128), torch.zeros(4, 8)
    W = moe.Experts(0, *W, None, 0)
    with pytest.raises(ValueError, match="8 experts of 128 x 256"):
        _layer().forward_train(logits, x, W)
    with pytest.raises(ValueError, match="8 experts of 128 x 256"):
        _layer().backward(logits, x, W, x)


@pytest.mark.parametrize("E", [7, 9])
def test_logits_of_another_layer(E):
    """More experts than the layer's would be counted past its buffers."""
    x, W = torch.zeros(4, 128), moe.Experts(0, 8, 128, 256, None, 0)
    with pytest.raises(ValueError, match="logits"):
        _layer().forward_train(torch.zeros(4, E), x, W)
    with pytest.raises(ValueError, match="logits"):
        _layer().backward(torch.zeros(4, E), x, W, x)
