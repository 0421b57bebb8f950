"""Calls that MoELayer refuses before it touches anything (no GPU needed)."""
from __future__ import annotations

import pytest

import moe_expert_ffn_router_amd as moe


def test_streamed_step_refuses_the_fp8_variant():
    layer = object.__new__(moe.MoELayer)       # no buffers: the refusal comes first
    with pytest.raises(ValueError, match="fp8"):
        layer.forward_streamed(None, None, 0, None, None, None, variant="fp8")
