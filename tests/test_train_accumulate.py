"""accumulate without weight gradients to add to: nothing is to be added, whatever their type would be."""
from __future__ import annotations

import ctypes

import pytest
import torch

import moe_expert_ffn_router_amd as moe


@pytest.mark.parametrize("kind", [0, 1])
def test_entry_point_takes_no_weight_gradients(kind):
    """No rows and no outputs: the call has nothing to do (no GPU needed)."""
    W = moe.Experts(0, 4, 256, 128, None, moe.moe_expert_layout_query("bf16", 256, 128)["stride"])
    call = lambda d13, d2: moe._lib.moe_expert_ffn_backward(  # noqa: E731
        ctypes.byref(W), None, 0, 2, None, None, None, None, None, None, d13, d2, kind, 1, None, 0, None)
    assert call(None, None) == moe.MOE_OK
    if kind == 0:                                # bf16 gradients that are there still do not accumulate
        for given in ((1 << 20, None), (None, 1 << 20), (1 << 20, 1 << 20)):
            assert call(*given) == moe.MOE_ERR_UNSUPPORTED


@pytest.mark.gpu
@pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU")
def test_frozen_weights_beside_accumulated_ones():
    """The layer's experts accumulate while the shared expert is frozen, and the other way round."""
    from gpu_cases import flush
    from test_gpu_layer_train import F32, Step
    flush("[layer train] frozen weights, accumulated gradients")
    s = Step(T=60, E=8, H=256, I=128, k=2, shared_I=128, seed=8)
    _, whole = s.run(F32)
    for names in (("d_w13", "d_w2"), ("d_s13", "d_s2"), ("d_w2",), ()):
        given = {n: torch.full_like(whole[n], 2.0) for n in names}
        s.layer.forward_train(s.logits, s.x, s.W, s.Ws)
        r = s.layer.backward(s.logits, s.x, s.W, s.d_y, Ws=s.Ws, accumulate=True, **given)
        for n in ("d_x", "d_logits", "d_topk_w"):
            assert torch.equal(r[n], whole[n]), (names, n)
        for n, t in given.items():
            assert torch.equal(t, 2.0 + whole[n]), (names, n)
