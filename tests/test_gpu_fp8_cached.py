"""The FP8 variant through the expert cache: forward_cached's slot table and fills, with a pool
smaller than the layer, give the bits of the run with every expert resident."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import synth
from gpu_cases import flush

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import moe_expert_ffn_router_amd as moe  # noqa: E402

DEV = torch.device("cuda")


@pytest.mark.parametrize("T,E,S,H,I", [
    (2, 32, 12, 512, 128),          # 16-row tiles
    (40, 8, 8, 1024, 256),          # 32-row gate/up tiles
    (400, 12, 12, 256, 640)])       # 64 x 256 gate/up tiles
def test_cached_forward(T, E, S, H, I):
    flush(f"[fp8 cached] T={T} E={E} S={S} H={H} I={I}")
    layers, k = 2, 4
    wl = synth.Workload("fp8_cached", T=T, H=H, E=E, I=I, k=k, fmt="fp8_b128", seed=31)
    stride = synth.record_layout(wl.fmt, H, I)["stride"]
    sets = [synth.make_expert_records(wl.fmt, E, H, I, wl.seed, layer=L).to(DEV) for L in range(layers)]
    bank = torch.empty((layers * E, stride), dtype=torch.uint8, pin_memory=True)
    bank.copy_(torch.cat(sets).cpu())
    pool = torch.zeros((S, stride), dtype=torch.uint8, device=DEV)
    table = torch.full((layers * E,), -1, dtype=torch.int32, device=DEV)
    cache = moe.ExpertCache(layers, E, S, stride, pool, bank, table)
    layer = moe.MoELayer(wl.fmt, E, H, I, k, T, stride)
    pool_W = moe.experts(wl.fmt, E, H, I, pool, stride)
    side = torch.cuda.Stream()
    fills = 0
    for b in range(6):
        L = b % layers
        lg = torch.from_numpy(synth.make_logits(wl, b)).to(DEV)
        x = torch.from_numpy(synth.make_x(wl, b).view(np.int16)).to(DEV).view(torch.bfloat16)
        y, info = layer.forward_cached(lg, x, L, cache, pool_W, table, side=side, variant="fp8")
        y = y.clone()
        torch.cuda.synchronize()
        fills += info["misses"]
        ref = layer.forward(lg, x, layer.weights(sets[L]), variant="fp8")
        torch.cuda.synchronize()
        assert torch.equal(y, ref), b
    assert fills > S                           # slots were refilled
    cache.close()
