"""MoELayer's router training and FP8 variant on a stream of the caller's: the memory that these
calls allocate is not memory that work pending on the current stream still uses."""
from __future__ import annotations

import pytest
import torch

import synth
from gpu_cases import Case, flush

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import moe_expert_ffn_router_amd as moe  # noqa: E402

DEV = torch.device("cuda")
WL = synth.Workload("streams", T=200, H=1024, E=16, I=256, k=4, fmt="fp8_b128", seed=5)


def _layer(case):
    layer = moe.MoELayer(WL.fmt, WL.E, WL.H, WL.I, WL.k, WL.T, case.stride)
    layer.route_permute(case.logits)
    return layer


def _pending_writes(sizes):
    """Blocks of these sizes, written late by the current stream and free again already."""
    junk = [torch.empty(n, dtype=torch.uint8, device=DEV) for n in sizes for _ in range(4)]
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)
    for j in junk:
        j.fill_(0x5a)


def _handle(s, raw):
    return s.cuda_stream if raw else s


@pytest.mark.parametrize("raw", [False, True])
def test_balance_loss_allocates_on_its_stream(raw):
    flush(f"[layer streams] balance loss, raw handle {raw}")
    case = Case(WL)
    layer = _layer(case)
    seq = torch.tensor([0, 70, 190], dtype=torch.int32, device=DEV)
    ref = layer.balance_loss(case.logits, None, seq)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    ws = max(moe.moe_balance_loss_workspace(WL.T, WL.E, 2), 256)
    _pending_writes([8, 8 * WL.E, ws])
    got = layer.balance_loss(case.logits, None, seq, _handle(s, raw))
    torch.cuda.synchronize()
    for name in ref:
        assert torch.equal(got[name], ref[name]), name


@pytest.mark.parametrize("raw", [False, True])
def test_balance_loss_results_freed_while_their_stream_works(raw):
    """Results dropped at once: their memory goes back to their own stream, not to the next
    allocation of the current one."""
    case = Case(WL)
    layer = _layer(case)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s):
            torch.cuda._sleep(5_000_000)
        layer.balance_loss(case.logits, None, None, _handle(s, raw))
        mine = [torch.full((n,), 7, dtype=torch.uint8, device=DEV) for n in (4, 4 * WL.E) for _ in range(8)]
        torch.cuda.synchronize()
        assert all(bool((t == 7).all()) for t in mine)


@pytest.mark.parametrize("raw", [False, True])
def test_balance_loss_results_read_by_the_current_stream(raw):
    """The current stream waits, reads the results late, and they are dropped before it has: the
    caller's stream does not write over them meanwhile."""
    case = Case(WL)
    layer = _layer(case)
    ref = layer.balance_loss(case.logits)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = layer.balance_loss(case.logits, None, None, _handle(s, raw))
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda._sleep(20_000_000)
    read = {name: t.clone() for name, t in got.items()}
    del got
    with torch.cuda.stream(s):
        for n in (4, 4 * WL.E, max(moe.moe_balance_loss_workspace(WL.T, WL.E, 1), 256)):
            for _ in range(4):
                torch.full((n,), 0x5a, dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    for name in ref:
        assert torch.equal(read[name], ref[name]), name


def test_handle_of_the_default_stream():
    """The current stream's raw handle (0) is the current stream."""
    case = Case(WL)
    layer = _layer(case)
    W = layer.weights(case.records)
    ref = layer.balance_loss(case.logits)
    layer.expert_ffn(W, case.x, WL.T, None, "fp8")
    torch.cuda.synchronize()
    y = layer.y_perm.clone()
    layer.fp8_ws = None
    raw = torch.cuda.current_stream().cuda_stream
    got = layer.balance_loss(case.logits, stream=raw)
    layer.expert_ffn(W, case.x, WL.T, None, "fp8", raw)
    torch.cuda.synchronize()
    assert all(torch.equal(got[name], ref[name]) for name in ref) and torch.equal(layer.y_perm, y)


def test_balance_loss_captured_on_its_stream():
    """Allocations and records inside a capture; two graphs, replayed with eager work between."""
    case = Case(WL)
    layer = _layer(case)
    ref = layer.balance_loss(case.logits)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    runs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.wait_stream(torch.cuda.current_stream())
            r = layer.balance_loss(case.logits, stream=s)
            torch.cuda.current_stream().wait_stream(s)
        runs.append((g, r))
    for _ in range(3):
        for g, r in runs:
            for t in r.values():
                t.zero_()
            g.replay()
            eager = layer.balance_loss(case.logits)
            torch.cuda.synchronize()
            for name in ref:
                assert torch.equal(r[name], ref[name]) and torch.equal(eager[name], ref[name]), name


@pytest.mark.parametrize("raw", [False, True])
def test_fp8_workspace_allocates_on_its_stream(raw):
    case = Case(WL)
    layer = _layer(case)
    W = layer.weights(case.records)
    layer.expert_ffn(W, case.x, WL.T, None, "fp8")
    torch.cuda.synchronize()
    ref = layer.y_perm.clone()
    layer.fp8_ws = None
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    _pending_writes([max(moe.moe_expert_ffn_fp8_workspace(W, WL.T, WL.k), 256)])
    layer.y_perm.record_stream(s)
    layer.expert_ffn(W, case.x, WL.T, None, "fp8", _handle(s, raw))
    torch.cuda.synchronize()
    assert torch.equal(layer.y_perm, ref)
