"""MoELayer: buffers + the call sequence of one layer forward.

Owns the device buffers of one layer (routing results, permutation,
workspaces, outputs) and issues route -> permute -> expert_ffn -> combine on
one stream through the C ABI.  With an expert cache, the slot-table path is
route -> permute -> counts to host -> expert_cache_lookup -> expert_cache_fill
-> expert_ffn (through the slot table) -> combine; the streamed variant hands
the whole step to moe_expert_ffn_streamed (waves, grouped fills on a side
stream, the FFN behind them).  forward_train and backward are a training step
over BF16 records.  No arithmetic happens here; it only sequences library calls.
"""
from __future__ import annotations

import contextlib

import numpy as np
import torch

from . import (Experts, experts, moe_balance_loss, moe_balance_loss_workspace, moe_combine,
               moe_combine_backward, moe_dispatch_backward, moe_expert_ffn, moe_expert_ffn_backward,
               moe_expert_ffn_backward_workspace, moe_expert_ffn_fp8, moe_expert_ffn_fp8_workspace,
               moe_expert_ffn_train, moe_expert_ffn_train_workspace,
               moe_expert_ffn_workspace, moe_expert_ffn_hybrid_host_bytes,
               moe_expert_ffn_streamed_workspace, moe_route_backward,
               moe_forward_decode, moe_forward_decode_supported, moe_forward_decode_workspace,
               moe_shared_ffn, moe_shared_ffn_workspace,
               moe_permute, moe_permute_workspace, moe_route, moe_route_permute)


def _i32(n, dev):
    return torch.empty(max(int(n), 1), dtype=torch.int32, device=dev)


def _on(stream):
    """Context in which torch allocates for work on `stream` (None: the current stream).  Memory
    allocated outside it could still be in use by work pending on the current stream, which a
    kernel on `stream` does not wait for."""
    if stream is None:
        return contextlib.nullcontext()
    return torch.cuda.stream(torch.cuda.ExternalStream(stream) if isinstance(stream, int)
                             else stream)


class MoELayer:
    def __init__(self, fmt: str, E: int, H: int, I: int, k: int, T_max: int, stride: int,
                 shared_I: int = 0, shared_stride: int = 0, renorm: bool = True,
                 device: str | torch.device = "cuda"):
        self.fmt, self.E, self.H, self.I, self.k = fmt, E, H, I, k
        self.T_max, self.stride, self.renorm = T_max, stride, renorm
        dev = torch.device(device)
        self.device = dev
        A = T_max * k
        self.ids = _i32(A, dev)
        self.w = torch.empty(max(A, 1), dtype=torch.float32, device=dev)
        self.counts = _i32(E, dev)
        self.offsets = _i32(E + 1, dev)
        self.sorted_idx = _i32(A, dev)
        self.inv_idx = _i32(A, dev)
        self.perm_ws = torch.empty(max(moe_permute_workspace(T_max, k, E), 256), dtype=torch.uint8,
                                   device=dev)
        probe = Experts(0, E, H, I, None, stride)
        from . import FMT
        probe.fmt = FMT[fmt]
        self.ffn_ws = torch.empty(max(moe_expert_ffn_workspace(probe, T_max, k), 256),
                                  dtype=torch.uint8, device=dev)
        self._probe = probe
        self.stream_ws = None                 # streamed cache path: made on first use
        self.fp8_ws = None                    # variant "fp8": made on first use
        self.train = None                     # training buffers: made on first use
        self.kept = None                      # (T, with shared expert) of what backward can use
        self.counts_host = torch.zeros(E, dtype=torch.int32).pin_memory()
        self.plan_out = tuple(torch.zeros(E, dtype=torch.int32) for _ in range(3))
        self.hybrid_out = tuple(torch.zeros(E, dtype=torch.int32) for _ in range(4))
        self.host_stage = None                # hybrid path: pinned staging, made on first use
        self.y_perm = torch.empty((max(A, 1), H), dtype=torch.bfloat16, device=dev)
        self.y = torch.empty((max(T_max, 1), H), dtype=torch.bfloat16, device=dev)
        self.shared_I = shared_I
        if shared_I:
            self.shared_stride = shared_stride
            sp = Experts(FMT["bf16"], 1, H, shared_I, None, shared_stride)
            self.s_ws = torch.empty(max(moe_shared_ffn_workspace(sp, T_max), 256),
                                    dtype=torch.uint8, device=dev)
            self.y_shared = torch.empty((T_max, H), dtype=torch.bfloat16, device=dev)
        # decode-sized batches: the two-launch whole-layer path
        self.decode_ws = None
        if moe_forward_decode_supported(H, I, T_max, k):
            self.decode_ws = torch.empty(max(moe_forward_decode_workspace(probe, T_max, k), 256),
                                         dtype=torch.uint8, device=dev)

    # -- individual steps ---------------------------------------------------
    def route(self, logits: torch.Tensor, stream=None):
        T = logits.shape[0]
        self.kept = None
        moe_route(logits, self.k, self.ids, self.w, self.renorm, stream)
        return T

    def permute(self, T: int, stream=None):
        self.kept = None
        moe_permute(self.ids, T, self.k, self.E, self.counts, self.offsets, self.sorted_idx,
                    self.inv_idx, self.perm_ws, stream)

    def expert_ffn(self, W: Experts, x: torch.Tensor, T: int, slot_of_expert=None,
                   variant="auto", stream=None):
        """The routed experts.  variant "fp8" (FP8 records only) takes the activations of both
        products in E4M3 (moe_expert_ffn_fp8); the others keep bf16 activations."""
        self.kept = None
        if variant == "fp8":
            if self.fp8_ws is None:
                with _on(stream):
                    self.fp8_ws = torch.empty(
                        max(moe_expert_ffn_fp8_workspace(self._probe, self.T_max, self.k), 256),
                        dtype=torch.uint8, device=self.device)
            moe_expert_ffn_fp8(W, slot_of_expert, x, T, self.k, self.counts, self.offsets,
                               self.sorted_idx, self.y_perm, self.fp8_ws, stream)
            return
        moe_expert_ffn(W, slot_of_expert, x, T, self.k, self.counts, self.offsets, self.sorted_idx,
                       self.y_perm, self.ffn_ws, variant, stream)

    def shared_ffn(self, Ws: Experts, x: torch.Tensor, T: int, variant="auto", stream=None):
        """The always-on shared expert (bf16 record): dense, every token (moe_shared_ffn)."""
        moe_shared_ffn(Ws, x, T, self.y_shared, self.s_ws, stream)

    def combine(self, T: int, with_shared: bool, stream=None):
        moe_combine(self.y_perm, self.inv_idx, self.w, T, self.k, self.H,
                    self.y_shared if with_shared else None, self.y, stream)

    def route_permute(self, logits: torch.Tensor, stream=None):
        self.kept = None
        moe_route_permute(logits, self.k, self.ids, self.w, self.counts, self.offsets,
                          self.sorted_idx, self.inv_idx, self.perm_ws, self.renorm, stream)
        return logits.shape[0]

    # -- router training ------------------------------------------------------
    def balance_loss(self, logits: torch.Tensor, token_mask=None, seq_offsets=None,
                     stream=None) -> dict:
        """Load-balance loss of the batch last routed (self.ids), per sequence, with the
        per-expert counts and probability sums (moe_balance_loss).  The results are
        memory of `stream`, recorded as used on the current stream too, which may read them
        once it has waited for `stream`."""
        T, E = logits.shape
        S = 1 if seq_offsets is None else seq_offsets.numel() - 1
        i32 = dict(dtype=torch.int32, device=self.device)
        f32 = dict(dtype=torch.float32, device=self.device)
        with _on(stream):
            r = {"n_tokens": torch.empty(S, **i32), "counts": torch.empty(S, E, **i32),
                 "probs": torch.empty(S, E, **f32), "loss": torch.empty(S, **f32)}
            ws = torch.empty(max(moe_balance_loss_workspace(T, E, S), 256), dtype=torch.uint8,
                             device=self.device)
        moe_balance_loss(logits, self.ids[:T * self.k], self.k, r["n_tokens"], r["counts"],
                         r["probs"], r["loss"], ws, token_mask, seq_offsets, stream)
        if stream is not None:
            for t in r.values():
                t.record_stream(torch.cuda.current_stream())
        return r

    def route_backward(self, logits: torch.Tensor, d_logits: torch.Tensor, d_topk_w=None,
                       balance: dict | None = None, d_loss=None, token_mask=None,
                       seq_offsets=None, stream=None) -> torch.Tensor:
        """Gradient of the routing weights last written (d_topk_w [T*k]) and of balance_loss's
        result (d_loss [S]) with respect to the logits, into d_logits (moe_route_backward)."""
        T = logits.shape[0]
        b = balance or {}
        moe_route_backward(logits, self.k, self.ids[:T * self.k], self.w[:T * self.k], d_topk_w,
                           b.get("n_tokens"), b.get("counts"), d_loss, d_logits, self.renorm,
                           token_mask, seq_offsets, stream)
        return d_logits

    # -- training the experts -------------------------------------------------
    def _train_buffers(self, stream) -> dict:
        """What a training step keeps: the gate and up products, the gradients of the rows in
        expert order, and the workspace of both directions."""
        if self.train is None:
            A, H, I, dev = max(self.T_max * self.k, 1), self.H, self.I, self.device
            bf = dict(dtype=torch.bfloat16, device=dev)
            with _on(stream):
                b = {"gate_up": torch.empty((A, 2 * I), **bf), "d_y_perm": torch.empty((A, H), **bf),
                     "d_x_perm": torch.empty((A, H), **bf)}
                size = max(moe_expert_ffn_train_workspace(self._probe, self.T_max, self.k),
                           moe_expert_ffn_backward_workspace(self._probe, self.T_max, self.k), 256)
                if self.shared_I:
                    sp = Experts(0, 1, H, self.shared_I, None, self.shared_stride)
                    b["shared_gate_up"] = torch.empty((max(self.T_max, 1), 2 * self.shared_I), **bf)
                    b["shared_counts"], b["shared_offsets"] = _i32(1, dev), _i32(2, dev)
                    size = max(size, moe_expert_ffn_train_workspace(sp, self.T_max, 1),
                               moe_expert_ffn_backward_workspace(sp, self.T_max, 1))
                b["ws"] = torch.empty(size, dtype=torch.uint8, device=dev)
            self.train = b
        return self.train

    def _check_step(self, logits: torch.Tensor, W: Experts) -> None:
        """The library takes the sizes of what it is given; the buffers are of the layer's."""
        if logits.dim() != 2 or logits.shape[1] != self.E:
            raise ValueError(f"logits: {tuple(logits.shape)}, expected [T][{self.E}]")
        if (W.E, W.H, W.I) != (self.E, self.H, self.I):
            raise ValueError(f"W: {W.E} experts of {W.H} x {W.I}, the layer has {self.E} experts of "
                             f"{self.H} x {self.I}")

    def forward_train(self, logits: torch.Tensor, x: torch.Tensor, W: Experts,
                      Ws: Experts | None = None, stream=None) -> torch.Tensor:
        """The layer's forward over BF16 records, keeping what `backward` needs until the next
        call on this layer (the routing, the gate and up products, the experts' outputs).  Ws: the
        shared expert's record."""
        T = logits.shape[0]
        assert T <= self.T_max and x.shape == (T, self.H)
        if Ws is not None and not self.shared_I:
            raise ValueError("forward_train: Ws given, but the layer was made without a shared expert")
        self._check_step(logits, W)
        b = self._train_buffers(stream)
        self.route_permute(logits, stream)
        if T == 0:
            self.kept = (0, Ws is not None)
            return self.y[:0]
        moe_expert_ffn_train(W, x, T, self.k, self.counts, self.offsets, self.sorted_idx, b["gate_up"],
                             self.y_perm, b["ws"], stream)
        if Ws is not None:
            with _on(stream):
                b["shared_counts"].fill_(T)
                b["shared_offsets"].copy_(torch.arange(2, dtype=torch.int32, device=self.device) * T)
            moe_expert_ffn_train(Ws, x, T, 1, b["shared_counts"], b["shared_offsets"], None,
                                 b["shared_gate_up"], self.y_shared, b["ws"], stream)
        self.combine(T, Ws is not None, stream)
        self.kept = (T, Ws is not None)
        return self.y[:T]

    def backward(self, logits: torch.Tensor, x: torch.Tensor, W: Experts, d_y: torch.Tensor,
                 d_w13=None, d_w2=None, Ws: Experts | None = None, d_s13=None, d_s2=None,
                 accumulate: bool = False, balance: dict | None = None, d_loss=None, token_mask=None,
                 seq_offsets=None, stream=None) -> dict:
        """Gradient of the last forward_train with the same logits, x, W and Ws: writes (or adds to)
        the weights' gradients that are given, d_s13 and d_s2 being the shared expert's, and
        returns {"d_x", "d_logits", "d_topk_w"}.  balance, d_loss, token_mask and seq_offsets as
        for route_backward.  The results are memory of `stream`, as balance_loss's are."""
        self._check_step(logits, W)
        T, E = logits.shape
        if self.kept != (T, Ws is not None):
            raise ValueError(f"backward of {T} tokens{' with' if Ws is not None else ' without'} a shared "
                             f"expert, but forward_train kept {self.kept}")
        if x.shape != (T, self.H) or d_y.shape != (T, self.H):
            raise ValueError(f"x, d_y: expected {(T, self.H)}, got {tuple(x.shape)}, {tuple(d_y.shape)}")
        b = self._train_buffers(stream)
        with _on(stream):
            r = {"d_x": torch.empty((T, self.H), dtype=torch.bfloat16, device=self.device),
                 "d_logits": torch.zeros((T, E), dtype=torch.float32, device=self.device),
                 "d_topk_w": torch.empty((T, self.k), dtype=torch.float32, device=self.device)}
        A = T * self.k
        w, inv = self.w[:A], self.inv_idx[:A]
        d_y_perm, d_x_perm = b["d_y_perm"][:A], b["d_x_perm"][:A]
        if T:
            moe_combine_backward(d_y, inv, w, self.k, d_y_perm, self.y_perm[:A], r["d_topk_w"], stream)
        moe_expert_ffn_backward(W, x, T, self.k, self.counts, self.offsets, self.sorted_idx,
                                b["gate_up"], d_y_perm, b["ws"], d_x_perm, d_w13, d_w2, accumulate,
                                stream)
        d_add = None
        if Ws is not None:
            moe_expert_ffn_backward(Ws, x, T, 1, b["shared_counts"], b["shared_offsets"], None,
                                    b["shared_gate_up"], d_y, b["ws"], r["d_x"], d_s13, d_s2,
                                    accumulate, stream)
            d_add = r["d_x"]
        if T:
            moe_dispatch_backward(d_x_perm, inv, self.k, r["d_x"], d_add=d_add, stream=stream)
            self.route_backward(logits, r["d_logits"], r["d_topk_w"], balance, d_loss, token_mask,
                                seq_offsets, stream)
        if stream is not None:
            for t in r.values():
                t.record_stream(torch.cuda.current_stream())
        return r

    # -- whole layer ----------------------------------------------------------
    def weights(self, base) -> Experts:
        return experts(self.fmt, self.E, self.H, self.I, base, self.stride)

    def forward_decode(self, logits: torch.Tensor, x: torch.Tensor, W: Experts,
                       slot_of_expert=None, y_shared=None, stream=None) -> torch.Tensor:
        """Whole layer in two launches (decode-sized batches)."""
        T = logits.shape[0]
        self.kept = None
        moe_forward_decode(W, slot_of_expert, logits, x, self.k, self.ids, self.w, self.counts,
                           self.offsets, self.sorted_idx, self.inv_idx, y_shared, self.y,
                           self.decode_ws, self.renorm, stream)
        return self.y[:T]

    def forward(self, logits: torch.Tensor, x: torch.Tensor, W: Experts, Ws: Experts | None = None,
                slot_of_expert=None, variant="auto", stream=None) -> torch.Tensor:
        T = logits.shape[0]
        assert T <= self.T_max and x.shape == (T, self.H)
        if self.decode_ws is not None and Ws is None and variant == "auto":
            return self.forward_decode(logits, x, W, slot_of_expert, None, stream)
        self.route_permute(logits, stream)
        self.expert_ffn(W, x, T, slot_of_expert, variant, stream)
        if Ws is not None:
            self.shared_ffn(Ws, x, T, variant, stream)
        self.combine(T, Ws is not None, stream)
        return self.y[:T]

    def forward_cached(self, logits: torch.Tensor, x: torch.Tensor, layer: int, cache,
                       pool_W: Experts, slot_table: torch.Tensor, side=None, variant="auto",
                       stream=None) -> tuple[torch.Tensor, dict]:
        """Slot-table path: misses are filled from the pinned bank before the FFN."""
        T = logits.shape[0]
        self.route_permute(logits, stream)
        counts_host = self.counts[:self.E].to("cpu")          # the one host sync of the step
        me, ms, n_miss, n_hit, _ = cache.expert_cache_lookup(layer, counts_host)
        cache.expert_cache_fill(layer, me, ms, side=side, compute=stream)
        row = slot_table[layer * self.E:(layer + 1) * self.E]
        self.expert_ffn(pool_W, x, T, row, variant, stream)
        self.combine(T, False, stream)
        return self.y[:T], {"misses": n_miss, "hits": n_hit, "fills": list(zip(me.tolist(), ms.tolist()))}

    def forward_streamed(self, logits: torch.Tensor, x: torch.Tensor, layer: int, cache,
                         pool_W: Experts, slot_table: torch.Tensor, side=None, groups: int = 4,
                         variant="auto", stream=None) -> tuple[torch.Tensor, dict]:
        """Slot-table path with the FFN behind the fills (moe_expert_ffn_streamed): waves of
        at most S (or S/2 when the step needs more than S experts), each wave's misses in
        `groups` copy groups on `side`, the FFN over the hits at once and over each group as
        it lands.  y is bit-identical to forward_cached whenever that one fits.  There is no
        streamed FFN with E4M3 activations: variant "fp8" is refused."""
        if variant == "fp8":
            raise ValueError('forward_streamed: variant "fp8" is not available; use forward_cached')
        T = logits.shape[0]
        E = self.E
        cs = stream if stream is not None else torch.cuda.current_stream()
        if self.stream_ws is None:
            with _on(cs):
                self.stream_ws = torch.empty(
                    max(moe_expert_ffn_streamed_workspace(self._probe, self.T_max, self.k), 256),
                    dtype=torch.uint8, device=self.device)
        self.route_permute(logits, cs)
        with torch.cuda.stream(cs):
            self.counts_host.copy_(self.counts[:E], non_blocking=True)
        cs.synchronize()                                 # the one host sync of the step
        nw, nh = cache.moe_expert_ffn_streamed(layer, pool_W, x, T, self.k, self.counts_host,
                                               self.offsets, self.sorted_idx, self.y_perm,
                                               groups, self.stream_ws, side=side, compute=cs,
                                               out=self.plan_out)
        fe, fs, we = self.plan_out
        n_fill = int(we[nw - 1]) if nw else 0
        fills = list(zip(fe[:n_fill].tolist(), fs[:n_fill].tolist()))
        self.combine(T, False, cs)
        return self.y[:T], {"misses": n_fill, "hits": nh, "waves": nw, "fills": fills}

    def forward_hybrid(self, logits: torch.Tensor, x: torch.Tensor, layer: int, cache, pool_W: Experts,
                       slot_table: torch.Tensor, cpu_pool, fetch_fraction: float,
                       max_fetch: int = -1, side=None, groups: int = 4,
                       stream=None) -> tuple[torch.Tensor, dict]:
        """Hybrid step (moe_expert_ffn_hybrid): ceil(fetch_fraction * misses) of the misses
        (the most recently active) are fetched and computed on the GPU behind their copies,
        the others computed on the CPU from the bank while the GPU runs; then combine."""
        T = logits.shape[0]
        E = self.E
        cs = stream if stream is not None else torch.cuda.current_stream()
        if self.stream_ws is None:
            with _on(cs):
                self.stream_ws = torch.empty(
                    max(moe_expert_ffn_streamed_workspace(self._probe, self.T_max, self.k), 256),
                    dtype=torch.uint8, device=self.device)
        if self.host_stage is None:
            self.host_stage = torch.empty(
                moe_expert_ffn_hybrid_host_bytes(self._probe, self.T_max, self.k),
                dtype=torch.uint8).pin_memory()
        self.route_permute(logits, cs)
        with torch.cuda.stream(cs):
            self.counts_host.copy_(self.counts[:E], non_blocking=True)
        cs.synchronize()                                 # the one host sync of the step
        nc, nw, nh = cache.moe_expert_ffn_hybrid(layer, pool_W, cpu_pool, x, T, self.k,
                                                 self.counts_host, self.offsets, self.sorted_idx,
                                                 self.y_perm, fetch_fraction, max_fetch, groups,
                                                 self.stream_ws, self.host_stage, side=side,
                                                 compute=cs, out=self.hybrid_out)
        ce, fe, fs, we = self.hybrid_out
        n_fill = int(we[nw - 1]) if nw else 0
        fills = list(zip(fe[:n_fill].tolist(), fs[:n_fill].tolist()))
        self.combine(T, False, cs)
        return self.y[:T], {"misses": n_fill + nc, "fetched": n_fill, "cpu": ce[:nc].tolist(),
                            "hits": nh, "waves": nw, "fills": fills}
