"""A mixture-of-experts layer on the library's kernels, forward and backward.

Y[t] = sum over the experts e a token t chose of w[t, e] W_out[e] h,
h = f(g) u with (g, u) = W_in[e] X[t]; routing (expert ids and weights) comes
from the caller.  The rows go to their experts (ufp4_expert_sort,
ufp4_expert_dispatch), every product runs on operands quantized by a training
recipe (ufp4_quantize_grouped, ufp4_gemm_grouped_nt / _dw; "Shrinkage Bias: The
Hidden Geometric Trap in FP4 Training" (zhichai.net), "Key points": the fix on
all three products of a linear layer, mixture-of-experts models), and the rows
come back weighted (ufp4_expert_combine).  No count of rows returns to the
host: segments are padded to the quantizer's block and the padding behind the
last one is a segment of its own.

What a forward pass keeps for the backward one: the tokens' input and the
gated activation's input in 8 bits, the experts' output in bf16 (the gradient
of the routing weights), and the sort.  The weight gradients' operands are
made again from the 8-bit values.

Streams.  load(), forward() and backward() run on `stream`, or on the current
stream if it is None.  A `stream` waits for what the current stream has been given
so far, so tensors made there can be passed at once, and may be dropped
after the call.  Memory that a call allocates, what it returns included, belongs
to the stream that it ran on: another stream that uses it waits for that one
first, like for any tensor.
"""
from __future__ import annotations

from contextlib import contextmanager

import torch

from . import (ACT_SILU, CKPT_INT8, GEMM_BWD_DW, GEMM_BWD_DX, GEMM_FWD_Y, OPERAND_A, OPERAND_B, RECIPE_UFP4, SCALE_NV16,
               QTensor, Workspace, alloc_checkpoint, alloc_layout, ufp4_checkpoint_save, ufp4_expert_combine,
               ufp4_expert_combine_backward, ufp4_expert_dispatch, ufp4_expert_dispatch_checkpoint, ufp4_expert_rows,
               ufp4_expert_sort, ufp4_gated_act, ufp4_gated_act_backward, ufp4_gemm_grouped_dw, ufp4_gemm_grouped_nt,
               ufp4_quantize_grouped, ufp4_recipe_config)

_BLOCK = 16


def _record(stream, *objects) -> None:
    """Keeps the memory of tensors, and of objects that hold some, from being
    used again before `stream` is through with it."""
    for o in objects:
        for t in (o,) if isinstance(o, torch.Tensor) else vars(o).values():
            if isinstance(t, torch.Tensor):
                t.record_stream(stream)


class ExpertLayer:
    """w_in: bf16 [experts, 2 hidden, width] (gate rows, then up rows); w_out:
    bf16 [experts, width, hidden]; width and hidden multiples of 32.  rht_seed
    is shared by all operands; sr_seed, below 2^63, keys the stochastic rounding
    of the output gradients (give each step and layer another one)."""

    def __init__(self, w_in: torch.Tensor, w_out: torch.Tensor, act: int = ACT_SILU, recipe: int = RECIPE_UFP4,
                 ckpt_format: int = CKPT_INT8, rht_seed: int = 0):
        self.experts, two, self.width = w_in.shape
        self.hidden = two // 2
        if two % 2 or tuple(w_out.shape) != (self.experts, self.width, self.hidden):
            raise ValueError("w_in must be [experts, 2 hidden, width] and w_out [experts, width, hidden]")
        if self.width % 32 or self.hidden % 32:
            raise ValueError("width and hidden must be multiples of 32")
        self.act, self.recipe, self.ckpt_format, self.rht_seed = act, recipe, ckpt_format, rht_seed
        self.device = w_in.device
        self.load(w_in, w_out)

    def load(self, w_in: torch.Tensor, w_out: torch.Tensor, stream=None) -> None:
        """Quantize (new) weights in both of the layouts the products read."""
        with self._on(stream, w_in, w_out) as run:
            self._w = {name: self._weights(w.contiguous()) for name, w in (("in", w_in), ("out", w_out))}
            self._loaded_on = run.cuda_stream

    @contextmanager
    def _on(self, stream, *inputs):
        """Runs the body, its allocations and torch operations among it, on
        `stream`; gives the stream that it is."""
        caller = torch.cuda.current_stream(self.device)
        if stream is None or stream.cuda_stream == caller.cuda_stream:
            yield caller
            return
        stream.wait_stream(caller)
        _record(stream, *inputs)
        with torch.cuda.stream(stream):
            yield stream

    def _cfg(self, gemm: int, operand: int, sr_seed: int = 0):
        return ufp4_recipe_config(self.recipe, gemm, operand, self.rht_seed, sr_seed)[0]

    def _weights(self, w: torch.Tensor):
        lines = w.shape[1]
        offsets = torch.arange(self.experts + 1, dtype=torch.int64, device=self.device) * lines
        flat = w.view(self.experts * lines, w.shape[2])
        ws = Workspace(flat.shape[0], flat.shape[1], self.experts, device=self.device)
        return (self._quantize(flat, offsets, self._cfg(GEMM_FWD_Y, OPERAND_B), True, ws),
                self._quantize(flat, offsets, self._cfg(GEMM_BWD_DX, OPERAND_B), False, ws))

    def _quantize(self, x: torch.Tensor, offsets: torch.Tensor, cfg, rowwise: bool, ws: Workspace) -> QTensor:
        rows, cols = x.shape
        lines, length = (rows, cols) if rowwise else (cols, rows)
        q = alloc_layout(lines, length, SCALE_NV16, offsets.numel() - 1, device=x.device)
        ufp4_quantize_grouped(x, offsets, rows, cfg, q if rowwise else None, None if rowwise else q, ws)
        return q

    def _nt(self, q: QTensor, b: QTensor, layout: int, offsets, K: int, N: int, gemm: int) -> torch.Tensor:
        c = torch.empty((q.codes.shape[0], N), dtype=torch.bfloat16, device=self.device)
        ufp4_gemm_grouped_nt(self._cfg(gemm, OPERAND_A), q, b, layout, offsets, K, c, self.experts)
        return c

    def forward(self, x: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, train: bool = True, stream=None):
        """x bf16 [tokens, width], ids int32 and weights float32 [tokens,
        slots] (an id outside the experts is a dropped slot).  Returns y bf16
        [tokens, width] and what backward() takes (None if not train)."""
        with self._on(stream, x, ids, weights) as run:
            self._use_weights(run)
            return self._forward(x, ids, weights, train, run)

    def backward(self, saved, dy: torch.Tensor, sr_seed: int = 0, stream=None):
        """Gradients (dx bf16, dw_in and dw_out float32 like the weights,
        dweights float32) for dy bf16 [tokens, width]."""
        *kept, home = saved
        with self._on(stream, dy) as run:
            if run.cuda_stream != home:
                _record(run, *kept)
            self._use_weights(run)
            return self._backward(kept, dy, sr_seed)

    def _use_weights(self, run) -> None:
        if run.cuda_stream != self._loaded_on:  # (load() drops them for new ones)
            _record(run, *(q for pair in self._w.values() for q in pair))

    def _forward(self, x: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, train: bool, run):
        (tokens, slots), dev = ids.shape, self.device
        R, E, F = ufp4_expert_rows(tokens, slots, self.experts, _BLOCK), self.experts, self.hidden
        offsets = torch.empty(E + 2, dtype=torch.int64, device=dev)
        row_of_slot = torch.empty((tokens, slots), dtype=torch.int32, device=dev)
        slot_of_row = torch.empty(R, dtype=torch.int32, device=dev)
        ufp4_expert_sort(ids, E, _BLOCK, offsets, row_of_slot, slot_of_row)
        rows = torch.empty((R, self.width), dtype=torch.bfloat16, device=dev)
        ufp4_expert_dispatch(x, row_of_slot, slot_of_row, rows)
        ws = Workspace(R, max(self.width, 2 * F), E + 1, device=dev)
        cfg = self._cfg(GEMM_FWD_Y, OPERAND_A)
        gu = self._nt(self._quantize(rows, offsets, cfg, True, ws), self._w["in"][0], 0, offsets, self.width,
                      2 * F, GEMM_FWD_Y)
        kept_x = kept_gu = None
        if train:
            kept_x = alloc_checkpoint(tokens, self.width, self.ckpt_format, device=dev)
            ufp4_checkpoint_save(x, kept_x)
            kept_gu = alloc_checkpoint(R, F, self.ckpt_format, halves=2, device=dev)
        h = torch.empty((R, F), dtype=torch.bfloat16, device=dev)
        ufp4_gated_act(gu, self.act, h, kept_gu)
        z = self._nt(self._quantize(h, offsets, cfg, True, ws), self._w["out"][0], 0, offsets, F, self.width,
                     GEMM_FWD_Y)
        y = torch.empty((tokens, self.width), dtype=torch.bfloat16, device=dev)
        ufp4_expert_combine(z, row_of_slot, weights, y)
        if not train:
            return y, None
        return y, (offsets, row_of_slot, slot_of_row, weights, kept_x, kept_gu, z, ws, run.cuda_stream)

    def _backward(self, kept, dy: torch.Tensor, sr_seed: int):
        offsets, row_of_slot, slot_of_row, weights, kept_x, kept_gu, z, ws = kept
        E, F, W, dev, R = self.experts, self.hidden, self.width, self.device, slot_of_row.numel()
        tokens = row_of_slot.shape[0]
        dz, dweights = torch.empty_like(z), torch.empty_like(weights)
        ufp4_expert_combine_backward(dy, z, row_of_slot, slot_of_row, weights, dz, dweights)

        # dgu depends on the rounded dz, so it is rounded by other random numbers:
        # by the same ones its mean would not be its value
        key_dz, key_dgu = int(sr_seed), int(sr_seed) ^ (1 << 63)

        def quantize(t, gemm, operand, rowwise, key=0):
            return self._quantize(t, offsets, self._cfg(gemm, operand, key), rowwise, ws)

        def dw(dout, key, inp, M, N):
            c = torch.empty((E, M, N), dtype=torch.float32, device=dev)
            ufp4_gemm_grouped_dw(self._cfg(GEMM_BWD_DW, OPERAND_A), quantize(dout, GEMM_BWD_DW, OPERAND_A, False, key),
                                 quantize(inp, GEMM_BWD_DW, OPERAND_B, False), offsets, c, E)
            return c

        dh = self._nt(quantize(dz, GEMM_BWD_DX, OPERAND_A, True, key_dz), self._w["out"][1], 1, offsets, W, F, GEMM_BWD_DX)
        dgu = torch.empty((R, 2 * F), dtype=torch.bfloat16, device=dev)
        h = torch.empty((R, F), dtype=torch.bfloat16, device=dev)
        ufp4_gated_act_backward(dh, kept_gu, self.act, dgu, h)
        dw_out = dw(dz, key_dz, h, W, F)
        rows = torch.empty((R, W), dtype=torch.bfloat16, device=dev)
        ufp4_expert_dispatch_checkpoint(kept_x, row_of_slot, slot_of_row, rows)
        dw_in = dw(dgu, key_dgu, rows, 2 * F, W)
        drows = self._nt(quantize(dgu, GEMM_BWD_DX, OPERAND_A, True, key_dgu), self._w["in"][1], 1, offsets, 2 * F, W,
                         GEMM_BWD_DX)
        dx = torch.empty((tokens, W), dtype=torch.bfloat16, device=dev)
        ufp4_expert_combine(drows, row_of_slot, None, dx)
        return dx, dw_in, dw_out, dweights
