"""MI355X (gfx950) fused random-Hadamard transform + 4-bit block quantization.

Thin Python layer over the C ABI of ``libufp4.so`` (include/ufp4.h): the
functions below marshal torch device tensors into pointers and call the
entry point of the same name.  PyTorch only provides device memory and
streams; every step of the quantization runs in the library's HIP kernels.
"""
from __future__ import annotations

import ctypes

import numpy as np
import torch

from ._lib import (GEMM_BWD_DW, GEMM_BWD_DX, GEMM_FWD_Y, OPERAND_A, OPERAND_B, RECIPE_NVFP4, RECIPE_UFP4,
                   RECIPE_UFP4_INT4, TENSOR_DY, TENSOR_W, TENSOR_X,
                   GRID_E1M2, GRID_E2M1, GRID_E2M1C, GRID_INT4, LIB_PATH, ROUND_RTNE, ROUND_STOCHASTIC,
                   ACT_GELU_TANH, ACT_SILU, CKPT_E4M3, CKPT_INT8, TYPE_BF16, TYPE_F32,
                   SCALE_MX32, SCALE_NV16, SCHEDULE_AUTO, SCHEDULE_SINGLE_PASS, SCHEDULE_TWO_PASS, Ufp4Error, check, lib, ufp4_config, ufp4_qtensor,
                   ufp4_stats_t)

__all__ = ["GRID_E1M2", "GRID_INT4", "GRID_E2M1", "GRID_E2M1C", "ROUND_RTNE", "ROUND_STOCHASTIC", "SCALE_NV16",
           "SCALE_MX32", "SCHEDULE_AUTO", "SCHEDULE_TWO_PASS", "SCHEDULE_SINGLE_PASS", "ufp4_set_schedule",
           "ufp4_schedule_of", "ufp4_amax_tiles", "ufp4_quantize_grouped_delayed", "ufp4_quantize_rowcol_noalloc", "ufp4_quantize_delayed", "ufp4_gemm_nt", "LIB_PATH", "Ufp4Error", "config", "QTensor", "Workspace", "alloc_layout",
           "ufp4_quantize", "ufp4_quantize_rowcol", "ufp4_quantize_grouped", "ufp4_dequantize",
           "ufp4_stats", "ufp4_round_f32", "ufp4_rht_signs", "ufp4_grouped_col_offsets", "ufp4_time_rowcol", "ufp4_roof_rowcol",
           "block_len", "ufp4_recipe_config", "RECIPE_UFP4", "RECIPE_UFP4_INT4", "RECIPE_NVFP4",
           "GEMM_FWD_Y", "GEMM_BWD_DX", "GEMM_BWD_DW", "OPERAND_A", "OPERAND_B", "TENSOR_X", "TENSOR_W",
           "TENSOR_DY", "ufp4_f32_to_bf16", "TYPE_BF16", "TYPE_F32", "CKPT_INT8", "CKPT_E4M3", "ACT_SILU",
           "ACT_GELU_TANH", "Checkpoint", "alloc_checkpoint", "ufp4_expert_rows", "ufp4_expert_sort",
           "ufp4_expert_dispatch", "ufp4_expert_dispatch_checkpoint", "ufp4_expert_combine",
           "ufp4_expert_combine_backward", "ufp4_checkpoint_save", "ufp4_checkpoint_load", "ufp4_gated_act",
           "ufp4_gated_act_backward", "ufp4_gemm_grouped_nt", "ufp4_gemm_grouped_dw"]


def config(grid: int = GRID_E1M2, rounding: int = ROUND_RTNE, scaling: int = SCALE_NV16,
           rht: int = 1, rht_seed: int = 0, sr_seed: int = 0) -> ufp4_config:
    return ufp4_config(int(grid), int(rounding), int(scaling), int(rht), int(rht_seed), int(sr_seed))


def block_len(scaling: int) -> int:
    return 32 if scaling == SCALE_MX32 else 16


# Addresses and stream handles go to ctypes as plain numbers, and the current
# stream is read as a handle: building a stream object and two wrapper objects
# took 3 us of a small call's 9.
def _ptr(t: torch.Tensor | None) -> int:
    return t.data_ptr() if t is not None else 0


def _stream(stream) -> int:
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _bf16_view(x: torch.Tensor):
    if x.dtype not in (torch.bfloat16, torch.int16, torch.uint16):
        raise TypeError("x must hold bf16 values (bfloat16, or their 16-bit patterns)")
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be a 2-D tensor with unit column stride")
    return x.shape[0], x.shape[1], x.stride(0)


class QTensor:
    """Device buffers of one quantized layout: packed codes, block scales and
    per-tensor scale(s)."""

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, tensor_scale: torch.Tensor):
        self.codes, self.scales, self.tensor_scale = codes, scales, tensor_scale

    def c(self) -> ufp4_qtensor:
        return ufp4_qtensor(self.codes.data_ptr(), self.scales.data_ptr(), self.tensor_scale.data_ptr())


def alloc_layout(lines: int, length: int, scaling: int, n_tensor_scales: int = 1,
                 device="cuda") -> QTensor:
    """Output buffers for `lines` block lines of `length` elements each."""
    B = block_len(scaling)
    return QTensor(torch.empty((lines, length // 2), dtype=torch.uint8, device=device),
                   torch.empty((lines, length // B), dtype=torch.uint8, device=device),
                   torch.empty(n_tensor_scales, dtype=torch.float32, device=device))


class Workspace:
    """Caller-owned device workspace (zeroed once by ufp4_workspace_init)."""

    def __init__(self, rows: int, cols: int, num_groups: int = 1, device="cuda", stream=None):
        self.nbytes = int(lib.ufp4_workspace_size(rows, cols, num_groups))
        if self.nbytes == 0:
            raise ValueError("invalid workspace shape")
        self.buf = torch.empty(self.nbytes, dtype=torch.uint8, device=device)
        check("ufp4_workspace_init", lib.ufp4_workspace_init(_ptr(self.buf), self.nbytes, _stream(stream)))

    @property
    def ptr(self):
        return _ptr(self.buf)

    def status(self, stream=None) -> int:
        st = ctypes.c_int(0)
        check("ufp4_workspace_status", lib.ufp4_workspace_status(self.ptr, self.nbytes, ctypes.byref(st),
                                                                   _stream(stream)))
        return st.value


def ufp4_quantize(x: torch.Tensor, cfg: ufp4_config, row_out: QTensor, ws: Workspace | None,
                  stream=None) -> None:
    rows, cols, ld = _bf16_view(x)
    check("ufp4_quantize", lib.ufp4_quantize(_ptr(x), rows, cols, ld, ctypes.byref(cfg), row_out.c(),
                                             ws.ptr if ws else None, ws.nbytes if ws else 0,
                                             _stream(stream)))


def ufp4_quantize_rowcol(x: torch.Tensor, cfg: ufp4_config, row_out: QTensor, col_out: QTensor,
                         ws: Workspace | None, stream=None) -> None:
    rows, cols, ld = _bf16_view(x)
    check("ufp4_quantize_rowcol",
          lib.ufp4_quantize_rowcol(_ptr(x), rows, cols, ld, ctypes.byref(cfg), row_out.c(), col_out.c(),
                                   ws.ptr if ws else None, ws.nbytes if ws else 0, _stream(stream)))


def ufp4_quantize_rowcol_noalloc(x: torch.Tensor, cfg: ufp4_config, row_out: QTensor, col_out: QTensor,
                                 stream=None) -> None:
    rows, cols, ld = _bf16_view(x)
    check("ufp4_quantize_rowcol_noalloc",
          lib.ufp4_quantize_rowcol_noalloc(_ptr(x), rows, cols, ld, ctypes.byref(cfg), row_out.c(), col_out.c(),
                                           _stream(stream)))


def ufp4_quantize_grouped(x: torch.Tensor, offsets_dev: torch.Tensor, padded_rows: int,
                          cfg: ufp4_config, row_out: QTensor | None, col_out: QTensor | None,
                          ws: Workspace | None, stream=None) -> None:
    rows, cols, ld = _bf16_view(x)
    if ld != cols:
        raise ValueError("grouped input must be contiguous")
    if offsets_dev.dtype != torch.int64:
        raise TypeError("offsets must be int64")
    E = offsets_dev.numel() - 1
    null = ufp4_qtensor(None, None, None)
    check("ufp4_quantize_grouped",
          lib.ufp4_quantize_grouped(_ptr(x), rows, cols, _ptr(offsets_dev), E, int(padded_rows),
                                    ctypes.byref(cfg), row_out.c() if row_out else null,
                                    col_out.c() if col_out else null, ws.ptr if ws else None,
                                    ws.nbytes if ws else 0, _stream(stream)))



def ufp4_quantize_grouped_delayed(x: torch.Tensor, offsets_dev: torch.Tensor, padded_rows: int,
                                  cfg: ufp4_config, amax_in: torch.Tensor, amax_out: torch.Tensor | None,
                                  row_out: QTensor | None, col_out: QTensor | None, ws: Workspace,
                                  stream=None) -> None:
    """amax_in / amax_out: float32 device tensors of num_groups (row, column) pairs."""
    rows, cols, ld = _bf16_view(x)
    if ld != cols:
        raise ValueError("grouped input must be contiguous")
    if offsets_dev.dtype != torch.int64 or amax_in.dtype != torch.float32:
        raise TypeError("offsets must be int64 and maxima float32")
    E = offsets_dev.numel() - 1
    if amax_in.numel() != 2 * E or (amax_out is not None and amax_out.numel() != 2 * E):
        raise ValueError("one (row, column) pair of maxima per segment")
    null = ufp4_qtensor(None, None, None)
    check("ufp4_quantize_grouped_delayed",
          lib.ufp4_quantize_grouped_delayed(_ptr(x), rows, cols, _ptr(offsets_dev), E, int(padded_rows),
                                            ctypes.byref(cfg), _ptr(amax_in), _ptr(amax_out),
                                            row_out.c() if row_out else null, col_out.c() if col_out else null,
                                            ws.ptr, ws.nbytes, _stream(stream)))

def ufp4_set_schedule(schedule: int, left_stride: int = 0) -> None:
    """Process-wide schedule of dense NV16 calls (SCHEDULE_AUTO, _TWO_PASS,
    _SINGLE_PASS); left_stride > 1 makes the single pass leave every tile whose
    index is not a multiple of it to the other workgroups (test hook)."""
    check("ufp4_set_schedule", lib.ufp4_set_schedule(int(schedule), int(left_stride)))


def ufp4_gemm_nt(cfg: ufp4_config, a: QTensor, b: QTensor, M: int, N: int, K: int, c: torch.Tensor,
                 stream=None) -> None:
    """c[m][n] = sum_k deq(a)[m][k] deq(b)[n][k] for NV16 row-wise layouts of
    an M x K and an N x K matrix; c float32 [M][ldc >= N] on the device."""
    assert c.dtype == torch.float32 and c.dim() == 2 and c.stride(1) == 1
    check("ufp4_gemm_nt", lib.ufp4_gemm_nt(ctypes.byref(cfg), int(M), int(N), int(K), a.c(), b.c(), _ptr(c),
                                           c.stride(0), _stream(stream)))


def ufp4_amax_tiles(rows: int, cols: int) -> int:
    """Pairs of tile maxima a delayed call on rows x cols writes."""
    return int(lib.ufp4_amax_tiles(int(rows), int(cols)))


def ufp4_quantize_delayed(x: torch.Tensor, cfg: ufp4_config, amax_in: torch.Tensor, amax_out,
                          row_out: QTensor, col_out: QTensor | None = None, stream=None) -> None:
    """Delayed scaling: tensor scales from amax_in (float32 [n, 2] on the
    device: row-wise, column-wise maxima); this call's tile maxima go to
    amax_out (float32 [ufp4_amax_tiles(rows, cols), 2], or None)."""
    rows, cols, ld = _bf16_view(x)
    assert amax_in.dtype == torch.float32 and amax_in.is_contiguous() and amax_in.numel() % 2 == 0
    if amax_out is not None:
        assert amax_out.dtype == torch.float32 and amax_out.is_contiguous()
        assert amax_out.numel() >= 2 * ufp4_amax_tiles(rows, cols)
    col = col_out.c() if col_out is not None else ufp4_qtensor(None, None, None)
    check("ufp4_quantize_delayed",
          lib.ufp4_quantize_delayed(_ptr(x), rows, cols, ld, ctypes.byref(cfg), _ptr(amax_in),
                                    amax_in.numel() // 2, _ptr(amax_out) if amax_out is not None else None,
                                    row_out.c(), col, _stream(stream)))


def ufp4_schedule_of(rows: int, cols: int, cfg: ufp4_config, num_groups: int = 1,
                     both_layouts: bool = True) -> int:
    """SCHEDULE_SINGLE_PASS or SCHEDULE_TWO_PASS: what a call on this shape
    and configuration (both layouts, or one) takes on the current device."""
    out = ctypes.c_int32(0)
    check("ufp4_schedule_of", lib.ufp4_schedule_of(int(rows), int(cols), int(num_groups), int(bool(both_layouts)),
                                                   ctypes.byref(cfg), ctypes.byref(out)))
    return out.value


def ufp4_time_rowcol(x: torch.Tensor, cfg: ufp4_config, row_out: QTensor, col_out: QTensor,
                     ws: Workspace, stream=None) -> tuple[float, float]:
    """One ufp4_quantize_rowcol call with hipEvents around each of its
    kernels; returns (ms of the tensor-maximum kernel, ms of the quantization
    kernel); under the single-pass schedule (0, ms of the one kernel).
    Synchronizes."""
    rows, cols, ld = _bf16_view(x)
    a, b = ctypes.c_float(0), ctypes.c_float(0)
    check("ufp4_time_rowcol", lib.ufp4_time_rowcol(_ptr(x), rows, cols, ld, ctypes.byref(cfg), row_out.c(),
                                                   col_out.c(), ws.ptr, ws.nbytes, _stream(stream),
                                                   ctypes.byref(a), ctypes.byref(b)))
    return a.value, b.value


def ufp4_roof_rowcol(x: torch.Tensor, row_out: QTensor, col_out: QTensor, stream=None) -> None:
    """The memory traffic of a row+col call on x with no arithmetic (a
    bandwidth reference): the quantization kernels' loads, and every byte of
    both layouts' codes and block scales written (as zeros, unless a lane's
    input words xor to one fixed constant).  rows % 128 == 0, cols % 256 == 0."""
    rows, cols, ld = _bf16_view(x)
    if ld != cols:
        raise ValueError("the roof hook takes a contiguous tensor")
    check("ufp4_roof_rowcol", lib.ufp4_roof_rowcol(_ptr(x), rows, cols, row_out.c(), col_out.c(), _stream(stream)))


def ufp4_dequantize(q: QTensor, rows: int, cols: int, cfg: ufp4_config, inverse_rht: bool,
                    out: torch.Tensor, stream=None) -> None:
    check("ufp4_dequantize",
          lib.ufp4_dequantize(_ptr(q.codes), _ptr(q.scales), _ptr(q.tensor_scale), rows, cols,
                              ctypes.byref(cfg), int(bool(inverse_rht)), _ptr(out), _stream(stream)))


def ufp4_stats(x: torch.Tensor, layout: int, cfg: ufp4_config, q: QTensor, ws: Workspace,
               stream=None) -> dict:
    rows, cols, ld = _bf16_view(x)
    out = ufp4_stats_t()
    check("ufp4_stats", lib.ufp4_stats(_ptr(x), rows, cols, ld, int(layout), ctypes.byref(cfg),
                                       _ptr(q.codes), _ptr(q.scales), _ptr(q.tensor_scale), ws.ptr,
                                       ws.nbytes, ctypes.byref(out), _stream(stream)))
    return out.as_dict()


def ufp4_round_f32(y: torch.Tensor, grid: int, rounding: int, sr_seed: int, codes: torch.Tensor,
                   stream=None) -> None:
    if y.dtype != torch.float32 or codes.dtype != torch.uint8 or codes.numel() != y.numel():
        raise TypeError("y must be float32 and codes uint8 of the same size")
    check("ufp4_round_f32", lib.ufp4_round_f32(_ptr(y), y.numel(), int(grid), int(rounding),
                                               int(sr_seed), _ptr(codes), _stream(stream)))


def ufp4_rht_signs(rht_seed: int) -> np.ndarray:
    s = np.zeros(16, dtype=np.int8)
    check("ufp4_rht_signs", lib.ufp4_rht_signs(int(rht_seed), s.ctypes.data_as(ctypes.c_void_p)))
    return s


def ufp4_grouped_col_offsets(offsets, block: int) -> np.ndarray:
    off = np.ascontiguousarray(offsets, dtype=np.int64)
    out = np.zeros(off.size, dtype=np.int64)
    check("ufp4_grouped_col_offsets",
          lib.ufp4_grouped_col_offsets(off.ctypes.data_as(ctypes.c_void_p), off.size - 1, int(block),
                                       out.ctypes.data_as(ctypes.c_void_p)))
    return out


def ufp4_recipe_config(recipe: int, gemm: int, operand: int, rht_seed: int = 0, sr_seed: int = 0):
    """(config, layout, tensor) of one operand of one training GEMM under a
    recipe: layout 0 row-wise / 1 column-wise, tensor TENSOR_X/W/DY."""
    cfg = ufp4_config()
    layout, tensor = ctypes.c_int32(), ctypes.c_int32()
    check("ufp4_recipe_config", lib.ufp4_recipe_config(int(recipe), int(gemm), int(operand), int(rht_seed),
                                                       int(sr_seed), ctypes.byref(cfg), ctypes.byref(layout),
                                                       ctypes.byref(tensor)))
    return cfg, layout.value, tensor.value


def ufp4_f32_to_bf16(x: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """bf16 (as int16 bit patterns) of a contiguous float32 device tensor,
    rounded to nearest even by the library's kernel."""
    if x.dtype != torch.float32 or not x.is_contiguous():
        raise TypeError("x must be a contiguous float32 tensor")
    if out is None:
        out = torch.empty(x.shape, dtype=torch.int16, device=x.device)
    check("ufp4_f32_to_bf16", lib.ufp4_f32_to_bf16(_ptr(x), x.numel(), _ptr(out), _stream(stream)))
    return out


# ---------------------------------------------------------------- expert layer

def _int32(t: torch.Tensor, name: str) -> torch.Tensor:
    if t.dtype != torch.int32 or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous int32 tensor")
    return t


def _int64(t: torch.Tensor, name: str) -> torch.Tensor:
    if t.dtype != torch.int64 or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous int64 tensor")
    return t


_TYPES = {torch.float32: TYPE_F32, torch.bfloat16: TYPE_BF16, torch.int16: TYPE_BF16, torch.uint16: TYPE_BF16}


def _rows(t: torch.Tensor, name: str):
    """(type, rows, cols, leading dimension) of a 2-D bf16 or float32 tensor
    with unit column stride."""
    kind = _TYPES.get(t.dtype)
    if kind is None:
        raise TypeError(f"{name} must hold bf16 or float32 values")
    if t.dim() != 2:
        raise ValueError(f"{name} must be a 2-D tensor with unit column stride")
    rows, cols = t.shape
    ld, step = t.stride()
    if step != 1 and rows and cols > 1:
        raise ValueError(f"{name} must be a 2-D tensor with unit column stride")
    return kind, rows, cols, (ld if rows > 1 else max(cols, 1))


def _bf16_rows(t: torch.Tensor, name: str):
    kind, rows, cols, ld = _rows(t, name)
    if kind != TYPE_BF16:
        raise TypeError(f"{name} must hold bf16 values")
    return rows, cols, ld


def _weights(w: torch.Tensor | None, shape) -> torch.Tensor | None:
    if w is not None and (w.dtype != torch.float32 or not w.is_contiguous() or tuple(w.shape) != tuple(shape)):
        raise TypeError("weights must be a contiguous float32 tensor of one weight a slot")
    return w


def ufp4_expert_rows(tokens: int, slots: int, num_experts: int, align: int = 1) -> int:
    """Rows that hold any routing of tokens x slots with segments padded to
    multiples of `align`."""
    n = int(lib.ufp4_expert_rows(int(tokens), int(slots), int(num_experts), int(align)))
    if n == 0 and tokens != 0:
        raise ValueError("invalid routing shape")
    return n


def ufp4_expert_sort(ids: torch.Tensor, num_experts: int, align: int, offsets: torch.Tensor,
                     row_of_slot: torch.Tensor, slot_of_row: torch.Tensor, stream=None) -> None:
    """ids int32 [tokens, slots] (unit column stride); writes offsets int64
    [num_experts + 2], row_of_slot int32 [tokens, slots] and slot_of_row int32
    [rows], rows >= ufp4_expert_rows(tokens, slots, num_experts, align)."""
    if ids.dtype != torch.int32 or ids.dim() != 2 or (ids.shape[0] and ids.shape[1] > 1 and ids.stride(1) != 1):
        raise TypeError("ids must be a 2-D int32 tensor with unit column stride")
    tokens, slots = ids.shape
    if tuple(row_of_slot.shape) != (tokens, slots) or offsets.numel() != num_experts + 2:
        raise ValueError("row_of_slot must have the shape of ids, offsets num_experts + 2 entries")
    check("ufp4_expert_sort",
          lib.ufp4_expert_sort(_ptr(ids), tokens, slots, ids.stride(0) if tokens > 1 else slots, int(num_experts),
                               int(align), slot_of_row.numel(), _ptr(_int64(offsets, "offsets")),
                               _ptr(_int32(row_of_slot, "row_of_slot")), _ptr(_int32(slot_of_row, "slot_of_row")),
                               _stream(stream)))


def ufp4_expert_dispatch(x: torch.Tensor, row_of_slot: torch.Tensor, slot_of_row: torch.Tensor, out: torch.Tensor,
                         stream=None) -> None:
    """out[r] = x[token of row r], zeros for padding rows."""
    tokens, cols, ld = _bf16_rows(x, "x")
    rows, ocols, ldo = _bf16_rows(out, "out")
    if row_of_slot.shape[0] != tokens or ocols != cols or slot_of_row.numel() != rows:
        raise ValueError("x, row_of_slot, slot_of_row and out disagree in their sizes")
    check("ufp4_expert_dispatch",
          lib.ufp4_expert_dispatch(_ptr(x), tokens, cols, ld, row_of_slot.shape[1],
                                   _ptr(_int32(row_of_slot, "row_of_slot")), _ptr(_int32(slot_of_row, "slot_of_row")),
                                   rows, _ptr(out), ldo, _stream(stream)))


def ufp4_expert_combine(z: torch.Tensor, row_of_slot: torch.Tensor, weights: torch.Tensor | None, out: torch.Tensor,
                        stream=None) -> None:
    """out[t] = sum over slots of weights[t, j] z[row_of_slot[t, j]] (weights
    None: all 1, the gradient of ufp4_expert_dispatch)."""
    zt, rows, cols, ldz = _rows(z, "z")
    ot, tokens, ocols, ldo = _rows(out, "out")
    if ocols != cols or row_of_slot.shape[0] != tokens:
        raise ValueError("z, row_of_slot and out disagree in their sizes")
    w = _weights(weights, row_of_slot.shape)
    check("ufp4_expert_combine",
          lib.ufp4_expert_combine(_ptr(z), zt, rows, cols, ldz, _ptr(_int32(row_of_slot, "row_of_slot")), _ptr(w),
                                  tokens, row_of_slot.shape[1], _ptr(out), ot, ldo, _stream(stream)))


def ufp4_expert_combine_backward(dout: torch.Tensor, z: torch.Tensor | None, row_of_slot: torch.Tensor,
                                 slot_of_row: torch.Tensor, weights: torch.Tensor | None, dz: torch.Tensor | None,
                                 dweights: torch.Tensor | None, stream=None) -> None:
    """Gradients of ufp4_expert_combine; dz (and with it weights) or dweights
    (and with it z) may be None."""
    dt, tokens, cols, ldd = _rows(dout, "dout")
    rows, kind, ldz, lddz = slot_of_row.numel(), None, cols, cols
    if z is not None:
        kind, zr, zc, ldz = _rows(z, "z")
        if (zr, zc) != (rows, cols):
            raise ValueError("z must have one row of dout's width for each entry of slot_of_row")
    elif dweights is not None:
        raise ValueError("dweights needs z")
    if dz is not None:
        k2, zr, zc, lddz = _rows(dz, "dz")
        if (zr, zc) != (rows, cols) or kind not in (None, k2):
            raise ValueError("dz must have the shape and type of z")
        kind = k2
    if row_of_slot.shape[0] != tokens:
        raise ValueError("row_of_slot must have one line a token")
    w, dw = _weights(weights, row_of_slot.shape), _weights(dweights, row_of_slot.shape)
    check("ufp4_expert_combine_backward",
          lib.ufp4_expert_combine_backward(_ptr(dout), dt, tokens, cols, ldd, row_of_slot.shape[1], _ptr(z),
                                           TYPE_BF16 if kind is None else kind, rows, ldz,
                                           _ptr(_int32(row_of_slot, "row_of_slot")),
                                           _ptr(_int32(slot_of_row, "slot_of_row")), _ptr(w), _ptr(dz), lddz, _ptr(dw),
                                           _stream(stream)))


class Checkpoint:
    """Device buffers of a matrix (or of the two halves of a gated
    activation's input) kept in 8 bits: codes uint8 [rows, cols], scales bf16
    [rows, blocks]."""

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, format: int, halves: int = 1):
        rows, cols = codes.shape
        if codes.dtype != torch.uint8 or scales.dtype not in (torch.bfloat16, torch.int16, torch.uint16):
            raise TypeError("codes must be uint8 and scales bf16")
        if cols % halves or tuple(scales.shape) != (rows, halves * -(-(cols // halves) // 32)):
            raise ValueError("one scale for each block of 32 of each half's columns")
        if not codes.is_contiguous() or not scales.is_contiguous():
            raise ValueError("codes and scales must be contiguous")
        self.codes, self.scales, self.format, self.halves = codes, scales, int(format), int(halves)
        self.rows, self.width = rows, cols // halves


def alloc_checkpoint(rows: int, width: int, format: int, halves: int = 1, device="cuda") -> Checkpoint:
    """Buffers for a rows x width matrix (halves 1), or for the gate and up
    halves of a rows x 2 width one (halves 2)."""
    return Checkpoint(torch.empty((rows, halves * width), dtype=torch.uint8, device=device),
                      torch.empty((rows, halves * -(-width // 32)), dtype=torch.bfloat16, device=device), format, halves)


def _checkpoint(c: Checkpoint, rows: int, width: int, halves: int) -> Checkpoint:
    if (c.rows, c.width, c.halves) != (rows, width, halves):
        raise ValueError(f"the checkpoint holds {c.halves} x [{c.rows}, {c.width}], not {halves} x [{rows}, {width}]")
    return c


def ufp4_checkpoint_save(x: torch.Tensor, ckpt: Checkpoint, stream=None) -> None:
    rows, cols, ld = _bf16_rows(x, "x")
    _checkpoint(ckpt, rows, cols, 1)
    check("ufp4_checkpoint_save", lib.ufp4_checkpoint_save(_ptr(x), rows, cols, ld, ckpt.format, _ptr(ckpt.codes),
                                                           _ptr(ckpt.scales), _stream(stream)))


def ufp4_checkpoint_load(ckpt: Checkpoint, out: torch.Tensor, stream=None) -> None:
    kind, rows, cols, ldo = _rows(out, "out")
    _checkpoint(ckpt, rows, cols, 1)
    check("ufp4_checkpoint_load", lib.ufp4_checkpoint_load(_ptr(ckpt.codes), _ptr(ckpt.scales), rows, cols,
                                                           ckpt.format, _ptr(out), kind, ldo, _stream(stream)))


def ufp4_expert_dispatch_checkpoint(ckpt: Checkpoint, row_of_slot: torch.Tensor, slot_of_row: torch.Tensor,
                                    out: torch.Tensor, stream=None) -> None:
    """ufp4_expert_dispatch of the kept matrix."""
    rows, cols, ldo = _bf16_rows(out, "out")
    tokens = row_of_slot.shape[0]
    _checkpoint(ckpt, tokens, cols, 1)
    if slot_of_row.numel() != rows:
        raise ValueError("slot_of_row must have one entry for each row of out")
    check("ufp4_expert_dispatch_checkpoint",
          lib.ufp4_expert_dispatch_checkpoint(_ptr(ckpt.codes), _ptr(ckpt.scales), ckpt.format, tokens, cols,
                                              row_of_slot.shape[1], _ptr(_int32(row_of_slot, "row_of_slot")),
                                              _ptr(_int32(slot_of_row, "slot_of_row")), rows, _ptr(out), ldo,
                                              _stream(stream)))


def ufp4_gated_act(gu: torch.Tensor, act: int, h: torch.Tensor, ckpt: Checkpoint | None = None, stream=None) -> None:
    """h = f(gate) up for gu = [gate | up]; keeps gu in ckpt (two halves) for
    the backward pass if given."""
    rows, two, ld = _bf16_rows(gu, "gu")
    hr, width, ldh = _bf16_rows(h, "h")
    if (hr, 2 * width) != (rows, two):
        raise ValueError("gu must have the rows of h and twice its width")
    if ckpt is not None:
        _checkpoint(ckpt, rows, width, 2)
    check("ufp4_gated_act",
          lib.ufp4_gated_act(_ptr(gu), rows, width, ld, int(act), _ptr(h), ldh, ckpt.format if ckpt else 0,
                             _ptr(ckpt.codes if ckpt else None), _ptr(ckpt.scales if ckpt else None),
                             _stream(stream)))


def ufp4_gated_act_backward(dh: torch.Tensor, ckpt: Checkpoint, act: int, dgu: torch.Tensor,
                            h: torch.Tensor | None = None, stream=None) -> None:
    """dgu = gradient of ufp4_gated_act at the kept values; h, if given, gets
    the activation's output at them."""
    rows, width, lddh = _bf16_rows(dh, "dh")
    gr, two, lddg = _bf16_rows(dgu, "dgu")
    if (gr, two) != (rows, 2 * width):
        raise ValueError("dgu must have the rows of dh and twice its width")
    _checkpoint(ckpt, rows, width, 2)
    ldho = width
    if h is not None:
        hr, hw, ldho = _bf16_rows(h, "h")
        if (hr, hw) != (rows, width):
            raise ValueError("h must have the shape of dh")
    check("ufp4_gated_act_backward",
          lib.ufp4_gated_act_backward(_ptr(dh), lddh, _ptr(ckpt.codes), _ptr(ckpt.scales), ckpt.format, rows, width,
                                      int(act), _ptr(dgu), lddg, _ptr(h), ldho, _stream(stream)))


def _lines(q: QTensor, lines: int, length: int, segments: int, name: str) -> None:
    if (tuple(q.codes.shape) != (lines, length // 2) or tuple(q.scales.shape) != (lines, length // 16)
            or not q.codes.is_contiguous() or not q.scales.is_contiguous()):
        raise ValueError(f"{name} must hold {lines} contiguous lines of {length} codes and their NV16 scales")
    if q.codes.element_size() != 1 or q.scales.element_size() != 1:
        raise ValueError(f"{name} must have codes and block scales of one byte")
    if q.tensor_scale.dtype != torch.float32 or q.tensor_scale.numel() < segments or not q.tensor_scale.is_contiguous():
        raise ValueError(f"{name} must have one float32 tensor scale a segment, side by side in memory")


def ufp4_gemm_grouped_nt(cfg: ufp4_config, a: QTensor, b: QTensor, b_layout: int, offsets: torch.Tensor, K: int,
                         c: torch.Tensor, num_groups: int | None = None, stream=None) -> None:
    """c[r] = (row r of a) times segment e's matrix of b transposed, for the
    rows r of segment e.  a: row-wise layout of c's rows; b_layout 0: b is the
    row-wise layout of the stacked matrices, 1: their column-wise layout.
    num_groups defaults to offsets.numel() - 1 (ufp4_expert_sort's array has
    one more entry: pass its number of experts)."""
    kind, rows, N, ldc = _rows(c, "c")
    E = offsets.numel() - 1 if num_groups is None else int(num_groups)
    if offsets.numel() < E + 1:
        raise ValueError("offsets must have num_groups + 1 entries")
    _lines(a, rows, K, E, "a")
    _lines(b, *((E * N, K) if b_layout == 0 else (N, E * K)), E, "b")
    check("ufp4_gemm_grouped_nt",
          lib.ufp4_gemm_grouped_nt(ctypes.byref(cfg), rows, N, int(K), a.c(), b.c(), int(b_layout),
                                   _ptr(_int64(offsets, "offsets")), E, _ptr(c), kind, ldc, _stream(stream)))


def ufp4_gemm_grouped_dw(cfg: ufp4_config, a: QTensor, b: QTensor, offsets: torch.Tensor, c: torch.Tensor,
                         num_groups: int | None = None, stream=None) -> None:
    """c[e] = a_e b_e^T over segment e's columns of two column-wise grouped
    layouts; c [num_groups, M, N] float32 or bf16, contiguous."""
    E = offsets.numel() - 1 if num_groups is None else int(num_groups)
    if c.dim() != 3 or not c.is_contiguous() or c.shape[0] != E or offsets.numel() < E + 1:
        raise ValueError("c must be a contiguous [num_groups, M, N] tensor, offsets num_groups + 1 entries")
    kind = _rows(c.view(-1, c.shape[2]), "c")[0] if c.numel() else TYPE_F32
    M, N = c.shape[1], c.shape[2]
    P = 2 * a.codes.shape[1]
    _lines(a, M, P, E, "a")
    _lines(b, N, P, E, "b")
    check("ufp4_gemm_grouped_dw",
          lib.ufp4_gemm_grouped_dw(ctypes.byref(cfg), M, N, P, a.c(), b.c(), _ptr(_int64(offsets, "offsets")), E,
                                   _ptr(c), kind, _stream(stream)))
