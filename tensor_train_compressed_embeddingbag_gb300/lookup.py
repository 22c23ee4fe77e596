"""Rows of a dense table by id, times a scale, and the table's gradient by sorted ids.

The table is the kind that the vocabulary head scores: tied, it is both ends of a language
model, and its two gradients add up in one array.

  tt_emb_lookup_forward / _backward   out[n] = scale weight[ids[n]], and the table's gradient
  vocab_embedding                     the same for autograd

Low-level functions carry the C ABI's names (``include/tt_emb.h``).
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import TT_ERR_ARG, TT_ERR_SHAPE, _check
from .head import _DTYPES, _c, _device, _err_word, _matrix, _on, _refuse, _row_stride, _stream_now

__all__ = ["tt_emb_lookup_workspace", "tt_emb_lookup_forward", "tt_emb_lookup_backward", "vocab_embedding"]


class _Lookup(ctypes.Structure):
    _fields_ = [
        ("weight_dev", ctypes.c_void_p),
        ("weight_stride", ctypes.c_int64),
        ("ids_dev", ctypes.c_void_p),
        ("rows", ctypes.c_int64),
        ("vocab", ctypes.c_int64),
        ("padding_idx", ctypes.c_int64),
        ("dim", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("scale", ctypes.c_float),
    ]


def _ids(ids, device) -> torch.Tensor:
    if not isinstance(ids, torch.Tensor) or ids.dtype != torch.int64 or ids.device != device:
        _refuse(TT_ERR_ARG, f"ids must be an int64 tensor on {device}")
    if ids.dim() != 1:
        _refuse(TT_ERR_SHAPE, "ids must be [rows]")
    return ids if ids.is_contiguous() else ids.contiguous()


def tt_emb_lookup_workspace(rows: int, vocab: int, dim: int, dtype: torch.dtype) -> int:
    """Bytes of workspace that a backward call of these sizes takes."""
    n = _c("tt_emb_lookup_workspace")(int(rows), int(vocab), int(dim), _DTYPES.get(dtype, -1))
    if n < 0:
        _refuse(TT_ERR_SHAPE, "tt_emb_lookup_workspace: sizes outside the limits")
    return n


def tt_emb_lookup_forward(weight: torch.Tensor, ids: torch.Tensor, scale: float = 1.0, err: Optional[torch.Tensor] = None,
                          stream=None) -> torch.Tensor:
    """scale * weight[ids], [rows, dim] of weight's type (float32, bfloat16, float16); ids int64 [rows].

    An id outside the table gives a row of zeros and sets bit 1 of err (int32, optional)."""
    device = _device(weight, "weight")
    with _on(stream, device):
        w = _matrix(weight, "weight")
        ids = _ids(ids, device)
        (vocab, dim), rows = w.shape, ids.shape[0]
        out = torch.empty((rows, dim), dtype=w.dtype, device=device)
        a = _Lookup(w.data_ptr(), _row_stride(w), ids.data_ptr(), rows, vocab, -1, dim, _DTYPES[w.dtype], scale)
        st = _c("tt_emb_lookup_forward")(ctypes.byref(a), out.data_ptr(), dim, _err_word(err, device), _stream_now(device.index))
        if st:
            _check(st, "tt_emb_lookup_forward")
    return out


def tt_emb_lookup_backward(grad_out: torch.Tensor, ids: torch.Tensor, vocab: int, scale: float = 1.0, padding_idx: int = -1,
                           grad_weight: Optional[torch.Tensor] = None, err: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The gradient [vocab, dim] of a table, of grad_out's type: scale times the sums of the rows of grad_out by id.

    Rows with padding_idx give none (below 0: every id counts).  With grad_weight (rows of contiguous elements) the sums are added to
    the rows of it that ids name, the others stay as they are: a tied table's other gradient, or the table itself for
    a step of gradient descent (scale times minus the learning rate)."""
    device = _device(grad_out, "grad_out")
    with _on(stream, device):
        g = _matrix(grad_out, "grad_out")
        ids = _ids(ids, device)
        vocab, (rows, dim) = int(vocab), g.shape
        if ids.shape[0] != rows:
            _refuse(TT_ERR_SHAPE, f"grad_out has {rows} rows, ids {ids.shape[0]}")
        n = tt_emb_lookup_workspace(rows, vocab, dim, g.dtype)
        out = grad_weight
        if out is None:
            out = torch.empty((vocab, dim), dtype=g.dtype, device=device)
        elif not isinstance(out, torch.Tensor) or out.dtype != g.dtype or out.device != device:
            _refuse(TT_ERR_ARG, "grad_weight must have grad_out's type and device")
        elif out.shape != (vocab, dim) or (dim > 1 and out.stride(1) != 1) or (vocab > 1 and out.stride(0) < dim):
            _refuse(TT_ERR_SHAPE, f"grad_weight must be [{vocab}, {dim}] with contiguous rows that do not overlap")
        ws = torch.empty(n, dtype=torch.uint8, device=device) if n else None
        a = _Lookup(None, dim, ids.data_ptr(), rows, vocab, int(padding_idx), dim, _DTYPES[g.dtype], scale)
        st = _c("tt_emb_lookup_backward")(ctypes.byref(a), g.data_ptr(), _row_stride(g), out.data_ptr(), _row_stride(out),
                                          int(grad_weight is not None), _err_word(err, device), ws.data_ptr() if n else None, n, _stream_now(device.index))
        if st:
            _check(st, "tt_emb_lookup_backward")
    return out


class _LookupFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, weight, ids, scale, padding_idx, err):
        out = tt_emb_lookup_forward(weight, ids, scale, err)
        ctx.save_for_backward(ids)
        ctx.vocab, ctx.scale, ctx.padding_idx, ctx.err = weight.shape[0], scale, padding_idx, err
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad):
        ids, = ctx.saved_tensors
        return tt_emb_lookup_backward(grad, ids, ctx.vocab, ctx.scale, ctx.padding_idx, err=ctx.err), None, None, None, None


def vocab_embedding(ids: torch.Tensor, weight: torch.Tensor, scale: float = 1.0, padding_idx: Optional[int] = None,
                    err: Optional[torch.Tensor] = None) -> torch.Tensor:
    """scale * weight[ids], [..., dim] for ids int64 [...], differentiable in weight [vocab, dim].

    padding_idx: an id that gives no gradient (looked up as any other), counted from the table's end if below 0; None: none.
    err (int32, optional): what the forward pass finds is ORed into it, and later what the backward pass does."""
    if not isinstance(ids, torch.Tensor):
        _refuse(TT_ERR_ARG, "ids must be an int64 tensor")
    pad = -1 if padding_idx is None else int(padding_idx)
    if padding_idx is not None and pad < 0:
        _device(weight, "weight")
        if weight.dim() != 2 or pad < -weight.shape[0]:
            _refuse(TT_ERR_SHAPE, "padding_idx must not be below -vocab, of weight [vocab, dim]")
        pad += weight.shape[0]
    out = _LookupFunction.apply(weight, ids.reshape(-1), float(scale), pad, err)
    return out.reshape(*ids.shape, weight.shape[1])
