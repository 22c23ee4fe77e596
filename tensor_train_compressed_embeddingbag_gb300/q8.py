"""Scores against a table held in 8-bit integers: a scale for each row of x and each row of the table.

  tt_emb_q8_quantize / tt_emb_q8_scores   an 8-bit copy of a table, and the scores of rows against it
  Q8Table                                 the same as an object

Beside the 4-bit table (head.py) it is the more exact copy, and the one for many rows: prompts,
batches and evaluation as well as single tokens.  Low-level functions carry the C ABI's names
(``include/tt_emb.h``).
"""
from __future__ import annotations

from typing import Optional, Tuple

import torch

from . import TT_ERR_ARG, TT_ERR_SHAPE, _check
from .head import _DTYPES, _c, _device, _err_word, _matrix, _on, _refuse, _row_stride, _stream_now, _vector

__all__ = ["tt_emb_q8_workspace", "tt_emb_q8_quantize", "tt_emb_q8_scores", "Q8Table"]


def tt_emb_q8_workspace(rows: int, dim: int) -> int:
    """Bytes of workspace that the scores of so many rows take."""
    n = _c("tt_emb_q8_workspace")(int(rows), int(dim))
    if n < 0:
        _refuse(TT_ERR_SHAPE, "tt_emb_q8_workspace: sizes outside the limits")
    return n


def tt_emb_q8_quantize(weight: torch.Tensor, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(codes int8 [rows, ceil(dim / 16) * 16], scales float32 [rows]) of the rows of a matrix."""
    with _on(stream, _device(weight, "weight")):
        w = _matrix(weight, "weight")
        rows, dim = w.shape
        codes = torch.empty((rows, (dim + 15) // 16 * 16), dtype=torch.int8, device=w.device)
        scales = torch.empty(rows, dtype=torch.float32, device=w.device)
        _check(_c("tt_emb_q8_quantize")(w.data_ptr(), _row_stride(w), rows, dim, _DTYPES[w.dtype], codes.data_ptr(), scales.data_ptr(),
                                        _stream_now(w.device.index)), "tt_emb_q8_quantize")
    return codes, scales


def tt_emb_q8_scores(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, out: Optional[torch.Tensor] = None,
                     err: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Scores float32 [rows, vocab] of the rows of x [rows, dim] (float32, bfloat16, float16) against an 8-bit table.

    The rows of x are quantized as tt_emb_q8_quantize does; the integer sums are exact.  A device wait
    that gave up sets 4 in err (int32, optional)."""
    device = _device(x, "x")
    with _on(stream, device):
        x = _matrix(x, "x")
        rows, dim = x.shape
        vocab = codes.shape[0] if isinstance(codes, torch.Tensor) and codes.dim() == 2 else 0
        if vocab < 1:
            _refuse(TT_ERR_SHAPE, "codes must be [vocab, bytes] with vocab >= 1")
        codes = _vector(codes, torch.int8, (vocab, (dim + 15) // 16 * 16), device, "codes")
        scales = _vector(scales, torch.float32, (vocab,), device, "scales")
        if out is None:
            out = torch.empty((rows, vocab), dtype=torch.float32, device=device)
        elif not isinstance(out, torch.Tensor) or out.shape != (rows, vocab) or out.dtype != torch.float32 or out.device != device or not out.is_contiguous():
            _refuse(TT_ERR_ARG, "out must be a contiguous float32 [rows, vocab] tensor on x's device")
        n = tt_emb_q8_workspace(rows, dim)
        ws = torch.empty(n, dtype=torch.uint8, device=device)
        st = _c("tt_emb_q8_scores")(x.data_ptr(), _row_stride(x), rows, _DTYPES[x.dtype], codes.data_ptr(), scales.data_ptr(), vocab, dim, out.data_ptr(),
                                    _err_word(err, device), ws.data_ptr(), n, _stream_now(device.index))
        if st:
            _check(st, "tt_emb_q8_scores")
    return out


class Q8Table:
    """An 8-bit copy of a dense table: ``Q8Table(weight).scores(x)``, float32 [..., vocab]."""

    def __init__(self, weight: torch.Tensor):
        self.codes, self.scales = tt_emb_q8_quantize(weight.detach() if isinstance(weight, torch.Tensor) else weight)
        self.vocab, self.dim = weight.shape

    def scores(self, x: torch.Tensor, err: Optional[torch.Tensor] = None) -> torch.Tensor:
        if not isinstance(x, torch.Tensor):
            _refuse(TT_ERR_ARG, "x must be a tensor")
        if x.dim() < 1 or x.shape[-1] != self.dim:
            _refuse(TT_ERR_SHAPE, f"x has shape {tuple(x.shape)}, expected [..., {self.dim}]")
        return tt_emb_q8_scores(x.reshape(-1, x.shape[-1]), self.codes, self.scales, err=err).reshape(*x.shape[:-1], self.vocab)
