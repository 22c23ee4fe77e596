"""The vocabulary head: losses and scores of rows against a whole table.

``z[n, v] = <hidden[n], weight[v]>`` over every row of ``weight``, which is any
dense table: an output projection, or the rows of a TT table themselves (a
``TTEmbeddingBag`` call with one bag per row, so that the loss trains its cores).

  tt_emb_xent_forward / _backward        softmax cross entropy, without an N x V
                                         array of logits
  tt_emb_distill_forward / _backward     the same against a teacher's top logits
  tt_emb_q4_quantize / tt_emb_q4_matvec  a 4-bit copy of a table for serving, and
                                         the scores of a few rows against it
  vocab_cross_entropy, vocab_distillation, Q4Table   the same for autograd and as
                                         an object

Low-level functions carry the C ABI's names (``include/tt_emb.h``, which also says what
each type's numbers keep); outputs and the workspace are torch allocations on the call's
stream, and so are copies of arguments whose rows are not contiguous.  Both gradients are
always formed, whichever are wanted.
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import Optional, Tuple

import torch

from . import TT_ERR_ARG, TT_ERR_SHAPE, TTError, _check, _stream, load_library

__all__ = [
    "tt_emb_head_workspace",
    "tt_emb_xent_forward",
    "tt_emb_xent_backward",
    "tt_emb_distill_forward",
    "tt_emb_distill_backward",
    "tt_emb_head_set_wait_limit",
    "tt_emb_q4_quantize",
    "tt_emb_q4_matvec",
    "vocab_cross_entropy",
    "vocab_distillation",
    "Q4Table",
]

TT_F32, TT_BF16, TT_F16 = 0, 1, 2
_DTYPES = {torch.float32: TT_F32, torch.bfloat16: TT_BF16, torch.float16: TT_F16}


class _Head(ctypes.Structure):
    _fields_ = [
        ("hidden_dev", ctypes.c_void_p),
        ("weight_dev", ctypes.c_void_p),
        ("rows", ctypes.c_int64),
        ("vocab", ctypes.c_int64),
        ("hidden_stride", ctypes.c_int64),
        ("weight_stride", ctypes.c_int64),
        ("dim", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
    ]


def _refuse(code: int, what: str):
    raise TTError(code, what)


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_calls = {}  # name -> bound C function (looked up once: the calls below are short)


def _c(name: str):
    fn = _calls.get(name)
    if fn is None:
        fn = _calls[name] = getattr(load_library(), name)
    return fn


def _stream_now(device_index: int):
    """The device's current stream as an address."""
    return _raw_stream(device_index) if _raw_stream is not None else _stream(None)


def _device(t: torch.Tensor, what: str) -> torch.device:
    """The device of a CUDA tensor of a supported type."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype not in _DTYPES:
        _refuse(TT_ERR_ARG, f"{what} must be a float32, bfloat16 or float16 CUDA tensor")
    return t.device


def _matrix(t: torch.Tensor, what: str) -> torch.Tensor:
    """A 2-D CUDA tensor of a supported type whose rows are contiguous (a copy where they are not)."""
    _device(t, what)
    if t.dim() != 2 or t.shape[1] < 1:
        _refuse(TT_ERR_SHAPE, f"{what} must be [rows, dim] with dim >= 1")
    if t.is_contiguous():
        return t
    if t.shape[0] > 1 and t.stride(0) < t.shape[1] or t.shape[1] > 1 and t.stride(1) != 1:
        return t.contiguous()
    return t


def _row_stride(t: torch.Tensor) -> int:
    rows, dim = t.shape
    return t.stride(0) if rows > 1 else dim


def _head(hidden: torch.Tensor, weight: torch.Tensor):
    h, w = _matrix(hidden, "hidden"), _matrix(weight, "weight")
    if h.dtype != w.dtype or h.device != w.device:
        _refuse(TT_ERR_ARG, "hidden and weight must have one type and one device")
    (rows, dim), (vocab, wdim) = h.shape, w.shape
    if dim != wdim or vocab < 1:
        _refuse(TT_ERR_SHAPE, "hidden is [rows, dim] and weight [vocab, dim]")
    return h, w, _Head(h.data_ptr(), w.data_ptr(), rows, vocab, _row_stride(h), _row_stride(w), dim, _DTYPES[h.dtype])


def _vector(t: torch.Tensor, dtype, shape, device, what: str) -> torch.Tensor:
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.device != device:
        _refuse(TT_ERR_ARG, f"{what} must be a {dtype} tensor on {device}")
    if t.shape != shape:
        _refuse(TT_ERR_SHAPE, f"{what} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t if t.is_contiguous() else t.contiguous()


def _err_word(err: Optional[torch.Tensor], device):
    if err is None:
        return None
    if not (isinstance(err, torch.Tensor) and err.device == device and err.dtype == torch.int32 and err.numel() >= 1):
        _refuse(TT_ERR_ARG, "err must be an int32 tensor on the inputs' device")
    return err.data_ptr()


@contextlib.contextmanager
def _current(stream, device):
    with torch.cuda.device(device):
        if stream is None:
            yield
        else:
            s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream), device=device)
            with torch.cuda.stream(s):
                yield


_here = contextlib.nullcontext()
_device_now = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)  # of tensors that are there: CUDA is up


def _on(stream, device):
    """The call's stream and device are current: what it allocates belongs to that stream, and what it copies of its
    arguments is copied there, before its kernels and with memory that no other stream takes meanwhile."""
    return _here if stream is None and device.index == _device_now() else _current(stream, device)


def tt_emb_head_workspace(hidden: torch.Tensor, weight: torch.Tensor, teacher_k: int = 1, backward: bool = False) -> int:
    """Bytes of workspace that a forward or backward call on these tensors takes."""
    with _on(None, _device(hidden, "hidden")):
        h, w, d = _head(hidden, weight)
        return _workspace_bytes(d, teacher_k, backward)


def _workspace_bytes(d: _Head, k: int, backward: bool) -> int:
    n = _c("tt_emb_head_workspace")(ctypes.byref(d), k, backward)
    if n < 0:
        _refuse(TT_ERR_SHAPE, "tt_emb_head_workspace: sizes outside the limits")
    return n


def _forward(name, hidden, weight, target, err, stream):
    device = _device(hidden, "hidden")
    with _on(stream, device):
        h, w, d = _head(hidden, weight)
        rows = d.rows
        k, args, keep = target(rows, device)
        n = _workspace_bytes(d, k, False)
        loss = torch.empty(rows, dtype=torch.float32, device=device)
        lse = torch.empty(rows, dtype=torch.float32, device=device)
        ws = torch.empty(n, dtype=torch.uint8, device=device)
        st = _c(name)(ctypes.byref(d), *args, loss.data_ptr(), lse.data_ptr(), _err_word(err, device), ws.data_ptr(), n,
                      _stream_now(device.index))
        if st:
            _check(st, name)
    return loss, lse


def _backward(name, hidden, weight, target, lse, grad_loss, err, stream):
    device = _device(hidden, "hidden")
    with _on(stream, device):
        h, w, d = _head(hidden, weight)
        rows = d.rows
        k, args, keep = target(rows, device)
        lse = _vector(lse, torch.float32, (rows,), device, "lse")
        grad_loss = _vector(grad_loss, torch.float32, (rows,), device, "grad_loss")
        n = _workspace_bytes(d, k, True)
        gh = torch.empty(h.shape, dtype=h.dtype, device=device)
        gw = torch.empty(w.shape, dtype=h.dtype, device=device)
        ws = torch.empty(n, dtype=torch.uint8, device=device)
        st = _c(name)(ctypes.byref(d), *args, lse.data_ptr(), grad_loss.data_ptr(), gh.data_ptr(), gw.data_ptr(), _err_word(err, device),
                      ws.data_ptr(), n, _stream_now(device.index))
        if st:
            _check(st, name)
    return gh, gw


def _ids(targets, ignore_index):
    def target(rows, device):
        t = _vector(targets, torch.int64, (rows,), device, "targets")
        return 1, (t.data_ptr(), ignore_index), t
    return target


def tt_emb_xent_forward(hidden: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor, ignore_index: int = -100,
                        err: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(loss, lse), float32 [rows], of softmax cross entropy over the whole table.

    hidden [rows, dim] and weight [vocab, dim] of one type (float32, bfloat16,
    float16), targets int64 [rows].  A row whose target is ignore_index has loss 0.  A
    target outside the table sets bit 1 of err (int32, optional) and counts as ignored."""
    return _forward("tt_emb_xent_forward", hidden, weight, _ids(targets, ignore_index), err, stream)


def tt_emb_xent_backward(hidden: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor, lse: torch.Tensor, grad_loss: torch.Tensor,
                         ignore_index: int = -100, err: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(grad_hidden, grad_weight) for lse of the forward call and the gradient of every row's loss."""
    return _backward("tt_emb_xent_backward", hidden, weight, _ids(targets, ignore_index), lse, grad_loss, err, stream)


def _teacher(teacher_ids, teacher_logits, temperature):
    def target(rows, device):
        if not isinstance(teacher_ids, torch.Tensor) or teacher_ids.dim() != 2 or teacher_ids.shape[1] < 1:
            _refuse(TT_ERR_SHAPE, "teacher_ids must be [rows, k] with k >= 1")
        k = teacher_ids.shape[1]
        ids = _vector(teacher_ids, torch.int64, (rows, k), device, "teacher_ids")
        logits = teacher_logits
        if isinstance(logits, torch.Tensor) and logits.dtype in (torch.bfloat16, torch.float16):
            logits = logits.float()
        logits = _vector(logits, torch.float32, (rows, k), device, "teacher_logits")
        return k, (ids.data_ptr(), logits.data_ptr(), k, temperature), (ids, logits)
    return target


def tt_emb_distill_forward(hidden: torch.Tensor, weight: torch.Tensor, teacher_ids: torch.Tensor, teacher_logits: torch.Tensor,
                           temperature: float = 1.0, err: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(loss, lse), float32 [rows]: T^2 KL(teacher's renormalised top entries || student) and log sum_v exp(z / T).

    teacher_ids int64 [rows, k] (negative: no entry), teacher_logits [rows, k]."""
    return _forward("tt_emb_distill_forward", hidden, weight, _teacher(teacher_ids, teacher_logits, temperature), err, stream)


def tt_emb_distill_backward(hidden: torch.Tensor, weight: torch.Tensor, teacher_ids: torch.Tensor, teacher_logits: torch.Tensor,
                            lse: torch.Tensor, grad_loss: torch.Tensor, temperature: float = 1.0, err: Optional[torch.Tensor] = None,
                            stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(grad_hidden, grad_weight); the teacher gets no gradient."""
    return _backward("tt_emb_distill_backward", hidden, weight, _teacher(teacher_ids, teacher_logits, temperature), lse, grad_loss, err,
                     stream)


def tt_emb_head_set_wait_limit(ns: int):
    """Bound of each device wait of the head's kernels in nanoseconds (default 2e9; 0 exercises the give-up path)."""
    _check(load_library().tt_emb_head_set_wait_limit(int(ns)), "tt_emb_head_set_wait_limit")


# ---------------------------------------------------------------- 4-bit tables


def tt_emb_q4_quantize(weight: torch.Tensor, group: int = 64, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(packed uint8 [vocab, ceil(dim / 32) * 16], scales bfloat16 [vocab, ceil(dim / group)]) of a dense table."""
    with _on(stream, _device(weight, "weight")):
        w = _matrix(weight, "weight")
        V, D, group = w.shape[0], w.shape[1], int(group)
        if V < 1 or group not in (32, 64, 128):
            _refuse(TT_ERR_SHAPE, "weight must have rows and group must be 32, 64 or 128")
        packed = torch.empty((V, (D + 31) // 32 * 16), dtype=torch.uint8, device=w.device)
        scales = torch.empty((V, (D + group - 1) // group), dtype=torch.bfloat16, device=w.device)
        _check(_c("tt_emb_q4_quantize")(w.data_ptr(), _row_stride(w), V, D, _DTYPES[w.dtype], group, packed.data_ptr(), scales.data_ptr(),
                                        _stream_now(w.device.index)), "tt_emb_q4_quantize")
    return packed, scales


def tt_emb_q4_matvec(x: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor, group: int, out: Optional[torch.Tensor] = None,
                     stream=None) -> torch.Tensor:
    """Scores float32 [rows, vocab] of the rows of x [rows, dim] (float32, bfloat16, float16) against a 4-bit table."""
    device = _device(x, "x")
    with _on(stream, device):
        x = _matrix(x, "x")
        M, D = x.shape
        if group not in (32, 64, 128):
            _refuse(TT_ERR_SHAPE, "group must be 32, 64 or 128")
        V = packed.shape[0] if isinstance(packed, torch.Tensor) and packed.dim() == 2 else 0
        if V < 1:
            _refuse(TT_ERR_SHAPE, "packed must be [vocab, bytes] with vocab >= 1")
        packed = _vector(packed, torch.uint8, (V, (D + 31) // 32 * 16), device, "packed")
        scales = _vector(scales, torch.bfloat16, (V, (D + group - 1) // group), device, "scales")
        if out is None:
            out = torch.empty((M, V), dtype=torch.float32, device=device)
        elif out.shape != (M, V) or out.dtype != torch.float32 or out.device != device or not out.is_contiguous():
            _refuse(TT_ERR_ARG, "out must be a contiguous float32 [rows, vocab] tensor on x's device")
        st = _c("tt_emb_q4_matvec")(x.data_ptr(), _row_stride(x), M, _DTYPES[x.dtype], packed.data_ptr(), scales.data_ptr(), V, D, group,
                                    out.data_ptr(), _stream_now(device.index))
        if st:
            _check(st, "tt_emb_q4_matvec")
    return out


# ---------------------------------------------------------------- autograd and objects


class _XentFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, hidden, weight, targets, ignore_index, err):
        loss, lse = tt_emb_xent_forward(hidden, weight, targets, ignore_index, err)
        ctx.save_for_backward(hidden, weight, targets, lse)
        ctx.ignore_index, ctx.err = ignore_index, err
        return loss

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad):
        hidden, weight, targets, lse = ctx.saved_tensors
        gh, gw = tt_emb_xent_backward(hidden, weight, targets, lse, grad, ctx.ignore_index, ctx.err)
        return gh, gw, None, None, None


class _DistillFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, hidden, weight, ids, logits, temperature, err):
        loss, lse = tt_emb_distill_forward(hidden, weight, ids, logits, temperature, err)
        ctx.save_for_backward(hidden, weight, ids, logits, lse)
        ctx.temperature, ctx.err = temperature, err
        return loss

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad):
        hidden, weight, ids, logits, lse = ctx.saved_tensors
        gh, gw = tt_emb_distill_backward(hidden, weight, ids, logits, lse, grad, ctx.temperature, ctx.err)
        return gh, gw, None, None, None, None


def _reduce(loss, counts, reduction):
    if reduction == "none":
        return loss
    total = loss.sum()
    return total if reduction == "sum" else total / counts.sum().clamp(min=1)


def _same_rows(a, b):
    """Shapes of the same rows in the same order: equal, or one of the two flattened (or the one row's, without a batch)."""
    return a == b or (min(len(a), len(b)) <= 1 and a.numel() == b.numel())


def _check_reduction(reduction):
    if reduction not in ("none", "sum", "mean"):
        raise ValueError("reduction must be 'none', 'sum' or 'mean'")


def vocab_cross_entropy(hidden: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor, ignore_index: int = -100,
                        reduction: str = "mean", err: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Softmax cross entropy of hidden [..., dim] against every row of weight [vocab, dim], differentiable in both.

    reduction 'mean' divides by the rows that count: a target in the table that is not ignore_index (0 when there are
    none).  err (int32, optional): what the forward pass finds is ORed into it, and later what the backward pass does;
    without it nothing tells of a target outside the table (a row that does not count) or of a device wait that gave up
    (results undefined)."""
    _check_reduction(reduction)
    if not _same_rows(hidden.shape[:-1], targets.shape):
        _refuse(TT_ERR_SHAPE, f"targets have shape {tuple(targets.shape)}, expected {tuple(hidden.shape[:-1])}")
    t = targets.reshape(-1)
    loss = _XentFunction.apply(hidden.reshape(-1, hidden.shape[-1]), weight, t, int(ignore_index), err)
    if reduction == "none":
        return loss.reshape(targets.shape)
    vocab = weight.shape[0]
    counts = t == t.clamp(0, vocab - 1)
    return _reduce(loss, counts & (t != ignore_index) if 0 <= ignore_index < vocab else counts, reduction)


def vocab_distillation(hidden: torch.Tensor, weight: torch.Tensor, teacher_ids: torch.Tensor, teacher_logits: torch.Tensor,
                       temperature: float = 1.0, reduction: str = "mean", err: Optional[torch.Tensor] = None) -> torch.Tensor:
    """T^2 KL(teacher's top entries || student) of hidden [..., dim] against weight [vocab, dim], differentiable in both.

    teacher_ids / teacher_logits [..., k]; negative ids are no entries.  reduction 'mean'
    divides by the rows that have an entry (0 when there are none).  err: as in vocab_cross_entropy."""
    _check_reduction(reduction)
    if teacher_ids.dim() < 1 or not _same_rows(hidden.shape[:-1], teacher_ids.shape[:-1]) or teacher_logits.shape != teacher_ids.shape:
        _refuse(TT_ERR_SHAPE, f"teacher_ids and teacher_logits have shapes {tuple(teacher_ids.shape)} and {tuple(teacher_logits.shape)}, "
                              f"expected {tuple(hidden.shape[:-1])} + [k]")
    k = teacher_ids.shape[-1]
    ids = teacher_ids.reshape(-1, k)
    loss = _DistillFunction.apply(hidden.reshape(-1, hidden.shape[-1]), weight, ids, teacher_logits.reshape(-1, k), float(temperature), err)
    if reduction == "none":
        return loss.reshape(teacher_ids.shape[:-1])
    have = ((ids >= 0) & (ids < weight.shape[0]) & (teacher_logits.reshape(-1, k) > -float("inf"))).any(1)
    return _reduce(loss, have, reduction)


class Q4Table:
    """A 4-bit copy of a dense table for serving: ``Q4Table(weight).scores(x)``, float32 [..., vocab]."""

    def __init__(self, weight: torch.Tensor, group: int = 64):
        self.vocab, self.dim, self.group = weight.shape[0], weight.shape[1], int(group)
        self.packed, self.scales = tt_emb_q4_quantize(weight.detach(), group)

    def scores(self, x: torch.Tensor) -> torch.Tensor:
        if x.dim() < 1 or x.shape[-1] != self.dim:
            _refuse(TT_ERR_SHAPE, f"x has shape {tuple(x.shape)}, expected [..., {self.dim}]")
        return tt_emb_q4_matvec(x.reshape(-1, x.shape[-1]), self.packed, self.scales, self.group).reshape(*x.shape[:-1], self.vocab)
