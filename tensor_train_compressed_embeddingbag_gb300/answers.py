"""Losses of answers from the log probabilities of their tokens: preference and policy.

An answer is a sequence of sampled tokens; their log probabilities under a vocabulary head
are minus its cross entropy (``-vocab_cross_entropy(..., reduction="none")``), so the
losses here train what is below the head without an array of logits.

  tt_emb_preference_forward / _backward   chosen against rejected answers, pair by pair
  tt_emb_policy_forward / _backward       clipped policy loss with a Kullback-Leibler term
  preference_loss, policy_loss            the same for autograd

Low-level functions carry the C ABI's names (``include/tt_emb.h``, which has the formulas).
Log probabilities are float32: [sequences, length] (a padded batch), or [tokens] with int64
``offsets`` [sequences + 1] (packed, as the bags of a table are).  ``mask`` (bool or uint8, of
the same shape) says which tokens count: an answer's own, not its prompt's or padding.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple, Union

import torch

from . import TT_ERR_ARG, TT_ERR_SHAPE, _check
from .head import _c, _check_reduction, _err_word, _on, _reduce, _refuse, _stream_now, _vector

__all__ = [
    "tt_emb_answers_workspace",
    "tt_emb_preference_forward",
    "tt_emb_preference_backward",
    "tt_emb_policy_forward",
    "tt_emb_policy_backward",
    "preference_loss",
    "policy_loss",
]

_KINDS = {"sigmoid": 0, "hinge": 1, "squared": 2}
_LEVELS = {"token": 0, "sequence": 1}
_KLS = {"k1": 1, "k2": 2, "k3": 3}


class _Answers(ctypes.Structure):
    _fields_ = [
        ("logp_dev", ctypes.c_void_p),
        ("reference_dev", ctypes.c_void_p),
        ("mask_dev", ctypes.c_void_p),
        ("offsets_dev", ctypes.c_void_p),
        ("tokens", ctypes.c_int64),
        ("sequences", ctypes.c_int64),
        ("average", ctypes.c_int32),
    ]


class _Preference(ctypes.Structure):
    _fields_ = [
        ("kind", ctypes.c_int32),
        ("beta", ctypes.c_double),
        ("label_smoothing", ctypes.c_double),
        ("margin", ctypes.c_double),
    ]


class _Policy(ctypes.Structure):
    _fields_ = [
        ("old_dev", ctypes.c_void_p),
        ("advantages_dev", ctypes.c_void_p),
        ("per_token", ctypes.c_int32),
        ("level", ctypes.c_int32),
        ("kl", ctypes.c_int32),
        ("clip_low", ctypes.c_double),
        ("clip_high", ctypes.c_double),
        ("dual_clip", ctypes.c_double),
        ("kl_weight", ctypes.c_double),
    ]


def tt_emb_answers_workspace(tokens: int, sequences: int) -> int:
    """Bytes of workspace that a forward call on so many tokens and sequences takes."""
    n = _c("tt_emb_answers_workspace")(tokens, sequences)
    if n < 0:
        _refuse(TT_ERR_SHAPE, "tt_emb_answers_workspace: sizes outside the limits")
    return n


def _device(logp) -> torch.device:
    if not isinstance(logp, torch.Tensor) or not logp.is_cuda or logp.dtype != torch.float32:
        _refuse(TT_ERR_ARG, "logp must be a float32 CUDA tensor")
    return logp.device


def _sequences(logp, offsets) -> int:
    if offsets is None:
        if logp.dim() != 2:
            _refuse(TT_ERR_SHAPE, "logp must be [sequences, length], or [tokens] with offsets")
        return logp.shape[0]
    if logp.dim() != 1 or not isinstance(offsets, torch.Tensor) or offsets.dim() != 1 or offsets.shape[0] < 1:
        _refuse(TT_ERR_SHAPE, "with offsets [sequences + 1], logp must be [tokens]")
    return offsets.shape[0] - 1


def _mask(mask, shape, device):
    if not isinstance(mask, torch.Tensor) or mask.dtype not in (torch.bool, torch.uint8) or mask.device != device:
        _refuse(TT_ERR_ARG, f"mask must be a bool or uint8 tensor on {device}")
    if mask.shape != shape:
        _refuse(TT_ERR_SHAPE, f"mask has shape {tuple(mask.shape)}, expected {tuple(shape)}")
    return mask if mask.is_contiguous() else mask.contiguous()


def _answers(logp, reference, mask, offsets, average, read_logp=True):
    """(struct, sequences, what it points to)."""
    device, count = logp.device, _sequences(logp, offsets)
    x = _vector(logp, torch.float32, logp.shape, device, "logp") if read_logp else None
    r = None if reference is None else _vector(reference, torch.float32, logp.shape, device, "reference")
    m = None if mask is None else _mask(mask, logp.shape, device)
    o = None if offsets is None else _vector(offsets, torch.int64, (count + 1,), device, "offsets")
    keep = x, r, m, o
    return _Answers(*[None if t is None else t.data_ptr() for t in keep], logp.numel(), count, bool(average)), count, keep


def _preference(beta, kind, label_smoothing, margin):
    if kind not in _KINDS:
        _refuse(TT_ERR_ARG, f"kind must be one of {', '.join(_KINDS)}")
    if kind != "sigmoid" and 0.0 <= label_smoothing < 1.0:
        label_smoothing = 0.0  # the other losses have no labels; the C ABI takes only 0 for them
    return _Preference(_KINDS[kind], beta, label_smoothing, margin)


def _policy(old_logp, advantages, logp, count, clip, dual_clip, kl, kl_weight, level, per_token):
    if level not in _LEVELS or kl not in _KLS:
        _refuse(TT_ERR_ARG, f"level must be one of {', '.join(_LEVELS)} and kl one of {', '.join(_KLS)}")
    low, high = clip if isinstance(clip, (tuple, list)) else (clip, clip)
    old = _vector(old_logp, torch.float32, logp.shape, logp.device, "old_logp")
    if per_token is None:
        shape = advantages.shape if isinstance(advantages, torch.Tensor) else None
        per_token = shape == logp.shape
        if per_token and shape == (count,):
            _refuse(TT_ERR_ARG, "as many tokens as sequences: say by per_token which of the two the advantages belong to")
    adv = _vector(advantages, torch.float32, logp.shape if per_token else (count,), logp.device, "advantages")
    return _Policy(old.data_ptr(), adv.data_ptr(), per_token, _LEVELS[level], _KLS[kl], low, high, dual_clip or 0.0, kl_weight), (old, adv)


def tt_emb_preference_forward(logp: torch.Tensor, reference: Optional[torch.Tensor] = None, mask: Optional[torch.Tensor] = None,
                              offsets: Optional[torch.Tensor] = None, beta: float = 0.1, kind: str = "sigmoid", label_smoothing: float = 0.0,
                              margin: float = 0.0, average: bool = False, err: Optional[torch.Tensor] = None,
                              stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
    """(loss [pairs], margins [pairs], rewards [2 pairs], counts int32 [2 pairs]) of sequences 0 .. pairs - 1 chosen
    over sequences pairs .. 2 pairs - 1.

    kind: "sigmoid", "hinge" or "squared".  label_smoothing, in [0, 1), belongs to the sigmoid loss; the others do not use it.  average: rewards by the mean over an answer's tokens, not their
    sum.  Malformed offsets set 2 in err (int32, optional)."""
    device = _device(logp)
    with _on(stream, device):
        how = _preference(beta, kind, label_smoothing, margin)
        a, count, keep = _answers(logp, reference, mask, offsets, average)
        if count % 2:
            _refuse(TT_ERR_SHAPE, "the number of sequences must be even: the chosen ones, then the rejected ones")
        n = tt_emb_answers_workspace(a.tokens, count)
        ws = torch.empty(n, dtype=torch.uint8, device=device) if n else None
        loss, rewards = torch.empty(count // 2, dtype=torch.float32, device=device), torch.empty(count, dtype=torch.float32, device=device)
        margins, counts = torch.empty_like(loss), torch.empty(count, dtype=torch.int32, device=device)
        st = _c("tt_emb_preference_forward")(ctypes.byref(a), ctypes.byref(how), loss.data_ptr(), margins.data_ptr(), rewards.data_ptr(),
                                             counts.data_ptr(), _err_word(err, device), ws.data_ptr() if n else None, n, _stream_now(device.index))
        if st:
            _check(st, "tt_emb_preference_forward")
    return loss, margins, rewards, counts


def tt_emb_preference_backward(logp: torch.Tensor, margins: torch.Tensor, counts: torch.Tensor, grad_loss: torch.Tensor,
                               mask: Optional[torch.Tensor] = None, offsets: Optional[torch.Tensor] = None, beta: float = 0.1,
                               kind: str = "sigmoid", label_smoothing: float = 0.0, margin: float = 0.0, average: bool = False,
                               stream=None) -> torch.Tensor:
    """The gradient of every token's log probability for margins and counts of the forward call (logp gives the shape only)."""
    device = _device(logp)
    with _on(stream, device):
        how = _preference(beta, kind, label_smoothing, margin)
        a, count, keep = _answers(logp, None, mask, offsets, average, read_logp=False)
        margins = _vector(margins, torch.float32, (count // 2,), device, "margins")
        counts = _vector(counts, torch.int32, (count,), device, "counts")
        grad_loss = _vector(grad_loss, torch.float32, (count // 2,), device, "grad_loss")
        grad = torch.empty(logp.shape, dtype=torch.float32, device=device)
        st = _c("tt_emb_preference_backward")(ctypes.byref(a), ctypes.byref(how), margins.data_ptr(), counts.data_ptr(), grad_loss.data_ptr(),
                                              grad.data_ptr(), _stream_now(device.index))
        if st:
            _check(st, "tt_emb_preference_backward")
    return grad


def tt_emb_policy_forward(logp: torch.Tensor, old_logp: torch.Tensor, advantages: torch.Tensor, reference: Optional[torch.Tensor] = None,
                          mask: Optional[torch.Tensor] = None, offsets: Optional[torch.Tensor] = None,
                          clip: Union[float, Tuple[float, float]] = 0.2, dual_clip: Optional[float] = None, kl: str = "k3",
                          kl_weight: float = 0.0, level: str = "token", average: bool = True, per_token: Optional[bool] = None,
                          err: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
    """(loss, kl, log_ratio, counts int32, clipped int32), each [sequences], of the clipped policy loss.

    advantages: [sequences], or of logp's shape (level "token" only); per_token says which where both fit.  clip: one bound for both
    sides or (low, high).  kl: "k1", "k2" or "k3", the estimate of the divergence from the reference.
    average: an answer's loss is the mean over its tokens, not their sum.  Malformed offsets set 2 in err."""
    device = _device(logp)
    with _on(stream, device):
        a, count, keep = _answers(logp, reference, mask, offsets, average)
        how, more = _policy(old_logp, advantages, logp, count, clip, dual_clip, kl, kl_weight, level, per_token)
        n = tt_emb_answers_workspace(a.tokens, count)
        ws = torch.empty(n, dtype=torch.uint8, device=device) if n else None
        loss, counts = torch.empty(count, dtype=torch.float32, device=device), torch.empty(count, dtype=torch.int32, device=device)
        kl_out, log_ratio, clipped = torch.empty_like(loss), torch.empty_like(loss), torch.empty_like(counts)
        st = _c("tt_emb_policy_forward")(ctypes.byref(a), ctypes.byref(how), loss.data_ptr(), kl_out.data_ptr(), log_ratio.data_ptr(),
                                         counts.data_ptr(), clipped.data_ptr(), _err_word(err, device), ws.data_ptr() if n else None, n,
                                         _stream_now(device.index))
        if st:
            _check(st, "tt_emb_policy_forward")
    return loss, kl_out, log_ratio, counts, clipped


def tt_emb_policy_backward(logp: torch.Tensor, old_logp: torch.Tensor, advantages: torch.Tensor, log_ratio: torch.Tensor,
                           counts: torch.Tensor, grad_loss: torch.Tensor, reference: Optional[torch.Tensor] = None,
                           mask: Optional[torch.Tensor] = None, offsets: Optional[torch.Tensor] = None,
                           clip: Union[float, Tuple[float, float]] = 0.2, dual_clip: Optional[float] = None, kl: str = "k3",
                           kl_weight: float = 0.0, level: str = "token", average: bool = True, per_token: Optional[bool] = None,
                           stream=None) -> torch.Tensor:
    """The gradient of every token's log probability for log_ratio and counts of the forward call."""
    device = _device(logp)
    with _on(stream, device):
        a, count, keep = _answers(logp, reference, mask, offsets, average)
        how, more = _policy(old_logp, advantages, logp, count, clip, dual_clip, kl, kl_weight, level, per_token)
        log_ratio = _vector(log_ratio, torch.float32, (count,), device, "log_ratio")
        counts = _vector(counts, torch.int32, (count,), device, "counts")
        grad_loss = _vector(grad_loss, torch.float32, (count,), device, "grad_loss")
        grad = torch.empty(logp.shape, dtype=torch.float32, device=device)
        st = _c("tt_emb_policy_backward")(ctypes.byref(a), ctypes.byref(how), log_ratio.data_ptr(), counts.data_ptr(), grad_loss.data_ptr(),
                                          grad.data_ptr(), _stream_now(device.index))
        if st:
            _check(st, "tt_emb_policy_backward")
    return grad


# ---------------------------------------------------------------- autograd


class _PreferenceFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logp, reference, mask, offsets, how, err):
        loss, margins, rewards, counts = tt_emb_preference_forward(logp, reference, mask, offsets, err=err, **how)
        ctx.save_for_backward(logp, mask, offsets, margins, counts)
        ctx.how = how
        ctx.mark_non_differentiable(rewards, counts)
        return loss, rewards, counts

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad, *_):
        logp, mask, offsets, margins, counts = ctx.saved_tensors
        return tt_emb_preference_backward(logp, margins, counts, grad, mask, offsets, **ctx.how), None, None, None, None, None


class _PolicyFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logp, old_logp, advantages, reference, mask, offsets, how, err):
        loss, kl, log_ratio, counts, clipped = tt_emb_policy_forward(logp, old_logp, advantages, reference, mask, offsets, err=err, **how)
        ctx.save_for_backward(logp, old_logp, advantages, reference, mask, offsets, log_ratio, counts)
        ctx.how = how
        ctx.mark_non_differentiable(kl, log_ratio, counts, clipped)
        return loss, counts, kl, log_ratio, clipped

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad, *_):
        logp, old_logp, advantages, reference, mask, offsets, log_ratio, counts = ctx.saved_tensors
        g = tt_emb_policy_backward(logp, old_logp, advantages, log_ratio, counts, grad, reference, mask, offsets, **ctx.how)
        return g, None, None, None, None, None, None, None


def preference_loss(logp: torch.Tensor, reference: Optional[torch.Tensor] = None, mask: Optional[torch.Tensor] = None,
                    offsets: Optional[torch.Tensor] = None, beta: float = 0.1, kind: str = "sigmoid", label_smoothing: float = 0.0,
                    margin: float = 0.0, average: bool = False, reduction: str = "mean", err: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Loss of pairs of answers (the first half of the sequences chosen over the second), differentiable in logp.

    label_smoothing, in [0, 1), belongs to kind "sigmoid"; "hinge" and "squared" do not use it.
    reduction 'mean' divides by the pairs that count: those with a token that counts in either answer (0 when
    there are none); pairs without one are in no sum."""
    _check_reduction(reduction)
    how = dict(beta=beta, kind=kind, label_smoothing=label_smoothing, margin=margin, average=average)
    loss, _, counts = _PreferenceFunction.apply(logp, reference, mask, offsets, how, err)
    if reduction == "none":
        return loss
    pairs = loss.shape[0]
    have = (counts[:pairs] > 0) | (counts[pairs:] > 0)
    return _reduce(torch.where(have, loss, torch.zeros_like(loss)), have, reduction)


def policy_loss(logp: torch.Tensor, old_logp: torch.Tensor, advantages: torch.Tensor, reference: Optional[torch.Tensor] = None,
                mask: Optional[torch.Tensor] = None, offsets: Optional[torch.Tensor] = None,
                clip: Union[float, Tuple[float, float]] = 0.2, dual_clip: Optional[float] = None, kl: str = "k3", kl_weight: float = 0.0,
                level: str = "token", average: bool = True, reduction: str = "mean", per_token: Optional[bool] = None,
                err: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Clipped policy loss with a Kullback-Leibler term, differentiable in logp.

    reduction: 'none' [sequences], 'sum', 'mean' over the sequences with a token that counts, or 'tokens', the mean over
    all tokens that count (whatever `average` says); 0 when there are none."""
    if reduction != "tokens":
        _check_reduction(reduction)
    how = dict(clip=clip, dual_clip=dual_clip, kl=kl, kl_weight=kl_weight, level=level,
               average=average and reduction != "tokens", per_token=per_token)
    loss, counts = _PolicyFunction.apply(logp, old_logp, advantages, reference, mask, offsets, how, err)[:2]
    if reduction == "tokens":
        return loss.sum() / counts.sum().clamp(min=1)
    return _reduce(loss, counts > 0, reduction)
