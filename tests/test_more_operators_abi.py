"""Lookups, losses of answers and 8-bit scores refuse bad arguments on the host, before any CUDA call."""
import ctypes
import math

import pytest
import torch

import tensor_train_compressed_embeddingbag_gb300 as tt
from tensor_train_compressed_embeddingbag_gb300.answers import _Answers, _Policy, _Preference
from tensor_train_compressed_embeddingbag_gb300.lookup import _Lookup


@pytest.fixture(scope="module")
def lib():
    tt.build()
    return tt.load_library()


def struct(cls, defaults, **kw):
    d = dict(defaults, **kw)
    return cls(*[d[name] for name, _ in cls._fields_])


LOOKUP = dict(weight_dev=4096, weight_stride=8, ids_dev=4096, rows=4, vocab=10, padding_idx=-1, dim=8, dtype=0, scale=1.0)


def test_lookup(lib):
    def forward(out=4096, stride=8, **kw):
        a = struct(_Lookup, LOOKUP, **kw)
        return lib.tt_emb_lookup_forward(ctypes.byref(a), out, stride, None, None)

    def backward(g=4096, gs=8, gw=4096, gws=8, ws=4096, n=1 << 40, err=None, **kw):
        a = struct(_Lookup, LOOKUP, **kw)
        return lib.tt_emb_lookup_backward(ctypes.byref(a), g, gs, gw, gws, 0, err, ws, n, None)

    for call in (forward, backward):
        for bad in (dict(rows=-1), dict(rows=134217729), dict(vocab=0), dict(vocab=(1 << 30) + 1), dict(dim=0), dict(dim=65537)):
            assert call(**bad) == tt.TT_ERR_SHAPE, bad
        for bad in (dict(dtype=3), dict(dtype=-1), dict(ids_dev=None), dict(ids_dev=4100)):
            assert call(**bad) == tt.TT_ERR_ARG, bad
    for bad in (dict(weight_stride=7), dict(stride=7)):
        assert forward(**bad) == tt.TT_ERR_SHAPE
    for bad in (dict(weight_dev=None), dict(weight_dev=4098), dict(out=None), dict(out=4097), dict(weight_dev=4097, dtype=1)):
        assert forward(**bad) == tt.TT_ERR_ARG, bad
    for bad in (dict(gs=7), dict(gws=7)):
        assert backward(**bad) == tt.TT_ERR_SHAPE
    for bad in (dict(g=None), dict(g=4098), dict(gw=None), dict(gw=4098), dict(ws=4096 + 128), dict(err=4097), dict(rows=5000, ws=None),
                dict(rows=5000, n=1000)):
        assert backward(**bad) == tt.TT_ERR_ARG, bad
    assert lib.tt_emb_lookup_forward(None, 4096, 8, None, None) == tt.TT_ERR_ARG
    assert lib.tt_emb_lookup_backward(None, 4096, 8, 4096, 8, 0, None, None, 0, None) == tt.TT_ERR_ARG
    assert forward(rows=0, ids_dev=None, out=None) == tt.TT_OK
    for bad in ((-1, 10, 8, 0), (4, 0, 8, 0), (4, 10, 0, 0), (4, 10, 8, 5)):
        assert lib.tt_emb_lookup_workspace(*bad) == -1
    assert lib.tt_emb_lookup_workspace(5000, 10, 8, 0) > 2 * 5000 * 8


ANSWERS = dict(logp_dev=4096, reference_dev=4096, mask_dev=4096, offsets_dev=None, tokens=12, sequences=4, average=0)
PREFERENCE = dict(kind=0, beta=0.1, label_smoothing=0.0, margin=0.0)
POLICY = dict(old_dev=4096, advantages_dev=4096, per_token=0, level=0, kl=3, clip_low=0.2, clip_high=0.2, dual_clip=0.0, kl_weight=0.1)


def _preference_forward(lib, out=(4096,) * 4, ws=4096, n=1 << 40, how=True, **kw):
    a = struct(_Answers, ANSWERS, **{k: v for k, v in kw.items() if k in ANSWERS})
    p = struct(_Preference, PREFERENCE, **{k: v for k, v in kw.items() if k in PREFERENCE})
    return lib.tt_emb_preference_forward(ctypes.byref(a), ctypes.byref(p) if how else None, *out, None, ws, n, None)


def _preference_backward(lib, ins=(4096,) * 3, grad=4096, how=True, **kw):
    a = struct(_Answers, ANSWERS, **{k: v for k, v in kw.items() if k in ANSWERS})
    p = struct(_Preference, PREFERENCE, **{k: v for k, v in kw.items() if k in PREFERENCE})
    return lib.tt_emb_preference_backward(ctypes.byref(a), ctypes.byref(p) if how else None, *ins, grad, None)


def _policy_forward(lib, out=(4096,) * 5, ws=4096, n=1 << 40, how=True, **kw):
    a = struct(_Answers, ANSWERS, **{k: v for k, v in kw.items() if k in ANSWERS})
    p = struct(_Policy, POLICY, **{k: v for k, v in kw.items() if k in POLICY})
    return lib.tt_emb_policy_forward(ctypes.byref(a), ctypes.byref(p) if how else None, *out, None, ws, n, None)


def _policy_backward(lib, ins=(4096,) * 3, grad=4096, how=True, **kw):
    a = struct(_Answers, ANSWERS, **{k: v for k, v in kw.items() if k in ANSWERS})
    p = struct(_Policy, POLICY, **{k: v for k, v in kw.items() if k in POLICY})
    return lib.tt_emb_policy_backward(ctypes.byref(a), ctypes.byref(p) if how else None, *ins, grad, None)


def test_answers(lib):
    for call in (_preference_forward, _preference_backward, _policy_forward, _policy_backward):
        for bad in (dict(tokens=-1), dict(sequences=-1), dict(tokens=13), dict(sequences=0), dict(sequences=(1 << 24) + 1), dict(tokens=(1 << 40) + 4),
                    dict(tokens=4 << 31)):
            assert call(lib, **bad) == tt.TT_ERR_SHAPE, (call, bad)
        assert call(lib, how=False) == tt.TT_ERR_ARG
        assert call(lib, offsets_dev=4100) == tt.TT_ERR_ARG
    for call in (_preference_forward, _policy_forward):
        many = 4 if call is _preference_forward else 5
        for i in range(many):
            assert call(lib, out=tuple(None if j == i else 4096 for j in range(many))) == tt.TT_ERR_ARG
            assert call(lib, out=tuple(4098 if j == i else 4096 for j in range(many))) == tt.TT_ERR_ARG
        for bad in (dict(logp_dev=None), dict(logp_dev=4098), dict(reference_dev=4098), dict(ws=4096 + 128), dict(tokens=40000, ws=None),
                    dict(tokens=40000, n=16)):
            assert call(lib, **bad) == tt.TT_ERR_ARG, bad
        assert call(lib, tokens=0, sequences=0, out=(None,) * many, ws=None, n=0) == tt.TT_OK
    for call in (_preference_backward, _policy_backward):
        for i in range(3):
            assert call(lib, ins=tuple(None if j == i else 4096 for j in range(3))) == tt.TT_ERR_ARG
            assert call(lib, ins=tuple(4097 if j == i else 4096 for j in range(3))) == tt.TT_ERR_ARG
        assert call(lib, grad=None) == tt.TT_ERR_ARG
        assert call(lib, tokens=0) == tt.TT_OK
    assert lib.tt_emb_answers_workspace(-1, 4) == -1 and lib.tt_emb_answers_workspace(4, -1) == -1
    assert lib.tt_emb_answers_workspace(0, 0) == 0 and lib.tt_emb_answers_workspace(100000, 7) >= 32 * (7 + 100000 // 2048)


def test_preference(lib):
    nan, inf = math.nan, math.inf
    for call in (_preference_forward, _preference_backward):
        for bad in (dict(kind=-1), dict(kind=3), dict(beta=0.0), dict(beta=-1.0), dict(beta=nan), dict(beta=inf), dict(label_smoothing=-0.1),
                    dict(label_smoothing=1.0), dict(label_smoothing=nan), dict(margin=nan), dict(margin=inf), dict(kind=1, label_smoothing=0.1)):
            assert call(lib, **bad) == tt.TT_ERR_ARG, bad
        assert call(lib, sequences=3) == tt.TT_ERR_SHAPE


def test_policy(lib):
    nan = math.nan
    for call in (_policy_forward, _policy_backward):
        for bad in (dict(level=2), dict(level=-1), dict(kl=0), dict(kl=4), dict(clip_low=-0.1), dict(clip_low=1.0), dict(clip_low=nan), dict(clip_high=-1.0),
                    dict(clip_high=nan), dict(dual_clip=1.0), dict(dual_clip=-2.0), dict(dual_clip=nan), dict(kl_weight=-1.0), dict(kl_weight=nan),
                    dict(level=1, per_token=1), dict(reference_dev=None), dict(old_dev=None), dict(advantages_dev=None), dict(old_dev=4097),
                    dict(advantages_dev=4097), dict(logp_dev=None)):
            assert call(lib, **bad) == tt.TT_ERR_ARG, bad


def test_q8(lib):
    def quant(w=4096, stride=64, rows=10, dim=64, dtype=0, codes=4096, scales=4096):
        return lib.tt_emb_q8_quantize(w, stride, rows, dim, dtype, codes, scales, None)

    for bad in (dict(stride=63), dict(rows=-1), dict(rows=(1 << 30) + 1), dict(dim=0), dict(dim=65537, stride=65537)):
        assert quant(**bad) == tt.TT_ERR_SHAPE, bad
    for bad in (dict(w=None), dict(w=4098), dict(dtype=4), dict(codes=None), dict(codes=4104), dict(scales=None), dict(scales=4098)):
        assert quant(**bad) == tt.TT_ERR_ARG, bad
    assert quant(rows=0) == tt.TT_OK

    def scores(x=4096, stride=64, rows=2, dtype=0, codes=4096, scales=4096, vocab=10, dim=64, out=4096, err=None, ws=4096, n=1 << 30):
        return lib.tt_emb_q8_scores(x, stride, rows, dtype, codes, scales, vocab, dim, out, err, ws, n, None)

    for bad in (dict(stride=63), dict(rows=-1), dict(rows=(1 << 24) + 1), dict(vocab=0), dict(vocab=(1 << 30) + 1), dict(dim=0)):
        assert scores(**bad) == tt.TT_ERR_SHAPE, bad
    for bad in (dict(x=None), dict(x=4097), dict(dtype=-1), dict(codes=None), dict(codes=4104), dict(scales=None), dict(scales=4098), dict(out=None),
                dict(out=4098), dict(err=4097), dict(ws=None), dict(ws=4100), dict(n=100)):
        assert scores(**bad) == tt.TT_ERR_ARG, bad
    assert scores(rows=0) == tt.TT_OK
    for bad in ((-1, 8), (2, 0), (2, 65537), ((1 << 24) + 1, 8)):
        assert lib.tt_emb_q8_workspace(*bad) == -1


def test_without_a_gpu_the_calls_say_so(lib):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    a = struct(_Lookup, LOOKUP)
    assert lib.tt_emb_lookup_forward(ctypes.byref(a), 4096, 8, None, None) == tt.TT_ERR_CUDA
    assert lib.tt_emb_lookup_backward(ctypes.byref(a), 4096, 8, 4096, 8, 0, None, 4096, 1 << 40, None) == tt.TT_ERR_CUDA
    for call in (_preference_forward, _preference_backward, _policy_forward, _policy_backward):
        assert call(lib) == tt.TT_ERR_CUDA
    assert lib.tt_emb_q8_quantize(4096, 64, 10, 64, 0, 4096, 4096, None) == tt.TT_ERR_CUDA
    assert lib.tt_emb_q8_scores(4096, 64, 2, 0, 4096, 4096, 10, 64, 4096, None, 4096, 1 << 30, None) == tt.TT_ERR_CUDA


def _refused(code, call, *args, **kw):
    with pytest.raises(tt.TTError) as e:
        call(*args, **kw)
    assert e.value.code == code


class _OnCuda(torch.Tensor):
    """A host tensor that passes for one on a GPU as far as the checks of shapes."""

    is_cuda = property(lambda self: True)


def cuda(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype).as_subclass(_OnCuda)


@pytest.fixture
def here(monkeypatch):
    """Calls stay on the host: no device is made current."""
    import contextlib

    from tensor_train_compressed_embeddingbag_gb300 import answers, lookup, q8

    for mod in (answers, lookup, q8):
        monkeypatch.setattr(mod, "_on", lambda stream, device: contextlib.nullcontext())
        monkeypatch.setattr(mod, "_stream_now", lambda index: None)


def test_wrong_tensors(here):
    ids = torch.zeros(4, dtype=torch.int64)
    host = torch.zeros((4, 8))
    _refused(tt.TT_ERR_ARG, tt.tt_emb_lookup_forward, host, ids)
    _refused(tt.TT_ERR_ARG, tt.tt_emb_lookup_backward, host, ids, 5)
    _refused(tt.TT_ERR_ARG, tt.tt_emb_q8_quantize, host)
    _refused(tt.TT_ERR_ARG, tt.tt_emb_q8_scores, host, host, host)
    _refused(tt.TT_ERR_ARG, tt.tt_emb_preference_forward, host)
    _refused(tt.TT_ERR_ARG, tt.tt_emb_policy_forward, host, host, host)
    _refused(tt.TT_ERR_ARG, tt.vocab_embedding, [1, 2], host)

    w = cuda(10, 8)
    for bad in (ids.int(), [1, 2]):
        _refused(tt.TT_ERR_ARG, tt.tt_emb_lookup_forward, w, bad)
    _refused(tt.TT_ERR_SHAPE, tt.tt_emb_lookup_forward, w, ids.reshape(2, 2))
    _refused(tt.TT_ERR_SHAPE, tt.tt_emb_lookup_forward, cuda(8), ids)
    _refused(tt.TT_ERR_SHAPE, tt.tt_emb_lookup_backward, w, ids, 5)
    g = cuda(4, 8)
    _refused(tt.TT_ERR_SHAPE, tt.tt_emb_lookup_backward, g, ids, 0)
    _refused(tt.TT_ERR_ARG, tt.tt_emb_lookup_backward, g, ids, 5, grad_weight=cuda(5, 8, dtype=torch.float16))
    for bad in (cuda(4, 8), cuda(5, 9), cuda(8, 5).t(), cuda(1, 8).expand(5, 8)):
        _refused(tt.TT_ERR_SHAPE, tt.tt_emb_lookup_backward, g, ids, 5, grad_weight=bad)


def test_wrong_answers(here):
    p, s = tt.tt_emb_preference_forward, tt.TT_ERR_SHAPE
    x = cuda(4, 6)
    _refused(s, p, cuda(4))
    _refused(s, p, cuda(3, 6))
    _refused(s, p, x, offsets=torch.zeros(5, dtype=torch.int64))
    _refused(s, p, cuda(24), offsets=torch.zeros(0, dtype=torch.int64))
    _refused(tt.TT_ERR_ARG, p, cuda(24), offsets=torch.zeros(5, dtype=torch.int32))
    _refused(s, p, x, reference=torch.zeros(6, 4))
    _refused(s, p, x, mask=torch.zeros((4, 5), dtype=torch.bool))
    for bad in (torch.zeros(4, 6), [1]):
        _refused(tt.TT_ERR_ARG, p, x, mask=bad)
    _refused(tt.TT_ERR_ARG, p, x, kind="other")
    _refused(tt.TT_ERR_ARG, p, cuda(4, 6, dtype=torch.float16))
    _refused(tt.TT_ERR_ARG, p, x, reference=torch.zeros((4, 6), dtype=torch.float16))
    _refused(tt.TT_ERR_ARG, p, x, beta=0.0)
    b = tt.tt_emb_preference_backward
    _refused(s, b, x, torch.zeros(3), torch.zeros(4, dtype=torch.int32), torch.zeros(2))
    _refused(s, b, x, torch.zeros(2), torch.zeros(2, dtype=torch.int32), torch.zeros(2))
    _refused(s, b, x, torch.zeros(2), torch.zeros(4, dtype=torch.int32), torch.zeros(4))
    _refused(tt.TT_ERR_ARG, b, x, torch.zeros(2), torch.zeros(4), torch.zeros(2))
    q, old, adv = tt.tt_emb_policy_forward, torch.zeros(4, 6), torch.zeros(4)
    _refused(s, q, x, torch.zeros(6, 4), adv)
    _refused(s, q, x, old, torch.zeros(5))
    _refused(s, q, x, old, adv, per_token=True)
    _refused(s, q, x, old, torch.zeros(4, 6), per_token=False)
    for bad in (dict(level="word"), dict(kl="k4"), dict(clip=-0.5), dict(clip=(0.2, math.nan)), dict(dual_clip=0.5), dict(kl_weight=0.1)):
        _refused(tt.TT_ERR_ARG, q, x, old, adv, **bad)
    _refused(tt.TT_ERR_ARG, q, x, old, torch.zeros(4, 6), level="sequence")
    # as many tokens as sequences: whose are the advantages?
    one = cuda(4)
    _refused(tt.TT_ERR_ARG, q, one, torch.zeros(4), adv, offsets=torch.arange(5))
    r = tt.tt_emb_policy_backward
    count = torch.zeros(4, dtype=torch.int32)
    _refused(s, r, x, old, adv, torch.zeros(3), count, torch.zeros(4))
    _refused(s, r, x, old, adv, torch.zeros(4), count[:3], torch.zeros(4))
    _refused(s, r, x, old, adv, torch.zeros(4), count, torch.zeros(5))


def test_wrong_8_bit_tables(here):
    x, codes, scales = cuda(2, 40), torch.zeros((5, 48), dtype=torch.int8), torch.zeros(5)
    s = tt.TT_ERR_SHAPE
    _refused(s, tt.tt_emb_q8_scores, x, codes[:, :40], scales)
    _refused(s, tt.tt_emb_q8_scores, x, codes[:0], scales[:0])
    _refused(s, tt.tt_emb_q8_scores, x, codes, scales[:4])
    _refused(tt.TT_ERR_ARG, tt.tt_emb_q8_scores, x, codes.to(torch.uint8), scales)
    _refused(tt.TT_ERR_ARG, tt.tt_emb_q8_scores, x, codes, scales.double())
    for bad in (torch.zeros(2, 6), torch.zeros((2, 5), dtype=torch.float16), torch.zeros(5, 2).t()):
        _refused(tt.TT_ERR_ARG, tt.tt_emb_q8_scores, x, codes, scales, out=bad)
    served = tt.Q8Table.__new__(tt.Q8Table)
    served.vocab, served.dim, served.codes, served.scales = 5, 40, codes, scales
    for width in (33, 41, 48):
        _refused(s, served.scores, torch.zeros((2, width)))
    _refused(s, served.scores, torch.zeros(()))


def test_what_is_no_table_is_refused_as_such(here):
    ids = torch.zeros(4, dtype=torch.int64)
    for bad in (None, [[1.0]], torch.zeros(2, 3)):
        _refused(tt.TT_ERR_ARG, tt.vocab_embedding, ids, bad)
        _refused(tt.TT_ERR_ARG, tt.Q8Table, bad)
    _refused(tt.TT_ERR_SHAPE, tt.vocab_embedding, ids, cuda(8))
    _refused(tt.TT_ERR_SHAPE, tt.vocab_embedding, ids, cuda(2, 3, 4))
    _refused(tt.TT_ERR_SHAPE, tt.Q8Table, cuda(8))
    _refused(tt.TT_ERR_SHAPE, tt.Q8Table, cuda(2, 3, 4))
    served = tt.Q8Table.__new__(tt.Q8Table)
    served.vocab, served.dim, served.codes, served.scales = 5, 40, None, None
    for bad in (None, [1.0] * 40):
        _refused(tt.TT_ERR_ARG, served.scores, bad)
