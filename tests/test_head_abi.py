"""The vocabulary head's C calls refuse bad arguments on the host, before any CUDA call."""
import ctypes

import pytest

import tensor_train_compressed_embeddingbag_gb300 as tt
from tensor_train_compressed_embeddingbag_gb300.head import _Head


@pytest.fixture(scope="module")
def lib():
    tt.build()
    return tt.load_library()


def head(**kw):
    d = dict(hidden_dev=4096, weight_dev=8192, rows=4, vocab=10, hidden_stride=8, weight_stride=8, dim=8, dtype=0)
    d.update(kw)
    return _Head(*[d[name] for name, _ in _Head._fields_])


def forward(lib, h, targets=4096, loss=4096, lse=4096, ws=4096):
    return lib.tt_emb_xent_forward(ctypes.byref(h) if h else None, targets, -100, loss, lse, None, ws, 1 << 30, None)


def backward(lib, h, targets=4096, lse=4096, grad=4096, gh=4096, gw=4096, ws=4096):
    return lib.tt_emb_xent_backward(ctypes.byref(h) if h else None, targets, -100, lse, grad, gh, gw, None, ws, 1 << 30, None)


@pytest.mark.parametrize("bad", [dict(rows=-1), dict(vocab=0), dict(dim=0), dict(hidden_stride=7), dict(weight_stride=7),
                                 dict(rows=16777217), dict(vocab=1073741825), dict(dim=65537, hidden_stride=65537, weight_stride=65537)])
def test_shapes(lib, bad):
    assert forward(lib, head(**bad)) == tt.TT_ERR_SHAPE
    assert backward(lib, head(**bad)) == tt.TT_ERR_SHAPE
    assert lib.tt_emb_head_workspace(ctypes.byref(head(**bad)), 1, 0) == -1


def test_arguments(lib):
    for call in (forward, backward):
        assert call(lib, None) == tt.TT_ERR_ARG
        assert call(lib, head(dtype=3)) == tt.TT_ERR_ARG
        assert call(lib, head(hidden_dev=None)) == tt.TT_ERR_ARG
        assert call(lib, head(weight_dev=None)) == tt.TT_ERR_ARG
        assert call(lib, head(hidden_dev=4098)) == tt.TT_ERR_ARG  # fp32 rows on a 2-byte boundary
        assert call(lib, head(), targets=None) == tt.TT_ERR_ARG
        assert call(lib, head(), lse=None) == tt.TT_ERR_ARG
        assert call(lib, head(), ws=None) == tt.TT_ERR_ARG
        assert call(lib, head(), ws=4096 + 128) == tt.TT_ERR_ARG
    assert forward(lib, head(), loss=None) == tt.TT_ERR_ARG
    assert backward(lib, head(), grad=None) == tt.TT_ERR_ARG
    assert backward(lib, head(), gh=None) == tt.TT_ERR_ARG
    assert backward(lib, head(), gw=None) == tt.TT_ERR_ARG
    assert lib.tt_emb_head_workspace(None, 1, 0) == -1


def test_teacher(lib):
    h = head()

    def call(ids=4096, logits=4096, k=4, temp=1.0):
        return lib.tt_emb_distill_forward(ctypes.byref(h), ids, logits, k, temp, 4096, 4096, None, 4096, 1 << 30, None)

    assert call(ids=None) == tt.TT_ERR_ARG
    assert call(logits=None) == tt.TT_ERR_ARG
    for temp in (0.0, -1.0, 1e-5, 2e4, float("nan"), float("inf")):
        assert call(temp=temp) == tt.TT_ERR_ARG
    assert call(k=0) == tt.TT_ERR_SHAPE
    assert call(k=1025) == tt.TT_ERR_SHAPE
    big = head(rows=16777216)
    assert lib.tt_emb_head_workspace(ctypes.byref(big), 1024, 0) == -1  # rows x entries past 2^31


def test_q4(lib):
    def call(x=4096, stride=64, rows=1, dtype=0, packed=4096, scales=4096, vocab=10, dim=64, group=32, out=4096):
        return lib.tt_emb_q4_matvec(x, stride, rows, dtype, packed, scales, vocab, dim, group, out, None)

    for bad in (dict(stride=63), dict(rows=-1), dict(rows=65537), dict(vocab=0), dict(dim=0), dict(group=48)):
        assert call(**bad) == tt.TT_ERR_SHAPE, bad
    for bad in (dict(x=None), dict(x=4097), dict(dtype=7), dict(packed=None), dict(packed=4104), dict(scales=None), dict(scales=4097),
                dict(out=None), dict(out=4098)):
        assert call(**bad) == tt.TT_ERR_ARG, bad
    assert call(rows=0) == tt.TT_OK

    def quant(w=4096, stride=64, vocab=10, dim=64, dtype=0, group=32, packed=4096, scales=4096):
        return lib.tt_emb_q4_quantize(w, stride, vocab, dim, dtype, group, packed, scales, None)

    for bad in (dict(stride=63), dict(vocab=0), dict(dim=70000, stride=70000), dict(group=0)):
        assert quant(**bad) == tt.TT_ERR_SHAPE, bad
    for bad in (dict(w=None), dict(packed=None), dict(packed=4100), dict(scales=None), dict(dtype=-1)):
        assert quant(**bad) == tt.TT_ERR_ARG, bad


def test_without_a_gpu_the_calls_say_so(lib):
    import torch

    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert forward(lib, head()) == tt.TT_ERR_CUDA
    assert backward(lib, head()) == tt.TT_ERR_CUDA
    assert lib.tt_emb_head_workspace(ctypes.byref(head()), 1, 1) == -1


def test_wrong_tensors_are_refused_without_a_gpu():
    import torch

    h = torch.ones((2, 4))
    with pytest.raises(tt.TTError) as e:
        tt.tt_emb_xent_forward(h, h, torch.zeros(2, dtype=torch.int64))
    assert e.value.code == tt.TT_ERR_ARG
    with pytest.raises(tt.TTError):
        tt.tt_emb_q4_quantize(h)


def _refused(code, call, *args):
    with pytest.raises(tt.TTError) as e:
        call(*args)
    assert e.value.code == code


def test_losses_refuse_shapes_that_do_not_match():
    """Also those that hold the right number of elements."""
    import torch

    h, w = torch.zeros((4, 6, 8)), torch.zeros((5, 8))
    t = torch.zeros((4, 6), dtype=torch.int64)
    for bad in (t.t(), t.reshape(3, 8), t[:, :5], t[..., None], t.reshape(-1)[1:]):
        _refused(tt.TT_ERR_SHAPE, tt.vocab_cross_entropy, h, w, bad)
    ids, logits = torch.zeros((4, 6, 3), dtype=torch.int64), torch.zeros((4, 6, 3))
    for bad_ids, bad_logits in ((ids.transpose(0, 1), logits.transpose(0, 1)), (ids, logits.transpose(1, 2)), (ids, logits.reshape(24, 3)), (ids.reshape(3, 8, 3), logits.reshape(3, 8, 3)),
                                (ids[..., :2], logits), (ids[..., 0], logits[..., 0])):
        _refused(tt.TT_ERR_SHAPE, tt.vocab_distillation, h, w, bad_ids, bad_logits)
    # rows flattened on one side only are the same rows: these go on to the next check, which wants a GPU
    for rows, ts in ((h, t.reshape(-1)), (h.reshape(24, 8), t)):
        _refused(tt.TT_ERR_ARG, tt.vocab_cross_entropy, rows, w, ts)
    _refused(tt.TT_ERR_ARG, tt.vocab_distillation, h, w, ids.reshape(24, 3), logits.reshape(24, 3))


def test_a_4_bit_table_refuses_rows_of_another_width():
    """Widths 33 to 64 have codes of one size: the table knows which is its own."""
    import torch

    table = tt.Q4Table.__new__(tt.Q4Table)
    table.vocab, table.dim, table.group = 10, 64, 32
    table.packed, table.scales = torch.zeros((10, 32), dtype=torch.uint8), torch.zeros((10, 2), dtype=torch.bfloat16)
    for width in (33, 60, 65, 128):
        _refused(tt.TT_ERR_SHAPE, table.scores, torch.zeros((2, width)))
    _refused(tt.TT_ERR_SHAPE, table.scores, torch.zeros(()))


@pytest.mark.parametrize("dtype", [0, 1, 2])
def test_no_rows_need_no_workspace(lib, dtype):
    """16-bit types take no workspace for a forward pass of no rows: a null one of 0 bytes is right."""
    h = head(rows=0, dtype=dtype, hidden_dev=None)
    n = 1 << 20 if dtype == 0 else 0  # fp32 copies the table whatever the rows
    for call in (lambda: lib.tt_emb_xent_forward(ctypes.byref(h), None, -100, None, None, None, 4096 if n else None, n, None),
                 lambda: lib.tt_emb_distill_forward(ctypes.byref(h), None, None, 3, 1.0, None, None, None, 4096 if n else None, n, None)):
        assert call() in (tt.TT_OK, tt.TT_ERR_CUDA)  # the latter without a GPU
    if dtype:
        assert forward(lib, head(dtype=dtype), ws=None) == tt.TT_ERR_ARG


def test_losses_take_one_row_without_a_batch():
    """Shapes that go on to the next check, which wants a GPU."""
    import torch

    h, w = torch.zeros(8), torch.zeros((5, 8))
    for rows, t in ((h, torch.tensor(1)), (h, torch.tensor([1])), (h[None], torch.tensor(1))):
        _refused(tt.TT_ERR_ARG, tt.vocab_cross_entropy, rows, w, t)
    ids, logits = torch.zeros(3, dtype=torch.int64), torch.zeros(3)
    for rows, i, x in ((h, ids, logits), (h, ids[None], logits[None]), (h[None], ids, logits)):
        _refused(tt.TT_ERR_ARG, tt.vocab_distillation, rows, w, i, x)
    _refused(tt.TT_ERR_SHAPE, tt.vocab_cross_entropy, h, w, torch.tensor([1, 2]))
    _refused(tt.TT_ERR_SHAPE, tt.vocab_distillation, h, w, torch.tensor(1), torch.tensor(1.0))
