"""A call on a stream of its own: what it copies of its arguments is copied on that stream.

A copy made on the current stream would be read by the call's kernels without waiting for
it, and its memory would go back to the current stream while they read it.  The order of
calls is shown on the CPU; on the GPU work is queued on the current stream that such a copy
would wait for, and its memory is written again at once."""
import contextlib

import pytest
import torch

import tensor_train_compressed_embeddingbag_gb300 as tt
from tensor_train_compressed_embeddingbag_gb300 import head


class _Copied(Exception):
    pass


class _OnCuda(torch.Tensor):
    """A host tensor that passes for one on a GPU; a copy of it says whether the call's stream is current."""

    inside = False
    is_cuda = property(lambda self: True)

    def is_contiguous(self, *a, **k):
        return False

    def contiguous(self, *a, **k):
        raise _Copied(_OnCuda.inside)


def _apart(rows, cols, dtype=torch.float32):
    return torch.zeros((cols, rows), dtype=dtype).t().as_subclass(_OnCuda)


def _calls(h, w, ids, logits, lse, dlse, rows, packed, scales):
    t = ids[:, 0]
    return {
        "tt_emb_xent_forward": lambda **kw: tt.tt_emb_xent_forward(h, w, t, **kw),
        "tt_emb_xent_backward": lambda **kw: tt.tt_emb_xent_backward(h, w, t, lse, rows, **kw),
        "tt_emb_distill_forward": lambda **kw: tt.tt_emb_distill_forward(h, w, ids, logits, **kw),
        "tt_emb_distill_backward": lambda **kw: tt.tt_emb_distill_backward(h, w, ids, logits, dlse, rows, **kw),
        "tt_emb_q4_quantize": lambda **kw: tt.tt_emb_q4_quantize(w, 32, **kw),
        "tt_emb_q4_matvec": lambda **kw: tt.tt_emb_q4_matvec(h, packed, scales, 32, **kw),
    }


NAMES = ["tt_emb_xent_forward", "tt_emb_xent_backward", "tt_emb_distill_forward", "tt_emb_distill_backward", "tt_emb_q4_quantize",
         "tt_emb_q4_matvec"]


@pytest.mark.parametrize("name", NAMES)
def test_copies_are_made_on_the_calls_stream(name, monkeypatch):
    @contextlib.contextmanager
    def on(stream, device):
        _OnCuda.inside = True
        try:
            yield
        finally:
            _OnCuda.inside = False

    monkeypatch.setattr(head, "_on", on)
    call = _calls(_apart(6, 40), _apart(9, 40), _apart(6, 3, torch.int64), _apart(6, 3), *[torch.zeros(6).as_subclass(_OnCuda)] * 3,
                  _apart(9, 32, torch.uint8), _apart(9, 2, torch.bfloat16))[name]
    with pytest.raises(_Copied) as e:
        call(stream=object())
    assert e.value.args == (True,)


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_copies_on_another_stream(name):
    n, v, d, k = 40, 600, 96, 4
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    h, w = (torch.randn((m, d), generator=g, device="cuda") for m in (n, v))
    w *= 0.2
    ids = torch.randint(0, v, (n, k), generator=g, device="cuda")
    logits, rows = torch.randn((n, k), generator=g, device="cuda"), torch.rand((n,), generator=g, device="cuda")
    packed, scales = tt.tt_emb_q4_quantize(w, 32)
    args = h, w, ids, logits, tt.tt_emb_xent_forward(h, w, ids[:, 0])[1], tt.tt_emb_distill_forward(h, w, ids, logits)[1], rows, packed, scales
    want = _calls(*args)[name]()
    apart = [x.t().contiguous().t() if x.dim() == 2 else x.repeat_interleave(2)[::2] for x in args]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)  # some 50 ms on the current stream
    got = _calls(*apart)[name](stream=side)
    junk = [torch.full_like(x, 7) for x in args]  # takes memory that the current stream has free
    side.synchronize()
    want, got = ((x,) if isinstance(x, torch.Tensor) else x for x in (want, got))
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    torch.cuda.synchronize()
    del junk
