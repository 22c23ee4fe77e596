"""Lookups of a dense table and their gradient on the GPU: what the sizes and arguments elsewhere leave out."""
import pytest
import torch

import tensor_train_compressed_embeddingbag_gb300 as tt

from test_lookup_gpu import check_grad, gen, popular

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [60, 3000])
def test_padding_below_zero_counts_from_the_end(n):
    v, d = 40, 24
    w = torch.randn((v, d), generator=gen(30), device="cuda").requires_grad_()
    ids = torch.randint(0, v, (n,), generator=gen(31), device="cuda")
    g = torch.randn((n, d), generator=gen(32), device="cuda")
    for pad in (-1, -v, -7):
        tt.vocab_embedding(ids, w, padding_idx=pad).backward(g)
        check_grad(w.grad, g, ids, 1.0, v + pad)
        assert not w.grad[v + pad].any()
        w.grad = None
    tt.vocab_embedding(ids, w).backward(g)
    check_grad(w.grad, g, ids, 1.0)


@pytest.mark.parametrize("n", [60, 3000])
def test_the_backward_pass_reports_ids_outside_the_table(n):
    """Into the caller's error word, as the head's losses do."""
    w = torch.randn((40, 24), generator=gen(33), device="cuda").requires_grad_()
    ids = popular(n, 40, 34)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    tt.vocab_embedding(ids, w, err=err).sum().backward()
    assert err.item() == 0
    ids[7] = 40
    out = tt.vocab_embedding(ids, w, err=err)
    assert err.item() == 1
    err.zero_()
    out.sum().backward()
    assert err.item() == 1
