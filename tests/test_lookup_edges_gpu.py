"""Lookups of a dense table and their gradient on the GPU: what the sizes and arguments elsewhere leave out."""
import pytest
import torch

import tensor_train_compressed_embeddingbag_gb300 as tt

from test_lookup_gpu import TYPES, check_grad, gen, popular

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


# around 65,536 lookups, 32 chunks of the sort, beyond which a launch of its own sums the chunks' histograms: one digit
# (8 and 11 bits: more than 32 bins), two (16 and 22 bits) and three (23 bits)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,v,d", [(65536, 200, 8), (65537, 200, 8), (65536, 2000, 8), (65537, 2000, 8), (65537, 3000, 8), (70000, 50001, 16),
                                   (131072, 2000000, 8), (200000, 4200000, 8), (200000, 5000000, 8), (300001, 70000, 33)])
def test_sorts_of_more_than_32_chunks(n, v, d, dtype):
    g = torch.randn((n, d), generator=gen(35), device="cuda").to(dtype)
    ids = popular(n, v, 36)
    got = tt.tt_emb_lookup_backward(g, ids, v, scale=0.7)
    check_grad(got, g, ids, 0.7)
    for _ in range(3):
        assert torch.equal(got, tt.tt_emb_lookup_backward(g, ids, v, scale=0.7))  # bit for bit
    # every id about as often: every digit has some
    ids = torch.randint(0, v, (n,), generator=gen(37), device="cuda")
    check_grad(tt.tt_emb_lookup_backward(g, ids, v), g, ids, 1.0)
    pad = v // 2
    ids = torch.where(torch.rand((n,), generator=gen(38), device="cuda") < 0.5, torch.full_like(ids, pad), ids)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ids[::1001] = v
    got = tt.tt_emb_lookup_backward(g, ids, v, padding_idx=pad, err=err)
    check_grad(got, g, ids, 1.0, pad)
    assert err.item() == 1 and not got[pad].any()
    into = torch.randn((v, d), generator=gen(39), device="cuda").to(dtype)
    old = into.clone()
    check_grad(tt.tt_emb_lookup_backward(g, ids, v, padding_idx=pad, grad_weight=into), g, ids, 1.0, pad, old)


@pytest.mark.parametrize("n", [1, 37, 1024])
def test_a_large_gradient_that_no_id_names(n):
    """All padding, or all outside: zeros, which the launch of the sums may not overtake."""
    v, d = 1_000_003, 64
    g = torch.randn((n, d), generator=gen(40), device="cuda")
    ids = torch.full((n,), 9, device="cuda")
    for i in range(30):
        held = torch.full((v, d), float("nan"), device="cuda")
        del held  # its memory is the gradient's next
        got = tt.tt_emb_lookup_backward(g, ids, v, padding_idx=9) if i % 2 else tt.tt_emb_lookup_backward(g, ids + v, v)
        assert not got.flip(0).any()
