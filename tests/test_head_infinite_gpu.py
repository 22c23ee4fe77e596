"""Infinities and NaN that count: a table row that is scored -inf drops out, NaN is not lost.

Rows are banned from a table as they are in practice: a column of biases, 0 or -inf, that hidden holds a 1 for.  Bounds are
_head_ref.py's for the table without the banned rows."""
import math

import pytest
import torch

import tensor_train_compressed_embeddingbag_gb300 as tt

import _head_ref as ref

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]


def banned_table(n, v, d, dtype, seed):
    """hidden, table, targets, grad, banned: every third row and one whole tile of the table."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    h = torch.randn((n, d), generator=g, device="cuda").to(dtype)
    w = (torch.randn((v, d), generator=g, device="cuda") * (2.0 / math.sqrt(d))).to(dtype)
    banned = torch.arange(v, device="cuda") % 3 == 1
    banned[256:384] = True
    h[:, -1], w[:, -1] = 1.0, torch.where(banned, -float("inf"), 0.0)
    free = (~banned).nonzero()[:, 0]
    t = free[torch.randint(0, free.numel(), (n,), generator=g, device="cuda")]
    if n > 2:
        t[n // 2] = -100
    return h, w, t, (torch.rand((n,), generator=g, device="cuda") + 0.5) / n, banned


def without_banned(h, w, t, grad, banned):
    """_head_ref's values and bounds over the rows that are not banned."""
    at = torch.cumsum(~banned, 0) - 1
    return ref.xent(h, w[~banned], torch.where(t >= 0, at[t.clamp(min=0)], t), grad=grad)


def check_forward(n, v, d, dtype):
    h, w, t, grad, banned = banned_table(n, v, d, dtype, 1)
    loss, lse = tt.tt_emb_xent_forward(h, w, t)
    ref.check({"loss": loss, "lse": lse}, without_banned(h, w, t, grad, banned))


NANS = [0x7FC00000, 0x7FFFFFFF, -1]  # a library's, this GPU's, the same with a sign


def check_nan(n, v, d, bits):
    """fp32: a NaN of these bits in the table makes every row NaN, in one hidden row that row."""
    h, w, t, _, _ = banned_table(n, v, d, torch.float32, 2)
    w = w[:, :-1].contiguous()
    h = h[:, :-1].contiguous()
    bad = w.clone()
    bad.view(torch.int32)[v // 2, 3] = bits
    assert torch.isnan(tt.tt_emb_xent_forward(h, bad, t)[1]).all()
    bad = h.clone()
    bad.view(torch.int32)[n - 1, d // 2] = bits
    lse = tt.tt_emb_xent_forward(bad, w, t)[1]
    assert torch.isnan(lse[n - 1]) and not torch.isnan(lse[:n - 1]).any()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,v,d", [(1, 1000, 256), (4, 1000, 64), (8, 3000, 320), (16, 2000, 300), (5, 700, 31)])
def test_few_rows_forward(n, v, d, dtype):
    check_forward(n, v, d, dtype)


@pytest.mark.parametrize("bits", NANS)
@pytest.mark.parametrize("n,v,d", [(1, 1000, 257), (8, 500, 65), (16, 2000, 301)])
def test_nan_in_few_rows(n, v, d, bits):
    check_nan(n, v, d, bits)


def test_few_rows_of_the_largest_values():
    """fp32's largest values are not rounded up to infinity."""
    w = torch.zeros((40, 64), device="cuda")
    w[3, 5], w[4, 5] = torch.finfo(torch.float32).max, torch.finfo(torch.float32).min
    h = torch.full((2, 64), 2.0 ** -126, device="cuda")
    lse = tt.tt_emb_xent_forward(h, w, torch.zeros(2, dtype=torch.int64, device="cuda"))[1]
    want = torch.logsumexp(ref.scores(h, w), 1)  # a score of 4, one of -4, 38 of 0
    assert ((lse.double() - want).abs() <= 2.0 ** -9 * 4).all()  # the largest values enter as TF32 holds them, cut: 2^-10


MANY = [(20, 1000, 64), (40, 3000, 128), (130, 2000, 100), (20, 1500, 300), (300, 2000, 200)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,v,d", MANY)
def test_many_rows_forward(n, v, d, dtype):
    check_forward(n, v, d, dtype)


@pytest.mark.parametrize("bits", NANS)
@pytest.mark.parametrize("n,v,d", [(20, 1000, 65), (40, 3000, 129), (20, 1500, 301)])
def test_nan_in_many_rows(n, v, d, bits):
    check_nan(n, v, d, bits)


def check_gradients(h, w, t, grad, banned):
    """The banned rows of dweight are 0, the column of biases aside (0 times -inf) dhidden is what it is without them."""
    loss, lse = tt.tt_emb_xent_forward(h, w, t)
    gh, gw = tt.tt_emb_xent_backward(h, w, t, lse, grad)
    want = without_banned(h, w, t, grad, banned)
    ref.check({"loss": loss, "lse": lse, "grad_weight": gw[~banned]}, want)
    ref.check({"grad_hidden": gh[:, :-1]}, {"grad_hidden": [x[:, :-1] for x in want["grad_hidden"]]})
    assert not gw[banned].any()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,v,d", MANY + [(5, 700, 32), (4, 600, 257), (128, 900, 48), (256, 384, 128)])
def test_gradients(n, v, d, dtype):
    h, w, t, grad, banned = banned_table(n, v, d, dtype, 3)
    t[t < 0] = 0
    check_gradients(h, w, t, grad, banned)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,v,d", MANY + [(5, 700, 32), (4, 600, 257), (128, 900, 48), (256, 384, 128)])
def test_gradients_beside_rows_that_do_not_count(n, v, d, dtype):
    """Rows that do not count, whatever they hold, get 0 in every column, that of the biases too, and give nothing; with none
    that counts dweight is 0."""
    h, w, t, grad, banned = banned_table(n, v, d, dtype, 6)
    t[::3] = -100
    ignored = t < 0
    h[ignored] = torch.tensor([float("nan"), float("inf"), -float("inf"), 0.0], dtype=dtype, device="cuda")[torch.arange(n, device="cuda") % 4][ignored, None]
    lse = tt.tt_emb_xent_forward(h, w, t)[1]
    gh, gw = tt.tt_emb_xent_backward(h, w, t, lse, grad)
    clean = torch.where(ignored[:, None], torch.zeros_like(h), h)
    want = without_banned(clean, w, t, grad, banned)
    assert not gh[ignored].any() and not gw[banned].any()
    ref.check({"grad_weight": gw[~banned]}, want)
    ref.check({"grad_hidden": gh[:, :-1]}, {"grad_hidden": [x[:, :-1] for x in want["grad_hidden"]]})
    t[:] = -100
    gh, gw = tt.tt_emb_xent_backward(h, w, t, tt.tt_emb_xent_forward(h, w, t)[1], grad)
    assert not gh.any() and not gw.any()


def test_an_infinite_hidden_row_is_its_own():
    """An infinity in one hidden row: scores of both infinities there, the others as they are."""
    for n, v, d in MANY:
        h, w, t, _, _ = banned_table(n, v, d, torch.float32, 4)
        h, w = h[:, :-1].contiguous(), w[:, :-1].contiguous()
        clean = tt.tt_emb_xent_forward(h, w, t)[1]
        h[7, 3] = -float("inf")
        lse = tt.tt_emb_xent_forward(h, w, t)[1]
        others = torch.arange(n, device="cuda") != 7
        assert not torch.isfinite(lse[7]) and torch.equal(lse[others], clean[others])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m", [1, 9, 40])
def test_4_bit_scores_of_an_infinity(m, dtype):
    """An infinity in x: the sign of its column's code where that is not 0, NaN where it is."""
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    packed, scales = tt.tt_emb_q4_quantize(torch.randn((300, 96), generator=g, device="cuda"), 32)
    x = torch.randn((m, 96), generator=g, device="cuda").to(dtype)
    x[0, 40] = float("inf")
    got = tt.tt_emb_q4_matvec(x, packed, scales, 32)
    column = ref.unpack_q4(packed, scales, 96, 32)[:, 40]
    assert torch.equal(got[0] == float("inf"), column > 0) and torch.equal(got[0] == -float("inf"), column < 0)
    assert torch.equal(torch.isnan(got[0]), column == 0)
    if m > 1:
        want, bound = ref.q4(x[1:], packed, scales, 32)
        assert ((got[1:].double() - want).abs() <= bound).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("group", [32, 64, 128])
def test_4_bit_tables_of_infinities_and_nan(group, dtype):
    """An infinite element keeps its sign and outweighs its group; a NaN makes its row's scores NaN; other rows are as they are."""
    g = torch.Generator(device="cuda")
    g.manual_seed(7)
    w = torch.randn((200, 150), generator=g, device="cuda").to(dtype)
    x = torch.randn((3, 150), generator=g, device="cuda").to(dtype)
    packed, scales = tt.tt_emb_q4_quantize(w, group)
    clean = tt.tt_emb_q4_matvec(x, packed, scales, group)
    bad = w.clone()
    bad[5, 149], bad[6, 0], bad[7, 70] = -float("inf"), float("inf"), float("nan")
    bad[8, 3], bad[8, 149] = float("inf"), -float("inf")
    packed, scales = tt.tt_emb_q4_quantize(bad, group)
    got = tt.tt_emb_q4_matvec(x, packed, scales, group)
    inf = torch.full((3,), float("inf"), device="cuda")
    assert torch.equal(got[:, 5], torch.copysign(inf, -x[:, 149].float())) and torch.equal(got[:, 6], torch.copysign(inf, x[:, 0].float()))
    assert torch.isnan(got[:, 7]).all()
    both = torch.copysign(inf, x[:, 3].float()) + torch.copysign(inf, -x[:, 149].float())
    assert torch.equal(torch.isnan(got[:, 8]), torch.isnan(both)) and torch.equal(got[:, 8].nan_to_num(0, 1, -1), both.nan_to_num(0, 1, -1))
    others = torch.ones(200, dtype=torch.bool, device="cuda")
    others[5:9] = False
    assert torch.equal(got[:, others], clean[:, others])
