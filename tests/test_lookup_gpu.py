"""Rows of a dense table by id and the table's gradient, on the GPU against float64.

Bounds.  u: half a unit in the last place, 2^-24 (fp32), 2^-8 (bf16), 2^-11 (f16).
  out       fp32 product, rounded: (u + 2^-24) |out|
  gradient  c rows in fp32, each addition off by at most 2^-24 of a partial sum, itself at most
            A = sum |g|: c 2^-24 A; times the scale (2^-24) and rounded (u)
  added     one fp32 multiply-add (2^-24 of the result) and the rounding
Half the smallest subnormal number of a type is added."""
import math

import pytest
import torch

import tensor_train_compressed_embeddingbag_gb300 as tt

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]
U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}
# lookups, table, width: no lookups, one, a block's, few and sorted (from 1,025 on), one digit and two and three
SIZES = [(0, 5, 8), (1, 1, 1), (2, 3, 5), (7, 120, 8), (8, 120, 3), (64, 50, 257), (1000, 70, 64), (1024, 4000, 40), (1025, 4000, 40),
         (3000, 2048, 33), (2049, 2049, 64), (5000, 100, 520), (20000, 70000, 16), (4097, 5000000, 8), (40000, 300, 2),
         (90, 5000, 38), (1500, 900, 38), (300, 2000, 2031), (2500, 9000, 102), (12000, 3000, 34)]


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def popular(n, v, seed=0):
    return (torch.rand((n,), generator=gen(seed), device="cuda") ** 3 * v).to(torch.int64).clamp_(max=v - 1)


def f32(x):
    return torch.tensor(x, dtype=torch.float32).item()


def exact_grad(grad, ids, v, scale, pad=-1):
    """(gradient, bound of the sums before the last rounding)."""
    keep = (ids >= 0) & (ids < v) & (ids != pad)
    d = grad.shape[1]
    total = torch.zeros((v, d), dtype=torch.float64, device="cuda").index_add_(0, ids[keep], grad[keep].double())
    size = torch.zeros((v, d), dtype=torch.float64, device="cuda").index_add_(0, ids[keep], grad[keep].double().abs())
    count = torch.bincount(ids[keep], minlength=v).double()[:, None]
    return total * f32(scale), count * 2.0 ** -24 * size * abs(f32(scale))


def check_grad(got, grad, ids, scale, pad=-1, old=None):
    want, off = exact_grad(grad, ids, got.shape[0], scale, pad)
    t = got.dtype
    if old is not None:
        want = want + old.double()
        off = off + 2.0 ** -24 * want.abs()
    bad = ~((got.double() - want).abs() <= off + (U[t] + 2.0 ** -23) * (want.abs() + off) + TINY[t])
    assert not bad.any(), (int(bad.sum()), got[bad][:4], want[bad][:4])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,v,d", SIZES)
def test_rows(n, v, d, dtype):
    w = torch.randn((v, d), generator=gen(1), device="cuda").to(dtype)
    ids = popular(n, v)
    for scale in (1.0, math.sqrt(d)):
        out = tt.tt_emb_lookup_forward(w, ids, scale=scale)
        want = w[ids].double() * f32(scale)
        assert out.shape == (n, d) and out.dtype == dtype
        assert ((out.double() - want).abs() <= (U[dtype] + 2.0 ** -23) * want.abs() + TINY[dtype]).all()
    assert torch.equal(tt.tt_emb_lookup_forward(w, ids), w[ids])  # as they are


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,v,d", SIZES)
def test_gradient(n, v, d, dtype):
    g = torch.randn((n, d), generator=gen(2), device="cuda").to(dtype)
    ids, scale = popular(n, v), 0.7
    got = tt.tt_emb_lookup_backward(g, ids, v, scale=scale)
    check_grad(got, g, ids, scale)
    assert torch.equal(got, tt.tt_emb_lookup_backward(g, ids, v, scale=scale))  # bit for bit
    pad = v // 2
    ids = torch.where(torch.rand((n,), generator=gen(3), device="cuda") < 0.5, torch.full_like(ids, pad), ids)
    g[ids == pad] = float("nan")  # whatever padding holds
    got = tt.tt_emb_lookup_backward(g, ids, v, scale=scale, padding_idx=pad)
    assert not got[pad].any()
    check_grad(got, g, ids, scale, pad)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,v,d", [(0, 9, 8), (5, 40, 8), (900, 60, 70), (3000, 500, 64), (3000, 10, 33)])
def test_added_to_a_gradient(n, v, d, dtype):
    """Rows that are not named are neither read nor written: they hold NaN."""
    g = torch.randn((n, d), generator=gen(4), device="cuda").to(dtype)
    ids = popular(n, v, 5) // 2 * 2
    wide = torch.full((v, d + 8), float("nan"), dtype=dtype, device="cuda")
    into = wide[:, :d]
    named = torch.zeros(v, dtype=torch.bool, device="cuda")
    named[ids] = True
    old = torch.randn((v, d), generator=gen(6), device="cuda").to(dtype)
    into[named] = old[named]
    got = tt.tt_emb_lookup_backward(g, ids, v, scale=-0.1, grad_weight=into)
    assert got is into
    check_grad(into[named], g, torch.cumsum(named, 0)[ids] - 1, -0.1, old=old[named])
    assert into[~named].isnan().all() and wide[:, d:].isnan().all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n", [700, 9000, 70000])
@pytest.mark.parametrize("d", [8, 96, 1030])
def test_one_id_has_all(n, d, dtype):
    """Every chunk is of one id; also with neighbours on both sides, and two ids that meet at a chunk's edge."""
    g = torch.randn((n, d), generator=gen(7), device="cuda").to(dtype)
    ids = torch.full((n,), 3, device="cuda")
    check_grad(tt.tt_emb_lookup_backward(g, ids, 9), g, ids, 1.0)
    ids[::n // 5] = 0
    ids[1] = 8
    check_grad(tt.tt_emb_lookup_backward(g, ids, 9), g, ids, 1.0)
    for edge in (16, 32, 64, 128, 256):
        ids = (torch.arange(n, device="cuda") >= 2 * edge).long()
        check_grad(tt.tt_emb_lookup_backward(g, ids, 2), g, ids, 1.0)


@pytest.mark.parametrize("n", [40, 5000])
def test_ids_outside_the_table(n):
    w = torch.randn((30, 24), generator=gen(8), device="cuda")
    ids = torch.randint(0, 30, (n,), generator=gen(9), device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = tt.tt_emb_lookup_forward(w, ids, err=err)
    g = torch.randn((n, 24), generator=gen(10), device="cuda")
    tt.tt_emb_lookup_backward(g, ids, 30, err=err)
    assert err.item() == 0
    bad = ids.clone()
    bad[5], bad[17], bad[-1] = -1, 30, 1 << 40
    got = tt.tt_emb_lookup_forward(w, bad, err=err)
    assert err.item() == 1
    out[[5, 17, n - 1]] = 0
    assert torch.equal(got, out)
    err.zero_()
    check_grad(tt.tt_emb_lookup_backward(g, bad, 30, err=err), g, bad, 1.0)
    assert err.item() == 1
    all_bad = torch.full((n,), 99, device="cuda")
    assert not tt.tt_emb_lookup_backward(g, all_bad, 30).any()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n", [50, 2000])
def test_strides(n, dtype):
    """Rows apart, unaligned, columns apart, one row for all, ids apart."""
    v, d = 300, 64
    w = torch.randn((v, d), generator=gen(11), device="cuda").to(dtype)
    g = torch.randn((n, d), generator=gen(12), device="cuda").to(dtype)
    ids = popular(n, v, 13)
    want, grad = w[ids], tt.tt_emb_lookup_backward(g, ids, v)
    apart = ids.repeat_interleave(2)[::2]
    for pad, at in ((8, 0), (13, 1), (8, 8), (4, 4), (2, 2), (6, 0)):
        ww = torch.full((v, d + pad), float("nan"), dtype=dtype, device="cuda")
        ww[:, at:at + d] = w
        gg = torch.full((n, d + pad), float("nan"), dtype=dtype, device="cuda")
        gg[:, at:at + d] = g
        assert torch.equal(tt.tt_emb_lookup_forward(ww[:, at:at + d], apart), want)
        check_grad(tt.tt_emb_lookup_backward(gg[:, at:at + d], apart, v), g, ids, 1.0)
    assert torch.equal(tt.tt_emb_lookup_forward(w.t().contiguous().t(), ids), want)
    assert torch.equal(tt.tt_emb_lookup_backward(g.t().contiguous().t(), ids, v), grad)
    one = g[:1].expand(n, d)
    check_grad(tt.tt_emb_lookup_backward(one, ids, v), one, ids, 1.0)


@pytest.mark.parametrize("dtype", TYPES)
def test_infinities_and_nan_stay_in_their_rows(dtype):
    for n in (200, 3000):
        g = torch.randn((n, 40), generator=gen(14), device="cuda").to(dtype)
        ids = popular(n, 50, 15)
        g[3, 7], g[4, 9] = float("inf"), float("nan")
        got = tt.tt_emb_lookup_backward(g, ids, 50)
        assert got[ids[3], 7] == float("inf") and got[ids[4], 9].isnan()
        clean = g.clone()
        clean[3, 7] = clean[4, 9] = 0
        want = tt.tt_emb_lookup_backward(clean, ids, 50)
        got[ids[3], 7], got[ids[4], 9] = want[ids[3], 7], want[ids[4], 9]
        assert torch.equal(got, want)


def test_tables_past_32_bit_offsets():
    v, d = 2_300_000, 1024  # 2.4 * 10^9 elements
    w = torch.zeros((v, d), dtype=torch.bfloat16, device="cuda")
    ids = torch.tensor([v - 1, 5, v - 2, v - 1], device="cuda")
    w[v - 1], w[v - 2], w[5] = 3.0, 2.0, 1.0
    assert torch.equal(tt.tt_emb_lookup_forward(w, ids)[:, 0].float().cpu(), torch.tensor([3.0, 1.0, 2.0, 3.0]))
    del w
    many = torch.cat([ids, torch.arange(7, 3007, device="cuda")])
    for each in (ids, many):
        got = tt.tt_emb_lookup_backward(torch.ones((each.shape[0], d), dtype=torch.bfloat16, device="cuda"), each, v)
        assert (got[v - 1] == 2).all() and (got[v - 2] == 1).all() and (got[5] == 1).all() and not got[v - 3].any()
        rows = got[:, 0].float()
        assert rows.sum().item() == each.shape[0]
        del got


@pytest.mark.parametrize("n", [30, 3000])
def test_graph_capture(n):
    """Captured calls follow what their inputs hold at the replay; two captures share no workspace."""
    v, d = 400, 48
    w = torch.randn((v, d), generator=gen(16), device="cuda")
    ids, g = popular(n, v, 17), torch.randn((n, d), generator=gen(18), device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        tt.tt_emb_lookup_backward(g, ids, v)
    s.synchronize()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            out, grad = tt.tt_emb_lookup_forward(w, ids, scale=2.0), tt.tt_emb_lookup_backward(g, ids, v, scale=2.0)
        graphs.append((graph, out, grad))
    for seed in (19, 20):
        ids.copy_(popular(n, v, seed))
        g.normal_(generator=gen(seed))
        for graph, out, grad in graphs:
            out.fill_(7), grad.fill_(7)
            graph.replay()
            assert torch.equal(out, w[ids] * 2)
            check_grad(grad, g, ids, 2.0)


@pytest.mark.parametrize("n", [30, 3000])
def test_another_stream(n):
    v, d = 400, 48
    w = torch.randn((v, d), generator=gen(21), device="cuda")
    ids, g = popular(n, v, 22), torch.randn((n, d), generator=gen(23), device="cuda")
    want = tt.tt_emb_lookup_forward(w, ids), tt.tt_emb_lookup_backward(g, ids, v)
    apart = w.t().contiguous().t(), ids.repeat_interleave(2)[::2], g.t().contiguous().t()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)  # some 50 ms on the current stream
    got = tt.tt_emb_lookup_forward(apart[0], apart[1], stream=side), tt.tt_emb_lookup_backward(apart[2], apart[1], v, stream=side)
    junk = [torch.full_like(x, 7) for x in apart]
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    torch.cuda.synchronize()
    del junk


@pytest.mark.parametrize("dtype", TYPES)
def test_vocab_embedding(dtype):
    v, d = 50, 24
    w = torch.randn((v, d), generator=gen(24), device="cuda").to(dtype).requires_grad_()
    ids = popular(42, v, 25).reshape(2, 3, 7)
    out = tt.vocab_embedding(ids, w, scale=3.0, padding_idx=1)
    assert out.shape == (2, 3, 7, d)
    assert torch.equal(out, (w[ids].float() * 3).to(dtype))
    weights = torch.randn((2, 3, 7, d), generator=gen(26), device="cuda").to(dtype)
    (out * weights).sum().backward()
    check_grad(w.grad, weights.reshape(-1, d), ids.reshape(-1), 3.0, 1)
    w.grad = None
    tt.vocab_embedding(ids, w).sum().backward()  # an expanded gradient
    check_grad(w.grad, torch.ones((42, d), device="cuda"), ids.reshape(-1), 1.0)
    one = tt.vocab_embedding(torch.tensor(4, device="cuda"), w)
    assert one.shape == (d,) and torch.equal(one, w[4])
    none = tt.vocab_embedding(torch.zeros((0, 5), dtype=torch.int64, device="cuda"), w)
    assert none.shape == (0, 5, d)
    none.sum().backward()


def test_differences():
    """The gradient against differences of a function of the rows."""
    v, d = 7, 5
    w = torch.randn((v, d), generator=gen(27), device="cuda").requires_grad_()
    ids = torch.tensor([0, 3, 3, 6, 0, 0], device="cuda")
    f = lambda x: (tt.vocab_embedding(ids, x, scale=1.5).double() ** 2).sum()  # noqa: E731
    f(w).backward()
    step = 2.0 ** -7
    for i, j in ((0, 0), (3, 2), (6, 4), (1, 1)):
        up, down = w.detach().clone(), w.detach().clone()
        up[i, j] += step
        down[i, j] -= step
        # a square's central difference is its slope; fp32 rows: 2^-22 of the values over the step
        size = 6 * (1.5 * w.detach().abs().max().item() + 1) ** 2
        assert abs((f(up) - f(down)).item() / (2 * step) - w.grad[i, j].item()) <= size * 2.0 ** -21 / step
