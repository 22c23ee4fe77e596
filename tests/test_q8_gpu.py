"""Scores against a table in 8-bit integers, on the GPU.

Codes are the exactly rounded quotients and integer sums are exact, so both, and the scores
(one rounding of the sum, one product of the scales, one product of the two), are known to
the last bit: there is no tolerance."""
import math

import pytest
import torch

import tensor_train_compressed_embeddingbag_gb300 as tt

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def quantized(x):
    """(codes, scales) of rows: 127 x / max|x| to the nearest, ties to even; in float64 the quotient's rounding
    cannot make a tie (numerators below 2^32, at least 2^-26 from one otherwise)."""
    y = x.double()
    top = y.abs().amax(1, keepdim=True)
    codes = torch.where(top > 0, torch.round(127.0 * y / torch.where(top > 0, top, torch.ones_like(top))), torch.zeros_like(y))
    return codes, (top[:, 0].float() / torch.full_like(top[:, 0], 127.0).float())


def product(xc, xs, wc, ws):
    total = torch.empty((xc.shape[0], wc.shape[0]), dtype=torch.float64, device="cuda")
    for r in range(0, wc.shape[0], 8192):
        total[:, r:r + 8192] = xc @ wc[r:r + 8192].double().t()
    return total.float() * (xs[:, None] * ws[None])


def table(v, d, seed=0, most=127):
    codes = torch.randint(-most, most + 1, (v, (d + 15) // 16 * 16), generator=gen(seed), device="cuda").to(torch.int8)
    return codes, torch.rand((v,), generator=gen(seed + 1), device="cuda") * 0.01


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,dim", [(0, 4), (1, 1), (3, 5), (33, 31), (100, 129), (70, 640), (5, 5000), (2000, 64), (40, 65536)])
def test_quantize(rows, dim, dtype):
    w = torch.randn((rows, dim), generator=gen(2), device="cuda").to(dtype)
    if rows > 2:
        w[1] = 0
        w[2] = torch.round(w[2].float() * 4).to(dtype) / 2  # halves: ties
        w[2, 0] = 63.5
    codes, scales = tt.tt_emb_q8_quantize(w)
    want, ws = quantized(w) if rows else (w.double(), w[:, 0].float())
    assert codes.shape == (rows, (dim + 15) // 16 * 16)
    assert torch.equal(codes[:, :dim].double(), want) and not codes[:, dim:].any()
    assert torch.equal(scales, ws)
    wide = torch.full((rows, dim + 3), float("nan"), dtype=dtype, device="cuda")
    wide[:, 1:dim + 1] = w
    again = tt.tt_emb_q8_quantize(wide[:, 1:dim + 1])
    assert torch.equal(again[0], codes) and torch.equal(again[1], scales)


def test_codes_next_to_a_tie():
    """Rows whose quotients are ties, or the next numbers to one, for many largest magnitudes."""
    g = gen(3)
    top = torch.rand((4000,), generator=g, device="cuda") * 3 + 0.1
    k = torch.randint(0, 127, (4000, 64), generator=g, device="cuda")
    x = ((k.double() + 0.5) * top.double()[:, None] / 127.0).float()
    x = torch.where(k % 3 == 0, torch.nextafter(x, torch.zeros_like(x)), torch.where(k % 3 == 1, torch.nextafter(x, x * 2), x))
    x = x * torch.where(torch.rand(x.shape, generator=g, device="cuda") < 0.5, -1.0, 1.0)
    x[:, 0] = top
    x = torch.cat([x, x * 2.0 ** -130, x * 2.0 ** 100, torch.round(x * 4096) * 254 / 2])
    codes, scales = tt.tt_emb_q8_quantize(x)
    want, ws = quantized(x)
    assert torch.equal(codes.double(), want) and torch.equal(scales, ws)


@pytest.mark.parametrize("dtype", TYPES)
def test_rows_that_are_not_finite(dtype):
    w = torch.randn((5, 40), generator=gen(4), device="cuda").to(dtype)
    clean = tt.tt_emb_q8_quantize(w)
    w[1, 3], w[1, 4], w[3, 7] = float("inf"), -float("inf"), float("nan")
    codes, scales = tt.tt_emb_q8_quantize(w)
    assert scales[1] == float("inf") and scales[3].isnan()
    assert codes[1].nonzero()[:, 0].tolist() == [3, 4] and codes[1, 3] == 1 and codes[1, 4] == -1
    for r in (0, 2, 4):
        assert torch.equal(codes[r], clean[0][r]) and scales[r] == clean[1][r]
    out = tt.tt_emb_q8_scores(w, *clean)
    assert torch.equal(out[[0, 2, 4]], tt.tt_emb_q8_scores(w[[0, 2, 4]], *clean)) and out[3].isnan().all()
    assert not out[1].isfinite().any()


# rows on both sides of each width of a tile, odd tables, widths of one range and more
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m,v,d", [(1, 1, 1), (1, 129, 16), (2, 50, 33), (5, 1000, 257), (16, 300, 64), (17, 127, 130), (32, 77, 1024), (33, 200, 1025),
                                   (64, 640, 96), (65, 33, 4096), (128, 128, 128), (129, 500, 2050), (192, 257, 100), (193, 400, 1030), (600, 1000, 300),
                                   (3, 20000, 40), (2, 40, 65536), (1000, 20011, 72), (9, 700, 256), (16, 300, 257), (8, 30000, 256),
                                   (12, 60000, 200), (40, 60000, 300), (100, 30000, 1100)])
def test_scores(m, v, d, dtype):
    x = torch.randn((m, d), generator=gen(5), device="cuda").to(dtype)
    codes, scales = table(v, d)  # padding columns hold something
    xc, xs = quantized(x)
    want = product(xc, xs, codes[:, :d], scales)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = tt.tt_emb_q8_scores(x, codes, scales, err=err)
    assert err.item() == 0
    assert torch.equal(got, want)
    into = torch.full((m, v), float("nan"), device="cuda")
    assert tt.tt_emb_q8_scores(x, codes, scales, out=into) is into and torch.equal(into, want)


@pytest.mark.parametrize("m", [4, 20, 50, 100, 129, 192])
def test_long_rows_of_many_tiles(m):
    """Every block takes many tiles of many steps: places of the rings are used hundreds of times."""
    x = torch.randn((m, 4096), generator=gen(20), device="cuda")
    codes, scales = table(60000, 4096)
    xc, xs = quantized(x)
    want = product(xc, xs, codes, scales)
    for _ in range(3):
        assert torch.equal(tt.tt_emb_q8_scores(x, codes, scales), want)


@pytest.mark.parametrize("m", [1, 20, 200])
@pytest.mark.parametrize("d", [1024, 1040, 4000, 20000])
def test_sums_that_fill_the_integers(m, d):
    """Codes of one sign and the largest size: sums past 2^24 (and 2^28), odd ones among them."""
    x = torch.ones((m, d), device="cuda")
    x[:, ::7] = 126 / 127
    codes = torch.full((300, (d + 15) // 16 * 16), 127, dtype=torch.int8, device="cuda")
    codes[1::3] = -128
    codes[2::5, ::3] = 125
    scales = torch.rand((300,), generator=gen(6), device="cuda")
    xc, xs = quantized(x)
    assert torch.equal(tt.tt_emb_q8_scores(x, codes, scales), product(xc, xs, codes[:, :d], scales))


@pytest.mark.parametrize("dtype", TYPES)
def test_strides(dtype):
    for m in (3, 150):
        x = torch.randn((m, 96), generator=gen(7), device="cuda").to(dtype)
        codes, scales = table(500, 96)
        want = tt.tt_emb_q8_scores(x, codes, scales)
        wide = torch.full((m, 109), float("nan"), dtype=dtype, device="cuda")
        wide[:, 5:101] = x
        assert torch.equal(tt.tt_emb_q8_scores(wide[:, 5:101], codes, scales), want)
        assert torch.equal(tt.tt_emb_q8_scores(x.t().contiguous().t(), codes.t().contiguous().t(), scales.repeat_interleave(2)[::2]), want)
        one = x[:1].expand(m, 96)
        assert torch.equal(tt.tt_emb_q8_scores(one, codes, scales), want[:1].expand(m, 500))
    assert tt.tt_emb_q8_scores(x[:0], codes, scales).shape == (0, 500)


def test_a_wait_that_gives_up():
    x = torch.randn((40, 3000), generator=gen(8), device="cuda")
    codes, scales = table(5000, 3000)
    want = tt.tt_emb_q8_scores(x, codes, scales)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    try:
        tt.tt_emb_head_set_wait_limit(0)
        tt.tt_emb_q8_scores(x, codes, scales, err=err)
        assert err.item() & 4
    finally:
        tt.tt_emb_head_set_wait_limit(2 * 10 ** 9)
    err.zero_()
    assert torch.equal(tt.tt_emb_q8_scores(x, codes, scales, err=err), want) and err.item() == 0


def test_tables_past_32_bit_offsets():
    """Codes past 2^31 bytes, scores past 2^31 elements."""
    v, d, m = 36_000_000, 64, 70
    codes = torch.zeros((v, d), dtype=torch.int8, device="cuda")
    codes[-300:] = table(300, d)[0]
    scales = torch.full((v,), 0.5, device="cuda")
    x = torch.randn((m, d), generator=gen(9), device="cuda")
    got = tt.tt_emb_q8_scores(x, codes, scales)
    assert torch.equal(got[:, -300:], product(*quantized(x), codes[-300:], scales[-300:]))
    assert not got[:, :-300].any()


@pytest.mark.parametrize("m", [1, 50, 300])
def test_streams_and_graphs(m):
    x = torch.randn((m, 320), generator=gen(10), device="cuda")
    codes, scales = table(3000, 320)
    want = tt.tt_emb_q8_scores(x, codes, scales)
    apart = x.t().contiguous().t(), codes.t().contiguous().t(), scales.repeat_interleave(2)[::2]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    got = tt.tt_emb_q8_scores(*apart, stream=side)
    junk = [torch.full_like(t, 7) for t in apart]
    side.synchronize()
    assert torch.equal(got, want)
    del junk
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = tt.tt_emb_q8_scores(x, codes, scales)
        graphs.append((graph, out))
    x.normal_(generator=gen(11))
    want = product(*quantized(x), codes, scales)
    for graph, out in graphs:
        graph.replay()
        assert torch.equal(out, want)


def test_two_streams_at_once():
    """Calls that overlap: each has its own workspace and tensor memory."""
    codes, scales = table(20000, 512)
    xs = [torch.randn((m, 512), generator=gen(12 + m), device="cuda") for m in (1, 40, 300, 20)]
    want = [tt.tt_emb_q8_scores(x, codes, scales) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got = [[tt.tt_emb_q8_scores(x, codes, scales, stream=s) for _ in range(5)] for x, s in zip(xs, streams)]
    torch.cuda.synchronize()
    for each, w in zip(got, want):
        for y in each:
            assert torch.equal(y, w)


@pytest.mark.parametrize("dtype", TYPES)
def test_q8_table(dtype):
    """Against the table it was made from: each code is off by at most half a step, of the row's largest magnitude
    over 127, in both operands."""
    v, d = 700, 200
    w = (torch.randn((v, d), generator=gen(13), device="cuda") / math.sqrt(d)).to(dtype)
    served = tt.Q8Table(w)
    x = torch.randn((2, 3, d), generator=gen(14), device="cuda").to(dtype)
    got = served.scores(x)
    assert got.shape == (2, 3, v)
    want = x.double() @ w.double().t()
    sw, sx = w.double().abs().amax(1) / 254, x.double().abs().amax(2, keepdim=True) / 254
    off = sx * w.double().abs().sum(1) + sw * x.double().abs().sum(2, keepdim=True) + d * sx * sw
    assert ((got.double() - want).abs() <= off + 2.0 ** -20 * (x.double().abs() @ w.double().abs().t())).all()
    assert torch.equal(served.scores(x[0, 0]), got[0, 0])
    with pytest.raises(tt.TTError):
        served.scores(x[..., :199])
