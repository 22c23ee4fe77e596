"""The vocabulary head on the GPU against its definition in float64 (_head_ref.py, which
derives the bounds): cross entropy, distillation, 4-bit scores."""
import math

import pytest
import torch

import tensor_train_compressed_embeddingbag_gb300 as tt

import _head_ref as ref

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]
# rows, table, width: one of each; a tile and one more; odd widths; each kernel's side
SIZES = [(1, 1, 1), (2, 3, 5), (8, 120, 8), (63, 65, 16), (128, 128, 64), (129, 257, 65), (130, 300, 64), (257, 700, 100),
         (200, 1000, 128), (140, 300, 129), (300, 1500, 200), (40, 260, 1000), (5, 4000, 256), (9, 3000, 320), (3000, 50, 33), (1, 5000, 64)]


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def inputs(n, v, d, dtype, seed=0, spread=2.0):
    g = gen(seed)
    h = torch.randn((n, d), generator=g, device="cuda").to(dtype)
    w = (torch.randn((v, d), generator=g, device="cuda") * (spread / math.sqrt(d))).to(dtype)
    t = torch.randint(0, v, (n,), generator=g, device="cuda")
    t = torch.where(torch.rand((n,), generator=g, device="cuda") < 0.2, torch.full_like(t, -100), t)
    grad = (torch.rand((n,), generator=g, device="cuda") - 0.3) / n  # of both signs
    return h, w, t, grad


def run_xent(h, w, t, grad, **kw):
    loss, lse = tt.tt_emb_xent_forward(h, w, t, **kw)
    gh, gw = tt.tt_emb_xent_backward(h, w, t, lse, grad, **kw)
    assert gh.dtype == h.dtype and gw.dtype == w.dtype
    return {"loss": loss, "lse": lse, "grad_hidden": gh, "grad_weight": gw}


def run_distill(h, w, ids, logits, temp, grad, **kw):
    loss, lse = tt.tt_emb_distill_forward(h, w, ids, logits, temp, **kw)
    gh, gw = tt.tt_emb_distill_backward(h, w, ids, logits, lse, grad, temp, **kw)
    return {"loss": loss, "lse": lse, "grad_hidden": gh, "grad_weight": gw}


def entries(n, v, k, seed=5):
    """Teacher entries with distinct ids, some of them missing, some rows with none."""
    g = gen(seed)
    ids = (torch.randint(0, v, (n, 1), generator=g, device="cuda") + torch.arange(k, device="cuda") * max(1, v // k)) % v
    logits = torch.randn((n, k), generator=g, device="cuda") * 2.0
    have = torch.randint(0, k + 1, (n, 1), generator=g, device="cuda")
    return torch.where(torch.arange(k, device="cuda") < have, ids, torch.full_like(ids, -1)), logits


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("size", SIZES)
def test_xent(size, dtype):
    h, w, t, grad = inputs(*size, dtype)
    ref.check(run_xent(h, w, t, grad), ref.xent(h, w, t, grad=grad))


@pytest.mark.parametrize("dtype", TYPES[1:])
@pytest.mark.parametrize("size", [(1, 5000, 300), (3, 4000, 64), (4, 9000, 200), (31, 2000, 129), (64, 700, 72)])
def test_few_targets_keep_their_low_bits(size, dtype):
    """The bound of the gradients without the 16-bit rounding of dz at the targets: in dweight's
    rows that a target names no entry of dz is rounded, in dhidden all others are."""
    h, w, t, grad = inputs(*size, dtype, seed=21)
    t[0], u = 7, ref.U[dtype]
    t[-1] = t[0]
    got = run_xent(h, w, t, grad)
    z = ref.scores(h, w)
    lse = torch.logsumexp(z, 1)
    keep = t >= 0
    q = torch.zeros_like(z)
    q[keep.nonzero()[:, 0], t[keep]] = 1.0
    g = torch.where(keep, grad.double(), torch.zeros_like(lse))[:, None]
    dz = g * (torch.exp(z - lse[:, None]) - q)
    ez, el = ref.bounds(h, w, lse)
    off = (ez + el + 2.0 ** -20)[:, None] * g.abs() * (torch.exp(z - lse[:, None]) + q) + 2.0 ** -38 * grad.abs().max()
    add = max(size) * 2.0 ** -27  # fp32 accumulation
    hd, wd = h.double(), w.double()
    want = dz.t() @ hd
    bound = u * want.abs() + (off + add * dz.abs()).t() @ hd.abs() + 2.0 ** -25
    rows = t[keep].unique()
    assert ((got["grad_weight"].double() - want).abs() <= bound)[rows].all()
    want = dz @ wd
    bound = u * want.abs() + (off + (add + u * (1 - q)) * dz.abs()) @ wd.abs() + 2.0 ** -25
    assert ((got["grad_hidden"].double() - want).abs() <= bound).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("size,k,temp", [((1, 1, 1), 1, 1.0), ((8, 120, 8), 5, 1.0), ((63, 65, 16), 65, 2.0), ((130, 300, 64), 8, 2.0),
                                         ((129, 257, 65), 32, 4.0), ((140, 300, 129), 100, 0.5), ((7, 900, 256), 64, 2.0),
                                         ((40, 260, 1000), 3, 1.0)])
def test_distill(size, k, temp, dtype):
    h, w, _, grad = inputs(*size, dtype, seed=1)
    ids, logits = entries(size[0], size[1], k)
    ref.check(run_distill(h, w, ids, logits, temp, grad), ref.distill(h, w, ids, logits, temp, grad))


@pytest.mark.parametrize("dtype", TYPES)
def test_pieces_of_the_vocabulary(dtype):
    """Wider than the fused kernels, and more dz than one piece holds (256 MB)."""
    n, v, d = 4096, 33000 if dtype != torch.float32 else 17000, 136
    h, w, t, grad = inputs(n, v, d, dtype, seed=2)
    got = run_xent(h, w, t, grad)
    want = ref.xent(h, w, t, grad=grad)
    ref.check(got, want)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n", [4, 130])
@pytest.mark.parametrize("d", [64, 200])
def test_strides(n, d, dtype):
    """Rows apart, rows that are not 16-byte aligned, columns apart, one row for all, all tensors of one storage."""
    h, w, t, grad = inputs(n, 300, d, dtype, seed=3)
    want = ref.xent(h, w, t, grad=grad)
    wide_h = torch.full((n, d + 8), float("nan"), dtype=dtype, device="cuda")
    wide_h[:, :d] = h
    wide_w = torch.full((300, d + 13), float("nan"), dtype=dtype, device="cuda")
    wide_w[:, 1:d + 1] = w
    ref.check(run_xent(wide_h[:, :d], wide_w[:, 1:d + 1], t, grad), want)
    ref.check(run_xent(h.t().contiguous().t(), w.t().contiguous().t(), t, grad), want)
    one = h[:1].expand(n, d)
    ref.check(run_xent(one, w, t, grad), ref.xent(one, w, t, grad=grad))
    both = torch.cat([h, w])
    ref.check(run_xent(both[:n], both[n:], t, grad), want)
    ref.check(run_xent(h, w, t.repeat_interleave(2)[::2], grad.repeat_interleave(2)[::2]), want)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("size", [(6, 90, 16), (150, 400, 64), (150, 400, 160), (5, 700, 320)])
def test_rows_that_do_not_count(size, dtype):
    """Whatever an ignored row holds, its gradient and what others get from it are 0."""
    h, w, t, grad = inputs(*size, dtype, seed=4)
    t[0], t[-1] = 1, -100
    clean = run_xent(h, w, t, grad)
    bad = h.clone()
    for i, x in enumerate([float("nan"), float("inf"), -float("inf"), 3e4]):
        rows = (t == -100).nonzero()[:, 0][i::4]
        bad[rows] = x
        grad = grad.clone()
        grad[rows] = float("nan")
    got = run_xent(bad, w, t, grad)
    keep = t != -100
    for name in ("grad_weight", "loss"):
        assert torch.equal(got[name], clean[name]), name
    assert torch.equal(got["lse"][keep], clean["lse"][keep])
    assert torch.equal(got["grad_hidden"][keep], clean["grad_hidden"][keep])
    assert not got["grad_hidden"][~keep].any() and not got["loss"][~keep].any()
    none = run_xent(bad, w, torch.full_like(t, -100), grad)
    assert not none["loss"].any() and not none["grad_hidden"].any() and not none["grad_weight"].any()


@pytest.mark.parametrize("dtype", TYPES)
def test_teacher_masks(dtype):
    """Missing entries (whatever their logits hold), logits of -inf and of the type's lowest value, repeated ids, no entry at all."""
    n, v, d, k = 40, 500, 64, 6
    h, w, _, grad = inputs(n, v, d, dtype, seed=6)
    g = gen(7)
    ids = torch.randint(0, v, (n, k), generator=g, device="cuda")
    logits = torch.randn((n, k), generator=g, device="cuda")
    low = torch.finfo(torch.float32).min
    ids[1] = -1                                                     # no entry
    logits[1] = float("nan")
    ids[2, 3:], logits[2, 3:] = -5, float("inf")                    # three entries
    logits[3] = -float("inf")                                       # none that counts
    logits[4, :5] = -float("inf")                                   # one
    logits[5] = low                                                 # all equal
    logits[6, 1:] = low                                             # one, the others underflow
    ids[7] = ids[7, 0]                                              # one id six times
    ids[8, 1], ids[8, 3] = ids[8, 0], ids[8, 2]
    ids[9] = torch.arange(k, device="cuda")                         # neighbours in one block of targets
    for temp in (1.0, 0.5, 3.0):
        got = run_distill(h, w, ids, logits, temp, grad)
        ref.check(got, ref.distill(h, w, ids, logits, temp, grad))
        assert not got["loss"][[1, 3]].any() and not got["grad_hidden"][[1, 3]].any()
    only = run_distill(h[1:2], w, ids[1:2], logits[1:2], 1.0, grad[1:2])
    assert not only["grad_weight"].any() and not only["grad_hidden"].any() and not only["loss"].any()


def test_a_nan_logit_that_counts_makes_its_row_nan():
    h, w, _, _ = inputs(4, 50, 16, torch.float32, seed=8)
    ids, logits = torch.arange(8, device="cuda").reshape(4, 2), torch.ones((4, 2), device="cuda")
    logits[2, 0] = float("nan")
    loss, _ = tt.tt_emb_distill_forward(h, w, ids, logits)
    assert torch.isnan(loss).tolist() == [False, False, True, False]


@pytest.mark.parametrize("d", [64, 136])
def test_many_targets_in_one_block(d):
    """Every row's target is the same id, and a teacher whose entries fill whole 32 x 32 blocks."""
    h, w, t, grad = inputs(300, 200, d, torch.bfloat16, seed=9)
    t[:] = 77
    ref.check(run_xent(h, w, t, grad), ref.xent(h, w, t, grad=grad))
    ids = torch.arange(200, device="cuda").repeat(300, 1)
    logits = torch.randn((300, 200), generator=gen(10), device="cuda")
    ref.check(run_distill(h, w, ids, logits, 1.0, grad), ref.distill(h, w, ids, logits, 1.0, grad))


@pytest.mark.parametrize("scale", [1e-30, 1e-6, 1e6, 1e15])
def test_fp32_magnitudes(scale):
    """Tables and gradients far from 1: the pieces are scaled by powers of two."""
    h, w, t, grad = inputs(140, 300, 96, torch.float32, seed=11)
    h, w, grad = h / scale, w * scale, grad * scale
    want = ref.xent(h, w, t, grad=grad)
    ref.check(run_xent(h, w, t, grad), want)


def test_fp32_blocks_of_different_size():
    """Rows of the table whose sizes differ by 2^30 between tiles and 2^10 within: bounds that go by the largest of a 128 x 128 block."""
    h, w, t, grad = inputs(140, 520, 200, torch.float32, seed=12)
    size = torch.tensor([2.0 ** -20, 1.0, 2.0 ** -6, 2.0 ** -30, 2.0 ** -10], device="cuda").repeat_interleave(128)[:520, None]
    w = w * size * torch.where(torch.arange(520, device="cuda") % 2 == 0, 1.0, 2.0 ** -10)[:, None]
    got, want = run_xent(h, w, t, grad), ref.xent(h, w, t, grad=grad)
    ref.check(got, want)


def test_extreme_scores():
    """Scores of some hundreds: one probability is 1 and the others underflow."""
    h, w, t, grad = inputs(130, 300, 64, torch.float32, seed=13, spread=200.0)
    ref.check(run_xent(h, w, t, grad), ref.xent(h, w, t, grad=grad))
    h, w, t, grad = inputs(4, 300, 512, torch.bfloat16, seed=13, spread=200.0)
    ref.check(run_xent(h, w, t, grad), ref.xent(h, w, t, grad=grad))


@pytest.mark.parametrize("op", ["xent", "distill"])
@pytest.mark.parametrize("size", [(6, 40, 8), (20, 150, 64), (12, 90, 140)])
def test_gradient_against_differences(op, size):
    """(L(x + e d) - L(x - e d)) / 2e along random directions d.  With s = max |change of a
    score| per unit of e, the third derivative of a row's loss is at most 8 s^3 (a third
    cumulant), so the difference is off by e^2 / 6 of it, and by the two losses' errors / 2e."""
    n, v, dim = size
    h, w, t, _ = inputs(n, v, dim, torch.float32, seed=14)
    g = gen(15)
    grad = torch.rand((n,), generator=g, device="cuda") + 0.5
    ids, logits = entries(n, v, 4)
    temp = 2.0 if op == "distill" else 1.0

    def loss(h, w):
        x, _ = tt.tt_emb_xent_forward(h, w, t) if op == "xent" else tt.tt_emb_distill_forward(h, w, ids, logits, temp)
        return (x.double() * grad.double()).sum().item()

    got = run_xent(h, w, t, grad) if op == "xent" else run_distill(h, w, ids, logits, temp, grad)
    want = ref.xent(h, w, t, grad=grad) if op == "xent" else ref.distill(h, w, ids, logits, temp, grad)
    e = 2.0 ** -6
    for which in (0, 1):
        d = torch.randn((h, w)[which].shape, generator=g, device="cuda")
        d = d / d.norm() * 4
        dh, dw = (d, torch.zeros_like(w)) if which == 0 else (torch.zeros_like(h), d)
        up = [(a + e * b) for a, b in ((h, dh), (w, dw))]
        down = [(a - e * b) for a, b in ((h, dh), (w, dw))]
        slope = (loss(*up) - loss(*down)) / (2 * e)
        name = ("grad_hidden", "grad_weight")[which]
        dot = (got[name].double() * d.double()).sum().item()
        s = (dh.double() @ w.double().t() + h.double() @ dw.double().t()).abs().amax(1) / temp
        noise = (want["loss"][1] * 1.2 * grad.double()).sum().item() / e
        # h +- e d are themselves rounded to fp32: by 2^-24 of an entry, through the gradient
        moved = 2.0 ** -23 / (2 * e) * (got[name].double().abs() * (h, w)[which].double().abs()).sum().item() * 2
        third = e * e / 6 * (8 * s ** 3 * grad.double() * temp * temp).sum().item()
        bound = noise + moved + third + (want[name][1] * d.double().abs()).sum().item()
        assert abs(slope - dot) <= bound, (slope, dot, bound)


def test_targets_outside_the_table():
    h, w, t, grad = inputs(20, 100, 64, torch.bfloat16, seed=16)
    t[3], t[5] = 100, -1
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run_xent(h, w, t, grad, err=err)
    assert err.item() == 1
    t2 = t.clone()
    t2[[3, 5]] = -100
    clean = run_xent(h, w, t2, grad, err=err.zero_())
    assert err.item() == 0
    for name in got:
        assert torch.equal(got[name], clean[name]), name
    # ignore_index may be any value, one inside the table among them
    t[5] = 7
    ref.check(run_xent(h, w, t, grad, ignore_index=7), ref.xent(h, w, t, ignore=7, grad=grad))
    ids, logits = entries(20, 100, 4)
    ids[2, 0] = 100
    got = run_distill(h, w, ids, logits, 1.0, grad, err=err)
    assert err.item() == 1
    ref.check(got, ref.distill(h, w, ids, logits, 1.0, grad))


def test_no_rows():
    w = torch.randn((50, 16), device="cuda")
    h = torch.empty((0, 16), device="cuda")
    t, grad = torch.empty(0, dtype=torch.int64, device="cuda"), torch.empty(0, device="cuda")
    got = run_xent(h, w, t, grad)
    assert got["loss"].shape == (0,) and got["grad_hidden"].shape == (0, 16)
    assert got["grad_weight"].shape == (50, 16) and not got["grad_weight"].any()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("size", [(200, 3000, 64), (300, 2000, 128), (260, 3000, 300), (4, 3000, 512)])
def test_results_repeat(size, dtype):
    """Bit for bit, with other work on the GPU in between and on another stream."""
    h, w, t, grad = inputs(*size, dtype, seed=17)
    ids, logits = entries(size[0], size[1], 16)
    first = run_xent(h, w, t, grad), run_distill(h, w, ids, logits, 2.0, grad)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for again in range(3):
        kw = {"stream": side} if again else {}
        got = run_xent(h, w, t, grad, **kw), run_distill(h, w, ids, logits, 2.0, grad, **kw)
        run_xent(h * 2, w, t, grad)
        torch.cuda.synchronize()
        for a, b in zip(first, got):
            for name in a:
                assert torch.equal(a[name], b[name]), name


def test_graph_capture():
    h, w, t, grad = inputs(200, 700, 64, torch.float32, seed=18)
    run_xent(h, w, t, grad)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run_xent(h, w, t, grad)
    h2, w2, t2, grad2 = inputs(200, 700, 64, torch.float32, seed=19)
    for a, b in ((h, h2), (w, w2), (t, t2), (grad, grad2)):
        a.copy_(b)
    graph.replay()
    torch.cuda.synchronize()
    ref.check(got, ref.xent(h, w, t, grad=grad))


@pytest.mark.parametrize("size,dtype", [((130, 300, 64), torch.float32), ((130, 300, 128), torch.bfloat16), ((130, 300, 200), torch.float16),
                                        ((130, 300, 200), torch.float32)])
def test_wait_that_gives_up(size, dtype):
    """A bound of 0 ns: the waits give up, the error word says so, nothing is left running and the next call is right."""
    h, w, t, grad = inputs(*size, dtype, seed=20)
    _, lse = tt.tt_emb_xent_forward(h, w, t)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    try:
        tt.tt_emb_head_set_wait_limit(0)
        tt.tt_emb_xent_forward(h, w, t, err=err)
        assert err.item() & 4
        err.zero_()
        tt.tt_emb_xent_backward(h, w, t, lse, grad, err=err)
        assert err.item() & 4
    finally:
        tt.tt_emb_head_set_wait_limit(2 * 10 ** 9)
    err.zero_()
    ref.check(run_xent(h, w, t, grad, err=err), ref.xent(h, w, t, grad=grad))
    assert err.item() == 0


@pytest.mark.parametrize("n", [3, 20])
def test_tables_past_32_bit_offsets(n):
    """35 million rows of 64: elements past 2^31.  The scores at the end of the table decide."""
    v, d = 35_000_000, 64
    w = torch.empty((v, d), dtype=torch.float16, device="cuda")
    w.normal_(0, 0.05, generator=gen(21))
    h = torch.randn((n, d), generator=gen(22), device="cuda").to(torch.float16)
    w[-n:] = h * 2  # each row's own score is far above the others
    t = torch.arange(v - n, v, device="cuda")
    loss, lse = tt.tt_emb_xent_forward(h, w, t)
    z = torch.empty(n, dtype=torch.float64, device="cuda").fill_(-float("inf"))
    for r in range(0, v, 1 << 21):
        z = torch.logaddexp(z, torch.logsumexp(h.double() @ w[r:r + (1 << 21)].double().t(), 1))
    own = (h.double() * w[-n:].double()).sum(1)
    a = (h.double().abs() * w[-n:].double().abs()).sum(1)
    bound = (2.0 ** -20 + d * 2.0 ** -27) * a + 2.0 ** -20 * (1 + z.abs())
    assert ((lse.double() - z).abs() <= bound).all()
    assert ((loss.double() - (z - own)).abs() <= 2 * bound).all()


# ---------------------------------------------------------------- autograd


@pytest.mark.parametrize("reduction", ["none", "sum", "mean"])
def test_vocab_cross_entropy(reduction):
    h, w, t, _ = inputs(24, 70, 32, torch.float32, seed=23)
    h3, t2 = h.reshape(4, 6, 32).requires_grad_(), t.reshape(4, 6)
    w = w.requires_grad_()
    loss = tt.vocab_cross_entropy(h3, w, t2, reduction=reduction)
    want = torch.nn.functional.cross_entropy(h.detach().double() @ w.detach().double().t(), t, reduction=reduction)
    assert loss.shape == (t2.shape if reduction == "none" else ())
    torch.testing.assert_close(loss.double().reshape(want.shape), want, rtol=2e-6, atol=2e-6)
    weights = torch.linspace(0.5, 1.5, 24, device="cuda").reshape(4, 6)
    (loss * weights if reduction == "none" else loss).sum().backward()
    scale = weights.reshape(-1) if reduction == "none" else torch.ones(24, device="cuda") / (1 if reduction == "sum" else (t != -100).sum())
    exact = ref.xent(h, w.detach(), t, grad=scale)
    ref.check({"grad_hidden": h3.grad.reshape(24, 32), "grad_weight": w.grad}, exact)


def test_losses_with_nothing_to_count():
    h, w, t, _ = inputs(5, 30, 8, torch.float32, seed=24)
    h.requires_grad_()
    loss = tt.vocab_cross_entropy(h, w, torch.full_like(t, -100))
    loss.backward()
    assert loss.item() == 0 and not h.grad.any()
    ids = torch.full((5, 3), -1, device="cuda")
    assert tt.vocab_distillation(h, w, ids, torch.zeros((5, 3), device="cuda")).item() == 0
    with pytest.raises(ValueError):
        tt.vocab_cross_entropy(h, w, t, reduction="max")


def test_vocab_distillation():
    h, w, _, _ = inputs(30, 200, 32, torch.bfloat16, seed=25)
    ids, logits = entries(30, 200, 8)
    h, w = h.requires_grad_(), w.requires_grad_()
    loss = tt.vocab_distillation(h, w, ids, logits.to(torch.bfloat16), temperature=2.0)
    loss.backward()
    have = (ids >= 0).any(1)
    lg = logits.to(torch.bfloat16).float()
    exact = ref.distill(h.detach(), w.detach(), ids, lg, 2.0, torch.full((30,), 1.0, device="cuda") / have.sum())
    total, off = exact["loss"][0].sum() / have.sum(), exact["loss"][1].sum() / have.sum() + 2.0 ** -20 * exact["loss"][0].sum()
    assert abs(loss.item() - total.item()) <= off.item()
    ref.check({"grad_hidden": h.grad, "grad_weight": w.grad}, exact)


def test_a_tt_table_under_its_own_head():
    """The table's rows as the head's weights: one bag per row, the cores' gradients by autograd against torch's."""
    E, D = 120, 8
    m = tt.TTEmbeddingBag(E, D, [4, 4], [4, 5, 6], [2, 2, 2], sparse=False, sigma=0.3, generator=torch.Generator().manual_seed(3))
    idx = torch.cat([torch.randint(0, E, (24,), generator=gen(26), device="cuda"), torch.arange(E, device="cuda")])
    off = torch.cat([torch.arange(0, 24, 3, device="cuda"), 24 + torch.arange(E, device="cuda")])
    t = torch.randint(0, E, (8,), generator=gen(27), device="cuda")
    out = m(idx, off)
    tt.vocab_cross_entropy(out[:8], out[8:], t).backward()
    got = [c.grad.double() for c in (m.G1, m.G2, m.G3)]
    cores = [c.detach().double().requires_grad_() for c in (m.G1, m.G2, m.G3)]
    full = torch.einsum("iaxb,jbyc,kczd->ijkxyz", *cores).reshape(E, D)
    hidden = full[idx[:24]].reshape(8, 3, D).sum(1)
    torch.nn.functional.cross_entropy(hidden @ full.t(), t).backward()
    for a, b in zip(got, cores):  # the framework's tolerance for its cores
        assert (a - b.grad).abs().max() <= 1e-4 * b.grad.abs().max()


# ---------------------------------------------------------------- 4 bits


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("shape", [(1, 1), (5, 32), (33, 31), (100, 129), (70, 640)])
def test_q4_quantize(shape, group, dtype):
    w = torch.randn(shape, generator=gen(28), device="cuda").to(dtype)
    w[0] = 0
    packed, scales = tt.tt_emb_q4_quantize(w, group)
    v, d = shape
    pad = torch.nn.functional.pad(w.float(), (0, -d % group)).reshape(v, -1, group)
    want = (pad.abs().amax(2) / 7.0).to(torch.bfloat16)
    assert torch.equal(scales, want)
    s = want.float()[:, :, None]
    code = torch.where(s > 0, torch.round(pad / torch.where(s > 0, s, torch.ones_like(s))).clamp(-8, 7), torch.zeros_like(pad))
    code = (code + 8).to(torch.uint8).reshape(v, -1)
    width = -(-d // 32) * 32
    code = torch.nn.functional.pad(code, (0, max(0, width - code.shape[1])), value=8)[:, :width]
    assert torch.equal(packed, code[:, 0::2] | (code[:, 1::2] << 4))
    wide = torch.zeros((v, d + 3), dtype=dtype, device="cuda")
    wide[:, :d] = w
    again = tt.tt_emb_q4_quantize(wide[:, :d], group)
    assert torch.equal(again[0], packed) and torch.equal(again[1], scales)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("m,v,d", [(1, 1, 1), (1, 50, 32), (3, 1000, 257), (8, 77, 64), (9, 333, 130), (17, 100, 4096), (33, 70, 300),
                                   (2, 40, 9000), (65, 33, 96)])
def test_q4_matvec(m, v, d, group, dtype):
    w = torch.randn((v, d), generator=gen(29), device="cuda") / math.sqrt(d)
    packed, scales = tt.tt_emb_q4_quantize(w, group)
    x = torch.randn((m, d), generator=gen(30), device="cuda").to(dtype)
    want, bound = ref.q4(x, packed, scales, group)
    got = tt.tt_emb_q4_matvec(x, packed, scales, group)
    assert got.dtype == torch.float32 and ((got.double() - want).abs() <= bound).all()
    wide = torch.full((m, d + 5), float("nan"), dtype=dtype, device="cuda")
    wide[:, 2:d + 2] = x
    assert torch.equal(tt.tt_emb_q4_matvec(wide[:, 2:d + 2], packed, scales, group), got)
    out = torch.full((m, v), float("nan"), device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert tt.tt_emb_q4_matvec(x, packed, scales, group, out=out, stream=side) is out
    torch.cuda.synchronize()
    assert torch.equal(out, got)


@pytest.mark.parametrize("dtype,scale", [(torch.float32, 1e-25), (torch.float32, 1e20), (torch.bfloat16, 1e-30), (torch.bfloat16, 1e25),
                                         (torch.float16, 1e-3), (torch.float16, 1e3)])
def test_q4_magnitudes(dtype, scale):
    packed, scales = tt.tt_emb_q4_quantize(torch.randn((60, 200), generator=gen(31), device="cuda"), 64)
    x = (torch.randn((4, 200), generator=gen(32), device="cuda") * scale).to(dtype)
    x[1] = 0
    want, bound = ref.q4(x, packed, scales, 64)
    got = tt.tt_emb_q4_matvec(x, packed, scales, 64)
    assert ((got.double() - want).abs() <= bound).all() and not got[1].any()


def test_q4_past_32_bit_offsets():
    v, d = 70_000_000, 64
    packed = torch.full((v, 32), 0x88, dtype=torch.uint8, device="cuda")
    packed[-1] = 0x99  # codes 9: one scale each
    scales = torch.full((v, 1), 0.5, dtype=torch.bfloat16, device="cuda")
    got = tt.tt_emb_q4_matvec(torch.ones((1, d), device="cuda"), packed, scales, 64)
    assert got[0, -1].item() == 32.0 and not got[0, :-1].any()


def test_q4_table():
    w = torch.randn((300, 96), generator=gen(33), device="cuda")
    table = tt.Q4Table(w, 32)
    x = torch.randn((2, 3, 96), generator=gen(34), device="cuda")
    got = table.scores(x)
    assert got.shape == (2, 3, 300)
    want, bound = ref.q4(x.reshape(6, 96), table.packed, table.scales, 32)
    assert ((got.reshape(6, 300).double() - want).abs() <= bound).all()
    # the stored table is within half a step of the dense one, and scale rounding (2^-9 of 7 steps)
    step = torch.repeat_interleave(table.scales.double(), 32, dim=1)
    assert ((ref.unpack_q4(table.packed, table.scales, 96, 32) - w.double()).abs() <= step * (0.5 + 8 * 2.0 ** -8)).all()


# ---------------------------------------------------------------- refusals


def refused(code, call, *args, **kw):
    with pytest.raises(tt.TTError) as e:
        call(*args, **kw)
    assert e.value.code == code


def test_refusals():
    h, w, t, grad = inputs(4, 20, 8, torch.float32, seed=35)
    f, b = tt.tt_emb_xent_forward, tt.tt_emb_xent_backward
    refused(tt.TT_ERR_ARG, f, h.double(), w.double(), t)
    refused(tt.TT_ERR_ARG, f, h, w.half(), t)
    refused(tt.TT_ERR_ARG, f, h.cpu(), w, t)
    refused(tt.TT_ERR_ARG, f, h, w, t.int())
    refused(tt.TT_ERR_ARG, f, h, w, t.cpu())
    refused(tt.TT_ERR_ARG, f, h, w, t, err=torch.zeros(1, device="cuda"))
    refused(tt.TT_ERR_SHAPE, f, h, w[:, :7], t)
    refused(tt.TT_ERR_SHAPE, f, h[0], w, t)
    refused(tt.TT_ERR_SHAPE, f, h, w[:0], t)
    refused(tt.TT_ERR_SHAPE, f, h, w, t[:3])
    lse = f(h, w, t)[1]
    refused(tt.TT_ERR_SHAPE, b, h, w, t, lse[:3], grad)
    refused(tt.TT_ERR_ARG, b, h, w, t, lse, grad.double())
    ids, logits = entries(4, 20, 3)
    d = tt.tt_emb_distill_forward
    refused(tt.TT_ERR_SHAPE, d, h, w, ids[:, 0], logits)
    refused(tt.TT_ERR_SHAPE, d, h, w, ids, logits[:, :2])
    refused(tt.TT_ERR_ARG, d, h, w, ids, logits.double())
    for temp in (0.0, -1.0, float("nan"), float("inf"), 1e-6):
        refused(tt.TT_ERR_ARG, d, h, w, ids, logits, temp)
    many = torch.zeros((4, 1025), dtype=torch.int64, device="cuda")
    refused(tt.TT_ERR_SHAPE, d, h, w, many, many.float())
    packed, scales = tt.tt_emb_q4_quantize(w, 32)
    q = tt.tt_emb_q4_matvec
    refused(tt.TT_ERR_SHAPE, tt.tt_emb_q4_quantize, w, 16)
    refused(tt.TT_ERR_SHAPE, q, h, packed, scales, 48)
    refused(tt.TT_ERR_SHAPE, q, torch.ones((1, 40), device="cuda"), packed, scales, 32)
    refused(tt.TT_ERR_ARG, q, h, packed, scales.float(), 32)
    refused(tt.TT_ERR_ARG, q, h, packed.int(), scales, 32)
    refused(tt.TT_ERR_ARG, q, h, packed, scales, 32, out=torch.empty((4, 21), device="cuda"))
    refused(tt.TT_ERR_ARG, q, h.double(), packed, scales, 32)


# ---------------------------------------------------------------- ranges of fp32


@pytest.mark.parametrize("d", [64, 128, 200])
@pytest.mark.parametrize("small", [1e-30, 1e-34, 1e-38, 3e-41])
@pytest.mark.parametrize("first", [0, 1])
def test_fp32_blocks_far_apart(d, small, first):
    """Every second 256 rows of the table next to nothing (decayed or subnormal rows): scores of one size after scores of
    another, in either order, many times in a block's run of tiles."""
    n, v = 20, 80_000
    h, w, t, grad = inputs(n, v, d, torch.float32, seed=36)
    w = w * torch.where(torch.arange(v, device="cuda") // 256 % 2 == first, 1.0, small)[:, None]
    got = run_xent(h, w, t, grad)
    ref.check(got, ref.xent(h, w, t, grad=grad))


# ---------------------------------------------------------------- few targets


@pytest.mark.parametrize("dtype", TYPES[1:])
@pytest.mark.parametrize("size", [(1, 100, 64), (3, 128, 128), (31, 60, 72), (64, 128, 16), (8, 9, 33), (3, 300, 64), (20, 500, 200)])
def test_few_targets_without_their_rounding(size, dtype):
    """One target for all rows, whose table row alone is large in column 0 (where hidden is 0): that column of dhidden is
    the target's dz times 91, rounded once.  Rounding is monotonic, so it lies between the roundings of the value less and plus
    what fp32 may be off; with dz rounded as well it does not."""
    n, v, d = size
    h, w, _, _ = inputs(*size, dtype, seed=37)
    h[:, 0], w[:, 0] = 0, w[:, 0] * 2.0 ** -10
    w[7, 0] = 91.0
    t = torch.full((n,), 7, device="cuda")
    grad = torch.rand((n,), generator=gen(38), device="cuda") + 0.5
    got = run_xent(h, w, t, grad)["grad_hidden"][:, 0].double()
    want = ref.xent(h, w, t, grad=grad)["grad_hidden"][0][:, 0]
    z = ref.scores(h, w)
    lse = torch.logsumexp(z, 1)
    ez, el = ref.bounds(h, w, lse)
    p = torch.exp(z - lse[:, None])
    off = grad.double() * 2 * (ez + el + 2.0 ** -20) * 91.0 + max(size) * 2.0 ** -27 * want.abs()
    rest = (p * w.double()[:, 0].abs())[:, torch.arange(v, device="cuda") != 7].sum(1)  # the others' dz, rounded
    off = off + ref.U[dtype] * grad.double() * rest
    low, high = (want - off).to(dtype).double(), (want + off).to(dtype).double()
    assert ((low <= got) & (got <= high)).all(), (got, low, high)


# ---------------------------------------------------------------- error words of the autograd functions


@pytest.mark.parametrize("op", ["xent", "distill"])
def test_a_backward_wait_that_gives_up_is_in_the_callers_err(op):
    """The word given to the loss is the backward pass's too: cleared in between, it holds what that found."""
    h, w, t, _ = inputs(130, 300, 64, torch.float32, seed=39)
    ids, logits = entries(130, 300, 4)
    h, w = h.requires_grad_(), w.requires_grad_()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    loss = tt.vocab_cross_entropy(h, w, t, err=err) if op == "xent" else tt.vocab_distillation(h, w, ids, logits, err=err)
    assert err.item() == 0
    try:
        tt.tt_emb_head_set_wait_limit(0)
        loss.backward()
        assert err.item() & 4
    finally:
        tt.tt_emb_head_set_wait_limit(2 * 10 ** 9)


@pytest.mark.parametrize("ignore", [-100, 7])
def test_mean_divides_by_the_rows_that_count(ignore):
    """A target outside the table counts as ignored: in the mean's denominator too."""
    h, w, t, _ = inputs(40, 100, 16, torch.float32, seed=40)
    t = torch.where(t == -100, torch.full_like(t, ignore), t)
    t[3], t[5], t[6], t[8] = 100, -1, 1 << 40, 7
    valid = (t >= 0) & (t < 100) & (t != ignore)
    got = tt.vocab_cross_entropy(h, w, t, ignore_index=ignore)
    want = ref.xent(h, w, t, ignore=ignore)["loss"]
    assert abs(got.item() - (want[0].sum() / valid.sum()).item()) <= (want[1].sum() / valid.sum()).item() + 2.0 ** -20 * got.item()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [16, 200])
def test_no_rows_of_any_type(dtype, d):
    w = torch.randn((50, d), device="cuda").to(dtype)
    h, t, grad = torch.empty((0, d), dtype=dtype, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda"), torch.empty(0, device="cuda")
    ids, logits = torch.empty((0, 3), dtype=torch.int64, device="cuda"), torch.empty((0, 3), device="cuda")
    for got in (run_xent(h, w, t, grad), run_distill(h, w, ids, logits, 2.0, grad)):
        assert got["loss"].shape == got["lse"].shape == (0,) and got["grad_hidden"].shape == (0, d)
        assert got["grad_weight"].shape == (50, d) and not got["grad_weight"].any()
    assert tt.vocab_cross_entropy(h, w, t).item() == 0 and tt.vocab_distillation(h, w, ids, logits).item() == 0
    assert tt.Q4Table(w, 32).scores(h).shape == (0, 50)


# ---------------------------------------------------------------- long rows


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,v,d", [(40, 700, 1100), (200, 2000, 4096), (40, 20000, 8192), (150, 3000, 20001)])
def test_wide_scores_of_one_sign(n, v, d, dtype):
    """All products positive, so every addition of a score's sum is cut the same way where the accumulator cuts: at most one
    unit (2^-23) of the sum per 16 columns within 512 of them, then one rounding (2^-24) per 512.  fp32 operands: 3 x 2^-22."""
    g = gen(41)
    h = torch.rand((n, d), generator=g, device="cuda").to(dtype)
    w = (torch.rand((v, d), generator=g, device="cuda") * (32.0 / d)).to(dtype)
    t = torch.randint(0, v, (n,), generator=g, device="cuda")
    _, lse = tt.tt_emb_xent_forward(h, w, t)
    z = ref.scores(h, w)
    want = torch.logsumexp(z, 1)
    unit = (3 * 2.0 ** -22 if dtype == torch.float32 else 0.0) + 32 * 2.0 ** -23 + (d / 512 + 1) * 2.0 ** -24
    bound = unit * z.amax(1) + 2.0 ** -21 * (1 + want)
    off = (lse.double() - want).abs()
    assert (off <= bound).all(), (off.max().item(), bound.min().item())


@pytest.mark.parametrize("dtype,v,d", [(torch.float32, 35_000_000, 64), (torch.float16, 35_000_000, 64), (torch.bfloat16, 17_000_000, 136)])
def test_gradients_past_32_bit_offsets(dtype, v, d):
    """Both gradients of tables with more than 2^31 elements: dhidden whole, dweight at both ends, around 2^31 elements
    and at the targets."""
    n = 20
    w = torch.empty((v, d), dtype=dtype, device="cuda")
    w.normal_(0, 0.05, generator=gen(42))
    h = torch.randn((n, d), generator=gen(43), device="cuda").to(dtype)
    w[-n:] = h
    t = torch.arange(v - n, v, device="cuda")
    t[:5] = torch.tensor([0, 1, (1 << 31) // d, (1 << 31) // d + 1, v // 2], device="cuda")
    grad = torch.rand((n,), generator=gen(44), device="cuda") + 0.5
    _, lse = tt.tt_emb_xent_forward(h, w, t)
    gh, gw = tt.tt_emb_xent_backward(h, w, t, lse, grad)
    step = 1 << 21
    z = torch.full((n,), -float("inf"), dtype=torch.float64, device="cuda")
    a = torch.zeros_like(z)
    for r in range(0, v, step):
        part = w[r:r + step].double()
        z = torch.logaddexp(z, torch.logsumexp(h.double() @ part.t(), 1))
        a = torch.maximum(a, (h.double().abs() @ part.abs().t()).amax(1))
    ez = (2.0 ** -20 + d * 2.0 ** -27) * a
    el = ez + 2.0 ** -21 * (1 + z.abs())
    assert ((lse.double() - z).abs() <= el).all()
    u, g = ref.U[dtype], grad.double()[:, None]
    want, size, off = (torch.zeros((n, d), dtype=torch.float64, device="cuda") for _ in range(3))

    def dz_of(rows):  # dz of some table rows, how far it may be off
        p = torch.exp(h.double() @ w[rows].double().t() - z[:, None])
        q = (t[:, None] == rows[None]).double()
        dz = g * (p - q)
        return dz, g * (p * 2 * (ez + el)[:, None] + q * 2.0 ** -20) + (u if u else 2.0 ** -21) * dz.abs() + 2.0 ** -38 * g.max()
    for r in range(0, v, step):
        rows = torch.arange(r, min(v, r + step), device="cuda")
        dz, e = dz_of(rows)
        part = w[rows].double()
        want += dz @ part
        size += dz.abs() @ part.abs()
        off += e @ part.abs()
    bound = off + (3 * 2.0 ** -22 + v * 2.0 ** -27) * size + (u + 2.0 ** -23) * want.abs() + 2.0 ** -25
    assert ((gh.double() - want).abs() <= bound).all()
    edge = (1 << 31) // d
    rows = torch.cat([torch.arange(0, 200, device="cuda"), torch.arange(edge - 200, edge + 200, device="cuda"), t, torch.arange(v - 200, v, device="cuda")])
    dz, e = dz_of(rows)
    want = dz.t() @ h.double()
    bound = e.t() @ h.double().abs() + (3 * 2.0 ** -22 + n * 2.0 ** -27) * (dz.abs().t() @ h.double().abs()) + (u + 2.0 ** -23) * want.abs() + 2.0 ** -25
    assert ((gw[rows].double() - want).abs() <= bound).all()
