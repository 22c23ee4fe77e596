"""Preference and policy losses on the GPU against their definitions in float64 (_answers_ref.py
derives the bounds)."""
import math

import pytest
import torch

import tensor_train_compressed_embeddingbag_gb300 as tt

import _answers_ref as ref

pytestmark = pytest.mark.gpu

# sequences, tokens, packed: nothing, single tokens, one block's, pieces of every length, many short and few long ones
SIZES = [(2, 0, False), (2, 2, False), (2, 0, True), (2, 1, True), (4, 12, False), (8, 777, True), (6, 6 * 255, False), (6, 6 * 257, False),
         (2, 8191, True), (2, 8193, True), (300, 301, True), (400, 2000, True), (2, 2 * 70001, False), (10, 100003, True), (5000, 30000, True),
         (1000, 1000, False), (2, 3000001, True), (64, 64 * 5000, False)]


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def inputs(sequences, tokens, packed, seed=0):
    f = dict(generator=gen(seed), device="cuda")
    shape = (tokens,) if packed else (sequences, tokens // sequences)
    logp = torch.rand(shape, **f).clamp_(min=1e-6).log_()
    s = {"logp": logp, "reference": logp + 0.1 * torch.randn(shape, **f), "mask": torch.rand(shape, **f) < 0.8, "offsets": None}
    if packed:
        cuts = torch.sort(torch.randint(0, tokens + 1, (sequences - 1,), **f)).values
        ends = torch.tensor([0, tokens], device="cuda")
        s["offsets"] = torch.cat([ends[:1], cuts, ends[1:]])
    s["old"] = logp + 0.2 * torch.randn(shape, **f)
    s["adv"] = torch.randn(shape, **f)
    s["seq_adv"] = torch.randn((sequences,), **f)
    s["grad"] = torch.randn((sequences,), **f)
    return s


def run_preference(s, train=True, **how):
    where = dict(mask=s["mask"], offsets=s["offsets"], **how)
    loss, margins, rewards, counts = tt.tt_emb_preference_forward(s["logp"], s["reference"], **where)
    out = {"loss": loss, "margins": margins, "rewards": rewards, "counts": counts}
    if train:
        out["grad"] = tt.tt_emb_preference_backward(s["logp"], margins, counts, s["grad"][:loss.shape[0]], **where)
    return out


def want_preference(s, beta=0.1, kind="sigmoid", label_smoothing=0.0, margin=0.0, average=False):
    return ref.preference(s["logp"], s["reference"], s["mask"], s["offsets"], beta, kind, label_smoothing, margin, average,
                          s["grad"][:s["grad"].shape[0] // 2])


POLICY = dict(clip=(0.2, 0.2), dual_clip=None, kl="k3", kl_weight=0.04, level="token", average=True)


def run_policy(s, per_token=False, **how):
    how = dict(POLICY, **how, mask=s["mask"], offsets=s["offsets"], reference=s["reference"], per_token=per_token)
    adv = s["adv"] if per_token else s["seq_adv"]
    names = ("loss", "kl", "log_ratio", "counts", "clipped")
    out = dict(zip(names, tt.tt_emb_policy_forward(s["logp"], s["old"], adv, **how)))
    out["grad"] = tt.tt_emb_policy_backward(s["logp"], s["old"], adv, out["log_ratio"], out["counts"], s["grad"], **how)
    return out


def want_policy(s, per_token=False, **how):
    how = dict(POLICY, **how)
    return ref.policy(s["logp"], s["old"], s["adv"] if per_token else s["seq_adv"], s["reference"], s["mask"], s["offsets"], per_token=per_token,
                      grad=s["grad"], **how)


KINDS = [dict(), dict(label_smoothing=0.1, beta=0.5), dict(kind="hinge", beta=1.0, margin=0.3), dict(kind="squared", average=True),
         dict(average=True, beta=2.0, margin=0.5)]


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("kind", KINDS)
def test_preference(size, kind):
    s = inputs(*size)
    got = run_preference(s, **kind)
    ref.check(got, want_preference(s, **kind))
    for name, value in run_preference(s, **kind).items():
        assert torch.equal(value, got[name]), name  # bit for bit


HOWS = [dict(), dict(per_token=True, average=False, kl="k1"), dict(kl="k2", clip=(0.1, 0.3), dual_clip=1.5), dict(level="sequence", clip=(0.01, 0.02)),
        dict(level="sequence", average=False, kl_weight=0.0, dual_clip=1.01), dict(per_token=True, kl_weight=2.0, dual_clip=1.1, clip=(0.0, 0.0))]


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("how", HOWS)
def test_policy(size, how):
    s = inputs(*size, seed=1)
    got = run_policy(s, **how)
    ref.check(got, want_policy(s, **how))
    for name, value in run_policy(s, **how).items():
        assert torch.equal(value, got[name]), name


def test_ratios_next_to_the_border():
    """Whether a ratio is clipped goes by the exact difference: pairs whose rounded difference is the rounded border."""
    for clip in ((0.2, 0.2), (0.1, 0.28), (0.0, 0.0)):
        lo, hi = math.log1p(-clip[0]), math.log1p(clip[1])
        g = gen(2)
        old = -torch.rand((4, 4096), generator=g, device="cuda") * 20
        border = torch.tensor([lo, hi, lo, hi], device="cuda")[:, None]
        logp = old + border  # within a rounding of it, some either side
        steps = torch.randint(-2, 3, logp.shape, generator=g, device="cuda")
        logp = torch.where(steps.abs() == 2, torch.nextafter(logp, logp + steps), logp)
        adv = torch.tensor([-1.0, 1.0, 1.0, -1.0], device="cuda")
        out = tt.tt_emb_policy_forward(logp, old, adv, clip=clip, average=False)
        x = logp.double() - old.double()
        over = torch.stack([x[0] < lo, x[1] > hi, x[2] > hi, x[3] < lo])
        assert torch.equal(out[4], over.sum(1).int())
        grad = tt.tt_emb_policy_backward(logp, old, adv, out[2], out[3], torch.ones(4, device="cuda"), clip=clip, average=False)
        assert torch.equal(grad == 0, over)


@pytest.mark.parametrize("size", [(4, 40, False), (40, 40000, False), (40, 39999, True)])
def test_what_masked_places_hold(size):
    s = inputs(*size, seed=3)
    clean = run_preference(s), run_policy(s, per_token=True)
    off = ~s["mask"]
    for i, x in enumerate([float("nan"), float("inf"), -float("inf"), torch.finfo(torch.float32).min]):
        for name in ("logp", "reference", "old", "adv"):
            places = off & (torch.arange(off.numel(), device="cuda").reshape(off.shape) % 4 == i)
            s[name] = torch.where(places, torch.full_like(s[name], x), s[name])
    for a, b in zip(clean, (run_preference(s), run_policy(s, per_token=True))):
        for name in a:
            assert torch.equal(a[name], b[name]), name
    # other types of mask, and none
    as_bytes = dict(s, mask=s["mask"].to(torch.uint8) * 255)
    assert torch.equal(run_preference(as_bytes)["grad"], clean[0]["grad"])


def test_sequences_with_nothing():
    """Masks that leave a sequence, a pair or everything empty."""
    s = inputs(6, 6 * 50, False, seed=4)
    s["mask"][0] = s["mask"][1] = s["mask"][4] = False  # pair 1 has none, pair 0 a rejected one
    for kind in KINDS:
        ref.check(run_preference(s, **kind), want_preference(s, **kind))
    for how in HOWS:
        got = run_policy(s, **how)
        ref.check(got, want_policy(s, **how))
        assert got["loss"][0] == 0 and got["kl"][0] == 0 and got["counts"][0] == 0 and not got["grad"][0].any()
    s["mask"][:] = False
    assert tt.preference_loss(s["logp"], s["reference"], s["mask"]).item() == 0
    assert tt.policy_loss(s["logp"], s["old"], s["seq_adv"], mask=s["mask"]).item() == 0
    assert tt.policy_loss(s["logp"], s["old"], s["seq_adv"], mask=s["mask"], reduction="tokens").item() == 0


def test_tokens_behind_the_last_sequence():
    for tokens, end in ((500, 300), (100000, 99990), (100000, 0)):
        s = inputs(8, tokens, True, seed=5)
        s["offsets"] = (s["offsets"].double() * end / tokens).long()
        for got, want in ((run_preference(s), want_preference(s)), (run_policy(s), want_policy(s))):
            ref.check(got, want)
            assert not got["grad"][s["offsets"][-1]:].any()


def test_malformed_offsets():
    """An error bit, and no access outside the buffers; other calls go on."""
    s = inputs(4, 6000, True, seed=6)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for offsets in ([0, 10, 5, 20, 30], [1, 10, 15, 20, 30], [0, 10, 15, 20, 6001], [0, -1, 15, 20, 30], [0, 1 << 50, 1 << 51, 3, 4]):
        err.zero_()
        bad = dict(s, offsets=torch.tensor(offsets, device="cuda"))
        where = dict(mask=bad["mask"], offsets=bad["offsets"])
        _, margins, _, counts = tt.tt_emb_preference_forward(bad["logp"], bad["reference"], err=err, **where)
        assert err.item() == 2
        tt.tt_emb_preference_backward(bad["logp"], margins, counts, bad["grad"][:2], **where)
        err.zero_()
        out = tt.tt_emb_policy_forward(bad["logp"], bad["old"], bad["seq_adv"], err=err, **where)
        assert err.item() == 2
        tt.tt_emb_policy_backward(bad["logp"], bad["old"], bad["seq_adv"], out[2], out[3], bad["grad"], **where)
    err.zero_()
    tt.tt_emb_policy_forward(s["logp"], s["old"], s["seq_adv"], err=err, mask=s["mask"], offsets=s["offsets"])
    assert err.item() == 0
    ref.check(run_policy(s), want_policy(s))


def test_extreme_numbers():
    """Far ratios, answers of probability 0, margins that are infinite: the formulas' own values, no NaN."""
    one = torch.ones((2, 1), device="cuda")
    inf = float("inf")
    for c, r, want, slope in ((1e4, -1e4, 0.0, 0.0), (-1e4, 1e4, 2e3, -1.0), (0.0, -inf, 0.0, 0.0), (-inf, 0.0, inf, -1.0)):
        logp = torch.tensor([[c], [r]], device="cuda")
        loss, margins, rewards, counts = tt.tt_emb_preference_forward(logp, beta=0.1)
        assert loss.item() == pytest.approx(want)
        grad = tt.tt_emb_preference_backward(logp, margins, counts, one[0], beta=0.1)
        assert torch.equal(grad, torch.tensor([[slope], [-slope]], device="cuda") * 0.1)
    logp = torch.tensor([[-inf, -1.0, -200.0]], device="cuda")
    old = torch.tensor([[-1.0, -1.0, -1.0]], device="cuda")
    for a, loss in ((1.0, -1.0), (-1.0, 0.8 + 1.0 + 0.8)):
        out = tt.tt_emb_policy_forward(logp, old, torch.tensor([a], device="cuda"), average=False)
        assert out[0].item() == pytest.approx(loss)
        grad = tt.tt_emb_policy_backward(logp, old, torch.tensor([a], device="cuda"), out[2], out[3], one[0], average=False)
        assert torch.equal(grad, torch.tensor([[0.0, -a, 0.0]], device="cuda"))
    # k3 of close and far log probabilities, relative to its own size
    y = torch.tensor([0.0, 1e-6, -1e-4, 1e-3, 0.02, -0.3, 0.99, 1.0, -1.0, 1.01, -1.01, 5.0, -30.0, 80.0], device="cuda")
    zero = torch.zeros((y.numel(), 1), device="cuda")
    k = tt.tt_emb_policy_forward(zero, zero, zero[:, 0], reference=y[:, None], per_token=False)[1].double()
    want = sum(y.double() ** i / float(math.factorial(i)) for i in range(2, 40))
    want = torch.where(y.abs() > 4, torch.expm1(y.double()) - y.double(), want)
    assert ((k - want).abs() <= 2.0 ** -21 * want).all()


@pytest.mark.parametrize("size", [(8, 8 * 33, False), (8, 777, True), (80, 80 * 900, False), (80, 70001, True)])
def test_views(size):
    """Slices of larger tensors: unaligned beginnings, rows apart, every second."""
    s = inputs(*size, seed=7)
    want = run_preference(s), run_policy(s, per_token=True)

    def unaligned(x):
        if x is None or x.dtype not in (torch.float32, torch.bool):
            return x
        wide = torch.zeros(x.shape[:-1] + (x.shape[-1] + 3,), dtype=x.dtype, device="cuda")
        wide[..., 1:-2] = x
        return wide[..., 1:-2]

    def apart(x):
        return None if x is None else x.repeat_interleave(2, -1)[..., ::2]

    for view in (unaligned, apart):
        v = {k: view(x) for k, x in s.items()}
        for a, b in zip(want, (run_preference(v), run_policy(v, per_token=True))):
            for name in a:
                assert torch.equal(a[name], b[name]), name


def test_a_stream_of_its_own_and_graphs():
    s = inputs(80, 70001, True, seed=8)
    want = run_policy(s)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    apart = {k: x.repeat_interleave(2)[::2] for k, x in s.items()}
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    how = dict(POLICY, reference=apart["reference"], mask=apart["mask"], offsets=apart["offsets"], stream=side)
    out = tt.tt_emb_policy_forward(apart["logp"], apart["old"], apart["seq_adv"], **how)
    grad = tt.tt_emb_policy_backward(apart["logp"], apart["old"], apart["seq_adv"], out[2], out[3], apart["grad"], **how)
    side.synchronize()
    assert torch.equal(grad, want["grad"]) and torch.equal(out[0], want["loss"])
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        run_policy(s), run_preference(s)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        a, b = run_policy(s), run_preference(s)
    other = inputs(80, 70001, True, seed=9)
    for name, x in other.items():
        s[name].copy_(x)
    graph.replay()
    ref.check(a, want_policy(s))
    ref.check(b, want_preference(s))


@pytest.mark.parametrize("reduction", ["none", "sum", "mean", "tokens"])
def test_policy_loss(reduction):
    s = inputs(12, 12 * 40, False, seed=10)
    s["mask"][3] = False
    logp = s["logp"].requires_grad_()
    loss = tt.policy_loss(logp, s["old"], s["adv"], s["reference"], s["mask"], kl_weight=0.1, reduction=reduction)
    r = torch.exp(logp.double() - s["old"].double())
    term = -torch.minimum(r * s["adv"], r.clamp(0.8, 1.2) * s["adv"])
    y = s["reference"].double() - logp.double()
    each = torch.where(s["mask"], term + 0.1 * (torch.exp(y) - 1 - y), torch.zeros_like(y))
    n = s["mask"].sum(1)
    if reduction == "tokens":
        want = each.sum() / n.sum()
    else:
        want = each.sum(1) / n.clamp(min=1)
        want = want if reduction == "none" else (want.sum() if reduction == "sum" else want.sum() / 11)
    torch.testing.assert_close(loss.double(), want, rtol=2e-6, atol=2e-6)
    weights = torch.linspace(0.5, 1.5, 12, device="cuda") if reduction == "none" else torch.ones((), device="cuda")
    g, = torch.autograd.grad((loss * weights).sum(), logp)
    wg, = torch.autograd.grad((want * weights).sum(), logp)
    torch.testing.assert_close(g, wg, rtol=4e-6, atol=1e-9)


@pytest.mark.parametrize("reduction", ["none", "sum", "mean"])
def test_preference_loss(reduction):
    s = inputs(12, 900, True, seed=11)
    logp = s["logp"].requires_grad_()
    loss = tt.preference_loss(logp, s["reference"], s["mask"], s["offsets"], beta=0.3, label_smoothing=0.2, reduction=reduction)
    of = torch.searchsorted(s["offsets"], torch.arange(900, device="cuda"), right=True) - 1
    d = torch.where(s["mask"], logp.double() - s["reference"].double(), torch.zeros((), dtype=torch.float64, device="cuda"))
    r = 0.3 * torch.zeros(12, dtype=torch.float64, device="cuda").index_add(0, of, d)
    h = r[:6] - r[6:]
    want = -0.8 * torch.nn.functional.logsigmoid(h) - 0.2 * torch.nn.functional.logsigmoid(-h)
    want = want if reduction == "none" else (want.sum() if reduction == "sum" else want.mean())
    torch.testing.assert_close(loss.double(), want, rtol=2e-5, atol=2e-6)
    g, = torch.autograd.grad(loss.sum(), logp)
    wg, = torch.autograd.grad(want.sum(), logp)
    torch.testing.assert_close(g, wg, rtol=1e-5, atol=1e-9)
    with pytest.raises(ValueError):
        tt.preference_loss(logp, reduction="max", offsets=s["offsets"])


@pytest.mark.parametrize("what", ["preference", "token", "sequence"])
def test_differences(what):
    """Gradients against central differences in float64 of the losses' definition at the kernels' precision."""
    s = inputs(4, 4 * 6, False, seed=12)
    one = torch.ones(4, device="cuda")

    def value(logp):
        if what == "preference":
            return tt.tt_emb_preference_forward(logp, s["reference"], beta=0.5)[0].double().sum()
        return tt.tt_emb_policy_forward(logp, s["old"], s["seq_adv"], reference=s["reference"], kl_weight=0.1, level=what, clip=0.9)[0].double().sum()

    logp = s["logp"]
    if what == "preference":
        _, margins, _, counts = tt.tt_emb_preference_forward(logp, s["reference"], beta=0.5)
        g = tt.tt_emb_preference_backward(logp, margins, counts, one[:2], beta=0.5)
    else:
        out = tt.tt_emb_policy_forward(logp, s["old"], s["seq_adv"], reference=s["reference"], kl_weight=0.1, level=what, clip=0.9)
        g = tt.tt_emb_policy_backward(logp, s["old"], s["seq_adv"], out[2], out[3], one, reference=s["reference"], kl_weight=0.1, level=what, clip=0.9)
    step = 2.0 ** -6
    for i, j in ((0, 0), (1, 5), (2, 3), (3, 1)):
        up, down = logp.clone(), logp.clone()
        up[i, j] += step
        down[i, j] -= step
        h = (up[i, j].double() - down[i, j].double()).item()
        # values of some 3 with 2^-21 of error over the step, and step^2 / 6 of a third derivative below 4
        assert abs((value(up) - value(down)).item() / h - g[i, j].item()) <= 2 * 4 * 3 * 2.0 ** -21 / h + 4 * step * step / 6


def test_more_tokens_than_32_bits_of_bytes():
    """A packed batch of 700 million tokens: byte offsets past 2^31."""
    n = 700_000_001
    logp = torch.zeros(n, device="cuda")
    logp[-5:] = 1.0
    offsets = torch.tensor([0, 3, n - 5, n - 2, n], device="cuda")
    loss, margins, rewards, counts = tt.tt_emb_preference_forward(logp, offsets=offsets, beta=1.0)
    assert rewards.tolist() == [0.0, 0.0, 3.0, 2.0] and counts.tolist() == [3, n - 8, 3, 2]
    grad = tt.tt_emb_preference_backward(logp, margins, counts, torch.ones(2, device="cuda"), offsets=offsets, beta=1.0)
    s = torch.sigmoid(torch.tensor([3.0, 2.0]))  # -slope at margins -3 and -2
    assert grad[[0, 3, n - 5, n - 2]].cpu() == pytest.approx(torch.tensor([-s[0], -s[1], s[0], s[1]]), rel=1e-6)
