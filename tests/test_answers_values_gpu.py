"""Losses of answers on the GPU: values and gradients of calls at the edges of their definitions."""
import pytest
import torch

import tensor_train_compressed_embeddingbag_gb300 as tt

from test_answers_gpu import inputs, run_policy, run_preference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["hinge", "squared"])
def test_label_smoothing_belongs_to_the_sigmoid_loss(kind):
    s = inputs(8, 777, True)
    plain, smoothed = run_preference(s, kind=kind), run_preference(s, kind=kind, label_smoothing=0.1)
    for name in plain:
        assert torch.equal(plain[name], smoothed[name]), name
    logp = s["logp"].requires_grad_()
    both = [tt.preference_loss(logp, s["reference"], s["mask"], s["offsets"], kind=kind, label_smoothing=x) for x in (0.0, 0.1)]
    assert torch.equal(*both) and torch.equal(*[torch.autograd.grad(x, logp)[0] for x in both])


@pytest.mark.parametrize("dual_clip", [None, 1.5])
@pytest.mark.parametrize("per_token", [True, False])
@pytest.mark.parametrize("level", ["token", "sequence"])
def test_advantages_that_are_not_a_number(level, per_token, dual_clip):
    """Whatever the ratio: the loss and the gradient are NaN too, no token counts as clipped, and the others are as they were."""
    if level == "sequence" and per_token:
        pytest.skip("an advantage for each sequence only")
    s = inputs(4, 4 * 9, False, seed=40)
    s["mask"][:] = True
    s["old"] = s["logp"] + torch.tensor([1.0, -1.0, 0.0], device="cuda").repeat(3)  # below the lower border, above the upper and dual_clip, between
    if level == "sequence":
        s["old"] = s["logp"] + torch.tensor([[1.0], [-1.0], [0.0], [1.0]], device="cuda")
    how = dict(per_token=per_token, level=level, dual_clip=dual_clip)
    clean = run_policy(s, **how)
    for row in range(4):
        for at in range(3 if per_token else 1):
            bad = {k: v if v is None else v.clone() for k, v in s.items()}
            if per_token:
                bad["adv"][row, at] = float("nan")
            else:
                bad["seq_adv"][row] = float("nan")
            got = run_policy(bad, **how)
            hit = torch.zeros((4, 9), dtype=torch.bool, device="cuda")
            hit[row, at:at + 1 if per_token else None] = True
            assert torch.equal(got["grad"].isnan(), hit) and torch.equal(got["grad"][~hit], clean["grad"][~hit])
            assert got["loss"][row].isnan() and torch.equal(got["loss"].isnan().sum(), torch.ones((), dtype=torch.int64, device="cuda"))
            x = s["logp"].double() - s["old"].double()
            if per_token:  # (one token's share of the clipped ones)
                over = (s["adv"][row, at] > 0 and x[row, at] > 0.5) or (s["adv"][row, at] < 0 and (x[row, at] < -0.5 or (bool(dual_clip) and x[row, at] > 0.5)))
                assert got["clipped"][row] == clean["clipped"][row] - int(over)
            else:
                assert got["clipped"][row] == 0


def exact_sums(shape, packed, seed):
    """Values of tokens whose sums are known to the last bit: 2^24 and its negative, far apart, and between them multiples
    of 2^-12 below 2^-9; a group of four has one of the large ones or four small, so its fp32 sum is exact, and the total of the
    small ones keeps within 24 bits.  A sum in one fp32 number loses them next to 2^24."""
    sequences, length = shape
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randint(1, 8, shape, generator=g, device="cuda").float() * 2.0 ** -12
    x[:, :4] = 0
    x[:, -4:] = 0
    x[:, 1], x[:, -2] = 2.0 ** 24, -2.0 ** 24
    want = x.double().sum(1)
    assert torch.equal(want.float().double(), want)
    offsets = torch.arange(sequences + 1, device="cuda") * length if packed else None
    return (x.reshape(-1) if packed else x), want, offsets


# one block, pieces of 256 to 2,048 tokens, a sequence of hundreds of pieces; the lengths are multiples of 4
@pytest.mark.parametrize("shape", [(2, 400), (2, 4096), (4, 20000), (2, 400000), (200, 8192), (2, 3_000_000)])
@pytest.mark.parametrize("packed", [False, True])
def test_sums_keep_what_one_float_would_lose(shape, packed):
    """2^24 and 2^-12 are 36 bits apart; the sums keep some 48."""
    x, want, offsets = exact_sums(shape, packed, 50)
    zero, n = torch.zeros_like(x), shape[1]
    rewards = tt.tt_emb_preference_forward(x, zero, offsets=offsets, beta=1.0)[2]
    assert torch.equal(rewards.double(), want)
    # the difference of log probabilities: its mean; inverse counts are good to some 2^-48
    none = torch.zeros(shape[0], device="cuda")
    log_ratio = tt.tt_emb_policy_forward(x, zero, none, offsets=offsets, average=False, level="sequence")[2]
    assert ((log_ratio.double() - want / n).abs() <= (2.0 ** -24 + 2.0 ** -40) * want / n).all()
    # the divergence (k1: log probability less reference), and the clipped term: minus the advantages where all ratios are 1
    loss, kl = tt.tt_emb_policy_forward(zero, zero, -x, reference=-x, offsets=offsets, average=False, kl="k1", kl_weight=1.0, per_token=True)[:2]
    assert torch.equal(kl.double(), want)
    assert ((loss.double() - 2 * want).abs() <= 2.0 ** -24 * 2 * want).all()


@pytest.mark.parametrize("size", [(8, 777, True), (6, 6 * 257, False), (10, 100003, True), (2, 3000001, True), (64, 64 * 5000, False)])
def test_sums_of_differences(size):
    """A difference is rounded once (2^-24 of it), then twice within its group of four (2^-24 of partial sums that are at most the group's
    magnitudes); the two floats and joins below 2^-40 of the magnitudes; the result is rounded to fp32."""
    s = inputs(*size, seed=51)
    got, pol = run_preference(s, beta=1.0), run_policy(s, kl="k1", average=False)
    m = s["mask"].reshape(-1)
    n = m.numel()
    of = (torch.searchsorted(s["offsets"], torch.arange(n, device="cuda"), right=True) - 1 if size[2] else torch.arange(n, device="cuda") // (n // size[0]))[m]

    def check(value, x, over=1.0):
        x = x.reshape(-1)[m]
        total, size_ = (torch.zeros(size[0], dtype=torch.float64, device="cuda").index_add_(0, of, y) / over for y in (x, x.abs()))
        assert ((value.double() - total).abs() <= (3 * 2.0 ** -24 + 2.0 ** -40) * size_ + 1.01 * 2.0 ** -24 * total.abs()).all()

    d = {k: s[k].double() for k in ("logp", "reference", "old")}
    check(got["rewards"], d["logp"] - d["reference"])
    check(pol["log_ratio"], d["logp"] - d["old"], pol["counts"].clamp(min=1).double())
    check(pol["kl"], d["logp"] - d["reference"])


@pytest.mark.parametrize("smoothing", [0.0, 0.1, 0.45])
@pytest.mark.parametrize("kind", ["sigmoid", "hinge", "squared"])
def test_pairs_are_rounded_once(kind, smoothing):
    """Answers of one token, whose rewards are exact but for one product: the loss and the gradient of a pair.

    Two floats keep what leads to them, but for one term of exp: some 2.5 roundings of a number that is at most a
    fifteenth of the result (0.7 for the smallest), 2^-26, and for as much in the logarithm: 2^-25 with the result's own 2^-24
    is a bound for both.  Where the two parts of a smoothed slope cancel, what they lose is of their own size.  The gradient is that
    of the margin which the forward call gave."""
    if kind != "sigmoid" and smoothing:
        pytest.skip("one loss without labels")
    n, beta = 20000, 0.1
    g = torch.Generator(device="cuda")
    g.manual_seed(52)
    size = 10.0 ** torch.linspace(-6, 2.9, n, device="cuda")
    h = size * torch.where(torch.rand((n,), generator=g, device="cuda") < 0.5, -1.0, 1.0)
    logp = torch.cat([h, torch.zeros_like(h)])[:, None]
    how = dict(beta=beta, kind=kind, label_smoothing=smoothing)
    loss, margins, rewards, counts = tt.tt_emb_preference_forward(logp, **how)
    x = beta * h.double()
    assert ((margins.double() - x).abs() <= 1.001 * 2.0 ** -24 * x.abs()).all()
    soft = torch.nn.functional.softplus
    want = {"sigmoid": (1 - smoothing) * soft(-x, threshold=1000.0) + smoothing * soft(x, threshold=1000.0), "hinge": (1 - x).clamp(min=0),
            "squared": ((x - 0.5) / beta) ** 2}[kind]
    # (a difference from 1 or 1/2 of a product that is itself rounded to 2^-47: of the numbers' size)
    assert ((loss.double() - want).abs() <= (2.0 ** -24 + 2.0 ** -25) * want + 2.0 ** -40 * (1 + x.abs()) / (beta if kind == "squared" else 1) ** 2 * (kind != "sigmoid")).all()
    grad = torch.rand((n,), generator=g, device="cuda") + 0.5
    got = tt.tt_emb_preference_backward(logp, margins, counts, grad, **how)[:, 0].double()
    m = margins.double()
    up, down = torch.sigmoid(m), torch.sigmoid(-m)
    slope = {"sigmoid": smoothing * up - (1 - smoothing) * down, "hinge": -(m < 1).double(), "squared": 2 * (m - 0.5) / beta ** 2}[kind]
    parts = (smoothing * up + (1 - smoothing) * down) if kind == "sigmoid" else slope.abs()
    c = grad.double() * beta
    off = c * (1.001 * 2.0 ** -24 * slope.abs() + 2.0 ** -25 * parts) + 2.0 ** -149
    assert ((got[:n] - c * slope).abs() <= off).all() and torch.equal(got[n:], -got[:n])


def test_gradients_of_long_answers_are_rounded_once():
    """A share of one over a number of tokens that is no fp32 number, and a beta that is none."""
    n = 16777217 + 2
    logp = torch.zeros((2, n), device="cuda")
    for beta in (0.1, 0.3, 7.7):
        _, margins, _, counts = tt.tt_emb_preference_forward(logp, beta=beta, average=True)
        assert counts.tolist() == [n, n]
        got = tt.tt_emb_preference_backward(logp, margins, counts, torch.ones(1, device="cuda"), beta=beta, average=True)
        want = -0.5 * beta / n
        assert (got[0] == got[0, 0]).all() and abs(got[0, 0].item() - want) <= (2.0 ** -24 + 2.0 ** -40) * abs(want) and torch.equal(got[1], -got[0])


@pytest.mark.parametrize("kind", ["sigmoid", "hinge", "squared"])
def test_margins_that_are_not_a_number(kind):
    """The loss and the gradient of such a pair are NaN, others are as they were."""
    s = inputs(8, 8 * 30, False, seed=53)
    s["mask"][:] = True
    s["grad"] = s["grad"].abs() + 0.5
    clean = run_preference(s, kind=kind)
    s["logp"][5, 7] = float("nan")  # of the second pair
    got = run_preference(s, kind=kind)
    assert got["loss"].isnan().tolist() == [False, True, False, False] and got["margins"][1].isnan()
    hit = torch.zeros((8, 30), dtype=torch.bool, device="cuda")
    hit[1], hit[5] = True, True
    assert torch.equal(got["grad"].isnan(), hit) and torch.equal(got["grad"][~hit], clean["grad"][~hit])
