"""Lookup, head, losses of answers and 8-bit scores together, as post-training uses them, and the example."""
import importlib.util
import math
import os

import pytest
import torch

import tensor_train_compressed_embeddingbag_gb300 as tt

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def step(table, mix, ids, mask, old, reference, advantage, how):
    """The loss of one tied-table step through the package."""
    rows = tt.vocab_embedding(ids[:, :-1], table, scale=2.0, padding_idx=0)
    hidden = torch.tanh(rows @ mix)
    logp = -tt.vocab_cross_entropy(hidden, table, ids[:, 1:], reduction="none")
    if how == "policy":
        return tt.policy_loss(logp, old, advantage, reference, mask, clip=(0.2, 0.3), kl_weight=0.1, reduction="tokens")
    n = logp.shape[0] // 2
    offsets = torch.arange(2 * n + 1, device="cuda") * logp.shape[1]  # packed, as answers of several lengths are
    return tt.preference_loss(logp.reshape(-1), reference.reshape(-1), mask.reshape(-1), offsets, beta=0.3, label_smoothing=0.1)


def exact(table, mix, ids, mask, old, reference, advantage, how):
    """The same in elementary float64 operations."""
    keep = (ids[:, :-1] != 0)[..., None]
    rows = 2.0 * table[ids[:, :-1]]
    rows = torch.where(keep, rows, rows.detach())
    logp = torch.log_softmax(torch.tanh(rows @ mix) @ table.t(), 2).gather(2, ids[:, 1:, None])[..., 0]
    m = mask.double()
    if how == "policy":
        a = advantage.double()[:, None]
        r = torch.exp(logp - old.double())
        y = reference.double() - logp
        each = -torch.minimum(r * a, r.clamp(0.8, 1.3) * a) + 0.1 * (torch.exp(y) - 1 - y)
        return (each * m).sum() / m.sum()
    s = 0.3 * ((logp - reference.double()) * m).sum(1)
    n = s.shape[0] // 2
    h = s[:n] - s[n:]
    return (-0.9 * torch.nn.functional.logsigmoid(h) - 0.1 * torch.nn.functional.logsigmoid(-h)).mean()


@pytest.mark.parametrize("how", ["policy", "preference"])
def test_a_step_of_a_tied_table(how):
    """Gradients of the table (from both its ends) and of what lies between.  Scores are sums of 48 products below some 8 in
    all, off by at most 2^-20 of that; log probabilities by twice that, losses' slopes and the gradients' own sums by
    as much again: 1e-4 of the largest element is several times their sum."""
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    v, d, rows, length = 300, 48, 16, 20
    table = (torch.randn((v, d), generator=g, device="cuda") * 0.3).requires_grad_()
    mix = (torch.randn((d, d), generator=g, device="cuda") / math.sqrt(d)).requires_grad_()
    ids = torch.randint(0, v, (rows, length), generator=g, device="cuda")
    ids[:, 3] = 0  # padding among them
    mask = torch.rand((rows, length - 1), generator=g, device="cuda") < 0.8
    mask[2] = False
    with torch.no_grad():
        rows_ = tt.vocab_embedding(ids[:, :-1], table, scale=2.0)
        logp = -tt.vocab_cross_entropy(torch.tanh(rows_ @ mix), table, ids[:, 1:], reduction="none")
    old = logp + 0.2 * torch.randn(logp.shape, generator=g, device="cuda")
    reference = logp + 0.2 * torch.randn(logp.shape, generator=g, device="cuda")
    advantage = torch.randn((rows,), generator=g, device="cuda")
    args = ids, mask, old, reference, advantage, how
    loss = step(table, mix, *args)
    got = torch.autograd.grad(loss, (table, mix))
    t64, m64 = table.detach().double().requires_grad_(), mix.detach().double().requires_grad_()
    want_loss = exact(t64, m64, *args)
    want = torch.autograd.grad(want_loss, (t64, m64))
    assert abs(loss.item() - want_loss.item()) <= 1e-5 * (1 + abs(want_loss.item()))
    for a, b in zip(got, want):
        assert (a - b).abs().max() <= 1e-4 * b.abs().max()
    # the same step again, from a graph (torch: no eager graph of the same leaves may live while a backward pass is captured)
    del loss
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.autograd.grad(step(table, mix, *args), (table, mix))
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        again = torch.autograd.grad(step(table, mix, *args), (table, mix))
    for x in again:
        x.zero_()
    graph.replay()
    for a, b in zip(got, again):
        assert torch.equal(a, b)


def test_rollout_and_log_probabilities_agree():
    """Scores of the 8-bit copy give the head's log probabilities up to the quantization: each code is off by at
    most half a step (the row's largest magnitude over 254) in both operands."""
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    table = torch.randn((500, 64), generator=g, device="cuda") * 0.3
    hidden = torch.tanh(torch.randn((40, 64), generator=g, device="cuda"))
    scores = tt.Q8Table(table).scores(hidden)
    ids = scores.argmax(1)
    mine = torch.log_softmax(scores.double(), 1).gather(1, ids[:, None])[:, 0]
    head = -tt.vocab_cross_entropy(hidden, table, ids, reduction="none").double()
    sw, sx = table.double().abs().amax(1) / 254, hidden.double().abs().amax(1, keepdim=True) / 254
    off = sx * table.double().abs().sum(1) + sw * hidden.double().abs().sum(1, keepdim=True) + 64 * sx * sw
    assert ((mine - head).abs() <= 2 * off.amax(1) + 1e-4).all()


def test_the_example_runs():
    spec = importlib.util.spec_from_file_location("post_training", os.path.join(ROOT, "examples", "post_training.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    lines = []
    got = example.main(tokens=500, dim=32, prompts=8, group=4, length=6, steps=3, log=lines.append)
    assert len(lines) == 2 and len(got["rewards"]) == 3 and all(math.isfinite(x) for x in got["rewards"] + got["losses"])
