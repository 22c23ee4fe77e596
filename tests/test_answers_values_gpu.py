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
