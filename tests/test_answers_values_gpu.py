"""Losses of answers on the GPU: values and gradients of calls at the edges of their definitions."""
import pytest
import torch

import tensor_train_compressed_embeddingbag_gb300 as tt

from test_answers_gpu import inputs, run_preference

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
