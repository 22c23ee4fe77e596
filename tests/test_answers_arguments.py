"""Arguments of the losses of answers, on the host."""
import pytest

import tensor_train_compressed_embeddingbag_gb300 as tt
from tensor_train_compressed_embeddingbag_gb300 import answers

from test_more_operators_abi import _refused, cuda, here  # noqa: F401


@pytest.mark.parametrize("kind", ["hinge", "squared"])
def test_label_smoothing_belongs_to_the_sigmoid_loss(kind, here):  # noqa: F811
    """The others take it and do not use it, as their definitions; what is no share is refused for all."""
    assert answers._preference(0.1, "sigmoid", 0.1, 0.0).label_smoothing == 0.1
    assert answers._preference(0.1, kind, 0.1, 0.0).label_smoothing == 0.0
    for bad in (-0.1, 1.0, float("nan")):
        for k in ("sigmoid", kind):
            _refused(tt.TT_ERR_ARG, tt.tt_emb_preference_forward, cuda(4, 6), kind=k, label_smoothing=bad)
