"""Arguments of the lookups of a dense table, on the host."""
import pytest
import torch

import tensor_train_compressed_embeddingbag_gb300 as tt
from tensor_train_compressed_embeddingbag_gb300 import lookup

from test_more_operators_abi import _refused, cuda, here  # noqa: F401


def test_padding_below_zero_counts_from_the_end(here, monkeypatch):  # noqa: F811
    """As an index does; without one there is none."""
    seen = []
    monkeypatch.setattr(lookup._LookupFunction, "apply", lambda w, ids, scale, pad, err: seen.append(pad) or torch.zeros((ids.shape[0], w.shape[1])))
    ids, w = torch.zeros(4, dtype=torch.int64), cuda(10, 8)
    for given, want in ((None, -1), (0, 0), (9, 9), (-1, 9), (-10, 0)):
        tt.vocab_embedding(ids, w, padding_idx=given)
        assert seen.pop() == want
    _refused(tt.TT_ERR_SHAPE, tt.vocab_embedding, ids, w, padding_idx=-11)
    for bad in (None, [[1.0]], torch.zeros(2, 3)):
        _refused(tt.TT_ERR_ARG, tt.vocab_embedding, ids, bad, padding_idx=-1)
    _refused(tt.TT_ERR_SHAPE, tt.vocab_embedding, ids, cuda(8), padding_idx=-1)
