"""8-bit scores of rows of many steps, again and again: every call the same exact numbers, and no wait given up.

A hand-over between the kernel's roles that goes wrong shows in single tiles of single calls; the message names them."""
import pytest
import torch

import tensor_train_compressed_embeddingbag_gb300 as tt

from test_q8_gpu import gen, product, quantized, table

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m,calls", [(20, 300), (33, 300), (50, 300), (64, 300), (100, 200), (129, 200), (192, 200), (400, 100)])
def test_every_call_is_exact(m, calls):
    v, d = 60000, 4096
    x = torch.randn((m, d), generator=gen(30), device="cuda")
    codes, scales = table(v, d, 31)
    want = product(*quantized(x), codes, scales)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    wrong = torch.zeros((calls, (v + 127) // 128), dtype=torch.bool, device="cuda")  # by call and table tile
    out = torch.empty((m, v), device="cuda")
    for i in range(calls):
        tt.tt_emb_q8_scores(x, codes, scales, out=out.fill_(float("nan")), err=err)
        bad = (out != want).any(0)
        wrong[i] = torch.nn.functional.pad(bad, (0, -v % 128)).reshape(-1, 128).any(1)
    assert err.item() == 0
    assert not wrong.any(), [(int(i), int(t)) for i, t in wrong.nonzero()[:20]]
