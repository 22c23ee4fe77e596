"""Rows of one batch whose weights (the gradients of their losses) are of very different size: dhidden of a row is as
exact as if the row were alone.

The bound is _head_ref.py's, but for what lies below the smallest f16 after scaling, which goes by the row's own weight:
2^-24 with the row's |g| at 2^14 or just below, hence 2^-38 |g_n| an element of dz, not of the batch's largest."""
import math

import pytest
import torch

import tensor_train_compressed_embeddingbag_gb300 as tt

import _head_ref as ref

pytestmark = pytest.mark.gpu


def hidden_bound(h, w, q, g, temp):
    """(grad_hidden, its bound) for a distribution q of every row's target and row weights g."""
    dt = h.dtype
    u = ref.U[dt]
    z = ref.scores(h, w, temp)
    lse = torch.logsumexp(z, 1)
    ez, el = ref.bounds(h, w, lse, temp)
    g = torch.where(q.sum(1) > 0, g.double() * temp, torch.zeros_like(lse))[:, None]
    p = torch.exp(z - lse[:, None])
    dz = g * (p - q)
    edz = g.abs() * (p * 2 * (ez + el)[:, None] + q * 2.0 ** -20) + (u if u else 2.0 ** -21) * dz.abs()
    if dt != torch.bfloat16:
        edz = edz + 2.0 ** -38 * g.abs()
    a = w.double().abs()
    gh = dz @ w.double()
    tiny = 2.0 ** -25 if dt == torch.float16 else 1e-40
    return gh, edz @ a + (3 * 2.0 ** -22 + w.shape[0] * 2.0 ** -27) * (dz.abs() @ a) + (u + 2.0 ** -23) * gh.abs() + tiny


def inputs(n, v, d, dtype, spread, largest, seed):
    """Row n's weight is 2^(spread n / (rows - 1)) of the largest; the table's rows have a common part, so that every
    row's gradient has one that no target gives."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    h = torch.randn((n, d), generator=g, device="cuda").to(dtype)
    w = ((torch.randn((v, d), generator=g, device="cuda") + 1.0) * (2.0 / math.sqrt(d))).to(dtype)
    t = torch.randint(0, v, (n,), generator=g, device="cuda")
    t[n // 2] = -100
    grad = largest * torch.exp2(torch.linspace(0.0, -spread, n, device="cuda"))
    return h, w, t, grad[torch.randperm(n, generator=g, device="cuda")] * (torch.randint(0, 2, (n,), generator=g, device="cuda") * 2 - 1)


CASES = [(torch.float32, 30, 1.0), (torch.float32, 60, 1.0), (torch.bfloat16, 30, 1.0), (torch.float16, 20, 4096.0)]


@pytest.mark.parametrize("dtype,spread,largest", CASES)
@pytest.mark.parametrize("n,v,d", [(20, 3000, 64), (130, 3000, 64), (130, 3000, 100), (20, 3000, 128), (20, 3000, 200), (130, 3000, 200),
                                   (700, 2000, 136), (130, 100, 32)])
def test_xent(n, v, d, dtype, spread, largest):
    h, w, t, grad = inputs(n, v, d, dtype, spread, largest, 1)
    loss, lse = tt.tt_emb_xent_forward(h, w, t)
    gh, gw = tt.tt_emb_xent_backward(h, w, t, lse, grad)
    q = torch.zeros((n, v), dtype=torch.float64, device="cuda")
    keep = t >= 0
    q[keep.nonzero()[:, 0], t[keep]] = 1.0
    ref.check({"grad_hidden": gh, "grad_weight": gw}, {"grad_hidden": hidden_bound(h, w, q, grad, 1.0),
                                                        "grad_weight": ref.xent(h, w, t, grad=grad)["grad_weight"]})


@pytest.mark.parametrize("dtype,spread,largest", CASES)
@pytest.mark.parametrize("n,v,d,k", [(8, 900, 64, 7), (130, 900, 64, 40), (130, 900, 300, 40), (200, 64, 16, 64)])
def test_distill(n, v, d, k, dtype, spread, largest):
    h, w, _, grad = inputs(n, v, d, dtype, spread, largest, 2)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    ids = torch.randint(0, v, (n, k), generator=g, device="cuda")
    logits = torch.randn((n, k), generator=g, device="cuda")
    ids[3] = -1
    temp = 2.0
    loss, lse = tt.tt_emb_distill_forward(h, w, ids, logits, temp)
    gh, gw = tt.tt_emb_distill_backward(h, w, ids, logits, lse, grad, temp)
    q, _ = ref.teacher(ids, logits, v, temp)
    ref.check({"grad_hidden": gh, "grad_weight": gw}, {"grad_hidden": hidden_bound(h, w, q, grad, temp),
                                                        "grad_weight": ref.distill(h, w, ids, logits, temp, grad)["grad_weight"]})


@pytest.mark.parametrize("d", [64, 128, 200])
def test_a_row_beside_a_much_heavier_one_is_as_it_would_be_alone(d):
    """The light row's dhidden does not depend on the other's weight: bit for bit."""
    h, w, t, _ = inputs(40, 3000, d, torch.float32, 1, 1.0, 4)
    _, lse = tt.tt_emb_xent_forward(h, w, t)
    light = torch.full((40,), 2.0 ** -9, device="cuda")
    heavy = light.clone()
    heavy[7] = 2.0 ** 20
    a, b = (tt.tt_emb_xent_backward(h, w, t, lse, x)[0] for x in (light, heavy))
    rows = torch.arange(40, device="cuda") != 7
    assert torch.equal(a[rows], b[rows])
