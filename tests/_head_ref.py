"""Plain float64 definitions of the vocabulary head's operators, and how far the
kernels may be from them.

Error bounds.  u: half a unit in the last place of the 16-bit types, 2^-8 (bf16) and
2^-11 (f16).
  scores   16-bit inputs enter the products exactly, fp32 inputs with 22 bits (each
           operand off by at most 2^-22 of itself, the product of the two remainders
           dropped): 3 x 2^-22.  fp32 accumulation, which may cut instead of round: at
           most one unit (2^-23) of the running sum, itself at most A = sum |h| |w|, per
           16 columns, hence D 2^-27 A; bound 2^-20 A + D 2^-27 A.
  lse      the largest score error, plus fp32 arithmetic of lse itself (2^-21 (1 + |lse|):
           a few roundings, the exponential's and logarithm's units and the sum's)
  loss     error of lse and of the target's score
  dz       p = exp(z - lse) is off by p times the errors of z and lse; rounding to 16 bits
           adds u |dz| (fp32: 2^-21 |dz|); what lies below the smallest f16 after scaling
           (2^-24 with the largest at 2^14) adds 2^-38 of the largest |g|
  gradient sum |dz error| |w|, accumulation as above over the rows of the sum (V or N:
           K 2^-27 sum |dz| |w|), fp32 operands 3 x 2^-22, and the rounding of the result
"""
import torch

U = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def scores(hidden, weight, temp=1.0):
    return hidden.double() @ weight.double().t() / temp


def bounds(hidden, weight, lse, temp=1.0):
    """Bound of the score error of every row (largest over the table), and of its lse."""
    a = (hidden.double().abs() @ weight.double().abs().t()).amax(1) / temp
    ez = (2.0 ** -20 + hidden.shape[1] * 2.0 ** -27) * a
    return ez, ez + 2.0 ** -21 * (1 + lse.abs())


def xent(hidden, weight, targets, ignore=-100, grad=None):
    return _soft(hidden, weight, *_onehot(targets, weight.shape[0], ignore), 1.0, grad)


def _onehot(targets, vocab, ignore):
    q = torch.zeros((targets.shape[0], vocab), dtype=torch.float64, device=targets.device)
    keep = (targets != ignore) & (targets >= 0) & (targets < vocab)
    rows = torch.arange(targets.shape[0], device=targets.device)[keep]
    q[rows, targets[keep]] = 1.0
    return q, torch.zeros(targets.shape[0], dtype=torch.float64, device=targets.device)


def teacher(ids, logits, vocab, temp):
    """(dense q [N, V], sum q log q [N]) of a teacher's entries."""
    have = (ids >= 0) & (ids < vocab) & (logits != -float("inf"))
    t = (logits.double() / temp).masked_fill(~have, -float("inf"))
    q = torch.where(have.any(1, keepdim=True), torch.softmax(t, 1), torch.zeros_like(t)).nan_to_num(0.0)
    dense = torch.zeros((ids.shape[0], vocab), dtype=torch.float64, device=ids.device)
    dense.scatter_add_(1, ids.clamp(0, vocab - 1), torch.where(have, q, torch.zeros_like(q)))
    return dense, torch.where(q > 0, q * torch.log(q.clamp(min=1e-320)), torch.zeros_like(q)).sum(1)


def distill(hidden, weight, ids, logits, temp, grad=None):
    return _soft(hidden, weight, *teacher(ids, logits, weight.shape[0], temp), temp, grad)


def _soft(hidden, weight, q, qlogq, temp, grad):
    """{name: (value, bound)} for targets q (rows sum to 1, or to 0: the row does not count)."""
    mass = q.sum(1)
    keep = mass > 0
    z = scores(hidden, weight, temp)
    lse = torch.logsumexp(z, 1)
    ez, el = bounds(hidden, weight, lse, temp)
    t2 = temp * temp
    loss = torch.where(keep, t2 * (qlogq - (q * z).sum(1) + lse), torch.zeros_like(lse))
    # distillation's own log q and the sum over entries: a few fp32 roundings of their size
    eloss = t2 * (ez + el + 2.0 ** -20 * (1 + qlogq.abs() + (q * z.abs()).sum(1) + lse.abs()))
    out = {"loss": (loss, torch.where(keep, eloss, torch.zeros_like(eloss))), "lse": (lse, el)}
    if grad is None:
        return out
    dt = hidden.dtype
    u = U[dt]
    g = torch.where(keep, grad.double() * temp, torch.zeros_like(lse))[:, None]
    h = torch.where(keep[:, None], hidden.double(), torch.zeros_like(hidden.double()))
    w = weight.double()
    p = torch.exp(z - lse[:, None])
    dz = torch.where(keep[:, None], g * (p - q), torch.zeros_like(p))
    edz = g.abs() * p * 2 * (ez + el)[:, None] + g.abs() * q * 2.0 ** -20 + (u if u else 2.0 ** -21) * dz.abs()
    if dt != torch.bfloat16:
        edz = edz + (2.0 ** -38 * g.abs().max() if g.numel() else 0.0)
    edz = torch.where(keep[:, None], edz, torch.zeros_like(edz))
    more = 3 * 2.0 ** -22
    gh, gw = dz @ w, dz.t() @ h
    eh = edz @ w.abs() + (more + weight.shape[0] * 2.0 ** -27) * (dz.abs() @ w.abs())
    ew = edz.t() @ h.abs() + (more + hidden.shape[0] * 2.0 ** -27) * (dz.abs().t() @ h.abs())
    tiny = 2.0 ** -25 if dt == torch.float16 else 1e-40  # half the smallest f16
    out["grad_hidden"] = (gh, eh + (u + 2.0 ** -23) * gh.abs() + tiny)
    out["grad_weight"] = (gw, ew + (u + 2.0 ** -23) * gw.abs() + tiny)
    return out


def check(got, want):
    for name, value in got.items():
        exact, bound = want[name]
        assert value.shape == exact.shape, name
        off = (value.double() - exact).abs()
        bad = ~(off <= bound)
        assert not bad.any(), (f"{name}: {int(bad.sum())} of {bad.numel()} beyond the bound; worst off "
                               f"{off[bad].max().item():.3e}, bound there {bound[bad].min().item():.3e}")


def unpack_q4(packed, scales, dim, group):
    code = torch.stack((packed & 15, packed >> 4), dim=2).reshape(packed.shape[0], -1)[:, :dim].double() - 8.0
    return code * torch.repeat_interleave(scales.double(), group, dim=1)[:, :dim]


def q4(x, packed, scales, group):
    """(scores, bound): exact products (fp32 x with 22 bits), fp32 sums."""
    w = unpack_q4(packed, scales, x.shape[1], group)
    a = x.double().abs() @ w.abs().t()
    return x.double() @ w.t(), (2.0 ** -20 + x.shape[1] * 2.0 ** -26) * a + 1e-38
