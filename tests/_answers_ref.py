"""Plain float64 definitions of the losses of answers, and how far the kernels may be from them.

Error bounds, e = 2^-24 a rounding of fp32.
  d, y       differences of two fp32 numbers: e |d|
  sums       eight terms at a time in fp32, then double: 8 e sum |terms|, plus the terms' errors
  exp        2 units (2^-22 of itself), and what an error of its argument makes of it; the ratio's: that of
             the difference, and e |x| of rounding x log2(e) (x log2(e) 2^-24 in the exponent of 2 is x 2^-24 in that of e)
  others     a few fp32 operations on numbers of one size: 2^-21 of it
"""
import math

import torch

E = 2.0 ** -24


def layout(shape, offsets, mask):
    """(sequence of every token that counts, indices of these tokens, sequences)."""
    n = math.prod(shape)
    if offsets is None:
        count = shape[0]
        of = torch.arange(n, device="cuda") // max(1, n // count if count else 1)
        keep = torch.ones(n, dtype=torch.bool, device="cuda")
    else:
        count = offsets.shape[0] - 1
        of = torch.searchsorted(offsets, torch.arange(n, device="cuda"), right=True) - 1
        keep = of < count
    if mask is not None:
        keep = keep & (mask.reshape(-1) != 0)
    at = keep.nonzero()[:, 0]
    return of[at], at, count


def _sum(of, x, count):
    return torch.zeros(count, dtype=torch.float64, device="cuda").index_add_(0, of, x)


def _share(of, count, average):
    n = torch.bincount(of, minlength=count) if count else torch.zeros(0, dtype=torch.int64, device="cuda")
    return n, (1.0 / n.clamp(min=1).double() if average else torch.ones(count, dtype=torch.float64, device="cuda"))


def preference(logp, reference, mask, offsets, beta, kind, label_smoothing, margin, average, grad=None):
    """{name: (value, bound)}; hinge margins within their bound of 1 are allowed either side."""
    of, at, count = layout(logp.shape, offsets, mask)
    d = logp.reshape(-1)[at].double() - (0.0 if reference is None else reference.reshape(-1)[at].double())
    n, share = _share(of, count, average)
    scale = beta * share
    rewards = scale * _sum(of, d, count)
    er = scale * 9 * E * _sum(of, d.abs(), count)
    p = count // 2
    h = rewards[:p] - rewards[p:] - margin
    eh = er[:p] + er[p:] + E * h.abs()
    s = label_smoothing
    up, down = torch.sigmoid(h), torch.sigmoid(-h)
    if kind == "sigmoid":
        loss = (1 - s) * torch.nn.functional.softplus(-h) + s * torch.nn.functional.softplus(h)
        el = eh + 2.0 ** -21 * (1 + h.abs())
        slope = s * up - (1 - s) * down
        es = (2.0 ** -21 + eh) * (s * up + (1 - s) * down)
    elif kind == "hinge":
        loss, el = (1 - h).clamp(min=0), eh + 2.0 ** -23 * (1 + h.abs())
        slope, es = -(h < 1).double(), ((h - 1).abs() <= eh).double()
    else:
        v = (h - 0.5) / beta
        ev = eh / beta + 2.0 ** -22 * v.abs()
        loss, el = v * v, 2 * v.abs() * ev + ev * ev + 2.0 ** -22 * v * v
        slope, es = 2 * v / beta, 2 * ev / beta + 2.0 ** -21 * (2 * v / beta).abs()
    tiny = 2.0 ** -149
    out = {"loss": (loss, el + tiny), "margins": (h, eh + tiny), "rewards": (rewards, er + E * rewards.abs() + tiny), "counts": (n, torch.zeros_like(n))}
    if grad is not None:
        c = grad.double() * slope * beta
        ec = (grad.double().abs() * es * beta + 2.0 ** -21 * c.abs() + tiny)
        c, ec = torch.cat([c, -c]) * share, torch.cat([ec, ec]) * share
        out["grad"] = _put(logp, at, c[of], ec[of] + 2.0 ** -22 * c[of].abs())
    return out


def _put(logp, at, value, bound):
    g = torch.zeros(logp.numel(), dtype=torch.float64, device="cuda")
    b = torch.zeros_like(g)
    g[at], b[at] = value, bound
    return g.reshape(logp.shape), b.reshape(logp.shape)


def policy(logp, old, adv, reference, mask, offsets, clip, dual_clip, kl, kl_weight, level, average, per_token, grad=None):
    of, at, count = layout(logp.shape, offsets, mask)
    n, share = _share(of, count, average)
    lp = logp.reshape(-1)[at].double()
    d = lp - old.reshape(-1)[at].double()
    mean = _sum(of, d, count) / n.clamp(min=1)
    em = 9 * E * _sum(of, d.abs(), count) / n.clamp(min=1) + E * mean.abs()
    a = (adv.reshape(-1)[at] if per_token else adv[of]).double()
    x, ex = (mean[of], em[of]) if level == "sequence" else (d, E * d.abs())
    low, high = clip
    over = ((a > 0) & (x > math.log1p(high))) | ((a < 0) & (x < math.log1p(-low)))
    bound = torch.where(a > 0, 1.0 + high, 1.0 - low)
    if dual_clip:
        twice = (a < 0) & (x > math.log(dual_clip))
        over, bound = over | twice, torch.where(twice, torch.full_like(bound, dual_clip), bound)
    ratio = torch.exp(x)
    term = -a * torch.where(over, bound, ratio)
    et = term.abs() * (torch.where(over, torch.zeros_like(ex), ex + E * x.abs()) + 2.0 ** -22)
    slope, eslope = torch.where(over, torch.zeros_like(term), term), torch.where(over, torch.zeros_like(et), et)
    k, kslope, ek, ekslope = (torch.zeros_like(lp) for _ in range(4))
    if reference is not None:
        y = reference.reshape(-1)[at].double() - lp
        if kl == "k1":
            k, kslope, ek = -y, torch.ones_like(y), E * y.abs()
        elif kl == "k2":
            k, kslope, ek, ekslope = y * y / 2, -y, 2.0 ** -22 * y * y, E * y.abs()
        else:
            m = torch.expm1(y)
            k, kslope = m - y, -m
            ek = m.abs() * E * y.abs() + 2.0 ** -21 * torch.where(y.abs() <= 1.001, k, torch.exp(y) + 1 + y.abs())
            ekslope = torch.exp(y) * E * y.abs() + 2.0 ** -21 * torch.where(y.abs() <= 1.001, k + y.abs(), torch.exp(y) + 1)
    add = 8 * E
    skl = share * _sum(of, k, count)
    ekl = share * _sum(of, ek + add * k.abs(), count)
    loss = share * _sum(of, term, count) + kl_weight * skl
    el = share * _sum(of, et + add * term.abs(), count) + kl_weight * (ekl + E * skl.abs())
    tiny = 2.0 ** -149
    clipped = _sum(of, over.double(), count)
    out = {"loss": (loss, el + E * loss.abs() + tiny), "kl": (skl, ekl + E * skl.abs() + tiny), "log_ratio": (mean, em + tiny),
           "counts": (n, torch.zeros_like(n)), "clipped": (clipped, torch.zeros_like(clipped))}
    if grad is not None:
        g = (grad.double() * share)[of]
        value = slope + kl_weight * kslope
        off = eslope + kl_weight * (ekslope + E * kslope.abs()) + 2.0 ** -23 * (slope.abs() + kl_weight * kslope.abs())
        out["grad"] = _put(logp, at, g * value, g.abs() * (off + 2.0 ** -22 * value.abs()) + tiny)
    return out


def check(got, want):
    for name, value in got.items():
        exact, bound = want[name]
        assert value.shape == exact.shape, name
        bad = ~((value.double() - exact.double()).abs() <= bound)
        assert not bad.any(), (name, int(bad.sum()), bad.numel(), value[bad][:3], exact[bad][:3], bound[bad][:3])
