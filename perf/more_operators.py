"""The operators around a table and the vocabulary head, and the cases they are measured on.

  lookup      rows of a dense table by id, times a scale; backward the table's gradient,
              scale times the sum of the rows of grad_out with that id
  preference  loss of pairs of sequences from the log ratios of their tokens (chosen
              against rejected), and the gradient of every token's log probability
  policy      clipped policy loss with a Kullback-Leibler term per sequence, and the same gradient
  q8          scores of rows against a table held in 8-bit integers: a scale for each row of x
              and for each row of the table, exact integer sums

With `own` false, `run` computes the plain form with elementary torch operations, in
float32 (float64 for sums over long sequences, differences next to a border, and the
choice of 8-bit codes); with `own` true it calls the package's operators.
"""
import math

import torch

own = False

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_BYTES = {"f32": 4, "bf16": 2, "f16": 2}


def listed():
    return [
        # one token of a request: launch latency
        {"name": "lookup_token", "op": "lookup", "n": 1, "v": 131072, "d": 2048, "type": "bf16", "train": False, "padded": 0.0},
        # prompts of 16,384 tokens, a wide table
        {"name": "lookup_prompt", "op": "lookup", "n": 16384, "v": 131072, "d": 4096, "type": "bf16", "train": False, "padded": 0.0},
        # the tiny configuration's table (E = 120, D = 8) and batch of 8: one step, launch latency
        {"name": "lookup_train_tiny", "op": "lookup", "n": 8, "v": 120, "d": 8, "type": "f32", "train": True, "padded": 0.0},
        # 512 x 20 lookups of a catalogue of 10^6 items of width 64, the tables' own type: the dense gradient is the cost
        {"name": "lookup_train_items", "op": "lookup", "n": 10240, "v": 1000000, "d": 64, "type": "f32", "train": True, "padded": 0.0},
        # a training batch of tokens, popular ids often, a tenth padding, odd sizes
        {"name": "lookup_train_tokens", "op": "lookup", "n": 65521, "v": 50001, "d": 2048, "type": "bf16", "train": True, "padded": 0.1},
        # four pairs of short answers: launch latency
        {"name": "preference_small", "op": "preference", "pairs": 4, "tokens": 777, "packed": True, "kind": "sigmoid", "smoothing": 0.0,
         "average": False, "train": True},
        # a large batch of long answers, packed one behind the other
        {"name": "preference_long", "op": "preference", "pairs": 1024, "tokens": 4194303, "packed": True, "kind": "sigmoid",
         "smoothing": 0.1, "average": False, "train": True},
        # a group of eight short answers: launch latency
        {"name": "policy_small", "op": "policy", "sequences": 8, "tokens": 8 * 64, "packed": False, "level": "token", "kl": "k3",
         "kl_weight": 0.04, "per_token": False, "average": True, "train": True},
        # rollouts of 1,024 prompts padded to 8,192 tokens, an advantage for every token
        {"name": "policy_rollouts", "op": "policy", "sequences": 1024, "tokens": 1024 * 8192, "packed": False, "level": "token",
         "kl": "k3", "kl_weight": 0.04, "per_token": True, "average": True, "train": True},
        # one token of a request against a wide vocabulary: 537 MB of codes
        {"name": "q8_token", "op": "q8", "m": 1, "v": 131072, "d": 4096, "type": "bf16"},
        # a few dozen requests, odd vocabulary and width
        {"name": "q8_requests", "op": "q8", "m": 33, "v": 50001, "d": 1000, "type": "f16"},
        # held-out rows of a batch against a wide vocabulary: 1.1 T operations
        {"name": "q8_batch", "op": "q8", "m": 2048, "v": 131072, "d": 2048, "type": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["lookup", "preference", "policy", "q8"])
    while True:
        if op == "lookup":
            c = {"op": op, "n": _log(rng, 1, 131072), "v": _log(rng, 50, 2000000), "d": _log(rng, 8, 8192), "type": rng.choice(list(_TYPES)),
                 "train": rng.random() < 0.7, "padded": rng.choice([0.0, 0.1, 0.5])}
            e = _BYTES[c["type"]]
            if c["n"] * c["d"] * e <= 1 << 28 and c["v"] * c["d"] * e <= 1 << 29:
                return c
        elif op == "q8":
            c = {"op": op, "m": _log(rng, 1, 4096), "v": _log(rng, 50, 1000000), "d": _log(rng, 16, 8192), "type": rng.choice(list(_TYPES))}
            if c["v"] * c["d"] <= 1 << 29 and c["m"] * c["v"] <= 1 << 28 and c["m"] * c["v"] * c["d"] <= 1 << 39:
                return c
        else:
            packed, sequences, length = rng.random() < 0.5, 2 * _log(rng, 1, 2048), _log(rng, 1, 32768)
            tokens = sequences * length - (rng.randint(0, sequences - 1) if packed else 0)
            if tokens > 1 << 22:
                continue
            c = {"op": op, "tokens": tokens, "packed": packed, "average": rng.random() < 0.5, "train": rng.random() < 0.8}
            if op == "preference":
                return {**c, "pairs": sequences // 2, "kind": rng.choice(["sigmoid", "sigmoid", "hinge", "squared"]), "smoothing": rng.choice([0.0, 0.1])}
            level = rng.choice(["token", "token", "sequence"])
            return {**c, "sequences": sequences, "level": level, "kl": rng.choice(["k1", "k2", "k3", "k3"]), "kl_weight": rng.choice([0.0, 0.001, 0.04]),
                    "per_token": level == "token" and rng.random() < 0.5}


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    f = dict(generator=g, device="cuda")
    s = dict(case)
    if case["op"] == "lookup":
        n, v, d, t = case["n"], case["v"], case["d"], _TYPES[case["type"]]
        ids = (torch.rand((n,), **f) ** 3 * v).to(torch.int64).clamp_(max=v - 1)  # low ids more often
        s["padding_idx"] = v // 2
        s["ids"] = torch.where(torch.rand((n,), **f) < case["padded"], torch.full_like(ids, v // 2), ids)
        s["weight"] = (torch.randn((v, d), **f) * (1.0 / math.sqrt(d))).to(t)
        s["scale"] = math.sqrt(d)
        if case["train"]:
            s["grad"] = (torch.randn((n, d), **f) * 1e-2).to(t)
        return s
    if case["op"] == "q8":
        m, v, d = case["m"], case["v"], case["d"]
        s["x"] = torch.randn((m, d), **f).to(_TYPES[case["type"]])
        # codes of normal weights, rows padded with zeros to a multiple of 16 columns
        s["codes"] = torch.zeros((v, (d + 15) // 16 * 16), dtype=torch.int8, device="cuda")
        for r in range(0, v, 1 << 16):
            rows = min(v, r + (1 << 16)) - r
            s["codes"][r:r + rows, :d] = (torch.randn((rows, d), **f) * 32.0).round().clamp_(-127, 127).to(torch.int8)
        s["scales"] = (torch.rand((v,), **f) + 0.5) * (0.03 / math.sqrt(d))
        return s
    n, count = case["tokens"], case["sequences"] if case["op"] == "policy" else 2 * case["pairs"]
    shape = (n,) if case["packed"] else (count, n // count)
    logp = torch.rand(shape, **f).clamp_(min=1e-6).log_()  # log probabilities of about -1
    s["logp"] = logp
    s["reference"] = (logp + 0.1 * torch.randn(shape, **f)).clamp_(max=0.0)
    s["mask"] = torch.rand(shape, **f) < 0.9
    s["offsets"] = None
    if case["packed"]:
        cuts = torch.sort(torch.randint(0, n + 1, (count - 1,), **f)).values
        s["offsets"] = torch.cat([torch.zeros_like(cuts[:1]) if count > 1 else torch.zeros((1,), dtype=torch.int64, device="cuda"),
                                  cuts, torch.full((1,), n, dtype=torch.int64, device="cuda")])
    if case["op"] == "preference":
        s["grad"] = (torch.rand((case["pairs"],), **f) + 0.5) / case["pairs"]
        return s
    s["old"] = logp + 0.15 * torch.randn(shape, **f)  # a few steps old: some ratios leave the clip range
    s["advantages"] = torch.randn(shape if case["per_token"] else (count,), **f)
    s["grad"] = (torch.rand((count,), **f) + 0.5) / count
    return s


BETA, CLIP = 0.1, (0.2, 0.28)


def _plain_lookup(s):
    w, ids = s["weight"], s["ids"]
    out = (w[ids].float() * s["scale"]).to(w.dtype)
    if not s["train"]:
        return {"out": out}
    g = torch.where((ids != s["padding_idx"])[:, None], s["grad"].float(), torch.zeros((), device="cuda"))
    gw = torch.zeros(w.shape, dtype=torch.float32, device="cuda").index_add_(0, ids, g).mul_(s["scale"])
    return {"out": out, "grad_weight": gw.to(w.dtype)}


class _Sequences:
    """Sums over sequences, and values of sequences at their tokens."""

    def __init__(self, s):
        self.keep, self.shape = s["mask"], s["mask"].shape
        if s["offsets"] is not None:
            self.first, self.last = s["offsets"][:-1], s["offsets"][1:]
            self.lengths = self.last - self.first

    def sum(self, x):
        x = torch.where(self.keep, x.double(), torch.zeros((), dtype=torch.float64, device="cuda"))
        if len(self.shape) == 2:
            return x.sum(1)
        total = torch.cat([torch.zeros((1,), dtype=torch.float64, device="cuda"), x.cumsum(0)])
        return total[self.last] - total[self.first]

    def spread(self, y):
        return y[:, None] if len(self.shape) == 2 else torch.repeat_interleave(y, self.lengths, output_size=self.shape[0])


def _plain_preference(s):
    q, pairs = _Sequences(s), s["pairs"]
    counts = q.sum(torch.ones((), device="cuda").expand(q.shape))
    share = 1.0 / counts.clamp(min=1.0) if s["average"] else torch.ones_like(counts)
    rewards = BETA * share * q.sum(s["logp"].double() - s["reference"].double())
    h, e = rewards[:pairs] - rewards[pairs:], s["smoothing"]
    if s["kind"] == "sigmoid":
        soft = torch.log1p(torch.exp(-h.abs()))
        loss = (1 - e) * (soft + (-h).clamp(min=0.0)) + e * (soft + h.clamp(min=0.0))
        slope = e / (1 + torch.exp(-h)) - (1 - e) / (1 + torch.exp(h))
    elif s["kind"] == "hinge":
        loss, slope = (1 - h).clamp(min=0.0), -(h < 1).double()
    else:
        u = (h - 0.5) / BETA
        loss, slope = u * u, 2.0 * u / BETA
    out = {"loss": loss.float(), "margins": h.float(), "rewards": rewards.float(), "counts": counts.to(torch.int32)}
    if s["train"]:
        c = s["grad"] * slope * BETA
        each = q.spread((torch.cat([c, -c]) * share).float())
        out["grad"] = torch.where(q.keep, each, torch.zeros_like(each))
    return out


def _plain_policy(s):
    q, lo, hi = _Sequences(s), math.log1p(-CLIP[0]), math.log1p(CLIP[1])
    counts = q.sum(torch.ones((), device="cuda").expand(q.shape))
    share = 1.0 / counts.clamp(min=1.0) if s["average"] else torch.ones_like(counts)
    delta = s["logp"].double() - s["old"].double()
    log_ratio = (q.sum(delta) / counts.clamp(min=1.0)).float()
    if s["level"] == "sequence":
        delta = q.spread(log_ratio.double())
    a = s["advantages"] if s["per_token"] else q.spread(s["advantages"])
    over = ((a > 0) & (delta > hi)) | ((a < 0) & (delta < lo))
    ratio = torch.exp(delta.float())
    bound = torch.where(a > 0, 1.0 + CLIP[1], 1.0 - CLIP[0])
    term = -a * torch.where(over, bound, ratio)
    x = s["reference"].double() - s["logp"].double()
    if s["kl"] == "k1":
        k, slope = -x, torch.ones_like(x)
    elif s["kl"] == "k2":
        k, slope = 0.5 * x * x, -x
    else:
        k, slope = torch.expm1(x) - x, -torch.expm1(x)
    kl = share * q.sum(k)
    loss = share * q.sum(term.expand(q.shape)) + s["kl_weight"] * kl
    out = {"loss": loss.float(), "kl": kl.float(), "log_ratio": log_ratio, "counts": counts.to(torch.int32),
           "clipped": q.sum(over.double().expand(q.shape)).to(torch.int32)}
    if s["train"]:
        each = torch.where(over, torch.zeros_like(term), -a * ratio) + s["kl_weight"] * slope.float()
        out["grad"] = torch.where(q.keep, q.spread(s["grad"] * share.float()) * each, torch.zeros((), device="cuda"))
    return out


def _plain_q8(s):
    d = s["d"]
    x = s["x"].double()
    top = x.abs().amax(1, keepdim=True)
    codes = torch.where(top > 0, torch.round(x * 127.0 / top), torch.zeros_like(x)).float()
    scale = (top / 127.0).float()
    return {"scores": (codes @ s["codes"][:, :d].float().t()) * (scale * s["scales"])}


def run(state):
    s = state
    if not own:
        return {"lookup": _plain_lookup, "preference": _plain_preference, "policy": _plain_policy, "q8": _plain_q8}[s["op"]](s)
    import tensor_train_compressed_embeddingbag_gb300 as tt

    if s["op"] == "lookup":
        out = tt.tt_emb_lookup_forward(s["weight"], s["ids"], scale=s["scale"])
        if not s["train"]:
            return {"out": out}
        gw = tt.tt_emb_lookup_backward(s["grad"], s["ids"], s["v"], scale=s["scale"], padding_idx=s["padding_idx"])
        return {"out": out, "grad_weight": gw}
    if s["op"] == "q8":
        return {"scores": tt.tt_emb_q8_scores(s["x"], s["codes"], s["scales"])}
    if s["op"] == "preference":
        how = dict(mask=s["mask"], offsets=s["offsets"], beta=BETA, kind=s["kind"], label_smoothing=s["smoothing"], average=s["average"])
        loss, margins, rewards, counts = tt.tt_emb_preference_forward(s["logp"], s["reference"], **how)
        out = {"loss": loss, "margins": margins, "rewards": rewards, "counts": counts}
        if s["train"]:
            out["grad"] = tt.tt_emb_preference_backward(s["logp"], margins, counts, s["grad"], **how)
        return out
    how = dict(reference=s["reference"], mask=s["mask"], offsets=s["offsets"], clip=CLIP, kl=s["kl"], kl_weight=s["kl_weight"], level=s["level"],
               average=s["average"], per_token=s["per_token"])
    loss, kl, log_ratio, counts, clipped = tt.tt_emb_policy_forward(s["logp"], s["old"], s["advantages"], **how)
    out = {"loss": loss, "kl": kl, "log_ratio": log_ratio, "counts": counts, "clipped": clipped}
    if s["train"]:
        out["grad"] = tt.tt_emb_policy_backward(s["logp"], s["old"], s["advantages"], log_ratio, counts, s["grad"], **how)
    return out


def work(case):
    if case["op"] == "lookup":
        n, v, d, e = case["n"], case["v"], case["d"], _BYTES[case["type"]]
        size = 8 * n + (min(n, v) + n) * d * e
        if not case["train"]:
            return {"bytes": size, "flops": 1.0 * n * d}
        return {"bytes": size + (n + v) * d * e, "flops": 2.0 * n * d}
    if case["op"] == "q8":
        m, v, d = case["m"], case["v"], case["d"]
        return {"bytes": m * d * _BYTES[case["type"]] + v * d + 4 * v + 4 * m * v, "flops": 2.0 * m * v * d}
    n = case["tokens"]
    if case["op"] == "preference":
        return {"bytes": 9 * n + 48 * case["pairs"] + (4 * n if case["train"] else 0), "flops": 3.0 * n}
    per_token = (17 if case["per_token"] else 13) * n
    return {"bytes": per_token + 32 * case["sequences"] + (4 * n if case["train"] else 0), "flops": 30.0 * n}


def exact(case, seed):
    s = prepare(case, seed)
    zero = torch.zeros((), dtype=torch.float64, device="cuda")
    if case["op"] == "lookup":
        out = {"out": torch.index_select(s["weight"], 0, s["ids"]).double() * s["scale"]}
        if case["train"]:
            count = s["ids"] != s["padding_idx"]
            gw = torch.zeros((case["v"], case["d"]), dtype=torch.float64, device="cuda")
            out["grad_weight"] = gw.index_add_(0, s["ids"][count], s["grad"][count].double() * s["scale"])
        return out
    if case["op"] == "q8":
        x, d = s["x"].double(), case["d"]
        top = x.abs().max(1).values
        step = top / 127.0
        codes = torch.round(torch.div(127.0 * x, torch.where(top > 0, top, torch.ones_like(top))[:, None]))
        scale = (step.float().double()[:, None]) * s["scales"].double()[None]
        for r in range(0, case["v"], 8192):
            scale[:, r:r + 8192] *= codes @ s["codes"][r:r + 8192, :d].double().t()
        return {"scores": scale}
    n, keep = case["tokens"], s["mask"].reshape(-1)
    count = case["sequences"] if case["op"] == "policy" else 2 * case["pairs"]
    if case["packed"]:
        of = torch.searchsorted(s["offsets"], torch.arange(n, device="cuda"), right=True) - 1
    else:
        of = torch.arange(n, device="cuda") // (n // count)

    def total(x):
        return torch.zeros((count,), dtype=torch.float64, device="cuda").index_add(0, of[keep], x[keep])

    logp = s["logp"].reshape(-1).double().requires_grad_()
    ref = s["reference"].reshape(-1).double()
    counts = torch.bincount(of[keep], minlength=count)
    size = counts.clamp(min=1).double() if case["average"] else torch.ones((count,), dtype=torch.float64, device="cuda")
    if case["op"] == "preference":
        rewards = BETA * total(logp - ref) / size
        h, e = rewards[:case["pairs"]] - rewards[case["pairs"]:], case["smoothing"]
        if case["kind"] == "sigmoid":
            loss = -(1 - e) * torch.nn.functional.logsigmoid(h) - e * torch.nn.functional.logsigmoid(-h)
        else:
            loss = torch.relu(1 - h) if case["kind"] == "hinge" else ((h - 0.5) / BETA) ** 2
        out = {"loss": loss.detach(), "margins": h.detach(), "rewards": rewards.detach(), "counts": counts.to(torch.int32)}
    else:
        delta = logp - s["old"].reshape(-1).double()
        log_ratio = total(delta) / counts.clamp(min=1).double()
        ratio = torch.exp(log_ratio[of] if case["level"] == "sequence" else delta)
        a = (s["advantages"].reshape(-1) if case["per_token"] else s["advantages"][of]).double()
        low, high = 1.0 - CLIP[0], 1.0 + CLIP[1]
        term = -torch.minimum(ratio * a, ratio.clamp(low, high) * a)
        x = ref - logp
        k = {"k1": -x, "k2": 0.5 * x ** 2, "k3": torch.expm1(x) - x}[case["kl"]]
        kl = total(k) / size
        loss = total(term) / size + case["kl_weight"] * kl
        clipped = torch.where(((a > 0) & (ratio > high)) | ((a < 0) & (ratio < low)), zero + 1.0, zero)
        out = {"loss": loss.detach(), "kl": kl.detach(), "log_ratio": log_ratio.detach(), "counts": counts.to(torch.int32),
               "clipped": total(clipped).to(torch.int32)}
    if case["train"]:
        out["grad"] = torch.autograd.grad((loss * s["grad"].double()).sum(), logp)[0].reshape(s["logp"].shape)
    return out
