"""The operators of the vocabulary head and the cases they are measured on.

The head scores hidden rows against every row of a table (items, tokens):
z[n, v] = <hidden[n], weight[v]>.

  xent      softmax cross entropy over the whole table, forward (loss and
            log-sum-exp per row) or forward and backward (and both gradients)
  distill   cross entropy against a teacher's top logits, the same two forms
  q4        scores of a few rows against a table held in 4 bits with one bf16
            scale per group of columns (serving)

With `own` false, `run` computes the plain form in float32 with elementary torch
operations; with `own` true it calls the package's operators.
"""
import math

import torch

own = False

IGNORE = -100
_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_BYTES = {"f32": 4, "bf16": 2, "f16": 2}


def listed():
    return [
        # the tiny configuration's table (E = 120, D = 8) and batch of 8: one step, launch latency
        {"name": "xent_train_tiny", "op": "xent", "n": 8, "v": 120, "d": 8, "type": "f32", "train": True, "ignored": 0.0},
        # next-item training: 512 histories against a catalogue of 10^6 rows of width 64, the tables' own type
        {"name": "xent_train_items", "op": "xent", "n": 512, "v": 1000000, "d": 64, "type": "f32", "train": True, "ignored": 0.0},
        # the same kind of head trained in bf16, more rows, an odd catalogue, a tenth of the rows padding
        {"name": "xent_train_items_bf16", "op": "xent", "n": 4096, "v": 100003, "d": 128, "type": "bf16", "train": True, "ignored": 0.1},
        # a wide token vocabulary: the largest training step
        {"name": "xent_train_tokens", "op": "xent", "n": 4096, "v": 131072, "d": 2048, "type": "bf16", "train": True, "ignored": 0.1},
        # held-out loss of a batch, forward only, odd vocabulary
        {"name": "xent_eval", "op": "xent", "n": 2047, "v": 50001, "d": 1024, "type": "f16", "train": False, "ignored": 0.3},
        # scoring of four single tokens: one pass over the table
        {"name": "xent_eval_few", "op": "xent", "n": 4, "v": 131072, "d": 4096, "type": "bf16", "train": False, "ignored": 0.0},
        # a small distillation check, forward only
        {"name": "distill_eval_small", "op": "distill", "n": 16, "v": 1000, "d": 64, "k": 8, "type": "f32", "train": False, "temp": 1.0},
        # distilling a dense item table's top 32 into a compressed one
        {"name": "distill_train_items", "op": "distill", "n": 512, "v": 100000, "d": 128, "k": 32, "type": "f32", "train": True, "temp": 2.0},
        # distilling a token model's top 64
        {"name": "distill_train_tokens", "op": "distill", "n": 2048, "v": 65537, "d": 1024, "k": 64, "type": "bf16", "train": True, "temp": 2.0},
        # one small request: launch latency
        {"name": "q4_small", "op": "q4", "m": 1, "v": 1000, "d": 256, "group": 64, "type": "f16"},
        # eight requests against the catalogue of 10^6 items of width 64
        {"name": "q4_items", "op": "q4", "m": 8, "v": 1000000, "d": 64, "group": 32, "type": "f32"},
        # one token against a wide vocabulary: 268 MB of weights
        {"name": "q4_token", "op": "q4", "m": 1, "v": 131072, "d": 4096, "group": 128, "type": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["xent", "xent", "distill", "q4"])
    while True:
        t = rng.choice(["f32", "bf16", "f16"])
        v = _log(rng, 50, 1000000)
        if op == "q4":
            c = {"op": op, "m": _log(rng, 1, 32), "v": v, "d": _log(rng, 32, 8192), "group": rng.choice([32, 64, 128]), "type": t}
            if c["v"] * c["d"] <= 1 << 29 and c["m"] * c["v"] <= 1 << 24:
                return c
            continue
        c = {"op": op, "n": _log(rng, 1, 8192), "v": v, "d": _log(rng, 8, 4096), "type": t, "train": rng.random() < 0.7}
        if op == "distill":
            c["k"], c["temp"] = min(v // 2, _log(rng, 1, 128)), rng.choice([1.0, 2.0, 4.0])
        else:
            c["ignored"] = rng.choice([0.0, 0.1, 0.5])
        if c["n"] * c["v"] <= 1 << 29 and c["v"] * c["d"] <= 1 << 29 and c["n"] * c["v"] * c["d"] <= 1 << 39:
            return c


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    f = dict(generator=g, device="cuda")
    s = dict(case)
    if case["op"] == "q4":
        m, v, d, gr = case["m"], case["v"], case["d"], case["group"]
        half, groups = (d + 31) // 32 * 16, (d + gr - 1) // gr
        s["x"] = torch.randn((m, d), **f).to(_TYPES[case["type"]])
        # two 4-bit codes to a byte, the even column in the low half; columns past d hold 8, which stands for 0
        s["packed"] = torch.randint(0, 256, (v, half), dtype=torch.uint8, **f)
        if d % 2:
            s["packed"][:, d // 2] = (s["packed"][:, d // 2] & 15) | 128
        s["packed"][:, (d + 1) // 2:] = 136
        s["scales"] = ((torch.rand((v, groups), **f) + 0.5) * (0.3 / math.sqrt(d))).to(torch.bfloat16)
        return s
    n, v, d = case["n"], case["v"], case["d"]
    s["hidden"] = torch.randn((n, d), **f).to(_TYPES[case["type"]])
    s["weight"] = (torch.randn((v, d), **f) * (2.0 / math.sqrt(d))).to(_TYPES[case["type"]])  # scores of about N(0, 4)
    s["grad"] = (torch.rand((n,), **f) + 0.5) / n  # per-row weights of a mean
    if case["op"] == "xent":
        t = (torch.rand((n,), **f) ** 3 * v).to(torch.int64).clamp_(max=v - 1)  # low ids more often
        s["targets"] = torch.where(torch.rand((n,), **f) < case["ignored"], torch.full_like(t, IGNORE), t)
    else:
        k = case["k"]
        step = torch.randint(1, v // k + 1, (n, k), **f)
        ids = (torch.randint(0, v, (n, 1), **f) + step.cumsum(1)) % v  # distinct within a row
        s["teacher_logits"] = torch.sort(torch.randn((n, k), **f) * 2.0, dim=1, descending=True).values
        have = torch.randint(0, k + 1, (n, 1), **f)  # some rows have fewer entries, some none
        have = torch.where(torch.rand((n, 1), **f) < 0.8, torch.full_like(have, k), have)
        s["teacher_ids"] = torch.where(torch.arange(k, device="cuda") < have, ids, torch.full_like(ids, -1))
    return s


def _plain_xent(s):
    h, w, t = s["hidden"].float(), s["weight"].float(), s["targets"]
    z = h @ w.t()
    m = z.amax(1, keepdim=True)
    e = torch.exp(z - m)
    total = e.sum(1, keepdim=True)
    lse = (m + torch.log(total))[:, 0]
    keep = t != IGNORE
    at = t.clamp(min=0)[:, None]
    loss = torch.where(keep, lse - z.gather(1, at)[:, 0], torch.zeros_like(lse))
    if not s["train"]:
        return {"loss": loss, "lse": lse}
    g = torch.where(keep, s["grad"], torch.zeros_like(lse))[:, None]
    dz = e * (g / total)
    dz.scatter_add_(1, at, -g)
    return {"loss": loss, "lse": lse, "grad_hidden": (dz @ w).to(s["hidden"].dtype),
            "grad_weight": (dz.t() @ h).to(s["weight"].dtype)}


def _plain_distill(s):
    h, w, ids, temp = s["hidden"].float(), s["weight"].float(), s["teacher_ids"], s["temp"]
    z = (h @ w.t()) / temp
    m = z.amax(1, keepdim=True)
    e = torch.exp(z - m)
    total = e.sum(1, keepdim=True)
    lse = m + torch.log(total)
    have = ids >= 0
    at = ids.clamp(min=0)
    t = torch.where(have, s["teacher_logits"].float() / temp, torch.full_like(lse, -math.inf))
    top = t.amax(1, keepdim=True)
    some = top > -math.inf
    a = torch.where(have & some, torch.exp(t - torch.where(some, top, torch.zeros_like(top))), torch.zeros_like(t))
    q = a / torch.where(some, a.sum(1, keepdim=True), torch.ones_like(top))
    logq = torch.where(q > 0, torch.log(q), torch.zeros_like(q))
    loss = (temp * temp) * (q * (logq - z.gather(1, at) + lse)).sum(1)
    lse = lse[:, 0]
    if not s["train"]:
        return {"loss": loss, "lse": lse}
    g = torch.where(some, s["grad"][:, None] * temp, torch.zeros_like(top))
    dz = e * (g / total)
    dz.scatter_add_(1, at, -g * q)
    return {"loss": loss, "lse": lse, "grad_hidden": (dz @ w).to(s["hidden"].dtype),
            "grad_weight": (dz.t() @ h).to(s["weight"].dtype)}


def _plain_q4(s):
    p, d = s["packed"], s["d"]
    q = torch.stack((p & 15, p >> 4), dim=2).reshape(p.shape[0], -1)[:, :d]
    scale = torch.repeat_interleave(s["scales"].float(), s["group"], dim=1)[:, :d]
    return {"scores": s["x"].float() @ ((q.float() - 8.0) * scale).t()}


def run(state):
    s = state
    if not own:
        return {"xent": _plain_xent, "distill": _plain_distill, "q4": _plain_q4}[s["op"]](s)
    import tensor_train_compressed_embeddingbag_gb300 as tt

    if s["op"] == "q4":
        return {"scores": tt.tt_emb_q4_matvec(s["x"], s["packed"], s["scales"], s["group"])}
    if s["op"] == "xent":
        loss, lse = tt.tt_emb_xent_forward(s["hidden"], s["weight"], s["targets"], ignore_index=IGNORE)
        if not s["train"]:
            return {"loss": loss, "lse": lse}
        gh, gw = tt.tt_emb_xent_backward(s["hidden"], s["weight"], s["targets"], lse, s["grad"], ignore_index=IGNORE)
    else:
        loss, lse = tt.tt_emb_distill_forward(s["hidden"], s["weight"], s["teacher_ids"], s["teacher_logits"], s["temp"])
        if not s["train"]:
            return {"loss": loss, "lse": lse}
        gh, gw = tt.tt_emb_distill_backward(s["hidden"], s["weight"], s["teacher_ids"], s["teacher_logits"], lse, s["grad"], s["temp"])
    return {"loss": loss, "lse": lse, "grad_hidden": gh, "grad_weight": gw}


def work(case):
    e = _BYTES[case["type"]]
    if case["op"] == "q4":
        m, v, d, gr = case["m"], case["v"], case["d"], case["group"]
        return {"bytes": m * d * e + v * ((d + 1) // 2) + 2 * v * ((d + gr - 1) // gr) + 4 * m * v, "flops": 2.0 * m * v * d}
    n, v, d, k = case["n"], case["v"], case["d"], case.get("k", 0)
    read = (n + v) * d * e + (12 * n * k if k else 8 * n)
    if not case["train"]:
        return {"bytes": read + 8 * n, "flops": 2.0 * n * v * d}
    return {"bytes": read + 12 * n + (n + v) * d * e, "flops": 6.0 * n * v * d}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "q4":
        x, p, v, d = s["x"].double(), s["packed"], case["v"], case["d"]
        out = torch.empty((case["m"], v), dtype=torch.float64, device="cuda")
        col = torch.arange(d, device="cuda")
        for r in range(0, v, 16384):
            byte = p[r:r + 16384][:, col // 2].to(torch.int32)
            code = torch.where(col % 2 == 0, byte % 16, byte // 16).double() - 8.0
            out[:, r:r + 16384] = x @ (code * s["scales"][r:r + 16384].double()[:, col // case["group"]]).t()
        return {"scores": out}
    n, v, d = case["n"], case["v"], case["d"]
    if n * v * d > 3 << 40:
        return None
    h, w, temp = s["hidden"].double(), s["weight"].double(), case.get("temp", 1.0)
    loss, lse = (torch.zeros(n, dtype=torch.float64, device="cuda") for _ in range(2))
    dh, dw = torch.zeros_like(h), torch.zeros_like(w)
    rows = max(1, (1 << 27) // v)
    for r in range(0, n, rows):
        a = slice(r, min(n, r + rows))
        target = torch.zeros((a.stop - a.start, v), dtype=torch.float64, device="cuda")
        if case["op"] == "xent":
            keep = s["targets"][a] >= 0
            target[keep, s["targets"][a][keep]] = 1.0
            entropy = 0.0
        else:
            have = s["teacher_ids"][a] >= 0
            q = torch.softmax((s["teacher_logits"][a].double() / temp).masked_fill(~have, -math.inf), 1).nan_to_num(0.0)
            target.scatter_add_(1, s["teacher_ids"][a].clamp(min=0), q)
            entropy = torch.special.entr(q).sum(1)
        mass = target.sum(1)
        z = (h[a] @ w.t()) / temp
        lse[a] = torch.logsumexp(z, 1)
        loss[a] = temp * temp * (mass * lse[a] - (target * z).sum(1) - entropy)
        if case["train"]:
            z.sub_(lse[a][:, None]).exp_().mul_(mass[:, None]).sub_(target).mul_((s["grad"][a].double() * temp)[:, None])
            dh[a] = z @ w
            dw.addmm_(z.t(), h[a])
    out = {"loss": loss, "lse": lse}
    return {**out, "grad_hidden": dh, "grad_weight": dw} if case["train"] else out
