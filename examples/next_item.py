"""Next-item prediction over a catalogue whose table is TT-compressed.

One TT table is both the input embedding and the output head: a step is one call over
the histories' bags and one bag per catalogue row, so the loss over the whole catalogue
trains the cores through the fused update.  A dense model of the same width is trained
first; the compressed one then learns from the items and from the dense one's top
scores (distillation).  For serving, the table's rows are expanded once and held in 4
bits, and a request is one pass over them.

    python examples/next_item.py [--items 4096] [--steps 300]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import tensor_train_compressed_embeddingbag_gb300 as tt  # noqa: E402


class Histories:
    """Synthetic sessions: a session follows one of `groups` fixed cycles through the catalogue, with some noise.
    Ids are grouped, as catalogue ids are: a cycle's items are neighbours."""

    def __init__(self, items: int, groups: int, length: int, seed: int, device):
        self.items, self.length, self.device = items, length, device
        self.gen = torch.Generator(device=device)
        self.gen.manual_seed(seed)
        self.span = items // groups

    def batch(self, rows: int):
        start = torch.randint(0, self.items, (rows, 1), generator=self.gen, device=self.device)
        step = torch.arange(self.length + 1, device=self.device)
        at = start // self.span * self.span + (start + step) % self.span
        seen = at % self.items
        noise = torch.rand(seen.shape, generator=self.gen, device=self.device) < 0.05
        seen = torch.where(noise, torch.randint(0, self.items, seen.shape, generator=self.gen, device=self.device), seen)
        return seen[:, :-1].contiguous(), at[:, -1] % self.items


def tt_step_inputs(history: torch.Tensor, items: int):
    """Indices and start offsets of one TT call: the histories' bags, then every row in a bag of its own."""
    rows, length = history.shape
    every = torch.arange(items, device=history.device)
    offsets = torch.cat([torch.arange(rows, device=history.device) * length, rows * length + every])
    return torch.cat([history.reshape(-1), every]), offsets


def main(items: int = 4096, dim: int = 32, rank: int = 16, rows: int = 512, steps: int = 300, top: int = 16, seed: int = 0, log=print):
    device = torch.device("cuda")
    torch.manual_seed(seed)
    data = Histories(items, groups=max(1, items // 64), length=4, seed=seed, device=device)

    # the dense teacher
    table = torch.nn.Parameter(torch.randn((items, dim), device=device) * 0.3)
    mix = torch.nn.Linear(dim, dim, device=device)
    opt = torch.optim.Adam([table, *mix.parameters()], lr=0.02)
    dense = []
    for _ in range(steps):
        history, target = data.batch(rows)
        hidden = mix(table[history].mean(1))
        loss = tt.vocab_cross_entropy(hidden, table, target)
        opt.zero_grad()
        loss.backward()
        opt.step()
        dense.append(loss.item())
    log(f"dense teacher: loss {dense[0]:.3f} -> {sum(dense[-10:]) / 10:.3f}, {table.numel()} parameters")

    # the TT student: items and the teacher's top scores
    m = tt.TTEmbeddingBag(items, dim, [rank, rank], learning_rate=0.2, optimizer="adagrad", weight_dist="approx-normal", sigma=0.5,
                          generator=torch.Generator().manual_seed(seed))
    smix = torch.nn.Linear(dim, dim, device=device)
    opt = torch.optim.Adam(smix.parameters(), lr=0.02)
    student = []
    for _ in range(steps):
        history, target = data.batch(rows)
        with torch.no_grad():
            scores, ids = torch.topk(mix(table[history].mean(1)) @ table.t(), top)
        out = m(*tt_step_inputs(history, items), mode="mean")
        hidden, weight = smix(out[:rows]), out[rows:]
        loss = tt.vocab_cross_entropy(hidden, weight, target)
        total = loss + 0.5 * tt.vocab_distillation(hidden, weight, ids, scores, temperature=2.0)
        opt.zero_grad()
        total.backward()  # the cores take their fused update here
        opt.step()
        student.append(loss.item())
    params = sum(c.numel() for c in (m.G1, m.G2, m.G3))
    log(f"TT student:    loss {student[0]:.3f} -> {sum(student[-10:]) / 10:.3f}, {params} parameters")

    # serving: the rows once, in 4 bits; then single requests
    with torch.no_grad():
        served = tt.Q4Table(m.full_weight(), group=32)
        history, target = data.batch(rows)
        offsets = torch.arange(rows, device=device) * history.shape[1]
        hidden = smix(m(history.reshape(-1), offsets, mode="mean"))
        exact = (hidden @ m.full_weight().t()).topk(10).indices
        quick = torch.cat([served.scores(hidden[i:i + 1]).topk(10).indices for i in range(rows)])
        hits = (quick == target[:, None]).any(1).float().mean().item()
        kept = sum(len(set(a) & set(b)) for a, b in zip(exact.tolist(), quick.tolist())) / (10.0 * rows)
    log(f"4-bit serving: target among the first 10 in {hits:.1%}, {kept:.1%} of the exact first 10 kept, "
        f"{served.packed.numel() + 2 * served.scales.numel()} bytes for {4 * items * dim} of fp32")
    return {"dense": dense, "student": student, "hits": hits, "kept": kept}


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--items", type=int, default=4096)
    ap.add_argument("--steps", type=int, default=300)
    a = ap.parse_args()
    main(items=a.items, steps=a.steps)
