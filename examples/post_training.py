"""Post-training of a small token model whose one table is both its input and its output.

A model (tied table, one hidden layer over the last tokens) answers prompts.  Answers are sampled
from the scores of an 8-bit copy of the table; a reward counts tokens of one class, and the policy
loss, with the log probabilities of the vocabulary head, trains the model under a Kullback-Leibler
term against where it began.  Then pairs of answers, ordered by reward, train it by the preference
loss.  Lookup and head both give the table its gradient.

    python examples/post_training.py [--tokens 2000] [--steps 20]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import tensor_train_compressed_embeddingbag_gb300 as tt  # noqa: E402


class Model(torch.nn.Module):
    """hidden[t] = tanh(mix(mean of the last `window` tokens' rows)); scores against the same table."""

    def __init__(self, tokens: int, dim: int, window: int = 4):
        super().__init__()
        self.table = torch.nn.Parameter(torch.randn((tokens, dim)) * 0.5)
        self.mix = torch.nn.Linear(dim, dim)
        self.window = window

    def hidden(self, ids: torch.Tensor) -> torch.Tensor:
        rows = tt.vocab_embedding(ids, self.table, scale=self.table.shape[1] ** 0.5)
        total = torch.nn.functional.pad(rows.cumsum(1), (0, 0, self.window, 0))
        return torch.tanh(self.mix((total[:, self.window:] - total[:, :-self.window]) / (self.window * self.table.shape[1] ** 0.5)))

    def log_probs(self, ids: torch.Tensor) -> torch.Tensor:
        """log p(ids[:, t] | ids[:, :t]) for t >= 1, without an array of scores."""
        return -tt.vocab_cross_entropy(self.hidden(ids[:, :-1]), self.table, ids[:, 1:], reduction="none")


@torch.no_grad()
def answer(model: Model, served: "tt.Q8Table", prompts: torch.Tensor, length: int) -> torch.Tensor:
    """Prompts with `length` sampled tokens behind them."""
    ids = prompts
    for _ in range(length):
        scores = served.scores(model.hidden(ids[:, -model.window:])[:, -1])
        noise = -torch.log(-torch.log(torch.rand_like(scores).clamp_(1e-20, 1 - 1e-7)))
        ids = torch.cat([ids, (scores + noise).argmax(1, keepdim=True)], 1)
    return ids


def main(tokens: int = 2000, dim: int = 64, prompts: int = 64, group: int = 8, length: int = 12, steps: int = 20, seed: int = 0, log=print):
    device = torch.device("cuda")
    torch.manual_seed(seed)
    model = Model(tokens, dim).to(device)
    start = Model(tokens, dim).to(device)
    start.load_state_dict(model.state_dict())
    opt = torch.optim.Adam(model.parameters(), lr=0.003)
    wanted = torch.rand(tokens, device=device) < 0.2  # the reward: tokens of this class
    rewards, losses = [], []

    def rollout():
        p = torch.randint(0, tokens, (prompts, model.window), device=device).repeat_interleave(group, 0)
        ids = answer(model, tt.Q8Table(model.table), p, length)
        mask = torch.arange(ids.shape[1] - 1, device=device).expand(ids.shape[0], -1) >= model.window - 1  # the answer's own tokens
        reward = wanted[ids[:, model.window:]].float().mean(1)
        with torch.no_grad():
            return ids, mask, reward, model.log_probs(ids), start.log_probs(ids)

    for _ in range(steps):
        ids, mask, reward, old, reference = rollout()
        each = reward.reshape(prompts, group)
        advantage = ((each - each.mean(1, keepdim=True)) / (each.std(1, keepdim=True) + 1e-4)).reshape(-1)
        for _ in range(2):
            loss = tt.policy_loss(model.log_probs(ids), old, advantage, reference, mask, clip=(0.2, 0.28), kl_weight=0.01)
            opt.zero_grad()
            loss.backward()
            opt.step()
        rewards.append(reward.mean().item())
    log(f"policy: reward {rewards[0]:.3f} -> {rewards[-1]:.3f}")

    for _ in range(steps):
        ids, mask, reward, _, reference = rollout()
        each = reward.reshape(prompts, group)
        first = torch.arange(prompts, device=device) * group
        pairs = torch.cat([first + each.argmax(1), first + each.argmin(1)])  # chosen, then rejected
        loss = tt.preference_loss(model.log_probs(ids[pairs]), reference[pairs], mask[pairs], beta=0.2)
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.item())
    log(f"preference: loss {losses[0]:.3f} -> {losses[-1]:.3f}, reward {reward.mean().item():.3f}")
    return {"rewards": rewards, "losses": losses}


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=2000)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args()
    main(tokens=a.tokens, steps=a.steps)
