"""Fine-tunes low-rank adapters of a frozen layer by policy gradient, twice, and
checks that the two runs agree bit for bit.

The model: token embedding -> RMS norm -> linear layer with an adapter per task
(the base frozen) on a residual stream -> RMS norm -> output layer over the
embedding's own table.  A step samples nothing: it scores given continuations
(their log probabilities and the entropy), weighs them by a reward, adds a
bonus for entropy, clips the adapters' gradients by their norm and steps.  Every
product, norm, lookup and gradient runs in this package's kernels.  The data are
synthetic: the reward of a token depends on its task.

    python examples/tune_adapters.py [--steps N] [--vocab V] [--width D]
"""
import argparse
import hashlib
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

from deterministic_invariant_gemm_fwd_gb300 import nn as cnn  # noqa: E402


class Policy(torch.nn.Module):
    def __init__(self, vocab, width, tasks, rank, dtype=torch.bfloat16):
        super().__init__()
        self.embed = cnn.Embedding(vocab, width, device="cuda", dtype=dtype)
        self.first = cnn.RMSNorm(width, device="cuda", dtype=dtype)
        self.layer = cnn.LoraLinear(cnn.Linear(width, width, tier="tc", device="cuda", dtype=dtype), tasks, rank)
        self.last = cnn.RMSNorm(width, device="cuda", dtype=dtype)
        for p in (self.embed.weight, self.first.weight, self.last.weight):
            p.requires_grad_(False)

    def forward(self, ids, tokens, tasks, temperature=1.0):
        """Log probabilities of tokens and entropies, [sequences, length]."""
        h = self.embed(ids)
        y, _ = self.last(self.layer(self.first(h), tasks), h)
        return cnn.linear_log_probs(y, self.embed.weight, tokens, temperature)

    @torch.no_grad()
    def alternatives(self, ids, tokens, tasks, top):
        h = self.embed(ids)
        y, _ = self.last(self.layer(self.first(h), tasks), h)
        return cnn.top_log_probs(y, self.embed.weight, tokens, top)


def batch(vocab, sequences, length, tasks, step):
    """Contexts, continuations of them, a task per sequence (one in eight has
    none) and the continuations' advantages; the first tokens are a prompt."""
    g = torch.Generator().manual_seed(2000 + step)
    ids = torch.randint(0, vocab, (sequences, length), generator=g)
    tokens = torch.randint(0, vocab, (sequences, length), generator=g)
    task = torch.randint(0, tasks, (sequences,), generator=g)
    task[torch.rand(sequences, generator=g) < 0.125] = -1
    advantage = ((tokens + task[:, None]) % 3 - 1).float()
    tokens[:, : length // 4] = -100
    return (t.cuda() for t in (ids, tokens, task[:, None].expand(-1, length).contiguous(), advantage))


def train(vocab, width, tasks, rank, sequences, length, steps, lr=0.5, seed=42):
    torch.manual_seed(seed)
    policy = Policy(vocab, width, tasks, rank)
    tuned = [p for p in policy.parameters() if p.requires_grad]
    optimizer = torch.optim.SGD(tuned, lr=lr, foreach=False)
    record = []
    for step in range(steps):
        ids, tokens, task, advantage = batch(vocab, sequences, length, tasks, step)
        logp, entropy = policy(ids, tokens, task)
        count = (tokens >= 0).sum()
        loss = -((advantage * logp).sum() + 0.01 * entropy.sum()) / count
        optimizer.zero_grad(set_to_none=True)
        loss.backward()
        norm = cnn.clip_grad_norm_(tuned, 0.1)
        optimizer.step()
        record.append((loss.detach(), norm))
    digest = hashlib.sha256()
    for w in tuned:
        digest.update(w.detach().cpu().view(torch.int16).numpy().tobytes())
    return [(float(a), float(b)) for a, b in record], digest.hexdigest(), policy


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--vocab", type=int, default=8191)
    ap.add_argument("--width", type=int, default=256)
    ap.add_argument("--tasks", type=int, default=4)
    ap.add_argument("--rank", type=int, default=16)
    ap.add_argument("--sequences", type=int, default=16)
    ap.add_argument("--length", type=int, default=48)
    a = ap.parse_args()
    runs = [train(a.vocab, a.width, a.tasks, a.rank, a.sequences, a.length, a.steps) for _ in range(2)]
    (record, digest, policy), (record2, digest2, _) = runs
    print(f"loss {record[0][0]:.4f} -> {record[-1][0]:.4f}, gradient norm {record[-1][1]:.4f}; adapters sha256 {digest[:16]}")
    ids, tokens, task, _ = batch(a.vocab, a.sequences, a.length, a.tasks, 0)
    best = policy.alternatives(ids, tokens.clamp(min=0), task, 3)
    print(f"most probable after the first context: {best.top_ids[0, 0].tolist()}")
    if record != record2 or digest != digest2:
        raise SystemExit("the two runs differ")
    print("two runs agree bit for bit")


if __name__ == "__main__":
    main()
