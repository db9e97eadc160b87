"""Trains a small language model with a tied table twice and checks that the
two runs agree bit for bit (the test the Carbon README gives its training
example: the hashes of all weights after two runs).

The model: token embedding -> blocks of [RMS norm + linear (8-bit checkpoint),
ReLU, linear] on a residual stream -> RMS norm -> output layer with softmax
cross entropy over the embedding's own table.  Every matrix product, norm,
lookup and gradient of them runs in this package's kernels.  The data are
synthetic: a fixed random walk over the vocabulary, so the loss can fall.

    python examples/train_tied_lm.py [--steps N] [--vocab V] [--width D] [--clip NORM]
"""
import argparse
import hashlib
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

from deterministic_invariant_gemm_fwd_gb300 import nn as cnn  # noqa: E402


class Block(torch.nn.Module):
    def __init__(self, width, hidden, tier, dtype):
        super().__init__()
        self.tier = tier
        self.gamma = torch.nn.Parameter(torch.ones(width, device="cuda", dtype=dtype))
        self.up = cnn.Linear(width, hidden, tier=tier, device="cuda", dtype=dtype)
        self.down = cnn.Linear(hidden, width, tier=tier, device="cuda", dtype=dtype)

    def forward(self, x, h):
        """x: what the last block adds to the residual stream h."""
        a, h = cnn.norm_linear(x, self.gamma, self.up.weight, self.up.bias, residual=h, tier=self.tier)
        return self.down(torch.relu(a)), h


class TiedLanguageModel(torch.nn.Module):
    def __init__(self, vocab, width, blocks, tier="tc", dtype=torch.bfloat16):
        super().__init__()
        self.embed = cnn.Embedding(vocab, width, scale=1.0, device="cuda", dtype=dtype)
        self.blocks = torch.nn.ModuleList(Block(width, 4 * width, tier, dtype) for _ in range(blocks))
        self.norm = cnn.RMSNorm(width, device="cuda", dtype=dtype)

    def forward(self, ids, targets):
        h = self.embed(ids)
        x = torch.zeros_like(h)
        for block in self.blocks:
            x, h = block(x, h)
        y, _ = self.norm(x, h)
        return cnn.linear_cross_entropy(y, self.embed.weight, targets)


def batch(vocab, tokens, step):
    """Next-token pairs: the successor of id i is a fixed function of i, and
    one position in sixteen is padding."""
    g = torch.Generator().manual_seed(1000 + step)
    ids = torch.randint(0, min(vocab, 512), (tokens,), generator=g)
    targets = (ids * 31 + 7) % min(vocab, 512)
    targets[torch.randperm(tokens, generator=g)[: tokens // 16]] = -100
    return ids.cuda(), targets.cuda()


def train(vocab, width, blocks, tokens, steps, lr=0.5, seed=42, clip=None):
    torch.manual_seed(seed)
    model = TiedLanguageModel(vocab, width, blocks)
    optimizer = torch.optim.SGD(model.parameters(), lr=lr, foreach=False)
    losses = []
    for step in range(steps):
        loss = model(*batch(vocab, tokens, step))
        optimizer.zero_grad(set_to_none=True)
        loss.backward()
        if clip is not None:
            cnn.clip_grad_norm_(model.parameters(), clip)
        optimizer.step()
        losses.append(loss.detach())
    digest = hashlib.sha256()
    for w in model.parameters():
        digest.update(w.detach().cpu().view(torch.int16).numpy().tobytes())
    return [float(v) for v in losses], digest.hexdigest()


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--vocab", type=int, default=8191)
    ap.add_argument("--width", type=int, default=256)
    ap.add_argument("--blocks", type=int, default=2)
    ap.add_argument("--tokens", type=int, default=1000)
    ap.add_argument("--clip", type=float, default=None, help="largest norm of all gradients")
    a = ap.parse_args()
    runs = [train(a.vocab, a.width, a.blocks, a.tokens, a.steps, clip=a.clip) for _ in range(2)]
    (losses, digest), (losses2, digest2) = runs
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {a.steps} steps; weights sha256 {digest[:16]}")
    if losses != losses2 or digest != digest2:
        raise SystemExit("the two runs differ")
    if not losses[-1] < losses[0]:
        raise SystemExit("the loss did not fall")
    print("two runs agree bit for bit")


if __name__ == "__main__":
    main()
