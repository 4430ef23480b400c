"""Train a small residual network with the library's operators alone: gated
feed-forward blocks behind layer norms, a linear head with cross entropy, the
Muon step for the blocks' matrices and AdamW for everything else.

    python examples/train_block.py [--steps 60] [--dtype bf16|f32]

Synthetic data: the next word is a fixed permutation of the current one, which
the network has to learn (the loss starts at log(vocab)).  Torch looks up and
scatters the embedding's rows and adds residuals; every product, norm,
activation, loss, gradient and update runs in the library.
"""

from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import matrix_orthogonalising_optimizer_amd as dm  # noqa: E402


class Net:
    def __init__(self, vocab=512, d=256, hidden=1024, layers=2, dtype=torch.bfloat16, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, std):
            return torch.empty(shape, device="cuda").normal_(0.0, std, generator=gen).to(dtype)

        ones = torch.ones(d, device="cuda", dtype=dtype)
        self.embed, self.head = normal(vocab, d, std=1.0), normal(vocab, d, std=d ** -0.5)
        self.norm, self.bias = [ones.clone() for _ in range(layers + 1)], [0 * ones for _ in range(layers + 1)]
        # per layer: gate, up (hidden x d) and down (d x hidden)
        self.ffn = [(normal(hidden, d, std=d ** -0.5), normal(hidden, d, std=d ** -0.5),
                     normal(d, hidden, std=hidden ** -0.5)) for _ in range(layers)]
        mats = [w for ws in self.ffn for w in ws]
        self.mats, self.momenta = mats, [torch.zeros(w.shape, device="cuda") for w in mats]
        self.plan = dm.Plan([tuple(w.shape) for w in mats], dtype=dtype)
        self.rest = [self.embed, self.head, *self.norm, *self.bias]
        self.m = [torch.zeros(p.shape, device="cuda") for p in self.rest]
        self.v = [torch.zeros(p.shape, device="cuda") for p in self.rest]
        self.t = 0

    def gradients(self, words, targets):
        """The loss of a batch and the gradients of ``mats`` and ``rest``."""
        x, kept = self.embed[words], []
        for (wg, wu, wd), w, b in zip(self.ffn, self.norm, self.bias):
            n, mean, rstd = dm.layer_norm(x, w, b)
            y, saved = dm.gated_ffn(n, wg, wu, wd, save=True)
            kept.append((x, n, mean, rstd, saved))
            x = x + y
        n, mean, rstd = dm.layer_norm(x, self.norm[-1], self.bias[-1])
        loss, _, dn, dhead = dm.linear_cross_entropy(n, self.head, targets)
        dx, dw, db = dm.layer_norm_backward(dn, x, self.norm[-1], mean, rstd)
        dnorm, dbias, dmats = [dw], [db], []
        for (wg, wu, wd), w, (x, n, mean, rstd, saved) in zip(self.ffn[::-1], self.norm[-2::-1], kept[::-1]):
            dn, *dws = dm.gated_ffn_backward(dx, n, wg, wu, wd, saved)
            dr, dw, db = dm.layer_norm_backward(dn, x, w, mean, rstd)
            dx = dx + dr
            dnorm.insert(0, dw)
            dbias.insert(0, db)
            dmats = [*dws, *dmats]
        dembed = torch.zeros(self.embed.shape, device="cuda").index_add_(0, words, dx.float()).to(self.embed.dtype)
        return loss, dmats, [dembed, dhead, *dnorm, *dbias]

    def step(self, words, targets, lr=0.02):
        loss, dmats, drest = self.gradients(words, targets)
        self.t += 1
        self.plan.step(self.mats, dmats, self.momenta, lr=lr, weight_decay=0.01, mu=0.95)
        dm.adamw_step(self.rest, drest, self.m, self.v, lr=0.1 * lr, step=self.t)
        return loss


def train(steps=60, dtype=torch.bfloat16, tokens=2048, vocab=512, report=None):
    """Losses of ``steps`` training steps."""
    net = Net(vocab=vocab, dtype=dtype)
    gen = torch.Generator(device="cuda").manual_seed(1)
    perm = torch.randperm(vocab, generator=gen, device="cuda")
    losses = []
    for i in range(steps):
        words = torch.randint(0, vocab, (tokens,), generator=gen, device="cuda")
        targets = perm[words]
        targets[::16] = -100  # some tokens do not count
        losses.append(net.step(words, targets))
        if report and i % 10 == 0:
            report(i, float(losses[-1]))
    return [float(x) for x in losses]


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--dtype", choices=["bf16", "f32"], default="bf16")
    a = ap.parse_args()
    out = train(a.steps, torch.bfloat16 if a.dtype == "bf16" else torch.float32,
                report=lambda i, x: print(f"step {i:3d}  loss {x:.4f}", flush=True))
    print(f"last loss {out[-1]:.4f}; a uniform guess costs {math.log(512):.4f}")
