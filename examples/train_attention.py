"""Train a small causal transformer on packed sequences: attention layers of grouped
heads with their norm and rotation, dropout into the residual stream, gated
feed-forward blocks, a linear head with cross entropy, the Muon step for the
layers' matrices and AdamW for everything else.

    python examples/train_attention.py [--steps 150] [--dtype bf16|f32]

Synthetic data: the word to predict is a fixed permutation of the one three places
before (which attention has to find; it counts from the fourth word of a
sequence on), in sequences of unlike lengths that one batch packs.  Torch looks up
and scatters the embedding's rows and multiplies by the projections; every norm,
rotation, attention, dropout, feed-forward block, loss, gradient of these and update
runs in the library.
"""

from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import matrix_orthogonalising_optimizer_amd as dm  # noqa: E402


class Layer:
    def __init__(self, normal, ones, d, hidden, heads, kv_heads, dim):
        self.w_qkv, self.w_out = normal((heads + 2 * kv_heads) * dim, d), normal(d, heads * dim)
        self.w_gate, self.w_up, self.w_down = normal(hidden, d), normal(hidden, d), normal(d, hidden)
        self.norm1, self.bias1, self.norm2, self.bias2 = ones(d), 0 * ones(d), ones(d), 0 * ones(d)
        self.norm_q, self.norm_k = ones(dim), ones(dim)
        self.split = (heads, kv_heads, kv_heads)
        self.dim = dim

    def mats(self):
        return [self.w_qkv, self.w_out, self.w_gate, self.w_up, self.w_down]

    def rest(self):
        return [self.norm1, self.bias1, self.norm_q, self.norm_k, self.norm2, self.bias2]

    def forward(self, x, positions, cu, p, seed, offset):
        n1, mean1, rstd1 = dm.layer_norm(x, self.norm1, self.bias1)
        # q, k and v stay where the projection wrote them
        q0, k0, v = (n1 @ self.w_qkv.T).view(len(x), -1, self.dim).split(self.split, 1)
        q, k = dm.qk_norm_rope(q0, k0, positions, self.norm_q, self.norm_k)
        y, lse = dm.attention(q, k, v, cu)
        a = dm.dropout(y.flatten(1) @ self.w_out.T, p, seed, offset=offset, residual=x)
        n2, mean2, rstd2 = dm.layer_norm(a, self.norm2, self.bias2)
        z, saved = dm.gated_ffn(n2, self.w_gate, self.w_up, self.w_down, save=True)
        groups = (x.numel() + 7) // 8
        out = dm.dropout(z, p, seed, offset=offset + groups, residual=a)
        self.kept = x, n1, mean1, rstd1, q0, k0, q, k, v, y, lse, a, n2, mean2, rstd2, saved
        return out, offset + 2 * groups

    def backward(self, dx, positions, cu, p, seed, offset):
        """The gradient of the layer's input, of ``mats`` and of ``rest``."""
        x, n1, mean1, rstd1, q0, k0, q, k, v, y, lse, a, n2, mean2, rstd2, saved = self.kept
        dz = dm.dropout_backward(dx, p, seed, offset=offset + (x.numel() + 7) // 8)
        dn2, dwg, dwu, dwd = dm.gated_ffn_backward(dz, n2, self.w_gate, self.w_up, self.w_down, saved)
        da, dnorm2, dbias2 = dm.layer_norm_backward(dn2, a, self.norm2, mean2, rstd2)
        da = da + dx
        do = dm.dropout_backward(da, p, seed, offset=offset)
        dy, dw_out = (do @ self.w_out).view_as(y), do.T @ y.flatten(1)
        dq, dk, dv = dm.attention_backward(dy, q, k, v, y, lse, cu)
        dq, dk, dnorm_q, dnorm_k = dm.qk_norm_rope_backward(dq, dk, q0, k0, positions, self.norm_q, self.norm_k)
        dqkv = torch.cat([dq, dk, dv], 1).flatten(1)
        dn1, dw_qkv = dqkv @ self.w_qkv, dqkv.T @ n1
        dr, dnorm1, dbias1 = dm.layer_norm_backward(dn1, x, self.norm1, mean1, rstd1)
        return da + dr, [dw_qkv, dw_out, dwg, dwu, dwd], [dnorm1, dbias1, dnorm_q, dnorm_k, dnorm2, dbias2]


class Net:
    def __init__(self, vocab=256, d=256, hidden=512, layers=2, heads=4, kv_heads=2, dim=64, dtype=torch.bfloat16,
                 seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, std=None):
            std = shape[1] ** -0.5 if std is None else std
            return torch.empty(shape, device="cuda").normal_(0.0, std, generator=gen).to(dtype)

        def ones(n):
            return torch.ones(n, device="cuda", dtype=dtype)

        self.embed, self.head = normal(vocab, d, std=1.0), normal(vocab, d)
        self.norm, self.bias = ones(d), 0 * ones(d)
        self.layers = [Layer(normal, ones, d, hidden, heads, kv_heads, dim) for _ in range(layers)]
        self.mats = [w for x in self.layers for w in x.mats()]
        self.rest = [self.embed, self.head, self.norm, self.bias, *(p for x in self.layers for p in x.rest())]
        self.plan = dm.Plan([tuple(w.shape) for w in self.mats], dtype=dtype)
        self.momenta = [torch.zeros(w.shape, device="cuda") for w in self.mats]
        self.m = [torch.zeros(p.shape, device="cuda") for p in self.rest]
        self.v = [torch.zeros(p.shape, device="cuda") for p in self.rest]
        self.t = 0

    def gradients(self, words, targets, positions, cu, p=0.0, seed=0):
        """The loss of a packed batch and the gradients of ``mats`` and ``rest``."""
        x, offsets = self.embed[words], [0]
        for layer in self.layers:
            x, end = layer.forward(x, positions, cu, p, seed, offsets[-1])
            offsets.append(end)
        n, mean, rstd = dm.layer_norm(x, self.norm, self.bias)
        loss, _, dn, dhead = dm.linear_cross_entropy(n, self.head, targets)
        dx, dnorm, dbias = dm.layer_norm_backward(dn, x, self.norm, mean, rstd)
        dmats, drest = [], []
        for layer, offset in zip(self.layers[::-1], offsets[-2::-1]):
            dx, mats, rest = layer.backward(dx, positions, cu, p, seed, offset)
            dmats, drest = [*mats, *dmats], [*rest, *drest]
        dembed = torch.zeros(self.embed.shape, device="cuda").index_add_(0, words, dx.float()).to(self.embed.dtype)
        return loss, dmats, [dembed, dhead, dnorm, dbias, *drest]

    def step(self, *batch, lr=0.02, p=0.0):
        self.t += 1  # (the step is the seed: each draws its own masks)
        loss, dmats, drest = self.gradients(*batch, p=p, seed=self.t)
        self.plan.step(self.mats, dmats, self.momenta, lr=lr, weight_decay=0.01, mu=0.95)
        dm.adamw_step(self.rest, drest, self.m, self.v, lr=0.1 * lr, step=self.t)
        return loss


def packed(lengths):
    """Positions in their sequences of a batch's words, and the sequences' first rows."""
    positions = torch.cat([torch.arange(n) for n in lengths])
    cu = torch.tensor([0, *torch.tensor(lengths).cumsum(0)], dtype=torch.int32)
    return positions.cuda(), cu.cuda()


def train(steps=150, dtype=torch.bfloat16, lengths=(700, 31, 1, 256, 412, 600), vocab=256, p=0.05, report=None):
    """Losses of ``steps`` training steps."""
    net = Net(vocab=vocab, dtype=dtype)
    gen = torch.Generator(device="cuda").manual_seed(1)
    perm = torch.randperm(vocab, generator=gen, device="cuda")
    positions, cu = packed(lengths)
    losses = []
    for i in range(steps):
        words = torch.randint(0, vocab, (sum(lengths),), generator=gen, device="cuda")
        targets = torch.where(positions >= 3, perm[words.roll(3)], -100)
        losses.append(net.step(words, targets, positions, cu, p=p))
        if report and i % 10 == 0:
            report(i, float(losses[-1]))
    return [float(x) for x in losses]


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=150)
    ap.add_argument("--dtype", choices=["bf16", "f32"], default="bf16")
    a = ap.parse_args()
    out = train(a.steps, torch.bfloat16 if a.dtype == "bf16" else torch.float32,
                report=lambda i, x: print(f"step {i:3d}  loss {x:.4f}", flush=True))
    print(f"last loss {out[-1]:.4f}; a uniform guess costs {math.log(256):.4f}")
