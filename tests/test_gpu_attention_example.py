"""The attention example: its gradients against torch's own in 64 bits, and its run."""

import importlib.util
import math
import os

import pytest
import torch

import heads_ref as hr

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_attention.py")


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("train_attention", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def rotated(x, w, positions):
    """Norm and rotation of heads as the formula has them, in differentiable torch."""
    n = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w
    half = x.shape[-1] // 2
    turn = positions[:, None].double() * 10000.0 ** (-torch.arange(half, device=x.device).double() / half)
    c, s = turn.cos()[:, None], turn.sin()[:, None]
    a, b = n[..., :half], n[..., half:]
    return torch.cat([a * c - b * s, b * c + a * s], -1)


@pytest.mark.parametrize("p", [0.0, 0.25])
def test_network_gradients_match_autograd(example, p):
    # fp32: the whole network's gradients, chained through every operator.  The relative
    # error of a chain of some 30 fp32 operators, each of a few 1e-7 relative to
    # its result's size, stays far below 1e-4; a wrong factor or operand anywhere is of
    # order 1.
    lengths, vocab, d, heads, kv, dim, seed = (70, 1, 33, 40), 61, 48, 4, 2, 20, 9
    net = example.Net(vocab=vocab, d=d, hidden=72, layers=2, heads=heads, kv_heads=kv, dim=dim, dtype=torch.float32,
                      seed=3)
    gen = torch.Generator(device="cuda").manual_seed(5)
    for w in net.rest[2:]:  # (norms that scale, biases that shift)
        w += 0.3 * torch.empty_like(w).normal_(generator=gen)
    tokens = sum(lengths)
    words = torch.randint(0, vocab, (tokens,), generator=gen, device="cuda")
    targets = torch.randint(0, vocab, (tokens,), generator=gen, device="cuda")
    targets[::7] = -100
    positions, cu = example.packed(lengths)
    loss, dmats, drest = net.gradients(words, targets, positions, cu, p=p, seed=seed)
    nn = torch.nn.functional
    rest = [w.double().requires_grad_() for w in net.rest]
    mats = [w.double().requires_grad_() for w in net.mats]
    x, groups = rest[0][words], (tokens * d + 7) // 8
    for i in range(2):
        wqkv, wo, wg, wu, wd = mats[5 * i:5 * i + 5]
        n1, b1, nq, nk, n2, b2 = rest[4 + 6 * i:10 + 6 * i]

        def drop(z, at):
            if p == 0.0:
                return z
            kept = hr.keep(z.numel(), p, seed, (2 * i + at) * groups)
            return z * torch.as_tensor(kept, device="cuda").view_as(z) / (1 - p)

        q, k, v = nn.linear(nn.layer_norm(x, (d,), n1, b1, 1e-5), wqkv).view(tokens, -1, dim).split((heads, kv, kv), 1)
        q, k = rotated(q, nq, positions), rotated(k, nk, positions)
        ys, at = [], 0
        for n in lengths:
            qs = q[at:at + n].transpose(0, 1)
            ks, vs = (t[at:at + n].transpose(0, 1).repeat_interleave(heads // kv, 0) for t in (k, v))
            s = (qs @ ks.transpose(1, 2)) * dim ** -0.5
            s = s.masked_fill(~torch.ones(n, n, dtype=torch.bool, device="cuda").tril(), -math.inf)
            ys.append((s.softmax(-1) @ vs).transpose(0, 1))
            at += n
        x = x + drop(nn.linear(torch.cat(ys).flatten(1), wo), 0)
        n = nn.layer_norm(x, (d,), n2, b2, 1e-5)
        x = x + drop(nn.linear(nn.silu(nn.linear(n, wg)) * nn.linear(n, wu), wd), 1)
    want = nn.cross_entropy(nn.linear(nn.layer_norm(x, (d,), rest[2], rest[3], 1e-5), rest[1]), targets,
                            ignore_index=-100)
    assert abs(float(loss) - float(want.detach())) < 1e-5
    for got, ref in zip(dmats + drest, torch.autograd.grad(want, mats + rest)):
        assert float((got.double() - ref).norm()) <= 1e-4 * float(ref.norm())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_example_runs(example, dtype):
    losses = example.train(steps=4, dtype=dtype)
    assert len(losses) == 4 and all(math.isfinite(x) for x in losses)
