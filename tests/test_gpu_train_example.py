"""The training example: its gradients against torch's own in 64 bits, and a
falling loss under the Muon and AdamW steps."""

import importlib.util
import math
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_block.py")


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("train_block", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_network_gradients_match_autograd(example):
    # fp32: the whole network's gradients, chained through every operator.  The
    # relative error of a chain of some 20 fp32 operators, each of a few 1e-7
    # relative to its result's size, stays far below 1e-4; a wrong factor or
    # operand anywhere is of order 1.
    net = example.Net(vocab=97, d=40, hidden=136, layers=2, dtype=torch.float32, seed=3)
    gen = torch.Generator(device="cuda").manual_seed(5)
    words = torch.randint(0, 97, (150,), generator=gen, device="cuda")
    targets = torch.randint(0, 97, (150,), generator=gen, device="cuda")
    targets[::7] = -100
    loss, dmats, drest = net.gradients(words, targets)
    nn = torch.nn.functional
    rest = [p.double().requires_grad_() for p in net.rest]
    mats = [w.double().requires_grad_() for w in net.mats]
    embed, head = rest[0], rest[1]
    norm, bias = rest[2:5], rest[5:8]
    x = embed[words]
    for i in range(2):
        wg, wu, wd = mats[3 * i:3 * i + 3]
        n = nn.layer_norm(x, (40,), norm[i], bias[i], 1e-5)
        x = x + nn.linear(nn.silu(nn.linear(n, wg)) * nn.linear(n, wu), wd)
    want = nn.cross_entropy(nn.linear(nn.layer_norm(x, (40,), norm[2], bias[2], 1e-5), head), targets,
                            ignore_index=-100)
    assert abs(float(loss) - float(want)) < 1e-5
    grads = torch.autograd.grad(want, mats + rest)
    for got, ref in zip(dmats + drest, grads):
        assert float((got.double() - ref).norm()) <= 1e-4 * float(ref.norm())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_training_lowers_the_loss(example, dtype):
    losses = example.train(steps=40, dtype=dtype, tokens=1024)
    assert abs(losses[0] - math.log(512)) < 1.5
    assert losses[-1] < 0.5 * losses[0]
