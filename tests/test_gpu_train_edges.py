"""Corners of the training operators on the GPU: widths of a few elements,
values at the ends of fp32's range, calls by keyword, very long batches."""

import pytest
import torch

import matrix_orthogonalising_optimizer_amd as dm
import train_ref as ref
from test_gpu_train import BF16, CE_NAMES, F32, ce_inputs, ffn_inputs, gen, kernels, run_ce, run_ffn

pytestmark = pytest.mark.gpu

inf = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dm.load_library()


# rows at any element, so narrow that a 16-byte chunk spans several: the rows behind the
# last whole step of K hold less than a chunk
@pytest.mark.parametrize("dtype,k", [(BF16, 65), (BF16, 66), (BF16, 70), (F32, 33), (F32, 34)])
@pytest.mark.parametrize("n", [1, 2, 3])
def test_narrow_rows_end_inside_a_chunk(n, k, dtype):
    args = ce_inputs(3, n, k, dtype, masked=0.0)
    _, names = kernels(lambda: run_ce(*args))
    assert any(", kr, out, raw>" in s for s in names), names
    run_ffn(*ffn_inputs(3, n, k, dtype), "silu")
    run_ffn(*ffn_inputs(3, k, n, dtype), "silu")


# fp32 products on planes: an infinite weight makes infinite logits and hidden values, as fp32 products do
def test_planes_words_that_cannot_be():
    x, w, y = ce_inputs(4001, 1030, 8203, F32)
    x[:, 7] = 1.0
    out = torch.zeros(8203, dtype=torch.bool, device="cuda")
    out[100:600] = out[8200] = True
    y[(y >= 0) & out[y.clamp(min=0)]] = 50
    keep = torch.nonzero(~out)[:, 0]
    place = torch.cumsum(~out, 0) - 1
    y2 = torch.where(y >= 0, place[y.clamp(min=0)], y)
    vals, errs = ref.cross_entropy(x, w[keep], y2, planes=True)
    w[out, 7] = -inf
    (loss, losses, dx, dw), names = kernels(lambda: dm.linear_cross_entropy(x, w, y))
    assert any(n.startswith("linear_kernel<split, 256, kk, xent") for n in names), names
    assert not dw[out].any()                     # probability 0
    assert torch.isnan(dx[y >= 0, 7]).all()      # 0 times -inf, as in the formula
    cols = [c for c in range(1030) if c != 7]
    ref.check([loss, losses, dx[:, cols], dw[keep]], [vals[0], vals[1], vals[2][:, cols], vals[3]],
              [errs[0], errs[1], errs[2][:, cols], errs[3]], CE_NAMES)


def test_planes_infinite_hidden_values():
    x, wg, wu, wd, dy = ffn_inputs(4001, 1030, 4100, F32)
    x[:, 3] = 1.0
    wu[9, 3] = inf
    y, names = kernels(lambda: dm.gated_ffn(x, wg, wu, wd))
    assert any(n.startswith("linear_kernel<split, 256, kk, gate") for n in names), names
    g = x.double() @ wg[9].double()
    sure = g.abs() > 1e-4
    want = torch.sign(g)[:, None] * torch.sign(wd[:, 9].double())[None, :] * inf
    assert torch.equal(y[sure].double(), want[sure])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("width", [100, 72, 500, 1001, 4100])
def test_layer_norm_gradient_of_huge_constant_rows(width, dtype):
    # 2^112 in every place: the mean is exact, xh is 0, and mean rstd (2^112 times 10^6) is past fp32's range
    x = torch.full((6, width), 2.0 ** 112, dtype=dtype, device="cuda")
    w, dy = gen(width, seed=2, dtype=dtype), gen(6, width, seed=4, dtype=dtype)
    y, mean, rstd = dm.layer_norm(x, w, eps=1e-12)
    assert torch.equal(mean, x[:, 0].float()) and not y.any()
    dx, dw, db = dm.layer_norm_backward(dy, x, w, mean, rstd)
    g = dy.double() * w.double()
    r, m = 1e-12 ** -0.5, g.mean(1, keepdim=True)
    want = r * (g - m)
    bound = (ref.ROUNDOFF[dtype] + 8 * 2.0 ** -24) * want.abs() + r * (
        ref.acc(width) * g.abs().mean(1, keepdim=True) + 8 * 2.0 ** -24 * (g.abs() + m.abs()))
    ref.check([dx, dw], [want, torch.zeros_like(w).double()], [1.01 * bound, torch.zeros_like(w).double()], ["dx", "dw"])


# more workgroups than one launch takes
def test_layer_norm_of_very_many_rows():
    rows = 2 ** 28 + 3
    x = torch.empty(rows, 2, dtype=BF16, device="cuda").normal_()
    w, b = gen(2, seed=1), gen(2, seed=2)
    y, mean, rstd = dm.layer_norm(x, w, b)
    for at in (0, 2 ** 25 - 500, 2 ** 27, rows - 1000):
        part = x[at:at + 1000].contiguous()
        for a, c in zip((y, mean, rstd), dm.layer_norm(part, w, b)):
            assert torch.equal(a[at:at + 1000], c)
    vals, errs = ref.layer_norm(x[-1000:], w, b, 1e-5)
    ref.check([y[-1000:]], vals, errs, ["y"])


def test_cross_entropy_of_very_many_tokens():
    run_ce(*ce_inputs(2 ** 24 + 5, 2, 3, BF16))


def test_weight_gradient_of_very_many_elements():
    v, d = 2 ** 22, 4096
    w = torch.empty(v, d, dtype=BF16, device="cuda").normal_(0.0, d ** -0.5)
    x = gen(512, d, seed=1)
    y = torch.randint(0, v, (512,), device="cuda")
    # two blocks of tokens, their sum rounded in one pass, against one block
    a = dm.linear_cross_entropy(x, w, y, max_block=1 << 30)
    b = dm.linear_cross_entropy(x, w, y, max_block=1 << 40)
    torch.testing.assert_close(a[1], b[1], rtol=1e-5, atol=1e-5)
    for r in (0, v // 2, v - 4096):
        p, q = a[3][r:r + 4096].float(), b[3][r:r + 4096].float()
        torch.testing.assert_close(p, q, rtol=2 ** -6, atol=1e-2 * float(q.abs().max()))


def test_cross_entropy_of_very_many_tiles():
    n = 2 ** 20
    x, w, y = ce_inputs(n, 8, n, BF16)
    loss, losses = dm.linear_cross_entropy(x, w, y, grad=False)
    at = torch.tensor([0, 1, 255, 256, 70001, 524288, n - 300, n - 1], device="cuda")
    vals, errs = ref.cross_entropy(x[at], w, y[at], grad=False)
    ref.check([losses[at]], vals[1:], errs[1:], ["losses"])
    assert abs(float(losses.double().sum() / (y >= 0).sum()) - float(loss)) < 1e-5 * float(loss)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("t,d,v,rows", [(900, 72, 777, 256), (2048, 256, 2000, 256), (3000, 64, 3000, 512),
                                        (5000, 512, 4000, 1024), (4001, 1030, 8203, 1100), (700, 2048, 520, 256)])
def test_loss_in_blocks_does_not_depend_on_gradients(t, d, v, rows, dtype):
    x, w, y = ce_inputs(t, d, v, dtype)
    block = rows * v * (2 if dtype is BF16 else 10)
    a = dm.linear_cross_entropy(x, w, y, max_block=block)
    b = dm.linear_cross_entropy(x, w, y, max_block=block, grad=False)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def activation(g, act, dtype=F32):
    """act(g) and its derivative by the block: u = dh = 1."""
    x = torch.stack([g, torch.ones_like(g)], 1).to(dtype)
    e = torch.eye(2, device="cuda", dtype=dtype)
    wg, wu, wd = e[:1].clone(), e[1:].clone(), e[:, :1].clone()
    y, saved = dm.gated_ffn(x, wg, wu, wd, act=act, save=True)
    dy = torch.zeros_like(x)
    dy[:, 0] = 1.0
    return y[:, 0], dm.gated_ffn_backward(dy, x, wg, wu, wd, saved, act=act)[0][:, 0]


# Relative to the value, far out too.  An exponential of z costs z 2^-24 for each
# rounding of its argument (z itself, its factors, log2 e); the rest, a
# polynomial's terms and quotients among them, less than 24 roundings.  The
# derivative is a sum of two terms, bounded by their magnitudes.
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_activation_tails(act):
    g = torch.linspace(-9.0, 9.0, 20001, device="cuda")
    a, da = activation(g, act)
    A, D, _ = ref.act(g.double(), act)
    z = g.double()
    if act == "gelu":
        e = 1.25 * z * z
        mag = 0.5 * torch.erfc(-z * 0.5 ** 0.5) + z.abs() * torch.exp(-0.5 * z * z) / (2 * torch.pi) ** 0.5
    elif act == "silu":
        e = 2.5 * z.abs()
        p = torch.sigmoid(z)
        mag = p + z.abs() * p * (1 - p)
    else:
        q = 2 * (2 / torch.pi) ** 0.5 * (z + 0.044715 * z ** 3)
        e = 6 * q.abs()
        p = torch.sigmoid(q)
        A = z * p  # (1 + tanh cancels in 64 bits too)
        D = p + z * p * torch.sigmoid(-q) * 2 * (2 / torch.pi) ** 0.5 * (1 + 0.134145 * z * z)
        mag = p + z.abs() * p * torch.sigmoid(-q) * 2 * (2 / torch.pi) ** 0.5 * (1 + 0.134145 * z * z)
    ref.check([a, da], [A, D], [(e + 24) * 2.0 ** -24 * A.abs(), (e + 24) * 2.0 ** -24 * mag], ["act", "derivative"])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_activations_of_huge_values(act, dtype):
    g = torch.tensor([1e20, -1e20, 3e38, -3e38, 200.0, -200.0], device="cuda")
    a, da = activation(g, act, dtype)
    assert torch.equal(a.float(), g.to(dtype).float().clamp(min=0) + 0.0)
    assert torch.equal(da.float(), (g > 0).float())
