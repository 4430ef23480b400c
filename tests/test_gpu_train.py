"""Training operators on the GPU against their 64-bit forms, element by element
(train_ref derives the bounds from the formulas and the types' roundings)."""

import pytest
import torch

import matrix_orthogonalising_optimizer_amd as dm
import train_ref as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dm.load_library()


def gen(*shape, seed, std=1.0, mean=0.0, dtype=BF16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(shape, device="cuda").normal_(mean, std, generator=g).to(dtype)


def offset_copy(t, k):
    """t's values in a contiguous tensor that starts k elements into its buffer."""
    buf = torch.empty(t.numel() + k, dtype=t.dtype, device=t.device)
    v = buf[k:].view(t.shape)
    v.copy_(t)
    return v


def kernels(fn):
    """fn()'s result and the names of the kernels it launched."""
    dm.timing_enable(True)
    try:
        out = fn()
        torch.cuda.synchronize()
    finally:
        dm.timing_enable(False)
    return out, [k["kernel"] for k in dm.timing_report()["kernels"]]


# ------------------------------------------------------------ layer norm
LN_NAMES = ["y", "mean", "rstd", "dx", "dw", "db"]


def run_ln(x, w, b, dy, eps=1e-5):
    y, mean, rstd = dm.layer_norm(x, w, b, eps=eps)
    dx, dw, db = dm.layer_norm_backward(dy, x, w, mean, rstd, bias=b is not None)
    got = [y, mean, rstd, dx, dw] + ([db] if db is not None else [])
    vals, errs = ref.layer_norm(x, w, b, eps, dy)
    ref.check(got, vals, errs, LN_NAMES)
    return got


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,width", [
    (1, 1), (1, 4096), (3, 2), (5, 7), (2, 8), (9, 511), (4, 512), (6, 513), (7, 1001), (300, 1024), (5, 1025),
    (33, 2048), (3, 2049), (1500, 4096), (4, 4097), (5, 8192), (3, 8200), (3, 9001), (2, 16384), (3, 16385),
    (70, 20000)])
def test_layer_norm(rows, width, dtype):
    x = gen(rows, width, seed=1, mean=0.7, dtype=dtype)
    x[:, ::17] *= 20
    run_ln(x, gen(width, seed=2, std=0.3, mean=1.0, dtype=dtype), gen(width, seed=3, dtype=dtype),
           gen(rows, width, seed=4, dtype=dtype))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_layer_norm_without_bias_and_unaligned(dtype):
    x, w, dy = gen(37, 264, seed=1, dtype=dtype), gen(264, seed=2, dtype=dtype), gen(37, 264, seed=3, dtype=dtype)
    a = run_ln(x, w, None, dy)
    b = run_ln(offset_copy(x, 1), offset_copy(w, 1), None, offset_copy(dy, 1))
    for p, q in zip(a[:2], b[:2]):
        torch.testing.assert_close(p, q, rtol=2 ** -7, atol=1e-6)


def test_layer_norm_offset_and_constant_rows():
    # a large common offset, a constant row (variance 0: eps decides), tiny and huge rows
    x = gen(6, 1000, seed=1, dtype=F32)
    x[0] += 300.0
    x[1] = 5.0
    x[2] *= 1e-12
    x[3] *= 1e12
    run_ln(x, gen(1000, seed=2, dtype=F32), gen(1000, seed=3, dtype=F32), gen(6, 1000, seed=4, dtype=F32))


def test_layer_norm_nonfinite_rows_stay_alone():
    x, w, b = gen(5, 300, seed=1), gen(300, seed=2), gen(300, seed=3)
    clean = dm.layer_norm(x, w, b)[0]
    x[1, 7], x[3, 299] = float("nan"), float("inf")
    y = dm.layer_norm(x, w, b)[0]
    assert torch.isnan(y[1]).all() and torch.isnan(y[3]).all()
    for r in (0, 2, 4):
        assert torch.equal(y[r], clean[r])


def test_layer_norm_shapes_and_no_rows():
    x, w = gen(2, 3, 40, seed=1), gen(40, seed=2)
    y, mean, rstd = dm.layer_norm(x, w)
    assert y.shape == x.shape and mean.shape == (2, 3) and rstd.shape == (2, 3)
    z = x[:0]
    y, mean, rstd = dm.layer_norm(z, w)
    dx, dw, db = dm.layer_norm_backward(z, z, w, mean, rstd)
    assert y.shape == z.shape and dx.shape == z.shape
    assert torch.equal(dw, torch.zeros_like(w)) and torch.equal(db, torch.zeros_like(w))


# ------------------------------------------------------------ gated block
FFN_NAMES = ["y", "dx", "dw_gate", "dw_up", "dw_down"]


def ffn_inputs(t, d, f, dtype, seed=0):
    return (gen(t, d, seed=seed + 1, dtype=dtype), gen(f, d, seed=seed + 2, std=1.5 * d ** -0.5, dtype=dtype),
            gen(f, d, seed=seed + 3, std=d ** -0.5, dtype=dtype), gen(d, f, seed=seed + 4, std=f ** -0.5, dtype=dtype),
            gen(t, d, seed=seed + 5, dtype=dtype))


def run_ffn(x, wg, wu, wd, dy, act):
    y0 = dm.gated_ffn(x, wg, wu, wd, act=act)
    y, saved = dm.gated_ffn(x, wg, wu, wd, act=act, save=True)
    assert torch.equal(y0, y)
    got = [y, *dm.gated_ffn_backward(dy, x, wg, wu, wd, saved, act=act)]
    vals, errs = ref.gated_ffn(x, wg, wu, wd, act, dy)
    ref.check(got, vals, errs, FFN_NAMES)
    return got


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("t,d,f", [(1, 1, 1), (1, 64, 128), (2, 72, 40), (63, 65, 33), (64, 64, 64), (65, 130, 259),
                                   (130, 256, 96), (300, 200, 520)])
def test_gated_ffn(t, d, f, act, dtype):
    run_ffn(*ffn_inputs(t, d, f, dtype), act)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("t,d,f", [(1, 1024, 4096), (5, 1030, 2051), (16, 4096, 512), (17, 512, 3000), (33, 1000, 1777),
                                   (100, 2048, 1024)])
def test_gated_ffn_few_tokens(t, d, f, dtype):
    run_ffn(*ffn_inputs(t, d, f, dtype), "silu")


@pytest.mark.parametrize("dtype,t,d,f,tile", [
    (BF16, 8192, 1024, 4096, "bf16, 256"), (BF16, 8189, 1032, 4100, "bf16, 256"), (BF16, 1000, 523, 2049, "bf16, 128"),
    (F32, 700, 520, 1300, "f32, 64"), (F32, 2100, 515, 1501, "f32, 64"), (F32, 2043, 515, 2010, "f32, 128"), (F32, 4096, 2048, 4096, "split, 256"),
    (F32, 4001, 1030, 4100, "split, 256")])
def test_gated_ffn_tiles(dtype, t, d, f, tile):
    args = ffn_inputs(t, d, f, dtype)
    _, names = kernels(lambda: run_ffn(*args, "silu"))
    assert any(n.startswith(f"linear_kernel<{tile}") for n in names), names


# more tiles than places on the GPU, and fewer with a long K: both depths of a tile's ring
@pytest.mark.parametrize("dtype,t,d,f", [(BF16, 1500, 128, 700), (BF16, 1531, 517, 2101), (BF16, 520, 2051, 640),
                                         (BF16, 700, 64, 4100), (F32, 1100, 300, 1501), (F32, 130, 1031, 515)])
def test_gated_ffn_rings(dtype, t, d, f):
    run_ffn(*ffn_inputs(t, d, f, dtype), "gelu")


# memory that a call was given holds NaN: what lies between a row's end and the next row reaches nothing
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("t,d,f", [(5, 515, 1030), (70, 1025, 517), (700, 523, 1100), (1100, 1032, 2052)])
def test_memory_given_may_hold_anything(t, d, f, dtype, monkeypatch):
    plain = torch.Tensor.new_empty
    monkeypatch.setattr(torch.Tensor, "new_empty", lambda self, *a, **k: plain(self, *a, **k).fill_(
        255 if k.get("dtype") == torch.uint8 else float("nan")))
    run_ffn(*ffn_inputs(t, d, f, dtype), "silu")
    args = ce_inputs(t, d, f, dtype)
    run_ce(*args)
    run_ce(*args, max_block=f * 4 * 256)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gated_ffn_unaligned_pointers(dtype):
    args = ffn_inputs(70, 72, 88, dtype)
    a = run_ffn(*args, "silu")
    b = run_ffn(*[offset_copy(t, 1) for t in args], "silu")
    for p, q in zip(a, b):
        assert torch.equal(p, q)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("t,d,f", [(10, 128, 257), (10, 65, 192), (3, 64, 9), (40, 521, 128), (1, 7, 64), (5, 130, 66)])
def test_gated_ffn_rows_at_any_element(t, d, f, dtype):
    # whole steps of K against ragged edges, and the other way round
    args = ffn_inputs(t, d, f, dtype)
    _, names = kernels(lambda: run_ffn(*args, "gelu"))
    assert any(n.endswith("raw>") for n in names), names


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("t", [9, 1500])
def test_one_unaligned_operand(t, dtype):
    args = list(ffn_inputs(t, 136, 520, dtype))
    want = run_ffn(*args, "silu")
    for k in range(5):
        part = list(args)
        part[k] = offset_copy(args[k], 1)
        got = run_ffn(*part, "silu")
        for a, b in zip(got, want):
            torch.testing.assert_close(a, b, rtol=2 ** -6 if dtype is BF16 else 1e-4, atol=1e-2 * float(b.abs().max()))


def test_gated_ffn_no_tokens():
    x, wg, wu, wd, _ = ffn_inputs(4, 24, 40, BF16)
    z = x[:0]
    y, saved = dm.gated_ffn(z, wg, wu, wd, save=True)
    dx, a, b, c = dm.gated_ffn_backward(z, z, wg, wu, wd, saved)
    assert y.shape == z.shape and dx.shape == z.shape
    assert not a.any() and not b.any() and not c.any()


def test_gated_ffn_nonfinite_tokens_stay_alone():
    # K tails and padded rows must not leak a NaN into other tokens
    x, wg, wu, wd, _ = ffn_inputs(70, 100, 52, BF16)
    clean = dm.gated_ffn(x, wg, wu, wd)
    x[3, 99], x[69, 0] = float("nan"), float("inf")
    y = dm.gated_ffn(x, wg, wu, wd)
    keep = [i for i in range(70) if i not in (3, 69)]
    assert torch.isnan(y[3]).all() and torch.isnan(y[69]).any()
    assert torch.equal(y[keep], clean[keep])


# ------------------------------------------------------------ cross entropy
CE_NAMES = ["loss", "losses", "dx", "dw"]


def ce_inputs(t, d, v, dtype, masked=0.2, seed=0):
    w = gen(v, d, seed=seed + 1, std=d ** -0.5, dtype=F32)
    g = torch.Generator(device="cuda").manual_seed(seed + 2)
    y = torch.randint(0, v, (t,), generator=g, device="cuda")
    sure = torch.rand(t, 1, generator=g, device="cuda") * 12
    x = gen(t, d, seed=seed + 3, dtype=F32) + sure * w[y]
    y[torch.rand(t, generator=g, device="cuda") < masked] = -100
    return x.to(dtype), w.to(dtype), y


def run_ce(x, w, y, planes=False, **kw):
    got = dm.linear_cross_entropy(x, w, y, **kw)
    if "max_block" not in kw:
        only = dm.linear_cross_entropy(x, w, y, grad=False)
        assert torch.equal(got[0], only[0]) and torch.equal(got[1], only[1])
    vals, errs = ref.cross_entropy(x, w, y, planes=planes)
    ref.check(got, vals, errs, CE_NAMES)
    return got


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("t,d,v", [(1, 1, 1), (1, 64, 100), (2, 33, 257), (64, 64, 1000), (65, 130, 4099), (130, 72, 31),
                                   (300, 256, 2048)])
def test_cross_entropy(t, d, v, dtype):
    run_ce(*ce_inputs(t, d, v, dtype, masked=0.0 if t == 1 else 0.2))


@pytest.mark.parametrize("dtype,t,d,v,tile", [
    (BF16, 8189, 1032, 16379, "bf16, 256"), (BF16, 1100, 515, 5003, "bf16, 128"), (F32, 700, 300, 3001, "f32, 64"),
    (F32, 4001, 1030, 8203, "split, 256")])
def test_cross_entropy_tiles(dtype, t, d, v, tile):
    args = ce_inputs(t, d, v, dtype)
    _, names = kernels(lambda: run_ce(*args))
    assert any(n.startswith(f"linear_kernel<{tile}, kk, xent") for n in names), names


@pytest.mark.parametrize("dtype,t,d,v", [(BF16, 1100, 100, 3001), (BF16, 2000, 600, 5003), (BF16, 130, 1031, 1500),
                                         (F32, 1100, 300, 3001)])
def test_cross_entropy_rings(dtype, t, d, v):
    run_ce(*ce_inputs(t, d, v, dtype))


def test_fp32_planes_hold_every_magnitude():
    # products on planes: values that round to infinity in bf16, and tiny ones
    x, w, y = ce_inputs(4001, 1030, 8203, F32, masked=0.0)
    x[:, 0] = torch.tensor([3.3999e38, -3.4028e38, 1e-30, 0.0], device="cuda").repeat(1001)[:4001]
    w[:, 0] *= 1e-37
    x[:, 1] *= 1e-25
    w[:, 1] *= 1e25
    _, names = kernels(lambda: run_ce(x, w, y, planes=True))
    assert any(n.startswith("linear_kernel<split") for n in names), names
    # an infinity or a NaN stays in its row
    x[5, 7], x[4000, 1029] = float("inf"), float("nan")
    clean = dm.linear_cross_entropy(x.nan_to_num(0.0, 0.0, 0.0), w, y, grad=False)[1]
    losses = dm.linear_cross_entropy(x, w, y, grad=False)[1]
    assert torch.isnan(losses[5]) and torch.isnan(losses[4000])
    keep = torch.ones(4001, dtype=torch.bool, device="cuda")
    keep[5] = keep[4000] = False
    assert torch.equal(losses[keep], clean[keep])


def test_fp32_planes_in_blocks_of_tokens():
    x, w, y = ce_inputs(4001, 1030, 8203, F32)
    a = run_ce(x, w, y)
    b = run_ce(x, w, y, max_block=1100 * 8203 * 10)  # four blocks, the last one smaller
    torch.testing.assert_close(a[1], b[1], rtol=1e-5, atol=1e-5)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_cross_entropy_in_blocks_of_tokens(dtype):
    x, w, y = ce_inputs(900, 72, 777, dtype)
    a = run_ce(x, w, y)
    b = run_ce(x, w, y, max_block=256 * 777 * 4)
    assert torch.equal(a[1], b[1])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("t,d,v", [(5, 131, 640), (20, 66, 1001), (3, 1, 64), (300, 77, 5000)])
def test_cross_entropy_rows_at_any_element(t, d, v, dtype):
    args = ce_inputs(t, d, v, dtype)
    _, names = kernels(lambda: run_ce(*args))
    assert any(n.endswith("raw>") for n in names), names


def test_cross_entropy_targets_that_do_not_count():
    x, w, y = ce_inputs(40, 64, 300, BF16, masked=0.0)
    y[0], y[1], y[2], y[39] = -1, 300, 2 ** 40, -(2 ** 40)
    got = run_ce(x, w, y)
    for i in (0, 1, 2, 39):
        assert got[1][i] == 0 and not got[2][i].any()
    y[:] = -100
    loss, losses, dx, dw = dm.linear_cross_entropy(x, w, y)
    assert loss == 0 and not losses.any() and not dx.any() and not dw.any()
    loss, losses, dx, dw = dm.linear_cross_entropy(x[:0], w, y[:0])
    assert loss == 0 and dx.shape == (0, 64) and not dw.any()


def test_cross_entropy_masked_tokens_may_hold_anything():
    x, w, y = ce_inputs(70, 40, 500, BF16, masked=0.0)
    y[5] = y[69] = -100
    want = dm.linear_cross_entropy(x, w, y)
    x[5], x[69, 3] = float("nan"), float("inf")
    loss, losses, dx, dw = dm.linear_cross_entropy(x, w, y)
    assert torch.equal(loss, want[0]) and torch.equal(losses, want[1]) and torch.equal(dx, want[2])
    # a NaN token times its zero gradient is NaN in the weight's sum, as in the formula
    assert torch.isnan(dw).any()


def test_cross_entropy_infinite_and_lowest_logits():
    # words that cannot be (logit -inf, or bf16's lowest value) have probability 0
    x = torch.ones(3, 8, dtype=BF16, device="cuda")
    w = gen(300, 8, seed=1)
    w[10:200, 0] = -float("inf")
    w[200:230, 0] = torch.finfo(BF16).min
    y = torch.tensor([0, 5, 299], device="cuda")
    loss, losses = dm.linear_cross_entropy(x, w, y, grad=False)
    l = x.double() @ w.double().T
    want = torch.logsumexp(l, 1) - l.gather(1, y[:, None])[:, 0]
    torch.testing.assert_close(losses.double(), want, rtol=1e-5, atol=1e-5)
    # a whole piece of words at -inf, the target among the others
    w[:256, 0] = -float("inf")
    loss, losses = dm.linear_cross_entropy(x, w, torch.full((3,), 299, device="cuda"), grad=False)
    l = x.double() @ w.double().T
    torch.testing.assert_close(losses.double(), torch.logsumexp(l, 1) - l[:, 299], rtol=1e-5, atol=1e-5)


def test_cross_entropy_sure_predictions_keep_their_gradient():
    # p = 1 - 1e-4 .. 1 - 1e-7: 1 - p lies below the 16-bit rounding of p
    d, v = 64, 512
    w = torch.zeros(v, d, dtype=BF16, device="cuda")
    w[0, 0] = 1.0
    w[1:, 1] = 1.0
    x = torch.zeros(4, d, dtype=BF16, device="cuda")
    x[:, 0] = torch.tensor([16.0, 18.0, 20.0, 22.0])
    run_ce(x, w, torch.zeros(4, dtype=torch.int64, device="cuda"))


# ------------------------------------------------------------ use
def test_other_streams_and_graph_replays():
    x, wg, wu, wd, dy = ffn_inputs(200, 136, 264, BF16)
    lw, lb = gen(136, seed=20), gen(136, seed=21)
    cx, cw, cy = ce_inputs(200, 136, 999, BF16)

    def step(**kw):
        n, mean, rstd = dm.layer_norm(x, lw, lb, **kw)
        y, saved = dm.gated_ffn(n, wg, wu, wd, save=True, **kw)
        out = [n, y, *dm.gated_ffn_backward(dy, n, wg, wu, wd, saved, **kw)]
        out += dm.layer_norm_backward(out[2], x, lw, mean, rstd, **kw)
        return out + list(dm.linear_cross_entropy(cx, cw, cy, **kw))

    want = step()
    again = step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, again))  # the same bits on every run
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(3):
        for t in out:
            t.zero_()
        junk = torch.randn(1 << 20, device="cuda").sum()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, out)), i
    del junk


def test_binding_refusals():
    x, wg, wu, wd, dy = ffn_inputs(4, 16, 24, BF16)
    w = gen(16, seed=1)
    y = torch.zeros(4, dtype=torch.int64, device="cuda")
    bad = [
        lambda: dm.layer_norm(x.t(), w[:4]), lambda: dm.layer_norm(x, w.float()), lambda: dm.layer_norm(x, w[:8]),
        lambda: dm.layer_norm(x, w.cpu()), lambda: dm.layer_norm_backward(dy[:2], x, w, y.float(), y.float()),
        lambda: dm.gated_ffn(x, wg, wu[:8], wd), lambda: dm.gated_ffn(x, wg, wu, wd.t().contiguous()),
        lambda: dm.gated_ffn(x, wg, wu.float(), wd), lambda: dm.gated_ffn(x, wg, wu, wd, act="relu"),
        lambda: dm.gated_ffn_backward(dy, x, wg, wu, wd, torch.empty(8, dtype=torch.uint8, device="cuda")),
        lambda: dm.linear_cross_entropy(x, wg, y.int()), lambda: dm.linear_cross_entropy(x, wg[:, :8], y),
        lambda: dm.linear_cross_entropy(x, wg, y[:2]), lambda: dm.linear_cross_entropy(x[:, ::2], wg[:, :8], y),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was accepted")
    with pytest.raises(TypeError):
        dm.layer_norm(x.half(), w.half())
