"""The training operators' 64-bit forms against differences and torch's own
derivatives, and the refusals of the entry points that need no device."""

import ctypes

import pytest
import torch

import matrix_orthogonalising_optimizer_amd as dm
import train_ref as ref


def close(a, b, tol=1e-10):
    assert torch.allclose(a, b, rtol=tol, atol=tol), float((a - b).abs().max())


def difference(f, x, i, h=1e-5):
    """Central difference of the scalar f along element i of x."""
    a, b = x.clone(), x.clone()
    a.view(-1)[i] += h
    b.view(-1)[i] -= h
    return float((f(a) - f(b)) / (2 * h))


def gen(*shape, seed, scale=1.0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64) * scale


@pytest.mark.parametrize("rows,width", [(1, 1), (3, 7), (5, 16)])
def test_layer_norm_form(rows, width):
    ref.ROUNDOFF[torch.float64] = 2.0 ** -53
    x, w, b, dy = gen(rows, width, seed=1), gen(width, seed=2), gen(width, seed=3), gen(rows, width, seed=4)
    (y, mean, rstd, dx, dw, db), _ = ref.layer_norm(x, w, b, 1e-5, dy)
    ts = [t.clone().requires_grad_() for t in (x, w, b)]
    z = torch.nn.functional.layer_norm(ts[0], (width,), ts[1], ts[2], 1e-5)
    close(y, z.detach())
    for a, c in zip((dx, dw, db), torch.autograd.grad(z, ts, dy)):
        close(a, c)
    f = lambda v: (ref.layer_norm(v, w, b, 1e-5)[0][0] * dy).sum()
    for i in range(0, x.numel(), 5):
        assert abs(difference(f, x, i) - float(dx.view(-1)[i])) < 1e-6 * (1 + float(rstd.max()) ** 2)


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("t,d,f", [(1, 1, 1), (3, 4, 5), (6, 5, 3)])
def test_gated_ffn_form(act, t, d, f):
    ref.ROUNDOFF[torch.float64] = 2.0 ** -53
    x, wg, wu, wd, dy = (gen(*s, seed=i) for i, s in enumerate([(t, d), (f, d), (f, d), (d, f), (t, d)]))
    vals, _ = ref.gated_ffn(x, wg, wu, wd, act, dy)
    for k, p in enumerate((x, wg, wu, wd)):
        def loss(v, k=k):
            ps = [x, wg, wu, wd]
            ps[k] = v
            return (ref.gated_ffn(*ps, act)[0][0] * dy).sum()
        for i in range(p.numel()):
            assert abs(difference(loss, p, i) - float(vals[1 + k].view(-1)[i])) < 1e-6


@pytest.mark.parametrize("t,d,v,masked", [(1, 1, 1, 0), (4, 3, 5, 0), (6, 4, 7, 3), (3, 2, 4, 3)])
def test_cross_entropy_form(t, d, v, masked):
    ref.ROUNDOFF[torch.float64] = 2.0 ** -53
    x, w = gen(t, d, seed=1), gen(v, d, seed=2)
    y = torch.randint(0, v, (t,), generator=torch.Generator().manual_seed(3))
    y[:masked] = torch.tensor([-100, v, -1])[:masked]
    (loss, losses, dx, dw), _ = ref.cross_entropy(x, w, y)
    close(losses, torch.nn.functional.cross_entropy(
        x @ w.T, torch.where((y >= 0) & (y < v), y, torch.full_like(y, -100)), ignore_index=-100, reduction="none"))
    for k, (p, gr) in enumerate(((x, dx), (w, dw))):
        def f(q, k=k):
            a, b = (q, w) if k == 0 else (x, q)
            return ref.cross_entropy(a, b, y)[0][0]
        for i in range(p.numel()):
            assert abs(difference(f, p, i) - float(gr.view(-1)[i])) < 1e-7


# ------------------------------------------------------------ refusals (nothing reaches a device)
P = ctypes.c_void_p(4096)   # never dereferenced: every call below is refused on the host
BAD = ctypes.c_void_p(4096 + 16)
N = None
BIG = 1 << 60


@pytest.fixture(scope="module")
def lib():
    return dm.load_library()


def refused(rc, text, lib):
    assert rc == dm.EINVAL
    assert text in lib.dmuon_last_error().decode()


def test_layer_norm_refusals(lib):
    f = lib.dmuon_layernorm_fwd
    refused(f(N, P, P, P, P, P, 4, 8, 1e-5, 0, N), "NULL", lib)
    refused(f(P, N, P, P, P, P, 4, 8, 1e-5, 0, N), "weight is NULL", lib)
    refused(f(P, P, P, P, P, N, 4, 8, 1e-5, 0, N), "NULL", lib)
    refused(f(P, P, P, P, P, P, -1, 8, 1e-5, 0, N), "out of range", lib)
    refused(f(P, P, P, P, P, P, 1 << 31, 8, 1e-5, 0, N), "out of range", lib)
    refused(f(P, P, P, P, P, P, 4, 0, 1e-5, 0, N), "width", lib)
    refused(f(P, P, P, P, P, P, 4, (1 << 20) + 1, 1e-5, 0, N), "width", lib)
    refused(f(P, P, P, P, P, P, 4, 8, 1e-5, 2, N), "dtype", lib)
    refused(f(P, P, P, P, P, P, 4, 8, -1.0, 0, N), "eps", lib)
    refused(f(P, P, P, P, P, P, 4, 8, float("nan"), 0, N), "eps", lib)
    assert f(N, P, N, N, N, N, 0, 8, 1e-5, 0, N) == dm.OK      # no rows
    b = lib.dmuon_layernorm_bwd
    need = lib.dmuon_layernorm_bwd_workspace(4, 8)
    assert need > 0
    refused(b(P, P, P, P, P, P, P, P, 4, 8, 0, P, need - 1, N), "workspace", lib)
    refused(b(P, P, P, P, P, P, P, P, 4, 8, 0, N, need, N), "workspace", lib)
    refused(b(P, P, P, P, P, P, P, P, 4, 8, 0, BAD, need, N), "workspace", lib)
    refused(b(N, P, P, P, P, P, P, P, 4, 8, 0, P, need, N), "NULL", lib)
    refused(b(P, P, P, P, P, P, N, P, 4, 8, 0, P, need, N), "NULL", lib)
    assert lib.dmuon_layernorm_bwd_workspace(-1, 8) == dm.EINVAL


def test_gated_ffn_refusals(lib):
    f = lib.dmuon_gated_ffn_fwd
    good = [P, P, P, P, P, N, 4, 8, 16, 0, 0, P, BIG, N]
    def call(**kw):
        a = list(good)
        for k, v in kw.items():
            a[int(k[1:])] = v
        return f(*a)
    for k in range(5):
        refused(call(**{f"_{k}": N}), "NULL", lib)
    refused(call(_5=BAD), "saved", lib)
    refused(call(_6=-1), "out of range", lib)
    refused(call(_7=0), "width", lib)
    refused(call(_8=0), "hidden", lib)
    refused(call(_8=(1 << 20) + 1), "hidden", lib)
    refused(call(_9=3), "activation", lib)
    refused(call(_10=7), "dtype", lib)
    refused(call(_12=0), "workspace", lib)
    refused(call(_11=BAD), "workspace", lib)
    assert f(N, P, P, P, N, N, 0, 8, 16, 0, 0, N, 0, N) == dm.OK
    b = lib.dmuon_gated_ffn_bwd
    need = lib.dmuon_gated_ffn_bwd_workspace(4, 8, 16, 0, 0)
    for k in range(10):
        a = [P] * 10 + [4, 8, 16, 0, 0, P, need, N]
        a[k] = N
        refused(b(*a), "NULL", lib)
    refused(b(*([P] * 10 + [4, 8, 16, 0, 0, P, need - 256, N])), "workspace", lib)
    # rows that are not 16-byte aligned need room for padded copies
    assert lib.dmuon_gated_ffn_bwd_workspace(4, 8, 16, 0, 1) > need
    assert lib.dmuon_gated_ffn_bwd_workspace(4, 9, 16, 0, 0) > need
    assert lib.dmuon_gated_ffn_saved(4, 17, 0) == 3 * 4 * 24 * 2 + 4 * 32
    assert lib.dmuon_gated_ffn_saved(4, 17, 1) == 3 * 4 * 20 * 4
    assert lib.dmuon_gated_ffn_saved(4, 0, 0) == dm.EINVAL


def test_linear_xent_refusals(lib):
    f = lib.dmuon_linear_xent
    need = lib.dmuon_linear_xent_workspace(4, 8, 100, 0, 1, 0, 0)
    good = [P, P, P, P, P, P, P, 4, 8, 100, 0, 0, P, need, N]
    def call(**kw):
        a = list(good)
        for k, v in kw.items():
            a[int(k[1:])] = v
        return f(*a)
    for k in range(5):
        refused(call(**{f"_{k}": N}), "NULL", lib)
    refused(call(_5=N), "both or neither", lib)
    refused(call(_6=N), "both or neither", lib)
    refused(call(_7=-1), "out of range", lib)
    refused(call(_8=0), "width", lib)
    refused(call(_9=0), "vocabulary", lib)
    refused(call(_9=(1 << 22) + 1), "vocabulary", lib)
    refused(call(_10=5), "dtype", lib)
    refused(call(_11=-1), "max_block", lib)
    refused(call(_13=need - 256), "workspace", lib)
    assert lib.dmuon_linear_xent_workspace(4, 8, 0, 0, 1, 0, 0) == dm.EINVAL
    # the exponentials of one block of tokens bound the workspace
    whole = lib.dmuon_linear_xent_workspace(8192, 64, 32000, 0, 1, 1 << 40, 0)
    part = lib.dmuon_linear_xent_workspace(8192, 64, 32000, 0, 1, 64 << 20, 0)
    assert whole > 8192 * 32000 * 2 and part < 160 << 20


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 8)
    for call in (lambda: dm.layer_norm(x, x[0]), lambda: dm.gated_ffn(x, x, x, x),
                 lambda: dm.linear_cross_entropy(x, x, torch.zeros(4, dtype=torch.int64)),
                 lambda: dm.layer_norm_backward(x, x, x[0], x[:, 0], x[:, 0]),
                 lambda: dm.gated_ffn_backward(x, x, x, x, x, x)):
        with pytest.raises(ValueError, match="GPU"):
            call()


def test_workspace_of_unaligned_calls_covers_every_choice(lib):
    # one misaligned pointer may change how all operands are taken: the size
    # asked with `unaligned` must be the one that the call checks against
    odd = ctypes.c_void_p(4096 + 2)
    for t, d, f in [(1, 64, 128), (10, 1000, 4096), (700, 1024, 4096), (5000, 512, 2048)]:
        for dt in (0, 1):
            need = lib.dmuon_gated_ffn_bwd_workspace(t, d, f, dt, 1)
            args = [P] * 10 + [t, d, f, 0, dt, P, need - 256, N]
            args[1] = odd
            refused(lib.dmuon_gated_ffn_bwd(*args), f"{need} needed", lib)
            need = lib.dmuon_gated_ffn_fwd_workspace(t, d, f, dt, 1)
            args = [P, P, odd, P, P, N, t, d, f, 0, dt, P, need - 256, N]
            refused(lib.dmuon_gated_ffn_fwd(*args), f"{need} needed", lib)
            need = lib.dmuon_linear_xent_workspace(t, d, 5000, dt, 1, 0, 1)
            args = [P, odd, P, P, P, P, P, t, d, 5000, dt, 0, P, need - 256, N]
            refused(lib.dmuon_linear_xent(*args), f"{need} needed", lib)


def test_products_of_too_many_tiles_are_refused(lib):
    assert lib.dmuon_linear_xent_workspace(1 << 30, 1, 1 << 22, 0, 0, 0, 0) == dm.EUNSUPPORTED
