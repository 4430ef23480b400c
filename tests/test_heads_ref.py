"""The attention block's 64-bit forms against differences and torch's own
derivatives, the generator's published values, and the refusals of the entry
points that need no device."""

import ctypes
import math

import pytest
import torch

import matrix_orthogonalising_optimizer_amd as dm
import heads_ref as ref

ref.ROUNDOFF[torch.float64] = 2.0 ** -53


def gen(*shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


def close(a, b, tol=1e-10):
    assert torch.allclose(a, b, rtol=tol, atol=tol), float((a - b).abs().max())


def difference(f, x, i, h=1e-5):
    a, b = x.clone(), x.clone()
    a.view(-1)[i] += h
    b.view(-1)[i] -= h
    return float((f(a) - f(b)) / (2 * h))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,keys,hq,hk", [([0, 4], [0, 4], 2, 1), ([1, 3, 2], [2, 5, 1], 2, 2), ([0, 5], [0, 2], 3, 1)])
def test_attention_form(lens, keys, hq, hk, causal):
    d, nq, nk = 3, sum(lens) + 1, sum(keys) + 1
    q, k, v, dy = (gen(*s, seed=i) for i, s in enumerate([(nq, hq, d), (nk, hk, d), (nk, hk, d), (nq, hq, d)]))
    vals, _ = ref.attention(q, k, v, lens, keys, causal, dy=dy)

    def loss(q, k, v):
        # row by row, from the definition
        total, a, b = 0.0, lens[0], keys[0]
        for n, m in zip(lens[1:], keys[1:]):
            for i in range(n):
                see = m if not causal else min(m, max(0, i + m - n + 1))
                for h in range(hq if see else 0):
                    p = torch.softmax(k[b:b + see, h * hk // hq] @ q[a + i, h] / math.sqrt(d), 0)
                    total = total + (p @ v[b:b + see, h * hk // hq] * dy[a + i, h]).sum()
            a, b = a + n, b + m
        return total
    leaves = [t.clone().requires_grad_() for t in (q, k, v)]
    want = loss(*leaves)
    close((vals[0] * dy).sum(), want.detach())
    for got, g in zip(vals[2:], torch.autograd.grad(want, leaves)):
        close(got, g)
    for j in range(3):
        def f(t, j=j):
            ts = [q, k, v]
            ts[j] = t
            return (ref.attention(*ts, lens, keys, causal)[0][0] * dy).sum()
        for i in range(0, vals[2 + j].numel(), 3):
            assert abs(difference(f, (q, k, v)[j], i) - float(vals[2 + j].view(-1)[i])) < 1e-7


@pytest.mark.parametrize("weights", [True, False])
@pytest.mark.parametrize("rot,sections,interleaved,per_axis", [(6, [3], False, False), (4, [2], True, False), (6, [1, 2], False, True),
                                                               (4, [1, 1], True, False), (0, [0], False, False)])
def test_norm_rope_form(rot, sections, interleaved, per_axis, weights):
    t, h, d = 4, 2, 6
    x, dy, w = gen(t, h, d, seed=1), gen(t, h, d, seed=2), gen(d, seed=3) if weights else None
    pos = torch.randint(0, 50, (t, len(sections)), generator=torch.Generator().manual_seed(4))
    how = dict(base=100.0, per_axis=per_axis, interleaved=interleaved)
    vals, _ = ref.norm_rope(x, w, pos, rot, sections, dy=dy, **how)
    # by complex numbers
    def loss(x, w):
        n = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w if weights else x
        total, p = (n[..., rot:] * dy[..., rot:]).sum(), 0
        for axis, count in enumerate(sections):
            for i in range(count):
                f = 100.0 ** (-i / count) if per_axis else 100.0 ** (-2 * p / rot)
                a, b = (2 * p, 2 * p + 1) if interleaved else (p, p + rot // 2)
                z = torch.complex(n[..., a], n[..., b]) * torch.exp(1j * (pos[:, axis, None].double() * f))
                total = total + (z.real * dy[..., a] + z.imag * dy[..., b]).sum()
                p += 1
        return total
    leaves = [x.clone().requires_grad_()] + ([w.clone().requires_grad_()] if weights else [])
    want = loss(leaves[0], leaves[-1])
    close((vals[0] * dy).sum(), want.detach())
    for got, g in zip(vals[1:], torch.autograd.grad(want, leaves)):
        close(got, g)
    f = lambda z: (ref.norm_rope(z, w, pos, rot, sections, **how)[0][0] * dy).sum()
    for i in range(0, x.numel(), 5):
        assert abs(difference(f, x, i) - float(vals[1].view(-1)[i])) < 1e-6


def test_generator_gives_the_published_values():
    # known answers of Philox 4x32-10 (counter words 2 and 3 are 0 here)
    assert ref.philox_words(0, 0) == [0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8]
    kept = ref.keep(8, 0.5, 0, 0)
    assert kept.tolist() == [w >= 0x8000 for w in (0xe8d5, 0x6627, 0xc58d, 0xe169, 0xac4c, 0xbc57, 0xdbd8, 0x9b00)]


def test_dropout_form():
    x, r = gen(40, seed=1), gen(40, seed=2)
    kept = ref.keep(40, 0.25, 9, 3)
    (y,), _ = ref.dropout(x, kept, 0.25, r)
    close(y, torch.where(kept, x / 0.75, 0.0) + r)
    assert torch.equal(ref.keep(24, 0.25, 9, 5), kept[16:40])


# ------------------------------------------------------------ refusals of the C entries
P, N, BAD, BIG = ctypes.c_void_p(4096), None, ctypes.c_void_p(4096 + 64), 1 << 40


@pytest.fixture(scope="module")
def lib():
    return dm.load_library()


def refused(rc, word, lib, code=dm.EINVAL):
    assert rc == code, rc
    assert word in lib.dmuon_last_error().decode(), lib.dmuon_last_error()


def att(**kw):
    d = dm._Attention()
    d.tokens_q, d.tokens_k, d.heads, d.kv_heads, d.head_dim, d.sequences = 8, 8, 4, 2, 64, 1
    for name, h in (("q_stride", 4), ("k_stride", 2), ("v_stride", 2), ("dy_stride", 4)):
        getattr(d, name)[:] = (h * 64, 64)
    d.scale, d.causal, d.dtype = 0.125, 1, 0
    for k, v in kw.items():
        if k.endswith("stride"):
            getattr(d, k)[:] = v
        else:
            setattr(d, k, v)
    return d


BAD_ATT = [(dict(tokens_q=-1), "tokens"), (dict(tokens_k=(1 << 30) + 1), "tokens"), (dict(heads=0), "heads"), (dict(kv_heads=0), "heads"),
           (dict(heads=5), "heads"), (dict(heads=2048), "heads"), (dict(head_dim=0), "head_dim"), (dict(sequences=0), "sequences"),
           (dict(sequences=3), "sequences"), (dict(cu_q=4096), "cu_q"), (dict(cu_k=4096), "cu_q"), (dict(scale=0.0), "scale"),
           (dict(scale=float("nan")), "scale"), (dict(scale=float("inf")), "scale"), (dict(scale=-1.0), "scale"), (dict(dtype=2), "dtype"),
           (dict(q_stride=(-64, 64)), "stride"), (dict(k_stride=(64, -1)), "stride"), (dict(v_stride=(1 << 50, 64)), "stride")]


def test_attention_refusals(lib):
    f, b = lib.dmuon_attention_fwd, lib.dmuon_attention_bwd
    for kw, word in BAD_ATT:
        refused(f(att(**kw), P, P, P, P, P, P, BIG, N), word, lib)
        refused(b(att(**kw), *[P] * 10, BIG, N), word, lib)
        assert lib.dmuon_attention_fwd_workspace(att(**kw), 0) == dm.EINVAL
        assert lib.dmuon_attention_bwd_workspace(att(**kw), 1) == dm.EINVAL
    for kw in (dict(head_dim=257), dict(head_dim=129, dtype=1), dict(tokens_q=1 << 30, heads=1024, kv_heads=1)):
        refused(f(att(**kw), P, P, P, P, P, P, BIG, N), "larger" if "head_dim" in kw else "2^36", lib, dm.EUNSUPPORTED)
    many = att(sequences=1 << 30, cu_q=P, cu_k=P)
    refused(f(many, P, P, P, P, P, P, BIG, N), "too many", lib, dm.EUNSUPPORTED)
    refused(b(many, *[P] * 10, BIG, N), "too many", lib, dm.EUNSUPPORTED)
    assert lib.dmuon_attention_bwd_workspace(att(sequences=1 << 20, cu_q=P, cu_k=P), 0) > 0
    refused(b(att(dy_stride=(-1, 1)), *[P] * 10, BIG, N), "stride", lib)
    refused(f(N, P, P, P, P, P, P, BIG, N), "NULL", lib)
    for k in range(5):
        a = [P] * 6
        a[k] = N
        refused(f(att(), *a, BIG, N), "NULL", lib)
    for k in range(9):
        a = [P] * 10
        a[k] = N
        refused(b(att(), *a, BIG, N), "NULL", lib)
    assert f(att(tokens_q=0), N, N, N, N, N, N, 0, N) == dm.OK


def test_attention_workspaces(lib):
    f, b = lib.dmuon_attention_fwd_workspace, lib.dmuon_attention_bwd_workspace
    assert f(att(), 0) == 0 and b(att(), 0) == 8 * 4 * 8
    # copies of operands that are not 16-byte aligned, or not whole 16-byte pieces
    copies = 8 * 64 * 2
    assert f(att(), 1) == copies * (4 + 2 + 2) and b(att(), 1) == copies * (4 + 2 + 2 + 4 + 4) + 256
    assert f(att(q_stride=(4 * 64 + 1, 64)), 0) == copies * 4
    assert f(att(k_stride=(128, 1 << 31)), 0) == copies * 2
    need = b(att(head_dim=60), 0)
    assert need > 256
    refused(lib.dmuon_attention_bwd(att(head_dim=60), *[P] * 10, need - 256, N), "workspace", lib)
    refused(lib.dmuon_attention_bwd(att(), *[P] * 9, N, 256, N), "workspace", lib)
    refused(lib.dmuon_attention_bwd(att(), *[P] * 9, BAD, 256, N), "workspace", lib)
    odd = ctypes.c_void_p(4096 + 2)
    refused(lib.dmuon_attention_fwd(att(), odd, P, P, P, P, P, 8, N), "workspace", lib)


def rope(**kw):
    d = dm._Rope()
    d.tokens, d.q_heads, d.k_heads, d.head_dim, d.rotary_dim = 8, 4, 2, 64, 64
    for name, h in (("q_stride", 4), ("k_stride", 2), ("dq_stride", 4), ("dk_stride", 2)):
        getattr(d, name)[:] = (h * 64, 64)
    d.sections[0], d.base, d.eps, d.axes, d.dtype = 32, 10000.0, 1e-6, 1, 0
    for k, v in kw.items():
        if k.endswith("stride"):
            getattr(d, k)[:] = v
        elif k == "sections":
            d.sections[:] = v
        else:
            setattr(d, k, v)
    return d


def test_norm_rope_refusals(lib):
    f, b = lib.dmuon_qk_norm_rope_fwd, lib.dmuon_qk_norm_rope_bwd
    for kw, word in [(dict(tokens=-1), "tokens"), (dict(q_heads=-1), "heads"), (dict(k_heads=2000), "heads"), (dict(head_dim=63), "head_dim"),
                     (dict(head_dim=258), "head_dim"), (dict(head_dim=0), "head_dim"), (dict(rotary_dim=66), "rotary_dim"),
                     (dict(rotary_dim=31), "rotary_dim"), (dict(rotary_dim=-2), "rotary_dim"), (dict(axes=0), "axes"), (dict(axes=5), "axes"),
                     (dict(sections=(31, 0, 0, 0)), "sections"), (dict(sections=(-1, 33, 0, 0), axes=2), "section"),
                     (dict(base=0.0), "base"), (dict(base=float("inf")), "base"), (dict(eps=-1.0), "eps"), (dict(eps=float("nan")), "eps"),
                     (dict(dtype=9), "dtype"), (dict(q_stride=(-1, 64)), "stride"), (dict(k_stride=(128, -64)), "stride")]:
        refused(f(rope(**kw), *[P] * 7, N), word, lib)
        refused(b(rope(**kw), *[P] * 12, BIG, N), word, lib)
        assert lib.dmuon_qk_norm_rope_bwd_workspace(rope(**kw)) == dm.EINVAL
    refused(b(rope(dq_stride=(-1, 1)), *[P] * 12, BIG, N), "stride", lib)
    refused(f(N, *[P] * 7, N), "NULL", lib)
    for k in (0, 1, 2, 5, 6):
        a = [P] * 7
        a[k] = N
        refused(f(rope(), *a, N), "NULL", lib)
    refused(f(rope(), P, P, P, P, N, P, P, N), "both or neither", lib)
    for k in (0, 1, 2, 3, 4, 7, 8, 9, 10):
        a = [P] * 12
        a[k] = N
        refused(b(rope(), *a, BIG, N), "NULL", lib)
    need = lib.dmuon_qk_norm_rope_bwd_workspace(rope())
    assert need > 0
    refused(b(rope(), *[P] * 12, need - 1, N), "workspace", lib)
    refused(b(rope(), *[P] * 11, BAD, need, N), "workspace", lib)
    assert f(rope(tokens=0), *[N] * 7, N) == dm.OK


def test_dropout_refusals(lib):
    f, b = lib.dmuon_dropout_fwd, lib.dmuon_dropout_bwd
    for p in (-0.1, 1.1, float("nan")):
        refused(f(P, N, P, 8, p, 0, 0, N, 0, N), "p must", lib)
        refused(b(P, P, 8, p, 0, 0, N, 0, N), "p must", lib)
    refused(f(N, N, P, 8, 0.1, 0, 0, N, 0, N), "NULL", lib)
    refused(f(P, N, N, 8, 0.1, 0, 0, N, 0, N), "NULL", lib)
    refused(f(P, N, P, -1, 0.1, 0, 0, N, 0, N), "range", lib)
    refused(f(P, N, P, (1 << 40) + 1, 0.1, 0, 0, N, 0, N), "range", lib)
    refused(b(P, P, 8, 0.1, 0, 0, N, 3, N), "dtype", lib)
    assert f(N, N, N, 0, 0.1, 0, 0, N, 0, N) == dm.OK


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 2, 8)
    pos = torch.zeros(4, dtype=torch.int64)
    for call in (lambda: dm.attention(x, x, x), lambda: dm.attention_backward(x, x, x, x, x, x[..., 0]),
                 lambda: dm.qk_norm_rope(x, x, pos), lambda: dm.qk_norm_rope_backward(x, x, x, x, pos),
                 lambda: dm.dropout(x, 0.1, 0), lambda: dm.dropout_backward(x, 0.1, 0)):
        with pytest.raises(ValueError, match="GPU"):
            call()


def test_evenly_spaced_tokens():
    x = torch.zeros(6, 5, 4, 8)
    assert dm._heads("t", "q", x, x, (6, 5), 4, 8) == (32, 8)
    assert dm._heads("t", "q", x[:, :1], x, (6, 1), 4, 8) == (160, 8)
    assert dm._heads("t", "q", x[:1, :1], x, (1, 1), 4, 8) == (0, 8)
    assert dm._heads("t", "q", x[:, :, :1], x, (6, 5), 1, 8) == (32, 0)
    assert dm._heads("t", "q", x[:1, :1].expand(6, 5, 4, 8), x, (6, 5), 4, 8) == (0, 8)
    for bad in (x[:, :3], x[:1].expand(6, 5, 4, 8), x[:, :1].expand(6, 5, 4, 8), x.transpose(0, 1)):
        with pytest.raises(ValueError, match="evenly"):
            dm._heads("t", "q", bad, x, tuple(bad.shape[:2]), 4, 8)
