"""The attention block's operators at the ends of their ranges: scores far from zero, rows whose every
score is -infinity, values that are not finite where the probability vanishes, lists that are not
as stated, sizes past 32 bits and past one launch, the work's counts; heads whose squares
fp32 does not hold."""

import math

import pytest
import torch

import matrix_orthogonalising_optimizer_amd as dm
import heads_ref as ref
from test_gpu_heads import BF16, F32, NAMES, edges, gen, inputs, rope_inputs, run

pytestmark = pytest.mark.gpu

inf, nan = math.inf, math.nan


# ------------------------------------------------------------ scores far from zero
def far_inputs(n, m, hq, hk, dim, dtype, sign=1, step=1, seed=0):
    """q, k, v, dy whose scores are sign 2^33 + a 2^10, a in 0 .. 7 step, exactly, whatever the
    order of their sums: products of powers of two and small integers in two places, zeros in the others."""
    q, k, v, dy = inputs(n, m, hq, hk, dim, dtype, seed=seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 9)
    a = step * torch.randint(0, 8, (m, hk), device="cuda", generator=g)
    q.zero_()
    k.zero_()
    q[..., 0], q[..., dim - 1] = sign * 2.0 ** 20, 32.0
    k[..., 0], k[..., dim - 1] = 2.0 ** 13, 32.0 * a.to(dtype)
    return q, k, v, dy, a


def far_values(q, a, v, lens, keys, causal, scale, sign=1, k=None, dy=None):
    """(values, bounds) of y and lse and, with k and dy, of dq, dk and dv.  (s - m) scale is off by two roundings of
    its size, of which 100 is the most that leaves a probability a bound notices, the exponential and a
    product by some 2^-24 each, p in bf16 by its rounding; lse by the rounding of its size, twice, and what the
    sum is off by.  The backward pass forms p from lse, whose multiple of log2 e is rounded once more, where that
    is below 4096, and has the sum's logarithm to 2^-19 above.  ds and the gradients as in heads_ref.
    An exponential below 2^-126, the least normal number, may be 0; as the row's reference is rounded by up to
    16 (half a step of 2^28 .. 2^29) that is a probability of up to 2^-110, which may be lost: `low`."""
    low = 2.0 ** -110
    u, up = ref.ROUNDOFF[q.dtype], ref.ROUNDOFF[q.dtype] if q.dtype is BF16 else 0.0
    hq, hk = q.shape[1], v.shape[1]
    y = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(hq, q.shape[0], dtype=torch.float64, device="cuda")
    ey, el = torch.zeros_like(y), torch.zeros_like(lse)
    if dy is not None:
        Q, K, G = q.double(), k.double(), dy.double()
        grads = [torch.zeros_like(Q), torch.zeros_like(K), torch.zeros_like(K)]
        eg = [torch.zeros_like(x) for x in grads]
    i, j = lens[0], keys[0]
    for n, m in zip(lens[1:], keys[1:]):
        mask = torch.ones(n, m, dtype=torch.bool, device="cuda")
        mask = mask.tril(m - n) if causal else mask
        for h in range(hq):
            g = h * hk // hq
            s = a[j:j + m, g].double()[None].expand(n, m) * (2.0 ** 10 * scale)
            s = torch.where(mask, s, -inf)
            p, V = s.softmax(1), v[j:j + m, g].double()
            Y, L = p @ V, s.logsumexp(1) + sign * 2.0 ** 33 * scale
            rel = 208 * 2.0 ** -24 + 2 * ref.acc(m)
            y[i:i + n, h], lse[h, i:i + n] = Y, L
            ey[i:i + n, h] = u * Y.abs() + (rel + up) * (p @ V.abs()) + low * V.abs().sum(0) + 2.0 ** -120
            el[h, i:i + n] = 2.0 ** -23 * L.abs() + rel + 2.0 ** -22
            if dy is None:
                continue
            E, ad, an = 2.0 ** -24, ref.acc(q.shape[2]), ref.acc(n * hq // hk)
            qh, kh, d = Q[i:i + n, h], K[j:j + m, g], G[i:i + n, h]
            dp, D = d @ V.T, (d * Y).sum(1, keepdim=True)
            e_d = (d.abs() * ey[i:i + n, h]).sum(1, keepdim=True) + ad * (d * Y).abs().sum(1, keepdim=True)
            near = (el[h, i:i + n] + 2 * E * (L.abs() + 1))[:, None] * (L.abs() < 4097 * math.log(2))[:, None]
            rp = rel + near + 2.0 ** -19
            ds = p * (dp - D)
            e_ds = p * (ad * (d.abs() @ V.abs().T) + e_d + 2 * E * (dp.abs() + D.abs())) + ds.abs() * (rp + up + 4 * E)
            e_ds, e_p, am = e_ds + low * mask * (dp.abs() + D.abs()), p * (rp + up) + low * mask, ref.acc(m)
            for out, err, where, x, e in (
                    (grads[0], eg[0], (slice(i, i + n), h), ds @ kh, e_ds @ kh.abs() + am * (ds.abs() @ kh.abs())),
                    (grads[1], eg[1], (slice(j, j + m), g), ds.T @ qh, e_ds.T @ qh.abs() + an * (ds.abs().T @ qh.abs()))):
                out[where] += scale * x
                err[where] += scale * e
            grads[2][j:j + m, g] += p.T @ d
            eg[2][j:j + m, g] += e_p.T @ d.abs() + an * (p.T @ d.abs())
        i, j = i + n, j + m
    vals, errs = [y, lse], [ey, el]
    if dy is not None:
        vals += grads
        errs += [e + u * x.abs() + 2.0 ** -120 for x, e in zip(grads, eg)]
    return vals, [1.01 * e for e in errs]


FAR = [([0, 70, 1], [0, 70, 1], True), ([0, 300], [0, 300], True), ([0, 40], [0, 90], False), ([0, 1], [0, 5000], True),
       ([0, 2, 1], [0, 3000, 700], False), ([0, 5], [0, 2100], True)]


@pytest.mark.parametrize("scale", [2.0 ** -22, 2.0 ** -20, 2.0 ** -12, 2.0 ** -9, 1.5 * 2.0 ** -9, 2.0 ** -6, 2.0 ** -3, 1.0, 2.0 ** 30, 2.0 ** 64])
@pytest.mark.parametrize("dtype,dim", [(BF16, 64), (BF16, 128), (BF16, 256), (F32, 64), (F32, 128)])
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_far_from_zero(sign, dtype, dim, scale):
    for lens, keys, causal in FAR:
        q, k, v, _, a = far_inputs(sum(lens), sum(keys), 4, 2, dim, dtype, sign)
        y, lse = dm.attention(q, k, v, edges(lens), edges(keys), causal=causal, scale=scale)
        ref.check([y, lse], *far_values(q, a, v, lens, keys, causal, scale, sign), NAMES)


@pytest.mark.parametrize("dtype,dim,n,heads", [(BF16, 128, 4200, 16), (BF16, 64, 2200, 32), (BF16, 96, 2200, 32), (F32, 128, 1000, 16)])
def test_scores_far_from_zero_in_wide_tiles(dtype, dim, n, heads):
    for scale in (2.0 ** -8, 1.0):
        q, k, v, _, a = far_inputs(n, n, heads, heads, dim, dtype, step=2)
        y, lse = dm.attention(q, k, v, scale=scale)
        ref.check([y, lse], *far_values(q, a, v, [0, n], [0, n], True, scale), NAMES)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_far_rows_leave_the_others_alone(dtype):
    n = 300
    q, k, v, _ = inputs(n, n, 2, 1, 64, dtype)
    z = q.clone()
    z[::3] *= 2.0 ** 34
    for causal in (True, False):
        (y, lse), (y2, lse2) = dm.attention(q, k, v, causal=causal), dm.attention(z, k, v, causal=causal)
        keep = torch.arange(n, device="cuda") % 3 != 0
        assert torch.equal(y[keep], y2[keep]) and torch.equal(lse[:, keep], lse2[:, keep])
        # (of such rows one key takes all but for ties)
        mask = torch.ones(n, n, device="cuda", dtype=torch.bool).tril(0 if causal else n)
        s = torch.einsum("qhd,kd->hqk", z.cpu().double(), k[:, 0].cpu().double()).cuda()
        top = s.masked_fill(~mask, -inf).argmax(2)
        assert torch.equal(y2[~keep], v[:, 0][top.T][~keep])


@pytest.mark.parametrize("scale", [2.0 ** -22, 2.0 ** -20, 2.0 ** -12, 2.0 ** -9, 1.5 * 2.0 ** -9, 2.0 ** -6, 2.0 ** -3, 1.0, 2.0 ** 30, 2.0 ** 64])
@pytest.mark.parametrize("dtype,dim", [(BF16, 64), (BF16, 96), (BF16, 128), (BF16, 256), (F32, 64), (F32, 96), (F32, 128)])
@pytest.mark.parametrize("sign", [1, -1])
def test_gradients_of_scores_far_from_zero(sign, dtype, dim, scale):
    for lens, keys, causal in FAR:
        q, k, v, dy, a = far_inputs(sum(lens), sum(keys), 4, 2, dim, dtype, sign)
        cu = edges(lens), edges(keys)
        y, lse = dm.attention(q, k, v, *cu, causal=causal, scale=scale)
        got = [y, lse, *dm.attention_backward(dy, q, k, v, y, lse, *cu, causal=causal, scale=scale)]
        ref.check(got, *far_values(q, a, v, lens, keys, causal, scale, sign, k, dy), NAMES)


@pytest.mark.parametrize("dtype,dim,n,heads", [(BF16, 128, 4200, 16), (BF16, 64, 2200, 32), (BF16, 96, 2200, 32), (F32, 128, 1000, 16)])
def test_gradients_of_scores_far_from_zero_in_wide_tiles(dtype, dim, n, heads):
    for scale in (2.0 ** -20, 2.0 ** -8, 1.0):
        q, k, v, dy, a = far_inputs(n, n, heads, heads, dim, dtype, step=2)
        y, lse = dm.attention(q, k, v, scale=scale)
        got = [y, lse, *dm.attention_backward(dy, q, k, v, y, lse, scale=scale)]
        ref.check(got, *far_values(q, a, v, [0, n], [0, n], True, scale, 1, k, dy), NAMES)


@pytest.mark.parametrize("dtype,dim", [(BF16, 64), (BF16, 128), (F32, 128)])
def test_far_rows_leave_the_others_gradients_alone(dtype, dim):
    # a far row whose dy is zero has no gradient and adds none
    n = 600
    q, k, v, dy = inputs(n, n, 4, 2, dim, dtype)
    far = torch.arange(n, device="cuda") % 3 == 0
    z = q.clone()
    z[far] *= 2.0 ** 34
    dy[far] = 0
    for causal in (True, False):
        outs = []
        for x in (q, z):
            y, lse = dm.attention(x, k, v, causal=causal)
            outs.append(dm.attention_backward(dy, x, k, v, y, lse, causal=causal))
        for a, b in zip(*outs):
            assert torch.equal(a, b)


# ------------------------------------------------------------ rows whose every score is -infinity
NONE = [([0, 5], [0, 70]), ([0, 300], [0, 300]), ([0, 1, 2], [0, 5000, 300]), ([0, 200, 64], [0, 90, 400])]


@pytest.mark.parametrize("dtype,dim", [(BF16, 64), (BF16, 96), (BF16, 128), (BF16, 256), (F32, 64), (F32, 128)])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("where", ["k", "q"])
def test_rows_of_infinite_scores_have_no_gradient(where, causal, dtype, dim):
    for lens, keys in NONE:
        q, k, v, dy = inputs(sum(lens), sum(keys), 4, 2, dim, dtype)
        q[..., 0], k[..., 0] = (1.0, -inf) if where == "k" else (-inf, 1.0)
        v[::7, :, 3], dy[::3, :, 1] = inf, nan  # (these meet zeros alone)
        cu = edges(lens), edges(keys)
        y, lse = dm.attention(q, k, v, *cu, causal=causal)
        assert not y.any() and bool((lse == -inf).all())
        for g in dm.attention_backward(dy, q, k, v, y, lse, *cu, causal=causal):
            assert not g.any()


@pytest.mark.parametrize("dtype,dim,heads,n", [(BF16, 64, 4, 300), (BF16, 128, 4, 300), (BF16, 256, 4, 200), (F32, 64, 4, 300), (F32, 128, 4, 300),
                                               (BF16, 128, 32, 2200), (BF16, 64, 32, 2200)])
@pytest.mark.parametrize("causal", [True, False])
def test_rows_of_infinite_scores_leave_the_others_alone(causal, dtype, dim, heads, n):
    q, k, v, dy = inputs(n, n, heads, heads // 2, dim, dtype)
    none = torch.arange(n, device="cuda") % 50 == 7
    k[..., 2] = 1.0
    z, dz = q.clone(), dy.clone()
    z[none, :, 2], dz[none, :, 5], dz[none, 1, 6] = -inf, inf, nan
    dy[none] = 0
    y, lse = dm.attention(q, k, v, causal=causal)
    want = dm.attention_backward(dy, q, k, v, y, lse, causal=causal)
    y2, lse2 = dm.attention(z, k, v, causal=causal)
    got = dm.attention_backward(dz, z, k, v, y2, lse2, causal=causal)
    assert not y2[none].any() and bool((lse2[:, none] == -inf).all()) and not got[0][none].any()
    assert torch.equal(y2[~none], y[~none]) and torch.equal(lse2[:, ~none], lse[:, ~none])
    for a, b in zip(got, want):
        assert torch.equal(a, b)


# ------------------------------------------------------------ a probability of zero meets what is not finite
@pytest.mark.parametrize("bad", [nan, inf, -inf])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("keys", [40, 5000])
def test_seen_values_that_are_not_finite_show(keys, dtype, bad):
    # the last key alone has a probability in fp32; keys in one part and, 5000 of them, in many
    q, k, v, _ = inputs(1, keys, 4, 2, 64, dtype)
    q[..., 0], k[..., 0], k[-1, :, 0] = 64.0, 0.0, 64.0
    v[3, :, 5] = bad
    y, _ = dm.attention(q, k, v)
    assert torch.isnan(y[..., 5]).all() and torch.isfinite(y[..., :5]).all() and torch.isfinite(y[..., 6:]).all()


# ------------------------------------------------------------ lists that are not as stated
BAD_LISTS = [[0, 150, 30, 200], [200, 100, 0], [-5, 100, 200], [0, 10 ** 9, 200], [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1, 5], [300, 400, 500],
             [0, 200] * 31, [0, 200, -7, 900] * 40, [5] * 9, [199, 0, 200, 1, 100]]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype,dim", [(BF16, 64), (BF16, 128), (BF16, 256), (F32, 72)])
def test_lists_that_are_not_as_stated_stay_within(dtype, dim, causal, monkeypatch):
    # results are unspecified, but nothing is written beside them
    around = []

    def middle(x):
        buf = torch.full((x.numel() + 8192,), 7.0, dtype=x.dtype, device="cuda")
        around.append(buf)
        return buf[4096:4096 + x.numel()].view(x.shape)
    monkeypatch.setattr(dm, "_dense", middle)
    for keys in (200, 3000):
        q, k, v, dy = inputs(200, keys, 4, 2, dim, dtype)
        for a in BAD_LISTS:
            for b in (a, [0] + [keys] * (len(a) - 1), [x * 15 for x in range(len(a))]):
                cu = [torch.tensor([min(max(z, -2 ** 31), 2 ** 31 - 1) for z in x], dtype=torch.int32, device="cuda") for x in (a, b)]
                for cq, ck in (cu, cu[::-1]):
                    y, lse = dm.attention(q, k, v, cq, ck, causal=causal)
                    dm.attention_backward(dy, q, k, v, y, lse, cq, ck, causal=causal)
        torch.cuda.synchronize()
        for buf in around:
            assert bool((buf[:4096] == 7).all()) and bool((buf[-4096:] == 7).all())
        around.clear()


# ------------------------------------------------------------ diagnostics
@pytest.mark.parametrize("causal,n,m", [(True, 70, 90), (True, 90, 70), (False, 70, 90)])
def test_timing_counts_the_work(causal, n, m):
    q, k, v, dy = (x.unflatten(0, (2, -1)) for x in inputs(2 * n, 2 * m, 4, 2, 64, BF16))
    pairs = sum(max(0, min(m, i + m - n + 1)) if causal else m for i in range(n))
    cu = edges([0, n, n]), edges([0, m, m])

    def flops(q, k, v, dy, *lists):
        dm.timing_report()
        dm.timing_enable(True)
        y, lse = dm.attention(q, k, v, *lists, causal=causal)
        dm.attention_backward(dy, q, k, v, y, lse, *lists, causal=causal)
        dm.timing_enable(False)
        got = {x["kernel"]: x["flops"] for x in dm.timing_report()["kernels"]}
        return [got["attn_rows_kernel<fwd>"], got["attn_rows_kernel<dq>"], got["attn_keys_kernel"]]
    # two products forward, three for dq, four for dk and dv, two operations a pair and element
    assert flops(q, k, v, dy) == [x * 2 * 64 * 4 * 2 * pairs for x in (2, 3, 4)]
    assert flops(*(x.flatten(0, 1) for x in (q, k, v, dy)), *cu) == [0, 0, 0]


def test_timing_counts_the_joins():
    q, k, v, _ = inputs(1, 5000, 4, 2, 64, BF16)
    dm.timing_report()
    dm.timing_enable(True)
    dm.attention(q, k, v)
    dm.timing_enable(False)
    got = {x["kernel"]: x["bytes"] for x in dm.timing_report()["kernels"]}
    parts = (got["attn_join_kernel<rows>"] - 4 * 64 * 2) / (4 * 64 * 4)  # (of 4 rows of 64, in fp32)
    assert parts == round(parts) and 2 <= parts <= 32


# ------------------------------------------------------------ sizes
def test_long_cache_offsets_backward():
    # rows of one head past 2^31 bytes from the first, in k, v, dk and dv
    t, hk, dim = 1 << 18, 64, 128
    k = torch.empty(t, hk, dim, dtype=BF16, device="cuda").normal_()
    v = torch.empty(t, hk, dim, dtype=BF16, device="cuda").normal_()
    q, dy = gen(3, 2 * hk, dim, seed=1), gen(3, 2 * hk, dim, seed=2)
    cu_q = torch.tensor([0, 0, 3], dtype=torch.int32, device="cuda")
    cu_k = torch.tensor([0, t - 500, t], dtype=torch.int32, device="cuda")
    y, lse = dm.attention(q, k, v, cu_q, cu_k)
    dq, dk, dv = dm.attention_backward(dy, q, k, v, y, lse, cu_q, cu_k)
    vals, errs = ref.attention(q, k[-500:], v[-500:], [0, 3], [0, 500], True, dy=dy)
    ref.check([y, lse, dq, dk[-500:], dv[-500:]], vals, errs, NAMES)
    assert not dk[:-500].any() and not dv[:-500].any()


def test_long_queries_offsets():
    # rows of q, dy, y and dq past 2^31 bytes; few of them belong to the sequence that has keys
    t, heads, dim = 1 << 17, 64, 160
    q = torch.empty(t, heads, dim, dtype=BF16, device="cuda").normal_()
    dy = torch.empty(t, heads, dim, dtype=BF16, device="cuda").normal_()
    k, v = gen(200, 8, dim, seed=3), gen(200, 8, dim, seed=4)
    cu_q = torch.tensor([0, t - 300, t], dtype=torch.int32, device="cuda")
    cu_k = torch.tensor([0, 0, 200], dtype=torch.int32, device="cuda")
    y, lse = dm.attention(q, k, v, cu_q, cu_k, causal=False)
    dq, dk, dv = dm.attention_backward(dy, q, k, v, y, lse, cu_q, cu_k, causal=False)
    vals, errs = ref.attention(q[-300:], k, v, [0, 300], [0, 200], False, dy=dy[-300:])
    ref.check([y[-300:], lse[:, -300:], dq[-300:], dk, dv], vals, errs, NAMES)
    assert not y[:-300].any() and not dq[:-300].any() and bool((lse[:, :-300] == -inf).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_more_workgroups_than_a_launch_takes(dtype):
    # sequences of one token: y = v and dv = dy, rounded as the sums are; no other gradient
    b, h, dim = (1 << 18) + 1, 8, 8
    q, k, v, dy = (x.view(b, 1, h, dim) for x in inputs(b, b, h, h, dim, dtype))
    y, lse = dm.attention(q, k, v)
    dq, dk, dv = dm.attention_backward(dy, q, k, v, y, lse)
    u = ref.ROUNDOFF[dtype] + 64 * 2.0 ** -24
    s = (q.double() * k.double()).sum(-1)[:, 0].T * dim ** -0.5
    assert bool(((lse[:, :, 0].double() - s).abs() <= 32 * 2.0 ** -24 * (1 + (q.double() * k.double()).abs().sum(-1)[:, 0].T)).all())
    assert bool(((y - v).abs().double() <= 2 * u * v.abs().double()).all())
    # p is off by the rounding of lse, relative; ds by what dp - D is off by, whose y is rounded
    size = 1 + (q.double() * k.double()).abs().sum(-1, keepdim=True)
    assert bool(((dv - dy).abs().double() <= (2 * u + 64 * 2.0 ** -24 * size) * dy.abs().double()).all())
    ds = 2 * u * (dy.double() * v.double()).abs().sum(-1, keepdim=True) + 2.0 ** -120
    assert bool((dq.abs().double() <= 2 * ds * k.double().abs()).all()) and bool((dk.abs().double() <= 2 * ds * q.double().abs()).all())


# tiles of 256 rows and keys: more sequences than one look at the list takes, batches of equal lengths
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dim", [64, 96, 128])
def test_wide_tiles_of_many_sequences(dim, causal):
    lens = [7] + [(i * 37) % 300 + 40 for i in range(70)]
    run(*inputs(sum(lens) + 5, sum(lens) + 5, 16, 8, dim, BF16), lens, causal=causal)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dim", [64, 128])
def test_wide_tiles_of_equal_lengths(dim, causal):
    b, n, m, heads = 5, 1000, 1100, 16
    q, k, v, dy = inputs(b * n, b * m, heads, heads, dim, BF16)
    cut = lambda t: t.view(b, -1, *t.shape[1:])
    y, lse = dm.attention(cut(q), cut(k), cut(v), causal=causal)
    got = [y, lse, *dm.attention_backward(cut(dy), cut(q), cut(k), cut(v), y, lse, causal=causal)]
    vals, errs = ref.attention(q, k, v, [0] + [n] * b, [0] + [m] * b, causal, None, dy)
    ref.check([g.reshape(w.shape) for g, w in zip(got, vals)], vals, errs, NAMES)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n", [5, 4096, 70001])
def test_dropout_in_place(n, dtype):
    # y may be x, or the residual
    lib, stream = dm.load_library(), torch.cuda.current_stream().cuda_stream
    x, r = gen(n, seed=1, dtype=dtype), gen(n, seed=2, dtype=dtype)
    want = dm.dropout(x, 0.3, 5, residual=r)
    for y in (0, 1):
        a = [x.clone(), r.clone()]
        assert lib.dmuon_dropout_fwd(a[0].data_ptr(), a[1].data_ptr(), a[y].data_ptr(), n, 0.3, 5, 0, None, dm._dtype_code(x), stream) == dm.OK
        assert torch.equal(a[y], want)


# ------------------------------------------------------------ heads whose squares fp32 does not hold
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dim,rot", [(64, 64), (128, 96), (256, 256), (72, 72), (80, 40), (6, 4)])
@pytest.mark.parametrize("power,eps", [(100, 0.0), (100, 1e-6), (64, 1e-6), (-80, 0.0), (-70, 1e-44)])
def test_norm_of_huge_and_tiny_heads(power, eps, dim, rot, dtype):
    # a power of two leaves y as it is and divides dx, bit for bit: x f / sqrt(mean (x f)^2 + eps)
    # is x / sqrt(mean x^2 + eps / f^2).  Every other head is scaled.
    q, k, pos, wq, wk, dq, dk = rope_inputs(40, 6, 2, dim, dtype)
    q[..., 0], k[..., 0] = 1.0, 1.0

    def both(q, k, eps):
        how = dict(eps=eps, rotary_dim=rot)
        return [*dm.qk_norm_rope(q, k, pos, wq, wk, **how), *dm.qk_norm_rope_backward(dq, dk, q, k, pos, wq, wk, **how)]
    want = both(q, k, float(torch.tensor(eps).double() * 2.0 ** (-2 * power)))
    for a, b in zip(want[:4], both(q, k, eps)):
        a[:, 1::2] = b[:, 1::2]
    factor = torch.ones(8, dtype=torch.float64, device="cuda")
    factor[::2] = 2.0 ** power
    scaled = lambda x, f: (x.double() * f[:, None]).to(dtype)
    got = both(scaled(q, factor[:6]), scaled(k, factor[6:]), eps)
    want[2], want[3] = scaled(want[2], 1 / factor[:6]), scaled(want[3], 1 / factor[6:])
    for a, b in zip(got[:4], want):
        assert torch.equal(a, b)
    for a, b in zip(got[4:], want[4:]):  # sums over all heads
        assert torch.equal(a, b) if eps == 0 else torch.isfinite(a).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_strides_past_32_bits(dtype):
    # heads, or tokens, so far apart that the loads' offsets do not reach: such operands are copied first
    lens = [0, 200, 60]
    q, k, v, dy = inputs(260, 260, 4, 2, 64, dtype)
    want = run(q, k, v, dy, lens)

    def spread(x, token, head):
        y = torch.empty((x.shape[0] - 1) * token + (x.shape[1] - 1) * head + x.shape[2], dtype=dtype, device="cuda").as_strided(
            x.shape, (token, head, 1))
        return y.copy_(x)
    # (bytes from token to token times 256 rows, or from head to head times the group, are 2^31 or more)
    far = 2 ** 31 // q.element_size()
    for a in ((spread(q, far // 256, 64), k, v, dy), (q, spread(k, 64, far // 2), spread(v, far // 256, 64), dy),
              (q, k, v, spread(dy, far // 256 + 1, 64))):
        y, lse = dm.attention(*a[:3], edges(lens))
        got = [y, lse, *dm.attention_backward(a[3], *a[:3], y, lse, edges(lens))]
        for g, w in zip(got, want):
            assert torch.equal(g.nan_to_num(neginf=0.0), w)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_far_and_empty_rows_in_replayed_graphs(dtype):
    # captured with rows of neither kind; each replay has others
    n, keys = 300, 400
    q, k, v, dy = inputs(n, keys, 4, 2, 64, dtype)
    plain, k_plain = q.clone(), k.clone()
    cu = edges([0, 290, 10]), edges([0, 100, 300])
    def both():
        y, lse = dm.attention(q, k, v, *cu)
        return [y, lse, *dm.attention_backward(dy, q, k, v, y, lse, *cu)]
    both()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    for i in range(5):
        q.copy_(plain)
        k.copy_(k_plain)
        if i % 2:
            q[i::7] *= 2.0 ** 34
        if i > 1:
            q[i::11, :, 3], k[..., 3] = -inf, 1.0
        want = both()
        for z in out:
            z.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, out):
            assert torch.equal(a.nan_to_num(neginf=0.0), b.nan_to_num(neginf=0.0)), i
        assert all(torch.isfinite(x).all() for x in (out[0], *out[2:])), i
