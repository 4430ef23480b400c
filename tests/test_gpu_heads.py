"""The attention block's operators on the GPU against their 64-bit forms,
element by element (heads_ref derives the bounds)."""

import pytest
import torch

import matrix_orthogonalising_optimizer_amd as dm
import heads_ref as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
inf, nan = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dm.load_library()


def gen(*shape, seed, std=1.0, mean=0.0, dtype=BF16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(shape, device="cuda").normal_(mean, std, generator=g).to(dtype)


def edges(lens):
    out, at = [], 0
    for n in lens:
        at += n
        out.append(at)
    return torch.tensor(out, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------ attention
NAMES = ["y", "lse", "dq", "dk", "dv"]


def inputs(tq, tk, hq, hk, dim, dtype, seed=0, std=1.5):
    return (gen(tq, hq, dim, seed=seed + 1, std=std, dtype=dtype), gen(tk, hk, dim, seed=seed + 2, dtype=dtype),
            gen(tk, hk, dim, seed=seed + 3, mean=0.3, dtype=dtype), gen(tq, hq, dim, seed=seed + 4, dtype=dtype))


def run(q, k, v, dy, lens, keys=None, causal=True, scale=None, tail=(0, 0)):
    """lens[0], keys[0]: rows before the first sequence; tail: rows behind the last."""
    keys = lens if keys is None else keys
    cu = (edges(lens), edges(keys))
    y, lse = dm.attention(q, k, v, *cu, causal=causal, scale=scale)
    got = [y, lse, *dm.attention_backward(dy, q, k, v, y, lse, *cu, causal=causal, scale=scale)]
    vals, errs = ref.attention(q, k, v, lens, keys, causal, scale, dy)
    none = vals[1] == -inf
    assert bool((got[1][none] == -inf).all())
    got[1], vals[1] = got[1].masked_fill(none, 0.0), vals[1].masked_fill(none, 0.0)
    ref.check(got, vals, errs, NAMES)
    return got


LENS = [[0, 1], [0, 5], [0, 64], [0, 65], [0, 1, 2, 3], [0, 130, 7, 63, 1], [0, 0, 33, 0, 129, 0], [0, 300, 128]]


@pytest.mark.parametrize("dtype,dim", [(BF16, 64), (BF16, 96), (BF16, 128), (BF16, 256), (F32, 64), (F32, 96), (F32, 128)])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_attention(lens, causal, dtype, dim):
    run(*inputs(sum(lens), sum(lens), 4, 2, dim, dtype), lens, causal=causal)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("hq,hk", [(1, 1), (3, 3), (7, 1), (6, 2), (16, 8), (10, 10), (24, 8), (65, 1)])
def test_attention_heads(hq, hk, dtype):
    lens = [0, 77, 1, 150]
    run(*inputs(228, 228, hq, hk, 64, dtype), lens)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dim", [1, 2, 3, 8, 31, 32, 40, 63, 72, 80, 100, 101, 120, 127])
def test_attention_widths(dim, dtype):
    run(*inputs(150, 150, 4, 2, dim, dtype), [0, 140, 10])


@pytest.mark.parametrize("dim", [130, 160, 200, 250])
def test_attention_wide_heads(dim):
    run(*inputs(150, 150, 4, 2, dim, BF16), [0, 140, 10])


# queries and keys of other lengths: causal rows that see nothing, keys that no row lacks, none at all
@pytest.mark.parametrize("dtype,dim", [(BF16, 128), (BF16, 64), (F32, 72)])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,keys", [([0, 1], [0, 700]), ([0, 1, 1, 1], [0, 300, 1, 65]), ([0, 100], [0, 3]),
                                       ([0, 200, 50], [0, 10, 0]), ([0, 0, 40], [0, 70, 170]), ([0, 33, 66], [0, 190, 67]),
                                       ([0, 300], [0, 257])], ids=str)
def test_attention_lengths(lens, keys, causal, dtype, dim):
    run(*inputs(sum(lens), sum(keys), 6, 2, dim, dtype), lens, keys, causal=causal)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_of_no_sequence(dtype):
    q, k, v, dy = inputs(200, 230, 4, 2, 64, dtype)
    lens, keys = [9, 60, 50], [70, 40, 90]
    for t in (q, k, v, dy):  # whatever those rows hold
        t[:9], t[-20:] = nan, inf
    k[:70] = v[:70] = nan
    y, *_ = run(q, k, v, dy, lens, keys)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("count", [61, 62, 63, 700])
def test_many_sequences(count, causal):
    lens = [3] + [(i * 7) % 5 + 200 * (i % 29 == 3) for i in range(count)]
    n = sum(lens) + 4
    run(*inputs(n, n, 2, 1, 64, BF16), lens, causal=causal)


# every way a pass may be cut: tiles of 128 and of 256, parts of the keys and of the rows
@pytest.mark.parametrize("dtype,dim,hq,hk,lens,keys", [
    (BF16, 128, 32, 8, [0, 1, 1, 1, 1], [0, 3000, 1, 70, 1501]), (BF16, 64, 8, 1, [0, 5, 3], [0, 4100, 2]), (F32, 72, 4, 2, [0, 3], [0, 2050]),
    (BF16, 256, 2, 1, [0, 40], [0, 1500]), (F32, 128, 2, 1, [0, 600, 31], None), (BF16, 96, 4, 1, [0, 1100, 700], None),
    (BF16, 128, 16, 16, [0, 4000, 300], None), (BF16, 128, 24, 8, [0, 2600, 2600], None), (BF16, 80, 20, 20, [0, 2100, 5, 1000], None),
    (BF16, 64, 16, 4, [0, 4097, 1, 511], None), (BF16, 256, 4, 2, [0, 1300], None), (F32, 64, 10, 5, [0, 900, 400], None)], ids=str)
@pytest.mark.parametrize("causal", [True, False])
def test_cuts_of_the_work(dtype, dim, hq, hk, lens, keys, causal):
    run(*inputs(sum(lens), sum(keys or lens), hq, hk, dim, dtype), lens, keys, causal=causal)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_equal_lengths(dtype):
    b, n, m = 3, 70, 90
    q, k, v, dy = inputs(b * n, b * m, 4, 2, 64, dtype)
    cut = lambda t: t.view(b, -1, *t.shape[1:])
    y, lse = dm.attention(cut(q), cut(k), cut(v))
    grads = dm.attention_backward(cut(dy), cut(q), cut(k), cut(v), y, lse)
    cu = torch.arange(b + 1, dtype=torch.int32, device="cuda")
    z, lse2 = dm.attention(q, k, v, cu * n, cu * m)
    want = [z, lse2, *dm.attention_backward(dy, q, k, v, z, lse2, cu * n, cu * m)]
    assert y.shape == (b, n, 4, 64) and lse.shape == (4, b, n)
    for got, w in zip([y, lse, *grads], want):
        assert torch.equal(got.reshape(w.shape), w)
    one = dm.attention(q[:n], k[:m], v[:m])
    assert torch.equal(one[0], z[:n])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_strided_and_unaligned_operands(dtype):
    t, hq, hk, dim = 150, 4, 2, 64
    lens = [0, 90, 60]
    q, k, v, dy = inputs(t, t, hq, hk, dim, dtype)
    want = run(q, k, v, dy, lens)
    x = torch.cat([q.flatten(1), k.flatten(1), v.flatten(1)], 1)
    views = [z.view(t, -1, dim) for z in x.split([hq * dim, hk * dim, hk * dim], 1)]
    heads_first = [z.transpose(0, 1).contiguous().transpose(0, 1) for z in (q, k, v)]
    off = []
    for z in (q, k, v, dy):
        buf = torch.full((z.numel() + 1,), nan, dtype=dtype, device="cuda")
        buf[1:] = z.flatten()
        off.append(buf[1:].view(z.shape))
    odd = torch.full((t, hq, dim + 1), nan, dtype=dtype, device="cuda")
    odd[..., :dim] = dy
    for a in ([*views, dy], [*heads_first, dy.transpose(0, 1).contiguous().transpose(0, 1)], off, [q, k, v, odd[..., :dim]]):
        y, lse = dm.attention(*a[:3], edges(lens))
        got = [y, lse, *dm.attention_backward(a[3], *a[:3], y, lse, edges(lens))]
        for g, w in zip(got, want):
            assert torch.equal(g, w) or g.dtype is F32 and torch.equal(g.nan_to_num(neginf=0.0), w)
    e = q[:, :1].expand(t, hq, dim)  # one head's queries for all
    y, lse = dm.attention(e, k, v, edges(lens))
    y2, lse2 = dm.attention(e.contiguous(), k, v, edges(lens))
    assert torch.equal(y, y2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_scores_far_apart(dtype):
    # maxima that keep growing along the keys, scores of +-hundreds, one key that takes all
    q, k, v, dy = inputs(200, 200, 2, 1, 64, dtype)
    k = k * torch.linspace(0.1, 20.0, 200, device="cuda").to(dtype)[:, None, None]
    run(q, k, v, dy, [0, 200])
    run(q, k, v, dy, [0, 200], scale=1.0)
    run(q, k.flip(0), v, dy, [0, 200], causal=False)


# what a row does not see reaches nothing of it
@pytest.mark.parametrize("bad", [nan, inf, -inf])
@pytest.mark.parametrize("dtype,dim", [(BF16, 64), (BF16, 128), (BF16, 256), (F32, 64), (F32, 128)])
def test_unseen_values_reach_nothing(dtype, dim, bad):
    n, at = 150, 101
    q, k, v, dy = inputs(n + 40, n + 40, 4, 2, dim, dtype)
    cu = edges([0, n, 40])
    def both(q, k, v, dy):
        y, lse = dm.attention(q, k, v, cu)
        return [y, lse, *dm.attention_backward(dy, q, k, v, y, lse, cu)]
    want = both(q, k, v, dy)
    rows, other = slice(0, at), slice(n, n + 40)
    for which in range(4):
        x = [t.clone() for t in (q, k, v, dy)]
        x[which][at, :, 3] = bad
        y, lse, dq, dk, dv = both(*x)
        # rows before it do not see key `at`
        assert torch.equal(y[rows], want[0][rows]) and torch.equal(lse[:, rows], want[1][:, rows])
        assert torch.equal(dq[rows], want[2][rows])
        # keys behind it are not seen by row `at`: nothing of its q and dy
        if which in (0, 3):
            assert torch.equal(dk[at + 1:n], want[3][at + 1:n]) and torch.equal(dv[at + 1:n], want[4][at + 1:n])
        for g, w in zip((y, dq, dk, dv), (want[0], want[2], want[3], want[4])):
            assert torch.equal(g[other], w[other])
        assert torch.equal(lse[:, other], want[1][:, other])
        if which in (1, 2):
            assert not torch.isfinite(y[at:n]).all()


def test_rows_whose_scores_are_all_infinite():
    q, k, v, _ = inputs(5, 70, 1, 1, 64, BF16)
    q[:, :, 0], k[:, :, 0] = 1.0, -inf
    y, lse = dm.attention(q, k, v, causal=False)
    assert not y.any() and bool((lse == -inf).all())


@pytest.mark.parametrize("dtype,hq,hk,dim", [(BF16, 32, 8, 128), (BF16, 12, 12, 64), (F32, 4, 2, 128)])
def test_attention_long(dtype, hq, hk, dim):
    lens = [0, 2500, 700, 33]
    run(*inputs(sum(lens), sum(lens), hq, hk, dim, dtype), lens)


def test_long_cache_offsets():
    # rows of one head past 2^31 bytes from the first
    t, hk, dim = 1 << 18, 64, 128
    k = torch.empty(t, hk, dim, dtype=BF16, device="cuda").normal_()
    v = torch.empty(t, hk, dim, dtype=BF16, device="cuda").normal_()
    q = gen(3, 2 * hk, dim, seed=1)
    cu_q = torch.tensor([0, 0, 3], dtype=torch.int32, device="cuda")
    cu_k = torch.tensor([0, t - 500, t], dtype=torch.int32, device="cuda")
    y, lse = dm.attention(q, k, v, cu_q, cu_k)
    vals, errs = ref.attention(q, k[-500:], v[-500:], [0, 3], [0, 500], True)
    ref.check([y, lse], vals, errs, NAMES)


# ------------------------------------------------------------ norm and rotation
def run_rope(q, k, pos, wq, wk, dq, dk, rot, sections, **how):
    hows = dict(how, rotary_dim=rot, sections=sections)
    yq, yk = dm.qk_norm_rope(q, k, pos, wq, wk, **hows)
    gq, gk, dwq, dwk = dm.qk_norm_rope_backward(dq, dk, q, k, pos, wq, wk, **hows)
    sec = [rot // 2] if sections is None else sections
    for x, w, dy, got in ((q, wq, dq, [yq, gq, dwq]), (k, wk, dk, [yk, gk, dwk])):
        vals, errs = ref.norm_rope(x, w, pos, rot, sec, dy=dy, **how)
        ref.check(got[:len(vals)], vals, errs, ["y", "dx", "dw"])
        assert (got[2] is None) == (w is None)
    return yq, yk, gq, gk, dwq, dwk


def rope_inputs(t, hq, hk, dim, dtype, axes=0, far=100000, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    pos = torch.randint(-5, far, (t, axes) if axes else (t,), device="cuda", generator=g)
    return (gen(t, hq, dim, seed=seed + 1, std=2.0, mean=0.3, dtype=dtype), gen(t, hk, dim, seed=seed + 2, dtype=dtype), pos,
            gen(dim, seed=seed + 3, std=0.3, mean=1.0, dtype=dtype), gen(dim, seed=seed + 4, std=0.3, mean=1.0, dtype=dtype),
            gen(t, hq, dim, seed=seed + 5, dtype=dtype), gen(t, hk, dim, seed=seed + 6, dtype=dtype))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rot", [(2, 2), (2, 0), (6, 4), (10, 10), (16, 16), (32, 16), (64, 64), (72, 72), (72, 36), (80, 64),
                                     (96, 96), (128, 128), (128, 40), (160, 160), (254, 254), (256, 256), (256, 0)])
def test_qk_norm_rope(dim, rot, interleaved, dtype):
    run_rope(*rope_inputs(37, 6, 2, dim, dtype), rot, None, interleaved=interleaved)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("t,hq,hk", [(1, 1, 1), (1, 32, 8), (2, 7, 3), (5, 64, 1), (1031, 4, 4), (5000, 12, 2)])
def test_qk_norm_rope_sizes(t, hq, hk, dtype):
    run_rope(*rope_inputs(t, hq, hk, 128, dtype), 128, None)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("per_axis", [False, True])
@pytest.mark.parametrize("dim,rot,sections", [(128, 128, [16, 24, 24]), (80, 64, [8, 12, 12]), (64, 64, [32]), (72, 72, [0, 18, 18]),
                                              (64, 40, [5, 5, 5, 5])])
def test_qk_norm_rope_axes(dim, rot, sections, per_axis, dtype):
    run_rope(*rope_inputs(53, 4, 2, dim, dtype, axes=len(sections)), rot, sections, per_axis=per_axis, base=500.0)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rotation_alone(dtype):
    q, k, pos, _, _, dq, dk = rope_inputs(41, 4, 2, 64, dtype)
    run_rope(q, k, pos, None, None, dq, dk, 64, None)


def test_far_positions():
    q, k, pos, wq, wk, dq, dk = rope_inputs(64, 2, 1, 128, F32)
    pos = pos + 2 ** 30
    run_rope(q, k, pos, wq, wk, dq, dk, 128, None, base=1e6)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_qk_norm_rope_views_and_shapes(dtype):
    q, k, pos, wq, wk, dq, dk = rope_inputs(60, 4, 2, 64, dtype)
    want = run_rope(q, k, pos, wq, wk, dq, dk, 64, None)
    x = torch.full((60, 6 * 64 + 3), nan, dtype=dtype, device="cuda")
    x[:, 1:257], x[:, 257:385] = q.flatten(1), k.flatten(1)
    vq, vk = x[:, 1:257].unflatten(1, (4, 64)), x[:, 257:385].unflatten(1, (2, 64))
    turn = lambda t: t.transpose(0, 1).contiguous().transpose(0, 1)
    got = [*dm.qk_norm_rope(vq, vk, pos, wq, wk), *dm.qk_norm_rope_backward(turn(dq), turn(dk), vq, vk, pos, wq, wk)]
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    cut = lambda t: t.view(5, 12, *t.shape[1:])
    got = dm.qk_norm_rope(cut(vq.contiguous()), cut(k), cut(pos), wq, wk)
    assert got[0].shape == (5, 12, 4, 64) and torch.equal(got[0].flatten(0, 1), want[0])


def test_no_tokens():
    q, k, pos, wq, wk, dq, dk = rope_inputs(3, 4, 2, 64, BF16)
    z = dm.qk_norm_rope_backward(dq[:0], dk[:0], q[:0], k[:0], pos[:0], wq, wk)
    assert z[0].shape == (0, 4, 64) and not z[2].any() and not z[3].any()
    y, lse = dm.attention(q[:0], k[:0], k[:0])
    assert y.shape == (0, 4, 64) and lse.shape == (4, 0)
    y, lse = dm.attention(q, k[:0], k[:0])
    assert not y.any() and bool((lse == -inf).all())
    g = dm.attention_backward(dq, q, k[:0], k[:0], y, lse)
    assert not g[0].any() and g[1].shape == (0, 2, 64)
    g = dm.attention_backward(dq[:0], q[:0], k, k, y[:0], lse[:, :0])
    assert not g[1].any() and not g[2].any()
    assert dm.dropout(q[:0], 0.1, 3).shape == (0, 4, 64)


def test_rope_nonfinite_heads_stay_alone():
    q, k, pos, wq, wk, dq, dk = rope_inputs(20, 4, 2, 128, BF16)
    want = dm.qk_norm_rope(q, k, pos, wq, wk, rotary_dim=64)
    q[3, 1, 5], q[7, 2, 100] = nan, inf
    got = dm.qk_norm_rope(q, k, pos, wq, wk, rotary_dim=64)
    keep = torch.ones(20, 4, dtype=torch.bool, device="cuda")
    keep[3, 1] = keep[7, 2] = False
    assert torch.equal(got[0][keep], want[0][keep]) and torch.equal(got[1], want[1])
    assert torch.isnan(got[0][3, 1]).all() and torch.isnan(got[0][7, 2, 100])


# ------------------------------------------------------------ dropout
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,p,seed,offset", [(1, 0.5, 0, 0), (7, 0.1, 1, 5), (8, 0.9, 2 ** 63 + 5, 2 ** 32 - 1), (1001, 0.25, -3, 2 ** 40),
                                             (4099, 0.1, 12345678901, 2 ** 64 - 2), (2048, 0.0, 7, 0), (2049, 1.0, 7, 0)])
def test_dropout(n, p, seed, offset, dtype):
    x, r, dy = gen(n, seed=1, dtype=dtype), gen(n, seed=2, dtype=dtype), gen(n, seed=3, dtype=dtype)
    kept = ref.keep(n, p, seed, offset).cuda()
    for got, src, res in ((dm.dropout(x, p, seed, offset=offset), x, None), (dm.dropout(x, p, seed, offset=offset, residual=r), x, r),
                          (dm.dropout_backward(dy, p, seed, offset=offset), dy, None)):
        ref.check([got], *ref.dropout(src, kept, p, res), ["y"])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_dropout_large_and_offsets(dtype):
    # more than one step of a thread; the second half's mask by its offset, the whole's
    x = torch.ones(5000, 8008, dtype=dtype, device="cuda")
    y = dm.dropout(x, 0.3, 99, offset=3)
    half = x.numel() // 2
    assert torch.equal(y.view(-1)[half:], dm.dropout(x.view(-1)[half:], 0.3, 99, offset=3 + half // 8))
    share = float((y == 0).double().mean())
    cut = round(0.3 * 65536) / 65536
    assert abs(share - cut) < 6 * (cut * (1 - cut) / x.numel()) ** 0.5
    assert torch.equal((y == 0), (dm.dropout_backward(x, 0.3, 99, offset=3) == 0))


def test_dropout_drops_anything_and_takes_any_address():
    x = gen(1003, seed=1)
    kept = ref.keep(1003, 0.5, 4, 0).cuda()
    z = x.masked_fill(~kept, nan)
    z[~kept] = torch.where(torch.arange(int((~kept).sum()), device="cuda") % 2 == 0, nan, inf).to(BF16)
    want = dm.dropout(x, 0.5, 4)
    assert torch.equal(dm.dropout(z, 0.5, 4), want)
    for k in (1, 3):
        buf = torch.zeros(1003 + k, dtype=BF16, device="cuda")
        buf[k:] = x
        assert torch.equal(dm.dropout(buf[k:], 0.5, 4), want)


def test_dropout_state_on_the_device():
    x = gen(999, seed=1)
    state = torch.tensor([77, 1000], dtype=torch.int64, device="cuda")
    assert torch.equal(dm.dropout(x, 0.4, state, offset=5), dm.dropout(x, 0.4, 77, offset=1005))
    assert torch.equal(dm.dropout_backward(x, 0.4, state), dm.dropout(x, 0.4, 77, offset=1000))


# ------------------------------------------------------------ use
def test_block_on_streams_and_in_graphs():
    t, hq, hk, dim, d = 300, 6, 2, 64, 384
    qkv = gen(t, (hq + 2 * hk) * dim, seed=1)
    q, k, v = (z.view(t, -1, dim) for z in qkv.split([hq * dim, hk * dim, hk * dim], 1))
    pos = torch.arange(t, device="cuda")
    wq, wk, x, dx = gen(dim, seed=2, mean=1.0, std=0.1), gen(dim, seed=3, mean=1.0, std=0.1), gen(t, d, seed=4), gen(t, d, seed=5)
    cu = edges([0, 100, 0, 170, 30])
    state = torch.tensor([5, 0], dtype=torch.int64, device="cuda")

    def step(**kw):
        a, b = dm.qk_norm_rope(q, k, pos, wq, wk, **kw)
        y, lse = dm.attention(a, b, v, cu, **kw)
        z = dm.dropout(y.view(t, d), 0.1, state, residual=x, **kw)
        dz = dm.dropout_backward(dx, 0.1, state, **kw)
        da, db, dv = dm.attention_backward(dz.view(t, hq, dim), a, b, v, y, lse, cu, **kw)
        return [a, b, y, lse, z, dz, da, db, dv, *dm.qk_norm_rope_backward(da, db, q, k, pos, wq, wk, **kw)]

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
    for i in range(4):
        # other sequences and another mask in the same graph
        cu.copy_(edges([0, 100, 0, 170, 30]) if i % 2 == 0 else edges([10, 1, 200, 9, 60]))
        state[1] = 1000 * (i // 2)
        want = step()
        for z in out:
            z.zero_()
        junk = torch.randn(1 << 20, device="cuda").sum()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, out)), i
    del junk


def test_memory_given_may_hold_anything(monkeypatch):
    plain = torch.Tensor.new_empty
    monkeypatch.setattr(torch.Tensor, "new_empty", lambda self, *a, **k: plain(self, *a, **k).fill_(
        255 if k.get("dtype") == torch.uint8 else nan))
    like = torch.empty_like
    monkeypatch.setattr(torch, "empty_like", lambda *a, **k: like(*a, **k).fill_(nan))
    for dtype, dim in ((BF16, 72), (BF16, 100), (BF16, 255), (F32, 50), (F32, 128)):
        run(*inputs(170, 170, 4, 2, dim, dtype), [5, 100, 0, 60])
    run_rope(*rope_inputs(30, 4, 2, 72, BF16), 36, None)


def test_refusals():
    q, k, v, dy = inputs(20, 20, 4, 2, 64, BF16)
    cu = edges([0, 20])
    y, lse = dm.attention(q, k, v)
    pos, w = torch.arange(20, device="cuda"), gen(64, seed=1)
    bad = [
        lambda: dm.attention(q, k, v[:10]), lambda: dm.attention(q, k.float(), v), lambda: dm.attention(q, k[..., :32], v),
        lambda: dm.attention(q.transpose(1, 2), k, v), lambda: dm.attention(q[..., ::2], k[..., ::2], v[..., ::2]),
        lambda: dm.attention(q, k, v, cu.long()), lambda: dm.attention(q, k, v, cu, cu[:1]),
        lambda: dm.attention(q, k, v, None, cu), lambda: dm.attention(q, k[:10], v[:10], cu),
        lambda: dm.attention(q, k, v, cu.cpu()), lambda: dm.attention(q[None], k, v),
        lambda: dm.attention(q.view(2, 10, 4, 64), k.view(1, 20, 2, 64), v.view(1, 20, 2, 64)),
        lambda: dm.attention(q.view(2, 10, 4, 64), k.view(2, 10, 2, 64), v.view(2, 10, 2, 64), cu),
        lambda: dm.attention_backward(dy[:10], q, k, v, y, lse), lambda: dm.attention_backward(dy, q, k, v, y, lse.T),
        lambda: dm.attention_backward(dy, q, k, v, y[..., :32], lse),
        lambda: dm.qk_norm_rope(q, k, pos, w), lambda: dm.qk_norm_rope(q, k, pos.int(), w, w),
        lambda: dm.qk_norm_rope(q, k, pos[:5], w, w), lambda: dm.qk_norm_rope(q, k[:5], pos, w, w),
        lambda: dm.qk_norm_rope(q, k, pos, w, w, sections=[16, 16]), lambda: dm.qk_norm_rope(q, k, pos, w[:32], w),
        lambda: dm.qk_norm_rope(q, k, pos[:, None].expand(20, 5), w, w, sections=[8, 8, 8, 4, 4]),
        lambda: dm.qk_norm_rope(q, k, pos, w.float(), w), lambda: dm.qk_norm_rope_backward(dy[:5], k, q, k, pos, w, w),
        lambda: dm.dropout(q.transpose(0, 1), 0.1, 0), lambda: dm.dropout(q, 0.1, 0, residual=k),
        lambda: dm.dropout(q, 0.1, pos), lambda: dm.dropout(q, 0.1, torch.zeros(2, dtype=torch.int64)),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was accepted")
    worse = [lambda: dm.attention(q, k[:, :1].expand(20, 3, 64), v[:, :1].expand(20, 3, 64)), lambda: dm.attention(q, k, v, scale=0.0),
             lambda: dm.attention(q, k, v, scale=nan), lambda: dm.attention(q, k, v, scale=-1.0),
             lambda: dm.attention(*inputs(4, 4, 1, 1, 257, BF16)[:3]), lambda: dm.attention(*inputs(4, 4, 1, 1, 129, F32)[:3]),
             lambda: dm.qk_norm_rope(q, k, pos, w, w, rotary_dim=66), lambda: dm.qk_norm_rope(q, k, pos, w, w, rotary_dim=33),
             lambda: dm.qk_norm_rope(q, k, pos, w, w, base=0.0), lambda: dm.qk_norm_rope(q, k, pos, w, w, eps=-1.0),
             lambda: dm.qk_norm_rope(q, k, pos[:, None], w, w, sections=[31]),
             lambda: dm.dropout(q, 1.5, 0), lambda: dm.dropout(q, -0.1, 0), lambda: dm.dropout(q, nan, 0)]
    for i, f in enumerate(worse):
        with pytest.raises(dm.DmuonError):
            f()
            pytest.fail(f"call {i} was accepted")
    with pytest.raises(TypeError):
        dm.attention(q.half(), k.half(), v.half())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_batch_of_no_sequences(dtype):
    q, k = torch.empty(0, 5, 4, 64, device="cuda", dtype=dtype), torch.empty(0, 7, 2, 64, device="cuda", dtype=dtype)
    y, lse = dm.attention(q, k, k)
    assert y.shape == q.shape and lse.shape == (4, 0, 5)
    dq, dk, dv = dm.attention_backward(q, q, k, k, y, lse)
    assert dq.shape == q.shape and dk.shape == dv.shape == k.shape
    rq, rk = dm.qk_norm_rope(q, k[:, :5], torch.empty(0, 5, device="cuda", dtype=torch.int64))
    assert rq.shape == q.shape and rk.shape == (0, 5, 2, 64)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("keys", [[0, 40, 3000, 1, 900], [0, 9000]], ids=str)
def test_single_tokens_in_many_parts(keys, dtype):
    lens = [0] + [1] * (len(keys) - 1)
    run(*inputs(sum(lens), sum(keys), 6, 2, 72, dtype), lens, keys, causal=True)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_parts_of_rows_that_see_little(dtype):
    # rows that see no key, few keys or all, each in several parts
    for causal in (True, False):
        lens, keys = [0, 3, 1, 2], [0, 2, 5000, 0]
        run(*inputs(sum(lens), sum(keys), 4, 1, 128, dtype), lens, keys, causal=causal)


@pytest.mark.parametrize("bad", [nan, inf, -inf])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_unseen_values_reach_no_part(dtype, bad):
    # four tokens on 4000 keys: the last key of each but the last token is not seen by those before
    q, k, v, dy = inputs(6, 4900, 4, 2, 72, dtype)
    cu = (edges([0, 4, 2]), edges([0, 4000, 900]))
    def both(q, k, v):
        y, lse = dm.attention(q, k, v, *cu)
        return [y, lse, *dm.attention_backward(dy, q, k, v, y, lse, *cu)]
    want = both(q, k, v)
    for which in (1, 2):
        x = [q.clone(), k.clone(), v.clone()]
        x[which][3999, :, 5] = bad  # seen by token 3 alone
        y, lse, dq, dk, dv = both(*x)
        for rows in (slice(0, 3), slice(4, 6)):
            assert torch.equal(y[rows], want[0][rows]) and torch.equal(lse[:, rows], want[1][:, rows])
            assert torch.equal(dq[rows], want[2][rows])
        assert torch.equal(dk[4000:], want[3][4000:]) and torch.equal(dv[4000:], want[4][4000:])
        if which == 2:
            assert not torch.isfinite(y[3]).all()


def test_parts_in_graphs():
    q, k, v, _ = inputs(8, 20000, 8, 2, 128, BF16)
    cu_q, cu_k = edges([0] + [1] * 8), edges([0] + [2500] * 8)
    y, lse = dm.attention(q, k, v, cu_q, cu_k)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = dm.attention(q, k, v, cu_q, cu_k)
    for i in range(4):  # other lengths in the same graph
        cu_k.copy_(edges([0] + [2500] * 8) if i % 2 == 0 else edges([100, 9000, 1, 0, 4000, 64, 3000, 700, 3000]))
        want = dm.attention(q, k, v, cu_q, cu_k)
        for z in out:
            z.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, out)), i
