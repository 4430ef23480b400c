"""The attention block's cases: queries and keys normed per head and rotated,
attention over packed sequences with grouped heads, and dropout from a
counter-based generator, each forward alone and with its backward pass.

``run`` computes a case in plain torch operations (32 bits, rounded once at the
end; angles in 64), or through matrix_orthogonalising_optimizer_amd where
``own`` is true; ``exact`` computes it in 64 bits with torch's own derivatives
and, for dropout, a generator of its own.
"""

from __future__ import annotations

import math

import numpy as np
import torch

own = False

EPS = 1e-6


def listed():
    return [
        # --- norm and rotation: tokens, heads of q and k, their width
        # one new token of a 7B-class layer: nothing but latency
        {"name": "rope_token", "op": "rope", "dir": "fwd", "tokens": 1, "hq": 32, "hk": 8, "dim": 128, "rot": 128,
         "sections": "", "base": 10000.0, "interleaved": False, "far": 4000, "dtype": "bf16"},
        # image and video tokens with time, height and width, an odd token count, fp32, rotated in part
        {"name": "rope_video_f32", "op": "rope", "dir": "train", "tokens": 4999, "hq": 12, "hk": 12, "dim": 80,
         "rot": 64, "sections": "8,12,12", "base": 10000.0, "interleaved": True, "far": 500, "dtype": "f32"},
        # a training step's batch of a 7B-class layer, positions of a long context
        {"name": "rope_7b", "op": "rope", "dir": "train", "tokens": 16384, "hq": 32, "hk": 8, "dim": 128, "rot": 128,
         "sections": "", "base": 500000.0, "interleaved": False, "far": 1000000, "dtype": "bf16"},
        # --- attention: lengths of the packed sequences' queries and (where they differ) keys
        # four short examples of a small model
        {"name": "att_short", "op": "att", "dir": "train", "lens": "64,17,300,131", "keys": "", "hq": 8, "hk": 8,
         "dim": 64, "causal": True, "fused": False, "dtype": "bf16"},
        # one new token for each of sixteen prompts of up to 8192 (evaluation, generation between training steps)
        {"name": "att_step", "op": "att", "dir": "fwd", "lens": ",".join(["1"] * 16),
         "keys": "8192,700,5003,1,4096,2222,64,7777,313,6000,1024,8191,3500,129,4500,2048", "hq": 32, "hk": 8,
         "dim": 128, "causal": True, "fused": False, "dtype": "bf16"},
        # fp32 and odd everywhere: an action head's queries on another model's longer prefix, nothing masked
        {"name": "att_cross_f32", "op": "att", "dir": "train", "lens": "701,50,333", "keys": "1100,1,515", "hq": 6,
         "hk": 3, "dim": 72, "causal": False, "fused": False, "dtype": "f32"},
        # a packed batch of a 7B-class layer, lengths as documents have them, q, k and v in one projection's output
        {"name": "att_packed", "op": "att", "dir": "train",
         "lens": "4096,37,901,2500,1,333,1800,64,2047,129,777,3100,600", "keys": "", "hq": 32, "hk": 8, "dim": 128,
         "causal": True, "fused": True, "dtype": "bf16"},
        # training on one long sequence
        {"name": "att_train", "op": "att", "dir": "train", "lens": "8192", "keys": "", "hq": 32, "hk": 8, "dim": 128,
         "causal": True, "fused": False, "dtype": "bf16"},
        # a whole long prompt, forward alone
        {"name": "att_prompt", "op": "att", "dir": "fwd", "lens": "16384", "keys": "", "hq": 32, "hk": 8, "dim": 128,
         "causal": True, "fused": False, "dtype": "bf16"},
        # --- dropout: rows x width
        # one example's activations
        {"name": "drop_row", "op": "drop", "dir": "fwd", "rows": 1, "width": 4096, "p": 0.1, "residual": True,
         "dtype": "bf16"},
        # fp32, a count that no vector width divides
        {"name": "drop_odd_f32", "op": "drop", "dir": "train", "rows": 5003, "width": 1001, "p": 0.25,
         "residual": False, "dtype": "f32"},
        # a sublayer's output on its way into the residual stream of a 7B-class layer
        {"name": "drop_7b", "op": "drop", "dir": "train", "rows": 16384, "width": 4096, "p": 0.1, "residual": True,
         "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _pairs(case):
    """(query, key) pairs that a case's attention computes, over its sequences."""
    total = 0
    for n, m in zip(*_lengths(case)):
        if not case["causal"]:
            total += n * m
        else:  # query i sees keys up to i + m - n
            full = min(n, m)
            total += full * (m - full) + full * (full + 1) // 2
    return total


def _lengths(case):
    n = [int(x) for x in case["lens"].split(",")]
    return n, ([int(x) for x in case["keys"].split(",")] if case["keys"] else n)


def draw(rng):
    op = rng.choice(["rope", "att", "att", "drop"])
    case = {"op": op, "dir": rng.choice(["fwd", "train"]), "dtype": rng.choice(["bf16", "bf16", "f32"])}
    while True:
        if op == "rope":
            dim = rng.choice([32, 64, 72, 80, 96, 128, 128, 160, 256])
            rot = rng.choice([dim, dim, dim // 2 & ~1])
            half = rot // 2
            a, b = half // 4, half // 3
            group = rng.choice([1, 2, 4, 8])
            hk = rng.choice([1, 2, 3, 4, 8])
            case.update(tokens=_log(rng, 1, 65536), hq=hk * group, hk=hk, dim=dim, rot=rot,
                        sections=rng.choice(["", "", f"{half - a},{a}", f"{half - a - b},{a},{b}"]),
                        base=rng.choice([10000.0, 500000.0]), interleaved=rng.random() < 0.3,
                        far=_log(rng, 100, 1000000))
            if case["tokens"] * (case["hq"] + hk) * dim <= 16384 * 40 * 128:
                return case
        elif op == "att":
            dim = rng.choice([32, 64, 64, 72, 80, 96, 128, 128, 128] + ([160, 256] if case["dtype"] == "bf16" else []))
            hk, group = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 1, 2, 4, 7])
            n = _log(rng, 1, 64)
            lens = [_log(rng, 1, 16384) for _ in range(n)]
            kind = rng.choice(["self", "self", "step", "cross"])
            keys = []
            if kind == "step":
                keys, lens, case["dir"] = lens, [1] * n, "fwd"
            elif kind == "cross":
                keys = [max(1, int(x * rng.uniform(0.3, 2.0))) for x in lens]
            case.update(lens=",".join(map(str, lens)), keys=",".join(map(str, keys)), hq=hk * group, hk=hk, dim=dim,
                        causal=kind != "cross" or rng.random() < 0.3, fused=kind == "self" and rng.random() < 0.5)
            work = _pairs(case) * case["hq"] * dim
            most = 8192 * 4096 * 32 * 128 // (1 if case["dtype"] == "bf16" else 16)
            if work <= most * (2 if case["dir"] == "fwd" else 1) and max(lens + keys) ** 2 * case["hq"] <= 2 ** 33 \
                    and sum(keys or lens) <= 131072:
                return case
        else:
            case.update(rows=_log(rng, 1, 65536), width=_log(rng, 32, 16384), p=rng.choice([0.05, 0.1, 0.3, 0.5]),
                        residual=rng.random() < 0.5)
            if case["rows"] * case["width"] <= 16384 * 4096:
                return case


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    train = case["dir"] == "train"

    def normal(*shape, std=1.0, mean=0.0):
        return torch.empty(shape, device="cuda").normal_(mean, std, generator=gen)

    st = dict(case)
    if case["op"] == "rope":
        t, dim = case["tokens"], case["dim"]
        sections = [int(x) for x in case["sections"].split(",")] if case["sections"] else None
        shape = (t, len(sections)) if sections else (t,)
        for name, h in (("q", case["hq"]), ("k", case["hk"])):
            # heads of different sizes, a few channels far larger than the others
            x = normal(t, h, dim) * torch.exp(normal(h, 1))
            x[..., :: max(1, dim // 4)] *= 8.0
            st[name] = x.to(dt)
            st["w" + name] = normal(dim, std=0.2, mean=1.0).to(dt)
            if train:
                st["d" + name] = normal(t, h, dim, std=0.01).to(dt)
        st["pos"] = torch.randint(0, case["far"], shape, device="cuda", generator=gen)
        st["section_list"] = sections
    elif case["op"] == "att":
        lens, keys = _lengths(case)
        tq, tk, hq, hk, dim = sum(lens), sum(keys), case["hq"], case["hk"], case["dim"]
        if case["fused"]:
            x = normal(tq, (hq + 2 * hk) * dim).to(dt)
            q, k, v = x.split([hq * dim, hk * dim, hk * dim], 1)
            q, k, v = q.view(tq, hq, dim), k.view(tq, hk, dim), v.view(tq, hk, dim)
        else:
            q, k = normal(tq, hq, dim, std=1.5).to(dt), normal(tk, hk, dim).to(dt)
            v = (normal(tk, hk, dim) + normal(hk, dim, std=0.5)).to(dt)
        edges = lambda ns: torch.tensor(np.cumsum([0] + ns), dtype=torch.int32, device="cuda")
        st.update(q=q, k=k, v=v, cu_q=edges(lens), cu_k=edges(keys), len_q=lens, len_k=keys)
        if train:
            st["dy"] = normal(tq, hq, dim, std=0.01).to(dt)
    else:
        rows, width = case["rows"], case["width"]
        st["x"] = normal(rows, width).to(dt)
        st["res"] = normal(rows, width, std=3.0).to(dt) if case["residual"] else None
        if train:
            st["dy"] = normal(rows, width, std=0.01).to(dt)
        st["seed"], st["offset"] = 0x9e3779b97f4a7c * (seed + 1) & (2 ** 63 - 1), 1000003 * (seed % 1000)
    return st


# ---------------------------------------------------------------- the framework's calls
def _run_own(st):
    import matrix_orthogonalising_optimizer_amd as dm
    train = st["dir"] == "train"
    if st["op"] == "rope":
        how = dict(eps=EPS, base=st["base"], rotary_dim=st["rot"], sections=st["section_list"],
                   interleaved=st["interleaved"])
        out = list(dm.qk_norm_rope(st["q"], st["k"], st["pos"], st["wq"], st["wk"], **how))
        if train:
            out += dm.qk_norm_rope_backward(st["dq"], st["dk"], st["q"], st["k"], st["pos"], st["wq"], st["wk"], **how)
        return out
    if st["op"] == "att":
        at = (st["cu_q"], st["cu_k"])
        y, lse = dm.attention(st["q"], st["k"], st["v"], *at, causal=st["causal"])
        if not train:
            return [y, lse]
        return [y, lse, *dm.attention_backward(st["dy"], st["q"], st["k"], st["v"], y, lse, *at, causal=st["causal"])]
    y = dm.dropout(st["x"], st["p"], st["seed"], offset=st["offset"], residual=st["res"])
    if not train:
        return [y]
    return [y, dm.dropout_backward(st["dy"], st["p"], st["seed"], offset=st["offset"])]


# ---------------------------------------------------------------- the plain forms
def _turn(x, c, s, rot, interleaved):
    """The first `rot` elements of heads turned, in pairs (i, i + rot / 2) or (2i, 2i + 1)."""
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    a, b = a * c - b * s, b * c + a * s
    r = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([r, x[..., rot:]], -1)


def _plain_rope(st):
    rot, inter = st["rot"], st["interleaved"]
    half = rot // 2
    i = torch.arange(half, device="cuda", dtype=torch.float64)
    freq = torch.exp(i * (-2.0 / rot * math.log(st["base"])))
    pos = st["pos"].double()
    if st["section_list"]:
        axis = torch.repeat_interleave(torch.arange(len(st["section_list"]), device="cuda"),
                                       torch.tensor(st["section_list"], device="cuda"), output_size=half)
        angle = pos[:, axis] * freq
    else:
        angle = pos[:, None] * freq
    c, s = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]

    def one(x, w, dy):
        dt = x.dtype
        x, w = x.float(), w.float()
        r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
        n = x * r
        y = _turn(n * w, c, s, rot, inter).to(dt)
        if dy is None:
            return y, None, None
        g = _turn(dy.float(), c, -s, rot, inter)
        gw = g * w
        return y, (r * (gw - n * (gw * n).mean(-1, keepdim=True))).to(dt), (g * n).sum((0, 1)).to(dt)

    q, dq, dwq = one(st["q"], st["wq"], st.get("dq"))
    k, dk, dwk = one(st["k"], st["wk"], st.get("dk"))
    return [q, k] if dq is None else [q, k, dq, dk, dwq, dwk]


def _plain_attention(st):
    dt, hq, hk, dim = st["q"].dtype, st["hq"], st["hk"], st["dim"]
    g, scale = hq // hk, dim ** -0.5
    heads = lambda x: x.float().view(x.shape[0], hk, -1, dim).permute(1, 2, 0, 3)  # (hk, group, tokens, dim)
    q, k, v = heads(st["q"]), heads(st["k"]), heads(st["v"])
    y = torch.zeros(q.shape, device="cuda")
    lse = torch.full(q.shape[:3], -math.inf, device="cuda")
    train = "dy" in st
    if train:
        dy, dq, dk, dv = heads(st["dy"]), torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    a = b = 0
    for n, m in zip(st["len_q"], st["len_k"]):  # one sequence after another
        if n > 0 and m > 0:
            qs = q[:, :, a:a + n].reshape(hk, g * n, dim)
            ks, vs = k[:, 0, b:b + m], v[:, 0, b:b + m]
            p = torch.bmm(qs, ks.transpose(1, 2)).mul_(scale).view(hk, g, n, m)
            if st["causal"]:
                row, col = torch.arange(n, device="cuda")[:, None], torch.arange(m, device="cuda")
                p.masked_fill_(col > row + (m - n), -math.inf)
            top = p.amax(-1, keepdim=True)
            top = torch.where(top == -math.inf, torch.zeros_like(top), top)
            p.sub_(top).exp_()
            total = p.sum(-1, keepdim=True)
            lse[:, :, a:a + n] = (torch.log(total) + top)[..., 0]
            p.div_(torch.where(total == 0, torch.ones_like(total), total))
            ys = torch.bmm(p.view(hk, g * n, m), vs)
            y[:, :, a:a + n] = ys.view(hk, g, n, dim)
            if train:
                ds = dy[:, :, a:a + n].reshape(hk, g * n, dim)
                dp = torch.bmm(ds, vs.transpose(1, 2)).sub_((ds * ys).sum(-1, keepdim=True))
                p = p.view(hk, g * n, m)
                dv[:, 0, b:b + m] = torch.bmm(p.transpose(1, 2), ds)
                dp.mul_(p).mul_(scale)
                dq[:, :, a:a + n] = torch.bmm(dp, ks).view(hk, g, n, dim)
                dk[:, 0, b:b + m] = torch.bmm(dp.transpose(1, 2), qs)
        a, b = a + n, b + m
    flat = lambda x: x.permute(2, 0, 1, 3).reshape(x.shape[2], -1, dim).to(dt)
    out = [flat(y), lse.view(hq, -1)]
    return out + [flat(dq), flat(dk), flat(dv)] if train else out


def _keep(st, n):
    """Which of n elements stay: Philox 4x32-10 of counter offset + i / 8 gives the 16-bit numbers of elements i .. i + 7."""
    low = 0xffffffff
    c = torch.arange((n + 7) // 8, device="cuda") + st["offset"]
    c0, c1 = c & low, (c >> 32) & low
    c2 = c3 = torch.zeros_like(c)
    k0, k1 = st["seed"] & low, (st["seed"] >> 32) & low
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57  # (modulo 2^64: the bits are those of the product without sign)
        c0, c1, c2, c3 = ((b >> 32) & low) ^ c1 ^ k0, b & low, ((a >> 32) & low) ^ c3 ^ k1, a & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    w = torch.stack([c0, c1, c2, c3], 1)
    u = torch.stack([w & 0xffff, w >> 16], 2).reshape(-1)[:n]
    return u >= round(st["p"] * 65536)


def _plain_dropout(st):
    dt, shape = st["x"].dtype, st["x"].shape
    keep = _keep(st, st["x"].numel()).view(shape)
    scale = 65536.0 / (65536 - round(st["p"] * 65536))

    def masked(x):
        return torch.where(keep, x.float() * scale, torch.zeros((), device="cuda"))

    y = masked(st["x"])
    out = [(y if st["res"] is None else y + st["res"].float()).to(dt)]
    return out + [masked(st["dy"]).to(dt)] if "dy" in st else out


def run(state):
    if own:
        return _run_own(state)
    return {"rope": _plain_rope, "att": _plain_attention, "drop": _plain_dropout}[state["op"]](state)


# ---------------------------------------------------------------- 64 bits
def _exact_rope(st, train):
    rot = st["rot"]
    freq = st["base"] ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    pos = st["pos"].double().reshape(st["tokens"], -1)
    parts, at = [], 0
    for axis, n in enumerate(st["section_list"] or [rot // 2]):
        parts.append(pos[:, axis, None] * freq[at:at + n])
        at += n
    z = torch.polar(torch.ones((), device="cuda", dtype=torch.float64), torch.cat(parts, 1))[:, None]
    out, grads = [], []
    for name in "qk":
        x, w = (st[n].double().requires_grad_(train) for n in (name, "w" + name))
        n = x / torch.sqrt(x.square().mean(2, keepdim=True) + EPS) * w
        r, rest = n[..., :rot], n[..., rot:]
        pair = r.unflatten(2, (rot // 2, 2)) if st["interleaved"] else r.unflatten(2, (2, rot // 2)).transpose(2, 3)
        turned = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * z)
        turned = turned if st["interleaved"] else turned.transpose(2, 3)
        y = torch.cat([turned.flatten(2), rest], 2)
        out.append(y.detach())
        if train:
            grads.append(torch.autograd.grad(y, (x, w), st["d" + name].double()))
    return out + [g[i] for i in range(2) for g in grads]


def _exact_attention(st, train):
    hq, hk, dim = st["hq"], st["hk"], st["dim"]
    g = hq // hk
    y = torch.zeros(st["q"].shape, device="cuda", dtype=torch.float64)
    lse = torch.full((hq, y.shape[0]), -math.inf, device="cuda", dtype=torch.float64)
    grads = [torch.zeros(st[n].shape, device="cuda", dtype=torch.float64) for n in "qkv"] if train else []
    a = b = 0
    for n, m in zip(st["len_q"], st["len_k"]):
        seen = torch.ones(n, m, device="cuda", dtype=torch.bool)
        seen = seen.tril(m - n) if st["causal"] else seen
        some = seen.any(1)
        for h in range(hq if n and m else 0):
            q, k, v = (st[x][s:s + c, j].double().requires_grad_(train)
                       for x, s, c, j in (("q", a, n, h), ("k", b, m, h // g), ("v", b, m, h // g)))
            s = (q @ k.T / math.sqrt(dim)).masked_fill(~seen, -math.inf)
            # (a row that sees nothing has no softmax: zeros, and no gradient)
            s = torch.where(some[:, None], s, torch.zeros_like(s))
            z = torch.softmax(s, 1) @ v * some[:, None]
            y[a:a + n, h] = z.detach()
            lse[h, a:a + n] = torch.where(some, torch.logsumexp(s.detach(), 1), lse[h, a:a + n])
            if train:
                for t, d, s_, c, j in zip(grads, torch.autograd.grad(z, (q, k, v), st["dy"][a:a + n, h].double()),
                                          (a, b, b), (n, m, m), (h, h // g, h // g)):
                    t[s_:s_ + c, j] += d
        a, b = a + n, b + m
    return [y, lse, *grads]


def _exact_dropout(st, train):
    n = st["x"].numel()
    c = np.arange((n + 7) // 8, dtype=np.uint64) + np.uint64(st["offset"])
    x = [(c & np.uint64(0xffffffff)).astype(np.uint32), (c >> np.uint64(32)).astype(np.uint32)]
    x += [np.zeros_like(x[0]), np.zeros_like(x[0])]
    key = [np.uint32(st["seed"] & 0xffffffff), np.uint32(st["seed"] >> 32)]
    with np.errstate(over="ignore"):
        for _ in range(10):
            left = x[0].astype(np.uint64) * np.uint64(0xD2511F53)
            right = x[2].astype(np.uint64) * np.uint64(0xCD9E8D57)
            x = [(right >> np.uint64(32)).astype(np.uint32) ^ x[1] ^ key[0], right.astype(np.uint32),
                 (left >> np.uint64(32)).astype(np.uint32) ^ x[3] ^ key[1], left.astype(np.uint32)]
            key = [key[0] + np.uint32(0x9E3779B9), key[1] + np.uint32(0xBB67AE85)]
    words = np.stack(x, 1).astype("<u4").reshape(-1).view("<u2")[:n]
    cut = int(round(st["p"] * 65536))
    keep = torch.from_numpy(words.astype(np.int32)).cuda().view(st["x"].shape) >= cut
    factor = keep.double() / (1.0 - cut / 65536)
    y = st["x"].double() * factor
    if st["res"] is not None:
        y = y + st["res"].double()
    return [y, st["dy"].double() * factor] if train else [y]


def exact(case, seed):
    st = prepare(case, seed)
    train = case["dir"] == "train"
    return {"rope": _exact_rope, "att": _exact_attention, "drop": _exact_dropout}[case["op"]](st, train)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    train = case["dir"] == "train"
    if case["op"] == "rope":  # q and k in and out, with training their gradients too; positions; weights
        n = case["tokens"] * (case["hq"] + case["hk"]) * case["dim"]
        axes = case["sections"].count(",") + 1
        return {"bytes": (4 if train else 2) * n * e + 8 * case["tokens"] * axes + (4 if train else 2) * case["dim"] * e,
                "flops": (25 if train else 9) * n}
    if case["op"] == "att":  # q, k, v in, y and lse out; with training dy in, three gradients out
        lens, keys = _lengths(case)
        q, k = sum(lens) * case["hq"] * case["dim"], sum(keys) * case["hk"] * case["dim"]
        pairs = _pairs(case) * case["hq"] * case["dim"]
        return {"bytes": ((4 * q + 4 * k) if train else (2 * q + 2 * k)) * e + 4 * sum(lens) * case["hq"],
                "flops": (14 if train else 4) * pairs}
    n = case["rows"] * case["width"]
    return {"bytes": ((3 if case["residual"] else 2) + (2 if train else 0)) * n * e, "flops": (4 if train else 2) * n}
