"""The training operators' cases: layer norm, the gated feed-forward block and
the linear cross entropy, each forward alone and with its backward pass.

``run`` computes a case in plain torch operations (32 bits, rounded once at the
end), or through matrix_orthogonalising_optimizer_amd where ``own`` is true;
``exact`` computes it in 64 bits with torch's own derivatives.
"""

from __future__ import annotations

import math

import torch

own = False

EPS = 1e-5


def listed():
    return [
        # --- layer norm: rows x width
        # one token of a 4096-wide model: nothing but latency
        {"name": "ln_token", "op": "ln", "dir": "fwd", "rows": 1, "width": 4096, "dtype": "bf16"},
        # fp32 parameters, a row count and a width that fill no tile
        {"name": "ln_ragged_f32", "op": "ln", "dir": "train", "rows": 5003, "width": 1001, "dtype": "f32"},
        # a training step's whole batch of a 7B-class layer
        {"name": "ln_7b", "op": "ln", "dir": "train", "rows": 32768, "width": 4096, "dtype": "bf16"},
        # --- gated feed-forward: tokens, model width, hidden width
        # a single token through the 7B-class block: the weights' bytes
        {"name": "ffn_token", "op": "ffn", "dir": "fwd", "tokens": 1, "d": 4096, "f": 11008, "act": "silu",
         "dtype": "bf16"},
        # a short batch through a 1024 x 4096 block, the mixed set's middle size
        {"name": "ffn_1024", "op": "ffn", "dir": "train", "tokens": 512, "d": 1024, "f": 4096, "act": "silu",
         "dtype": "bf16"},
        # sizes that no tile divides and rows that are not 16-byte aligned
        {"name": "ffn_odd", "op": "ffn", "dir": "train", "tokens": 1531, "d": 2050, "f": 5461, "act": "gelu",
         "dtype": "bf16"},
        # fp32 training of a small block
        {"name": "ffn_f32", "op": "ffn", "dir": "train", "tokens": 777, "d": 1000, "f": 2730, "act": "gelu_tanh",
         "dtype": "f32"},
        # the 7B-class layer's block on a batch of 8192 tokens
        {"name": "ffn_7b", "op": "ffn", "dir": "train", "tokens": 8192, "d": 4096, "f": 11008, "act": "silu",
         "dtype": "bf16"},
        # the 70B-class block
        {"name": "ffn_70b", "op": "ffn", "dir": "train", "tokens": 4096, "d": 8192, "f": 28672, "act": "silu",
         "dtype": "bf16"},
        # --- linear cross entropy: tokens, width, vocabulary, share of tokens that do not count
        # the loss of a few tokens (evaluation)
        {"name": "ce_eval", "op": "ce", "dir": "fwd", "tokens": 64, "d": 1024, "vocab": 32000, "masked": 0.0,
         "dtype": "bf16"},
        # fp32 training, odd everywhere, half of the tokens are prompt
        {"name": "ce_f32", "op": "ce", "dir": "train", "tokens": 515, "d": 1000, "vocab": 10007, "masked": 0.5,
         "dtype": "f32"},
        # a training batch at 4096 wide and an odd vocabulary
        {"name": "ce_train", "op": "ce", "dir": "train", "tokens": 8192, "d": 4096, "vocab": 50257, "masked": 0.1,
         "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi):
    """A size spread over the logarithm: half of them 4, 5 or 7 times a power of two, half of them not divisible by 4."""
    n = _log(rng, lo, hi)
    if rng.random() < 0.5:
        return n | rng.choice([1, 2])
    p = 1 << max(n.bit_length() - 3, 4)
    return max(m * p for m in (4, 5, 7) if m * p <= max(n, 4 * p))


def draw(rng):
    case = {"op": rng.choice(["ln", "ffn", "ce"]), "dir": rng.choice(["fwd", "train"]),
            "dtype": rng.choice(["bf16", "bf16", "f32"])}
    while True:
        if case["op"] == "ln":
            case.update(rows=_log(rng, 1, 65536), width=_size(rng, 64, 16384))
            if case["rows"] * case["width"] <= 32768 * 4096:
                return case
        elif case["op"] == "ffn":
            case.update(tokens=_log(rng, 1, 16384), d=_size(rng, 64, 8192), f=_size(rng, 64, 28672),
                        act=rng.choice(["silu", "gelu", "gelu_tanh"]))
            if case["tokens"] * case["d"] * case["f"] <= 8192 * 4096 * 11008:
                return case
        else:
            case.update(tokens=_log(rng, 1, 16384), d=_size(rng, 64, 4096), vocab=_size(rng, 128, 131072),
                        masked=rng.choice([0.0, 0.1, 0.5]))
            if case["tokens"] * case["d"] * case["vocab"] <= 8192 * 4096 * 50257:
                return case


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32

    def normal(*shape, std=1.0, mean=0.0):
        return torch.empty(shape, device="cuda").normal_(mean, std, generator=gen)

    st = dict(case)
    if case["op"] == "ln":
        rows, width = case["rows"], case["width"]
        # a residual stream: an offset, and a few channels far larger than the others
        x = normal(rows, width) + normal(width, std=0.5)
        x[:, :: max(1, width // 4)] *= 20.0
        st.update(x=x.to(dt), w=normal(width, std=0.2, mean=1.0).to(dt), b=normal(width, std=0.2).to(dt))
        if case["dir"] == "train":
            st["dy"] = normal(rows, width, std=0.01).to(dt)
    elif case["op"] == "ffn":
        t, d, f = case["tokens"], case["d"], case["f"]
        st.update(x=normal(t, d).to(dt), wg=normal(f, d, std=1.5 / math.sqrt(d)).to(dt),
                  wu=normal(f, d, std=1.0 / math.sqrt(d)).to(dt), wd=normal(d, f, std=1.0 / math.sqrt(f)).to(dt))
        if case["dir"] == "train":
            st["dy"] = normal(t, d, std=0.01).to(dt)
    else:
        t, d, v = case["tokens"], case["d"], case["vocab"]
        w = normal(v, d, std=1.0 / math.sqrt(d))
        # frequent words are more frequent; some tokens are predicted well, some not at all
        u = torch.rand(t, device="cuda", generator=gen)
        y = ((v + 1.0) ** u - 1.0).long().clamp_(0, v - 1)
        sure = torch.rand(t, 1, device="cuda", generator=gen) * 12.0
        x = normal(t, d) + sure * w[y]
        y[torch.rand(t, device="cuda", generator=gen) < case["masked"]] = -100
        st.update(x=x.to(dt), w=w.to(dt), y=y)
    return st


# ---------------------------------------------------------------- the framework's calls
def _run_own(st):
    import matrix_orthogonalising_optimizer_amd as dm
    train = st["dir"] == "train"
    if st["op"] == "ln":
        y, mean, rstd = dm.layer_norm(st["x"], st["w"], st["b"], eps=EPS)
        if not train:
            return [y, mean, rstd]
        return [y, *dm.layer_norm_backward(st["dy"], st["x"], st["w"], mean, rstd)]
    if st["op"] == "ffn":
        ws = (st["wg"], st["wu"], st["wd"])
        if not train:
            return [dm.gated_ffn(st["x"], *ws, act=st["act"])]
        y, saved = dm.gated_ffn(st["x"], *ws, act=st["act"], save=True)
        return [y, *dm.gated_ffn_backward(st["dy"], st["x"], *ws, saved, act=st["act"])]
    if not train:
        return list(dm.linear_cross_entropy(st["x"], st["w"], st["y"], grad=False))
    return list(dm.linear_cross_entropy(st["x"], st["w"], st["y"]))


# ---------------------------------------------------------------- the plain forms
def _act(g, act):
    """act(g) and its derivative."""
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-g))
        return g * s, s * (1.0 + g * (1.0 - s))
    if act == "gelu":
        p = 0.5 * (1.0 + torch.erf(g * math.sqrt(0.5)))
        return g * p, p + g * torch.exp(-0.5 * g * g) * (1.0 / math.sqrt(2.0 * math.pi))
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * c * (1.0 + 3.0 * 0.044715 * g * g)


def _run_plain(st):
    dt = st["x"].dtype
    train = st["dir"] == "train"
    x = st["x"].float()
    if st["op"] == "ln":
        w, b = st["w"].float(), st["b"].float()
        mean = x.mean(1)
        xc = x - mean[:, None]
        rstd = 1.0 / torch.sqrt((xc * xc).mean(1) + EPS)
        xh = xc * rstd[:, None]
        y = (xh * w + b).to(dt)
        if not train:
            return [y, mean, rstd]
        dy = st["dy"].float()
        g = dy * w
        dx = rstd[:, None] * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
        return [y, dx.to(dt), (dy * xh).sum(0).to(dt), dy.sum(0).to(dt)]
    if st["op"] == "ffn":
        wg, wu, wd = st["wg"].float(), st["wu"].float(), st["wd"].float()
        g, u = x @ wg.t(), x @ wu.t()
        a, da = _act(g, st["act"])
        h = a * u
        y = (h @ wd.t()).to(dt)
        if not train:
            return [y]
        dy = st["dy"].float()
        dh = dy @ wd
        dg, du = dh * u * da, dh * a
        dx = dg @ wg + du @ wu
        return [y, dx.to(dt), (dg.t() @ x).to(dt), (du.t() @ x).to(dt), (dy.t() @ h).to(dt)]
    w, y = st["w"].float(), st["y"]
    counts = y >= 0
    n = counts.sum().clamp(min=1).float()
    word = torch.where(counts, y, torch.zeros_like(y))[:, None]
    logits = x @ w.t()
    top = logits.max(1, keepdim=True).values
    e = torch.exp(logits - top)
    s = e.sum(1, keepdim=True)
    at = logits.gather(1, word)
    row = torch.where(counts, (torch.log(s) + top - at)[:, 0], torch.zeros_like(top[:, 0]))
    loss = row.sum() / n
    if not train:
        return [loss, row]
    dl = e / s
    # the target's p - 1, without the cancellation of a sure prediction
    dl.scatter_(1, word, torch.expm1(at - top - torch.log(s)))
    dl = dl * (counts.float() / n)[:, None]
    return [loss, row, (dl @ w).to(dt), (dl.t() @ x).to(dt)]


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    nn = torch.nn.functional
    st = prepare(case, seed)
    train = case["dir"] == "train"

    def leaf(k):
        return st[k].double().requires_grad_(train)

    x = leaf("x")
    if case["op"] == "ln":
        w, b = leaf("w"), leaf("b")
        y = nn.layer_norm(x, (case["width"],), w, b, EPS)
        if not train:
            return [y, x.mean(1), (x.var(1, unbiased=False) + EPS).rsqrt()]
        return [y.detach(), *torch.autograd.grad(y, (x, w, b), st["dy"].double())]
    if case["op"] == "ffn":
        wg, wu, wd = leaf("wg"), leaf("wu"), leaf("wd")
        act = {"silu": nn.silu, "gelu": nn.gelu, "gelu_tanh": lambda g: nn.gelu(g, approximate="tanh")}[case["act"]]
        y = nn.linear(act(nn.linear(x, wg)) * nn.linear(x, wu), wd)
        if not train:
            return [y]
        return [y.detach(), *torch.autograd.grad(y, (x, wg, wu, wd), st["dy"].double())]
    w = leaf("w")
    row = nn.cross_entropy(nn.linear(x, w), st["y"], ignore_index=-100, reduction="none")
    loss = row.sum() / max(1, int((st["y"] >= 0).sum()))
    if not train:
        return [loss, row]
    return [loss.detach(), row.detach(), *torch.autograd.grad(loss, (x, w))]


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    train = case["dir"] == "train"
    if case["op"] == "ln":
        n, k = case["rows"] * case["width"], case["width"]
        if train:  # x, dy in; y, dx out; w, b in, their gradients out
            return {"bytes": 4 * n * e + 4 * k * e, "flops": 20 * n}
        return {"bytes": 2 * n * e + 2 * k * e + 8 * case["rows"], "flops": 8 * n}
    if case["op"] == "ffn":
        t, d, f = case["tokens"], case["d"], case["f"]
        if train:  # x, dy in; y, dx out; three weights in, three gradients out
            return {"bytes": (4 * t * d + 6 * d * f) * e, "flops": 18 * t * d * f}
        return {"bytes": (2 * t * d + 3 * d * f) * e, "flops": 6 * t * d * f}
    t, d, v = case["tokens"], case["d"], case["vocab"]
    if train:  # x, w, targets in; the losses and both gradients out
        return {"bytes": 2 * (t * d + v * d) * e + 12 * t + 4, "flops": 6 * t * d * v}
    return {"bytes": (t * d + v * d) * e + 12 * t + 4, "flops": 2 * t * d * v}
