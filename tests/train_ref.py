"""64-bit forms of the training operators and bounds on the kernels' error
(not a test module).

Bounds.  u is the unit roundoff of the caller's type: 2^-p for a significand of
p bits (2^-8 for bf16, whose 1 + 2^-8 rounds to 1; 2^-24 for fp32).  A sum of K products accumulated in fp32 is off by at
most a = (K + 8) 2^-24 of the sum of their magnitudes (K - 1 additions, and a
margin for the exponential, error function and division around it); the
products of bf16 values are exact in fp32.  Every value that is rounded to the
caller's type on the way (h, dg, du; the softmax, twice) adds u of its
magnitude (g and u, saved with 12 bits for the backward pass, 2^-12).  The bounds below carry these errors through the formulas in first
order, magnitudes in place of signed terms, and are multiplied by 1.01 for the
second order.  Large fp32 products take each operand as three bf16 planes,
which hold a value to the smaller of 2^-24 of it and bf16's least step, half of
2^-133 (``planes`` below).  Nothing in the bounds is fitted to a result.
"""

import math

import torch

ROUNDOFF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def acc(k):
    return (k + 8) * 2.0 ** -24


def act(g, name):
    """act(g), act'(g) and a bound of |act''|."""
    if name == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s)), 0.5
    if name == "gelu":
        p = 0.5 * torch.erfc(-g * math.sqrt(0.5))
        return g * p, p + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi), 0.8
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 0.134145 * g * g), 0.8


def layer_norm(x, w, b, eps, dy=None):
    """(values, bounds) of y, mean, rstd and, with dy, of dx, dw, db."""
    hu = ROUNDOFF[x.dtype]
    x, w = x.double(), w.double()
    b = torch.zeros_like(w) if b is None else b.double()
    n = x.shape[-1]
    a = acc(n)
    mean = x.mean(-1, keepdim=True)
    xc = x - mean
    var = (xc * xc).mean(-1, keepdim=True)
    rstd = 1 / torch.sqrt(var + eps)
    xh = xc * rstd
    y = xh * w + b
    # the mean's error shifts every xc; the variance about the shifted mean
    # gains its square and the cross term with the sum of xc (zero)
    e_mean = a * x.abs().mean(-1, keepdim=True)
    e_xc = e_mean + 2.0 ** -24 * (x.abs() + mean.abs())
    e_var = a * var + 2 * (xc.abs() * e_xc).mean(-1, keepdim=True) + (e_xc ** 2).mean(-1, keepdim=True)
    e_rstd = rstd * (0.5 * e_var / (var + eps) + 8 * 2.0 ** -24)
    e_xh = e_xc * rstd + xc.abs() * e_rstd
    e_y = hu * y.abs() + e_xh * w.abs() + 4 * 2.0 ** -24 * ((xh * w).abs() + b.abs())
    vals, errs = [y, mean[..., 0], rstd[..., 0]], [e_y, e_mean[..., 0], e_rstd[..., 0]]
    if dy is not None:
        dy = dy.double()
        g = dy * w
        m1, m2 = g.mean(-1, keepdim=True), (g * xh).mean(-1, keepdim=True)
        dx = rstd * (g - m1 - xh * m2)
        e_m1 = a * g.abs().mean(-1, keepdim=True)
        e_m2 = a * (g * xh).abs().mean(-1, keepdim=True) + (g.abs() * e_xh).mean(-1, keepdim=True)
        size = g.abs() + m1.abs() + (xh * m2).abs()
        e_dx = (hu * dx.abs() + rstd * (e_m1 + xh.abs() * e_m2 + e_xh * m2.abs() + 8 * 2.0 ** -24 * size)
                + e_rstd * (dx / rstd).abs())
        rows = x.reshape(-1, n).shape[0]
        flat = lambda t: t.reshape(-1, n)
        dw, db = flat(dy * xh).sum(0), flat(dy).sum(0)
        ar = acc(rows)
        e_dw = hu * dw.abs() + ar * flat((dy * xh).abs()).sum(0) + flat(dy.abs() * e_xh).sum(0)
        e_db = hu * db.abs() + ar * flat(dy.abs()).sum(0)
        vals += [dx, dw, db]
        errs += [e_dx, e_dw, e_db]
    return vals, [1.01 * e for e in errs]


def gated_ffn(x, wg, wu, wd, name, dy=None):
    """(values, bounds) of y and, with dy, of dx, dwg, dwu, dwd; 2-D x."""
    hu = ROUNDOFF[x.dtype]
    x, wg, wu, wd = x.double(), wg.double(), wu.double(), wd.double()
    d, f, t = x.shape[1], wg.shape[0], x.shape[0]
    ad, af, at = acc(d), acc(f), acc(t)
    g, u = x @ wg.T, x @ wu.T
    e_g, e_u = ad * (x.abs() @ wg.abs().T), ad * (x.abs() @ wu.abs().T)
    A, D, D2 = act(g, name)
    # an activation is evaluated to a few fp32 units of max(|g|, its value)
    e_A = D.abs() * e_g + D2 * e_g ** 2 + 8 * 2.0 ** -24 * (A.abs() + 0.5 * g.abs())
    h = A * u
    e_h = hu * h.abs() + e_A * u.abs() + A.abs() * e_u
    y = h @ wd.T
    e_y = hu * y.abs() + e_h @ wd.abs().T + af * (h.abs() @ wd.abs().T)
    vals, errs = [y], [e_y]
    if dy is not None:
        dy = dy.double()
        dh = dy @ wd
        e_dh = ad * (dy.abs() @ wd.abs())
        # the backward pass reads g and u rounded (bf16: to 12 bits)
        hs = 2.0 ** -12 if hu > 2.0 ** -12 else hu
        r_g, r_u = e_g + hs * g.abs(), e_u + hs * u.abs()
        e_D = D2 * r_g + 16 * 2.0 ** -24
        e_A2 = D.abs() * r_g + D2 * r_g ** 2 + 8 * 2.0 ** -24 * (A.abs() + 0.5 * g.abs())
        dg, du = dh * u * D, dh * A
        e_dg = hu * dg.abs() + e_dh * (u * D).abs() + dh.abs() * (r_u * D.abs() + u.abs() * e_D + r_u * e_D)
        e_du = hu * du.abs() + e_dh * A.abs() + dh.abs() * e_A2
        dx = dg @ wg + du @ wu
        e_dx = (hu * dx.abs() + e_dg @ wg.abs() + e_du @ wu.abs()
                + acc(2 * f) * (dg.abs() @ wg.abs() + du.abs() @ wu.abs()))
        vals.append(dx)
        errs.append(e_dx)
        for left, e_left, right, e_right in ((dg, e_dg, x, None), (du, e_du, x, None), (dy, None, h, e_h)):
            v = left.T @ right
            e = hu * v.abs() + at * (left.abs().T @ right.abs())
            if e_left is not None:
                e = e + e_left.T @ right.abs()
            if e_right is not None:
                e = e + left.abs().T @ e_right
            vals.append(v)
            errs.append(e)
    return vals, [1.01 * e for e in errs]


def cross_entropy(x, w, y, grad=True, planes=False):
    """(values, bounds) of loss, losses and, with grad, dx and dw; 2-D x."""
    hu = ROUNDOFF[x.dtype]
    least = 2.0 ** -134 if planes else 0.0
    x, w = x.double(), w.double()
    t, d = x.shape
    v = w.shape[0]
    counts = (y >= 0) & (y < v)
    n = max(1, int(counts.sum()))
    word = torch.where(counts, y, torch.zeros_like(y))[:, None]
    l = x @ w.T
    e_l = acc(d) * (x.abs() @ w.abs().T) + least * (x.abs().sum(1, keepdim=True) + w.abs().sum(1)[None, :])
    lse = torch.logsumexp(l, 1, keepdim=True)
    p = torch.exp(l - lse)
    # fp32 rounding of the logits' differences, then the sum of exponentials
    e_d = e_l + 2.0 ** -23 * (l.abs() + lse.abs() + 1)
    e_lse = (p * e_d).sum(1, keepdim=True) + acc(v if v < 4096 else 4096) + 2.0 ** -23 * (lse.abs() + 1)
    at, e_at = l.gather(1, word), e_d.gather(1, word)
    cf = counts.double()
    losses = (lse - at)[:, 0] * cf
    e_losses = (e_lse + e_at)[:, 0] * cf
    loss, e_loss = losses.sum() / n, e_losses.sum() / n + 4 * 2.0 ** -24 * losses.abs().sum() / n
    vals, errs = [loss, losses], [e_loss, e_losses]
    if grad:
        q = p.scatter(1, word, torch.expm1(at - lse)) * cf[:, None]
        # rounded as the exponential and again as the softmax; the fp32 rest
        # is relative to the softmax (to 1 at the target)
        rel = e_d + e_lse + 16 * 2.0 ** -24
        e_q = 2 * hu * q.abs() + rel * p.scatter(1, word, torch.ones_like(at) * p.gather(1, word))
        e_q = e_q * cf[:, None] + 2.0 ** -126
        dx, dw = q @ w / n, q.T @ x / n
        e_q = e_q + least
        e_dx = hu * dx.abs() + (e_q @ w.abs() + acc(v) * (q.abs() @ w.abs()) + least * q.abs().sum(1, keepdim=True)) / n
        e_dw = hu * dw.abs() + (e_q.T @ x.abs() + acc(t) * (q.abs().T @ x.abs()) + least * q.abs().sum(0)[:, None]) / n
        vals += [dx, dw]
        errs += [e_dx, e_dw]
    return vals, [1.01 * e for e in errs]


def check(got, vals, errs, names):
    """Every element within its bound (and not NaN)."""
    for g, v, e, name in zip(got, vals, errs, names):
        assert tuple(g.shape) == tuple(v.shape), (name, tuple(g.shape), tuple(v.shape))
        off = (g.double() - v).abs()
        bad = ~(off <= e + 2.0 ** -126)
        if bool(bad.any()):
            i = int(torch.argmax((off / (e + 2.0 ** -126)).nan_to_num(float("inf")).reshape(-1)))
            raise AssertionError(f"{name}: {int(bad.sum())} of {g.numel()} out of bound; worst at {i}: got "
                                 f"{g.reshape(-1)[i].item()}, want {v.reshape(-1)[i].item()}, bound "
                                 f"{e.expand_as(v).reshape(-1)[i].item()}")
