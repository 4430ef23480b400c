"""64-bit forms of the attention block's operators and bounds on the kernels'
error (not a test module).

Bounds as in train_ref: u is the caller's type's unit roundoff, a sum of K products in
fp32 is off by at most acc(K) of the sum of their magnitudes, and these errors
are carried through the formulas in first order, magnitudes in place of signed
terms.  Nothing in the bounds is fitted to a result.

Attention.  A score is off by scale acc(D) |q| |k|; in the exponent come the
rounding of the row's reference and of the scaling, 2^-23 of the row's largest
score, and the exponential's own (2^-22).  For bf16 the probabilities and ds are
rounded once more (u) as operands.  A row's keys may be walked in parts that are put
together with weights exp(lse of the part - lse): these are off by what both
logarithms are, and lse by what a part's is once more.
"""

import math

import torch

from train_ref import ROUNDOFF, acc, check  # noqa: F401

E = 2.0 ** -24


def attention(q, k, v, lens, keys, causal, scale=None, dy=None, seen=None):
    """(values, bounds) of y, lse and, with dy, of dq, dk, dv.  lens and keys: rows of
    each sequence, the first behind lens[0] (keys[0]) rows that belong to none."""
    u = ROUNDOFF[q.dtype]
    up = u if q.dtype == torch.bfloat16 else 0.0
    q, k, v = q.double(), k.double(), v.double()
    hq, hk, dim = q.shape[1], k.shape[1], q.shape[2]
    g = hq // hk
    scale = dim ** -0.5 if scale is None else scale
    y, lse = torch.zeros_like(q), torch.full((hq, q.shape[0]), -math.inf, dtype=torch.float64, device=q.device)
    ey, else_ = torch.zeros_like(y), torch.zeros_like(lse)
    vals, errs = [y, lse], [ey, else_]
    if dy is not None:
        dy = dy.double()
        dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
        edq, edk, edv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
        vals += [dq, dk, dv]
        errs += [edq, edk, edv]
    ad = acc(dim)
    a, b = lens[0], keys[0]
    for n, m in zip(lens[1:], keys[1:]):
        for h in range(hq if n and m else 0):
            Q, K, V = q[a:a + n, h], k[b:b + m, h // g], v[b:b + m, h // g]
            mask = torch.ones(n, m, dtype=torch.bool, device=q.device)
            mask = mask.tril(m - n) if causal else mask
            some = mask.any(1, keepdim=True)
            zero = torch.zeros((), dtype=torch.float64, device=q.device)
            S = torch.where(mask, scale * (Q @ K.T), -math.inf)
            top = torch.where(some, S.amax(1, keepdim=True), zero)
            big = torch.where(mask, S.abs(), zero).amax(1, keepdim=True)
            p = torch.where(mask, torch.exp(S - top), zero)
            l = torch.where(some, p.sum(1, keepdim=True), zero + 1)
            p = p / l
            L = torch.log(l) + top
            rel = torch.where(mask, scale * ad * (Q.abs() @ K.abs().T), zero) + 2 * E * big + 4 * E
            am = acc(m)
            rel_l = (p * rel).sum(1, keepdim=True) + am
            Y = p @ V
            size = p @ V.abs()
            e_part = rel_l + 2 * E * (L.abs() + big + 1)
            eY = u * Y.abs() + (p * (rel + up)) @ V.abs() + (am + rel_l + 2 * e_part + 4 * E) * size + 2.0 ** -120
            eL = 2 * e_part + 4 * E
            y[a:a + n, h], ey[a:a + n, h] = Y, eY
            lse[h, a:a + n], else_[h, a:a + n] = torch.where(some, L, -math.inf)[:, 0], torch.where(some, eL, zero)[:, 0]
            if dy is None:
                continue
            G = dy[a:a + n, h]
            dp, D = G @ V.T, (G * Y).sum(1, keepdim=True)
            e_d = (G.abs() * eY).sum(1, keepdim=True) + ad * (G * Y).abs().sum(1, keepdim=True)
            rel_p = rel + eL + 2 * E * (L.abs() + big + 1)
            ds = p * (dp - D)
            e_ds = p * (ad * (G.abs() @ V.abs().T) + e_d + 2 * E * (dp.abs() + D.abs())) + ds.abs() * (rel_p + up + 4 * E)
            e_p = p * (rel_p + up)
            dq[a:a + n, h] = scale * ds @ K
            edq[a:a + n, h] = scale * (e_ds @ K.abs() + am * (ds.abs() @ K.abs()))
            an = acc(n * g)
            dk[b:b + m, h // g] += scale * ds.T @ Q
            edk[b:b + m, h // g] += scale * (e_ds.T @ Q.abs() + an * (ds.abs().T @ Q.abs()))
            dv[b:b + m, h // g] += p.T @ G
            edv[b:b + m, h // g] += e_p.T @ G.abs() + an * (p.T @ G.abs())
        a, b = a + n, b + m
    for x, e in zip(vals[2:], errs[2:]):
        e += u * x.abs() + 2.0 ** -120
    return vals, [1.01 * e for e in errs]


def turns(positions, rot, sections, base, per_axis):
    """(angle, bound of the angle's error) of every token and pair, in 64 bits."""
    pos = positions.double().reshape(positions.shape[0], -1)
    parts, at = [], 0
    for axis, n in enumerate(sections):
        i = torch.arange(n, dtype=torch.float64, device=pos.device)
        f = base ** (-i / max(1, n)) if per_axis else base ** (-2 * (at + i) / max(1, rot))
        parts.append(pos[:, axis, None] * f)
        at += n
    angle = torch.cat(parts, 1)
    return angle, angle.abs() * 2.0 ** -50 + 2.0 ** -22


def rotate(x, c, s, rot, interleaved):
    z, rest = x[..., :rot], x[..., rot:]
    a, b = (z[..., 0::2], z[..., 1::2]) if interleaved else z.chunk(2, -1) if rot else (z, z)
    a, b = a * c - b * s, b * c + a * s
    z = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([z[..., :rot], rest], -1)


def norm_rope(x, w, positions, rot, sections, *, eps=1e-6, base=10000.0, per_axis=False, interleaved=False, dy=None):
    """(values, bounds) of y and, with dy, of dx and dw; x (tokens, heads, dim), w or None."""
    u = ROUNDOFF[x.dtype]
    x = x.double()
    dim = x.shape[-1]
    ang, e_ang = turns(positions, rot, sections, base, per_axis)
    c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
    one = torch.ones_like(c)
    def spread(t):
        """Of t >= 0: the pairs' sums in both places, the rest as it is."""
        z = t.clone()
        if rot:
            a, b = (t[..., 0:rot:2], t[..., 1:rot:2]) if interleaved else (t[..., :rot // 2], t[..., rot // 2:rot])
            q = torch.stack([a + b, a + b], -1).flatten(-2) if interleaved else torch.cat([a + b, a + b], -1)
            z[..., :rot] = q
        return z
    e_cs = torch.zeros_like(x[:, :1])
    if rot:
        e = e_ang[:, None] + 4 * E
        e_cs[..., :rot] = torch.stack([e, e], -1).flatten(-2) if interleaved else torch.cat([e, e], -1)
    if w is None:
        W, r, n, rel_r = 1.0, torch.ones_like(x[..., :1]), x, 0.0
    else:
        W = w.double()
        r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
        n, rel_r = x * r, 0.5 * acc(dim) + 4 * E
    y = rotate(n * W, c, s, rot, interleaved)
    size = spread((n * W).abs())
    vals, errs = [y], [u * y.abs() + size * (e_cs + rel_r + 4 * E)]
    if dy is not None:
        dy = dy.double()
        g = rotate(dy, c, -s, rot, interleaved)
        e_g = spread(dy.abs()) * (e_cs + 4 * E)
        if w is None:
            vals.append(g)
            errs.append(u * g.abs() + e_g)
        else:
            gw, e_gw = g * W, e_g * W.abs() + E * (g * W).abs()
            m = (gw * n).mean(-1, keepdim=True)
            e_m = acc(dim) * (gw * n).abs().mean(-1, keepdim=True) + ((e_gw + gw.abs() * (rel_r + E)) * n.abs()).mean(-1, keepdim=True)
            dx = r * (gw - n * m)
            vals.append(dx)
            errs.append(u * dx.abs() + r * (e_gw + n.abs() * e_m + (rel_r + 4 * E) * (gw.abs() + 2 * (n * m).abs())))
            dw = (g * n).sum((0, 1))
            e_dw = acc(x.shape[0] * x.shape[1]) * (g * n).abs().sum((0, 1)) + (e_g * n.abs() + (g * n).abs() * (rel_r + E)).sum((0, 1))
            vals.append(dw)
            errs.append(u * dw.abs() + e_dw)
    return vals, [1.01 * e + 2.0 ** -120 for e in errs]


def philox_words(counter, key):
    """Philox 4x32-10 in Python integers: the four words of a 64-bit counter and key."""
    c = [counter & 0xffffffff, counter >> 32 & 0xffffffff, 0, 0]
    k = [key & 0xffffffff, key >> 32 & 0xffffffff]
    for _ in range(10):
        a, b = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(b >> 32) ^ c[1] ^ k[0], b & 0xffffffff, (a >> 32) ^ c[3] ^ k[1], a & 0xffffffff]
        k = [(k[0] + 0x9E3779B9) & 0xffffffff, (k[1] + 0xBB67AE85) & 0xffffffff]
    return c


def keep(n, p, seed, offset):
    """Which of n elements dropout keeps (bool, on the host)."""
    cut = round(p * 65536)
    out = []
    for g in range((n + 7) // 8):
        for w in philox_words((offset + g) & (2 ** 64 - 1), seed & (2 ** 64 - 1)):
            out += [(w & 0xffff) >= cut, (w >> 16) >= cut]
    return torch.tensor(out[:n], dtype=torch.bool)


def dropout(x, kept, p, residual=None):
    """(value, bound) of dropout's result."""
    u = ROUNDOFF[x.dtype]
    cut = round(p * 65536)
    z = torch.where(kept.view(x.shape), x.double() * (65536 / max(1, 65536 - cut)), torch.zeros((), dtype=torch.float64, device=x.device))
    y = z if residual is None else z + residual.double()
    size = z.abs() + (0 if residual is None else residual.double().abs())
    return [y], [1.01 * (u * y.abs() + 4 * E * size) + 2.0 ** -140]
