"""float64 CPU oracle of the operators between an attention block's projections: the norm of each head
with the rotation by position, and causal attention over packed sequences, with their backward passes.
Plain and slow; shares no code with the CUDA path."""
from __future__ import annotations

import numpy as np


def rope_table(n_pos: int, inv_freq):
    a = np.arange(n_pos, dtype=np.float64)[:, None] * np.asarray(inv_freq, np.float64)[None]
    return np.stack([np.cos(a), np.sin(a)], axis=-1)


def _pairs(dim: int, pairs: bool):
    """Indices of the first and the second elements of the pairs."""
    i = np.arange(dim // 2)
    return (2 * i, 2 * i + 1) if pairs else (i, i + dim // 2)


def _turn(x, cs, pairs: bool, sign: float):
    a, b = _pairs(x.shape[-1], pairs)
    c, s = cs[:, None, :, 0], sign * cs[:, None, :, 1]
    y = np.empty_like(x)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., a] * s + x[..., b] * c
    return y


def rope_forward(x, gamma, cs, eps: float, pairs: bool):
    """x [T, heads, dim], cs [T, dim / 2, 2] the tokens' rows of the table."""
    x = np.asarray(x, np.float64)
    if gamma is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(gamma, np.float64)
    return _turn(x, np.asarray(cs, np.float64), pairs, 1.0)


def rope_backward(x, gamma, cs, dy, eps: float, pairs: bool):
    """(dx, dgamma); dgamma None without a weight."""
    h = _turn(np.asarray(dy, np.float64), np.asarray(cs, np.float64), pairs, -1.0)
    if gamma is None:
        return h, None
    x = np.asarray(x, np.float64)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    xhat = x * r
    g = h * np.asarray(gamma, np.float64)
    return r * (g - xhat * (g * xhat).mean(-1, keepdims=True)), (h * xhat).sum((0, 1))


def attention_forward(q, k, v, starts, scale: float):
    """(o, lse [heads, T]) of q [T, heads, dim] and k, v [T, kv heads, dim]; rows of no sequence are NaN."""
    q, k, v = (np.asarray(a, np.float64) for a in (q, k, v))
    T, H, _ = q.shape
    per = H // k.shape[1]
    o, lse = np.full_like(q, np.nan), np.full((H, T), np.nan)
    for a, b in zip(starts, starts[1:]):
        for h in range(H):
            s = scale * q[a:b, h] @ k[a:b, h // per].T
            s[np.triu_indices(b - a, 1)] = -np.inf
            if b == a:
                continue
            top = s.max(1, keepdims=True)
            p = np.exp(s - top)
            z = p.sum(1, keepdims=True)
            o[a:b, h] = (p / z) @ v[a:b, h // per]
            lse[h, a:b] = (top + np.log(z))[:, 0]
    return o, lse


def attention_backward(q, k, v, o, lse, do, starts, scale: float):
    """(dq, dk, dv) from the forward's inputs, its output and log sums; zeros in rows of no sequence."""
    q, k, v, o, do = (np.asarray(a, np.float64) for a in (q, k, v, o, do))
    H, per = q.shape[1], q.shape[1] // k.shape[1]
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    for a, b in zip(starts, starts[1:]):
        for h in range(H):
            g = h // per
            s = scale * q[a:b, h] @ k[a:b, g].T
            s[np.triu_indices(b - a, 1)] = -np.inf
            p = np.exp(s - lse[h, a:b, None])
            dv[a:b, g] += p.T @ do[a:b, h]
            delta = (do[a:b, h] * o[a:b, h]).sum(1, keepdims=True)
            ds = p * (do[a:b, h] @ v[a:b, g].T - delta) * scale
            dq[a:b, h] = ds @ k[a:b, g]
            dk[a:b, g] += ds.T @ q[a:b, h]
    return dq, dk, dv


def attention_bounds(q, k, v, o, lse, do, starts, scale: float, backward: bool):
    """How far each output may be off the exact value, element by element, beyond its own rounding.

    A score is a sum of dim products in fp32, each addition off by at most 2^-23 of the sum of their sizes:
    e_s = dim 2^-23 scale sum |q k|. P = exp(S - lse) is off by a factor e_s, by the rounding of the
    exponent's argument (2^-22 of |S| and |lse|) and of the exponential (2^-21): e_p in all; as an operand it
    is rounded to bf16, 2^-8. Sums of n such terms in fp32 add n 2^-23, at most 2^-10 here (n <= 8192).
    dS = P (dP - delta) carries P's factor, the roundings of dP and delta (dim 2^-23 of their terms' sizes)
    and its own to bf16. The exponential gives 0 below the smallest normal number, 2^-126: P may be off by
    that much besides, and dS by that times |dP - delta|; with the subnormal roundings of the two operands
    (2^-134) and products with at least as small a term, `tiny` = 2^-125 of the other factors holds it."""
    tiny = 2.0 ** -125
    q, k, v, o, do = (np.asarray(a, np.float64) for a in (q, k, v, o, do))
    H, per, dim = q.shape[1], q.shape[1] // k.shape[1], q.shape[2]
    u = dim * 2.0 ** -23
    outs = [np.zeros_like(q), np.zeros((H, q.shape[0]))] if not backward else \
        [np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)]
    for a, b in zip(starts, starts[1:]):
        for h in range(H):
            g = h // per
            s = scale * q[a:b, h] @ k[a:b, g].T
            size = scale * np.abs(q[a:b, h]) @ np.abs(k[a:b, g]).T
            late = np.triu_indices(b - a, 1)
            s[late], size[late] = -np.inf, 0.0
            if b == a:
                continue
            p = np.exp(s - lse[h, a:b, None])
            e_s = u * size
            e_p = e_s + 2.0 ** -22 * (np.abs(np.where(p > 0, s, 0.0)) + np.abs(lse[h, a:b, None])) + 2.0 ** -21
            n = (b - a) * 2.0 ** -23
            if not backward:
                # the sum of P is off by the mean of e_p at most; the running reference rescales both alike
                mean = (p * e_p).sum(1, keepdims=True)
                outs[0][a:b, h] = (p * (e_p + mean + 2.0 ** -8 + 2 * n) + tiny) @ np.abs(v[a:b, g])
                outs[1][h, a:b] = mean[:, 0] + n + 2.0 ** -21 * (1 + np.abs(lse[h, a:b]))
                continue
            outs[2][a:b, g] += (p * (e_p + 2.0 ** -8 + n) + tiny).T @ np.abs(do[a:b, h])
            ad, av = np.abs(do[a:b, h]), np.abs(v[a:b, g])
            delta = (do[a:b, h] * o[a:b, h]).sum(1, keepdims=True)
            dp = np.abs(do[a:b, h] @ v[a:b, g].T - delta)
            e_ds = p * dp * (e_p + 2.0 ** -8 + n) + tiny * (1 + dp)
            e_ds += p * u * (ad @ av.T + (ad * np.abs(o[a:b, h])).sum(1, keepdims=True)) * 1.01
            outs[0][a:b, h] = scale * e_ds @ np.abs(k[a:b, g])
            outs[1][a:b, g] += scale * e_ds.T @ np.abs(q[a:b, h])
    return outs
