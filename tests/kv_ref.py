"""Plain 64-bit forms of the attention layer's operators, the cache's bytes read
by the header's words, and the error a right kernel may make, for the tests of
the norm, rotation, cache and attention calls.

Error model.  Norm and rotation of queries and keys run in binary32: each of
square, sum, root, quotient, the two products with the weight and the two
products and the sum of the rotation is within 2^-24 of its result (the sum of
128 squares within 16 * 2^-24, positive terms), and the rotated value is a sum
of two products: (24 * 2^-24) * (|a cos| + |b sin|), then the store's rounding.
What goes into the cache runs in 64 bits, so its codes are those of the 64-bit
form wherever that is more than 1e-9 from a border.

Attention.  Operands are fp16 at worst: a key or value read from the cache may be
rounded once (2^-11 relative, half a subnormal step 2^-25 below 2^-14), a
probability once (relative to the largest of the row, 2^-11 and 2^-25); queries
are exact (bfloat16 ones scaled by a power of two lose at most 2^-25 of the
row's largest).  Sums of binary32 products in any order are within terms * 2^-23
of the sum of their magnitudes.  So a logit is off by
    d = scale * (sum |q||k| * (2^-11 + D * 2^-23) + sum |q| * 2^-25 + max|q| * 2^-25 * sum |k|)
plus 2^-22 of its magnitude from the scale and the exponent's argument (relative to
the row's largest, which is as far off), a probability by exp(2d) - 1, and the output by
that, the two roundings and 2^-23 for each key times sum p |v|, plus 2^-25 for each key
times the largest |v| over the sum of probabilities (at least 1), plus the store's rounding.
"""
from __future__ import annotations

import math

import numpy as np
import torch

U32 = 2.0 ** -24
HALF = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
SUB = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -150}


def store_err(y, d, dtype):
    return d + HALF[dtype] * (y.abs() + d) + SUB[dtype]


def turn64(x, weight, rope, positions, eps, interleaved):
    """x [T, H, D] normed and rotated, and the sum of magnitudes of its terms."""
    x = x.double().cpu()
    T, H, D = x.shape
    if eps is not None:
        x = x / torch.sqrt((x ** 2).mean(-1, keepdim=True) + eps)
        if weight is not None:
            x = x * weight.double().cpu()
    y, mag = x.clone(), x.abs()
    if rope is not None:
        table, pos = rope.double().cpu(), positions.cpu().tolist()
        rot = table.shape[1]
        for t in range(T):
            if not 0 <= pos[t] < table.shape[0]:
                y[t] = 0
                mag[t] = 0
                continue
            for i in range(rot // 2):
                a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
                c, s = table[pos[t], i], table[pos[t], rot // 2 + i]
                y[t, :, a] = x[t, :, a] * c - x[t, :, b] * s
                y[t, :, b] = x[t, :, b] * c + x[t, :, a] * s
                mag[t, :, a] = (x[t, :, a] * c).abs() + (x[t, :, b] * s).abs()
                mag[t, :, b] = (x[t, :, b] * c).abs() + (x[t, :, a] * s).abs()
    return y, mag


def quantize64(x):
    """x [..., D] (float64) -> codes, scales, minima (numpy), and how far each code is from a border."""
    g = x.double().cpu().numpy().reshape(*x.shape[:-1], -1, 32)
    g = np.clip(np.where(np.isnan(g), 0.0, g), -32768.0, 32768.0)
    m = g.min(-1).astype(np.float32).astype(np.float16)
    s = ((g.max(-1) - m.astype(np.float64)) / 15.0).astype(np.float32).astype(np.float16)
    sd = np.where(s > 0, s.astype(np.float64), 1.0)[..., None]
    t = np.where(s[..., None] > 0, (g - m.astype(np.float64)[..., None]) / sd, 0.0)
    c = np.clip(np.rint(t), 0, 15)
    edge = np.abs(np.abs(t - np.floor(t)) - 0.5)
    return c.reshape(x.shape).astype(np.uint8), s, m, edge.reshape(x.shape)


def held64(x):
    """What the cache holds of x [..., D]."""
    c, s, m, _ = quantize64(x)
    s, m = np.repeat(s.astype(np.float64), 32, -1), np.repeat(m.astype(np.float64), 32, -1)
    return torch.from_numpy(c * s + m)


def token_fields(cache, page_id, H, page, D, place, head):
    """(key codes, key scales, key minima, value codes, value scales, value minima) of one token's
    head, from the cache's bytes (numpy [pages][bytes]) by the header's description."""
    tile = cache[page_id].reshape(H, page // 16, 20 * D)[head, place % page // 16]
    r, E = place % 16, D // 16
    kc, vc = np.zeros(D, np.uint8), np.zeros(D, np.uint8)
    for d in range(D):
        h, x = d // (D // 4), d % (D // 4)
        at = (16 * h + r) * (D // 8) + 4 * (x // 8)
        w = int.from_bytes(bytes(tile[at:at + 4]), "little")
        kc[d] = (w >> (4 * (x % 8 // 2) + 16 * (x % 2))) & 15
        n, e, i = d // E, d % E, r % 4
        at = 10 * D + (16 * (r // 4) + n) * (D // 8) + 4 * (e // 2)
        w = int.from_bytes(bytes(tile[at:at + 4]), "little")
        vc[d] = (w >> (4 * (2 * (e % 2) + i // 2) + 16 * (i % 2))) & 15

    def heads(base):
        f = np.frombuffer(bytes(tile[base:base + 2 * D]), np.float16).reshape(D // 32, 16, 2)
        return f[:, r, 0], f[:, r, 1]

    return (kc, *heads(8 * D), vc, *heads(18 * D))


def attention64(q, k, v, places, scale, window, dtype):
    """One sequence: q [n, heads, D], k and v [L, H, D] (float64, as the cache holds them), places
    [n].  (outputs [n, heads, D], their error bound)."""
    q, k, v = q.double().cpu(), k.double().cpu(), v.double().cpu()
    n, heads, D = q.shape
    L, H = k.shape[:2]
    y, e = torch.zeros_like(q), torch.zeros_like(q)
    for i in range(n):
        p = places[i]
        lo = max(0, p - window + 1) if window else 0
        if p < 0 or lo > p or L == 0:
            e[i] = 0
            continue
        for h in range(heads):
            j = h // (heads // H)
            kk, vv, qq = k[lo:p + 1, j], v[lo:p + 1, j], q[i, h]
            x = scale * (kk @ qq)
            mag = kk.abs() @ qq.abs()
            d = (abs(scale) * (mag * (2.0 ** -11 + D * 2.0 ** -23) + qq.abs().sum() * 2.0 ** -25
                               + qq.abs().max() * 2.0 ** -25 * kk.abs().sum(1)) + x.abs() * 2.0 ** -22).max()
            w = torch.exp(x - x.max())
            pr = w / w.sum()
            y[i, h] = pr @ vv
            rel = math.expm1(min(2 * float(d) + 2.0 ** -21, 50.0)) + 2 * 2.0 ** -11 + kk.shape[0] * 2.0 ** -23
            e[i, h] = rel * (pr @ vv.abs()) + kk.shape[0] * 2.0 ** -25 * vv.abs().max() / w.sum() + 2.0 ** -25
    return y, store_err(y, e, dtype)
