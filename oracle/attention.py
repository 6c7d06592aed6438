"""fp64 oracle of the full-attention layers' operators (rotary positions, paged cache, attention): plain
numpy and exact rationals, token by token, from the definitions.  Arguments and results are float64 arrays but
where said."""
from __future__ import annotations

import math
from fractions import Fraction

import numpy as np

TURN = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494")


def cos_sin(position, freq):
    """Cosine and sine of position * freq radians: whole turns are taken out in exact arithmetic."""
    turn = (Fraction(int(position)) * Fraction(float(freq)) / TURN) % 1
    a = 2.0 * math.pi * float(turn)
    return math.cos(a), math.sin(a)


def rope(x, positions, freqs, interleaved=False, magnitude=1.0, back=False):
    """x [T, H, D], positions [T], freqs [R / 2]."""
    y = np.array(x, np.float64)
    half = len(freqs)
    for t in range(y.shape[0]):
        for i, f in enumerate(freqs):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            c, s = cos_sin(positions[t], f)
            s = -s if back else s
            u, w = np.array(x[t, :, a], np.float64), np.array(x[t, :, b], np.float64)
            y[t, :, a], y[t, :, b] = magnitude * (u * c - w * s), magnitude * (u * s + w * c)
    return y


def rows_of(cache, table, n):
    """The n rows [n, H, D] that a sequence with these pages has in a cache [pages, H, P, D]; a page outside the
    cache is rows of 0."""
    pages, H, P, D = cache.shape
    out = np.zeros((n, H, D))
    for j in range(n):
        page = int(table[j // P])
        if 0 <= page < pages:
            out[j] = cache[page, :, j % P]
    return out


def attention(q, k, v, n, scale, causal=True, window=0):
    """One sequence: q [n, Hq, D] new tokens, k and v [L, Hk, D].  Returns o [n, Hq, D], lse [n, Hq], and for
    error bounds: mean [n, Hq, D] (the weighted mean of |v|) and size [n, Hq] (the largest sum of |q_d k_d| over the
    keys seen, times scale)."""
    Hq, D = q.shape[1:]
    L, Hk = k.shape[:2]
    G = Hq // Hk
    o, mean = np.zeros((n, Hq, D)), np.zeros((n, Hq, D))
    lse, size = np.full((n, Hq), -np.inf), np.zeros((n, Hq))
    for t in range(n):
        at = L - n + t
        seen = np.arange(L) if not causal else np.arange(max(0, at - window + 1) if window else 0, at + 1)
        if len(seen) == 0:
            continue
        for h in range(Hq):
            kk, vv = k[seen, h // G], v[seen, h // G]
            z = scale * (kk @ q[t, h])
            top = z.max()
            p = np.exp(z - top)
            s = p.sum()
            o[t, h], mean[t, h] = p @ vv / s, p @ np.abs(vv) / s
            lse[t, h] = top + np.log(s)
            size[t, h] = scale * (np.abs(kk) @ np.abs(q[t, h])).max()
    return o, lse, mean, size
