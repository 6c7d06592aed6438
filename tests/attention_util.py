"""Caches, comparison rules and tolerances of the full-attention layers' GPU tests.

Rotary positions: a result is m (u c - w s) with c and s off by at most 5 u (u = 2^-24): two roundings of the
angle (at most pi / 4, so 1.6 u), the polynomial's own (1.5 u), its last step and the product with m (1 u
each); and two roundings of its own: 8 u m (|u| + |w|) in all.

Attention: with weights p_j off by a relative d_j and outputs o = sum p v / sum p, the error is at most
2 max d * mean, mean = sum p |v| / sum p.  d is the score's error (D + 4 roundings of partial sums of
|q_d k_d| scale, at most size each: (D + 4) u size), the exponential's (2 u), one for each addition into the
running sums and each rescaling of them (at most two for each of L keys: 2 L u).  bf16 weights are off by
2^-8 more in the numerator (half a step, torch.finfo(bfloat16).eps / 2).  Scales of 8-bit rows add two
roundings.  Outputs' own rounding: half a step of their type.
"""
import numpy as np
import torch

from oracle import attention as O

DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
E4M3 = torch.float8_e4m3fn
U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def f64(t):
    return t.detach().float().cpu().double().numpy()


def within(name, got, ref, bound):
    """|got - ref| <= bound + half a step of got's type, elementwise; equal where ref is not finite."""
    g, ref, bound = f64(got), np.asarray(ref), np.asarray(bound)
    fin = np.isfinite(ref)
    assert g.shape == ref.shape, (name, g.shape, ref.shape)
    assert np.array_equal(g[~fin], ref[~fin], equal_nan=True), "%s: values that are not finite differ" % name
    bound = np.broadcast_to(bound, ref.shape)[fin]
    err = np.abs(g[fin] - ref[fin])
    limit = bound + HALF[got.dtype] * (np.abs(ref[fin]) + bound)
    worst = float((err / np.maximum(limit, 1e-300)).max()) if err.size else 0.0
    print("  %-4s error at most %.3f of its bound" % (name, worst), flush=True)
    assert worst <= 1.0, "%s: error %.3f of its bound" % (name, worst)


def quantised(x):
    """(e4m3 values, scales) of rows x [.., D] in fp32, the definition's steps in torch on the CPU."""
    x = x.float()
    scale = x.abs().amax(-1).clamp(min=1e-12) / 448
    return (x / scale[..., None]).clamp(-448, 448).to(E4M3), scale


class Cache:
    """A cache of random rows on the GPU; `values`: what its rows stand for (fp64, [pages, H, P, D])."""

    def __init__(self, g, pages, H, P, D, kind, dtype=torch.bfloat16, fill=None):
        self.kind, self.P = kind, P
        self.shape = (pages, H, P, D)
        self.t, self.s, self.values = {}, {}, {}
        for n in "kv":
            x = torch.randn(*self.shape, generator=g) if fill is None else torch.full(self.shape, fill)
            self.put(n, x, dtype)

    def put(self, n, x, dtype):
        if self.kind == "e4m3":
            q, s = quantised(x)
            self.t[n], self.s[n] = q.to(DEV), s.to(DEV)
            self.values[n] = q.float().double().numpy() * s.double().numpy()[..., None]
        else:
            x = x.to(dtype)
            self.t[n], self.s[n] = x.to(DEV), None
            self.values[n] = x.double().numpy()

    def args(self):
        return self.t["k"], self.t["v"]

    def scales(self):
        return {} if self.kind != "e4m3" else {"k_scale": self.s["k"], "v_scale": self.s["v"]}


def pages_of(g, pages, lens, P, extra=0):
    """A table of pages, taken from all over the cache, for sequences of these lengths (-7 behind them)."""
    need = [-(-n // P) for n in lens]
    assert sum(need) <= pages
    order = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.full((len(lens), max(1, max(need)) + extra), -7, dtype=torch.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    return table


def reference(q, cache, table, lens, new, scale, causal=True, window=0):
    """The oracle over packed queries q [T, Hq, D]: o, lse, and the bounds of both."""
    T, Hq, D = q.shape
    qn = f64(q)
    o, lse, bound, lbound = np.zeros((T, Hq, D)), np.zeros((T, Hq)), np.zeros((T, Hq, D)), np.zeros((T, Hq))
    t0 = 0
    for i, (n, L) in enumerate(zip(new, lens)):
        k, v = (O.rows_of(cache.values[c], table[i].tolist(), L) for c in "kv")
        a, b, mean, size = O.attention(qn[t0:t0 + n], k, v, n, scale, causal, window)
        d = (D + 4) * U * size + (4 + 2 * L) * U
        o[t0:t0 + n], lse[t0:t0 + n] = a, b
        bound[t0:t0 + n] = (2 * d[..., None] + (2.0 ** -8 if q.dtype == torch.bfloat16 else 0.0)) * mean
        # the log of a sum off by d, and the roundings of the maximum and the result
        lbound[t0:t0 + n] = d + 4 * U * (size + np.where(np.isfinite(b), np.abs(b), 0.0) + 1)
        t0 += n
    return o, lse, bound, lbound
