"""fp64 oracle of the layer operators (short causal convolution, selective scan, residual RMS norm)
and their gradients: plain numpy, token by token, from the definitions.  Sequences are given by
their lengths; every tensor is [tokens, ..] with the sequences' tokens in order.  Arguments and results
are float64 arrays; None stands for an absent input."""
from __future__ import annotations

import numpy as np


def _f(x):
    return None if x is None else np.asarray(x, np.float64)


def sigmoid(x):
    return 0.5 * (1.0 + np.tanh(0.5 * x))


def softplus(x):
    return np.logaddexp(0.0, x)


def _bounds(lens):
    ends = np.cumsum(lens)
    return [(int(e - n), int(e)) for n, e in zip(lens, ends)]


def conv(lens, x, w, bias=None, init=None, silu=True):
    """(y [T,D], last [n,W-1,D])."""
    x, w, bias, init = _f(x), _f(w), _f(bias), _f(init)
    (_, D), W = x.shape, w.shape[1]
    y, last = np.zeros_like(x), np.zeros((len(lens), W - 1, D))
    for i, (a, b) in enumerate(_bounds(lens)):
        line = np.concatenate([np.zeros((W - 1, D)) if init is None else init[i], x[a:b]])
        for t in range(b - a):
            u = (line[t:t + W] * w.T).sum(0) + (0.0 if bias is None else bias)
            y[a + t] = u * sigmoid(u) if silu else u
        last[i] = line[b - a:]
    return y, last


def conv_bwd(lens, dy, x, w, bias=None, init=None, dlast=None, silu=True):
    """dict(dx, dw, dbias, dinit)."""
    dy, x, w, bias, init, dlast = (_f(v) for v in (dy, x, w, bias, init, dlast))
    (_, D), W = x.shape, w.shape[1]
    dx, dw, db = np.zeros_like(x), np.zeros_like(w), np.zeros(D)
    dinit = np.zeros((len(lens), W - 1, D))
    for i, (a, b) in enumerate(_bounds(lens)):
        line = np.concatenate([np.zeros((W - 1, D)) if init is None else init[i], x[a:b]])
        dl = np.zeros_like(line)
        if dlast is not None:
            dl[b - a:] += dlast[i]
        for t in range(b - a):
            u = (line[t:t + W] * w.T).sum(0) + (0.0 if bias is None else bias)
            s = sigmoid(u)
            du = dy[a + t] * (s + u * s * (1.0 - s) if silu else 1.0)
            dl[t:t + W] += w.T * du
            dw += (line[t:t + W] * du).T
            db += du
        dinit[i], dx[a:b] = dl[:W - 1], dl[W - 1:]
    return dict(dx=dx, dw=dw, dbias=db, dinit=dinit)


def scan(lens, x, dt, A, Bm, Cm, skip=None, z=None, dt_bias=None, h0=None, use_softplus=True, chunk=None):
    """(y [T,D], ht [n,D,N], h): h the states entering each chunk of `chunk` tokens of each sequence,
    in order, where chunk is given."""
    x, dt, A, Bm, Cm, skip, z, dt_bias, h0 = (_f(v) for v in (x, dt, A, Bm, Cm, skip, z, dt_bias, h0))
    (T, D), N = x.shape, A.shape[1]
    raw = dt + (0.0 if dt_bias is None else dt_bias)
    de = softplus(raw) if use_softplus else raw
    y, ht, saved = np.zeros_like(x), np.zeros((len(lens), D, N)), []
    for i, (a, b) in enumerate(_bounds(lens)):
        h = np.zeros((D, N)) if h0 is None else h0[i].copy()
        for t in range(a, b):
            if chunk and (t - a) % chunk == 0:
                saved.append(h.copy())
            h = np.exp(de[t][:, None] * A) * h + (de[t] * x[t])[:, None] * Bm[t]
            y[t] = h @ Cm[t] + (0.0 if skip is None else skip * x[t])
        ht[i] = h
    if z is not None:
        y = y * z * sigmoid(z)
    return y, ht, np.array(saved) if chunk else None


def scan_bwd(lens, dy, x, dt, A, Bm, Cm, skip=None, z=None, dt_bias=None, h0=None, dht=None, use_softplus=True):
    """dict(dx, ddt, dA, dB, dC, dD, dz, ddt_bias, dh0)."""
    dy, x, dt, A, Bm, Cm, skip, z, dt_bias, h0, dht = (
        _f(v) for v in (dy, x, dt, A, Bm, Cm, skip, z, dt_bias, h0, dht))
    (T, D), N = x.shape, A.shape[1]
    raw = dt + (0.0 if dt_bias is None else dt_bias)
    de = softplus(raw) if use_softplus else raw
    sk = np.zeros(D) if skip is None else skip
    o = dict(dx=np.zeros_like(x), ddt=np.zeros_like(x), dA=np.zeros_like(A), dB=np.zeros_like(Bm),
             dC=np.zeros_like(Cm), dD=np.zeros(D), dz=np.zeros_like(x), dh0=np.zeros((len(lens), D, N)))
    for i, (a, b) in enumerate(_bounds(lens)):
        states = [np.zeros((D, N)) if h0 is None else h0[i]]
        for t in range(a, b):
            states.append(np.exp(de[t][:, None] * A) * states[-1] + (de[t] * x[t])[:, None] * Bm[t])
        g = np.zeros((D, N)) if dht is None else dht[i].copy()
        for t in reversed(range(a, b)):
            h, prev = states[t - a + 1], states[t - a]
            gy = dy[t]
            if z is not None:
                s = sigmoid(z[t])
                o["dz"][t] = dy[t] * (h @ Cm[t] + sk * x[t]) * (s + z[t] * s * (1.0 - s))
                gy = dy[t] * z[t] * s
            g = g + gy[:, None] * Cm[t]
            o["dC"][t] = gy @ h
            o["dB"][t] = (de[t] * x[t]) @ g
            gb = g @ Bm[t]
            o["dx"][t] = de[t] * gb + sk * gy
            o["dD"] += gy * x[t]
            e = np.exp(de[t][:, None] * A)
            o["ddt"][t] = x[t] * gb + (g * e * prev * A).sum(1)
            o["dA"] += g * e * prev * de[t][:, None]
            g = g * e
        o["dh0"][i] = g
    if use_softplus:
        o["ddt"] = o["ddt"] * sigmoid(raw)
    o["ddt_bias"] = o["ddt"].sum(0)
    return o


def norm(s, w, eps):
    """(y, rstd) of the rows of s."""
    s, w = _f(s), _f(w)
    rstd = 1.0 / np.sqrt((s * s).mean(-1) + eps)
    return s * rstd[:, None] * w, rstd


def norm_scales(y, block):
    """8-bit scales of the rows of y: one a row (block 0) or one for each `block` columns."""
    y = _f(y)
    parts = [y] if not block else [y[:, c:c + block] for c in range(0, y.shape[1], block)]
    return np.stack([np.maximum(np.abs(p).max(-1), 1e-12) / 448.0 for p in parts], 1)


def norm_bwd(dy, s, w, eps, dsum=None):
    """dict(ds, dw)."""
    dy, s, w, dsum = _f(dy), _f(s), _f(w), _f(dsum)
    rstd = norm(s, w, eps)[1][:, None]
    gw = dy * w
    ds = rstd * (gw - s * rstd ** 2 * (gw * s).mean(-1, keepdims=True))
    return dict(ds=ds if dsum is None else ds + dsum, dw=(dy * s * rstd).sum(0))
