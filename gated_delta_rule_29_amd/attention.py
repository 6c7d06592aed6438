"""Operators of the full-attention layers that stand between recurrent ones: rotary positions with their
gradient, the paged cache of keys and values (8-bit or not) as it is written and read back, and the attention
of new tokens over it, for chunks and for single tokens.

As everywhere in the binding, arguments are marshalled and shapes checked here; every step of the
method runs in the library.  Head inputs [.., H, D] may be columns of a wider tensor or a heads-first layout:
a head's columns have to be dense, tokens and heads evenly spaced.  Everything else is contiguous.  Calls run on
the inputs' device, on its current stream.
"""
from __future__ import annotations

import math
from fractions import Fraction

import torch

from . import _lib
from .layer import _CPU, _DT, _INT, F32, _act, _call, _int32, _large, _like, _need, _refuse, _workspace

__all__ = ["rope_freqs", "rope_table", "rope_fwd", "rope_bwd", "kv_cache_write", "kv_cache_read", "paged_attn_fwd",
           "paged_attn_fwd_varlen", "paged_attn_step"]

E4M3 = torch.float8_e4m3fn
I32 = torch.int32


def _heads(t, name, shape, dtype, dev):
    """(pitch, head pitch) of a head tensor [.., H, D]: elements from token to token and from head to head."""
    if not (isinstance(t, torch.Tensor) and t.shape == shape and t.dtype is dtype and t.device == dev):
        _refuse(t, name, shape, dtype, dev, None)
    H, D = shape[-2:]
    if t.is_contiguous():
        return H * D, D
    strides = t.stride()
    head = strides[-2] if H > 1 else D
    pitch, span = None, None  # of the innermost token dimension with more than one token; tokens so far
    for n, s in zip(reversed(shape[:-2]), reversed(strides[:-2])):
        if n == 1:
            continue
        if pitch is None:
            pitch, span = s, n
        elif s != pitch * span:
            raise ValueError("%s must have evenly spaced tokens (strides %s of shape %s)"
                             % (name, tuple(strides), tuple(shape)))
        else:
            span *= n
    if pitch is None:
        pitch = D
    if (strides[-1] != 1 and D != 1) or pitch < D or head < D:
        raise ValueError("%s must have dense heads that do not overlap (strides %s of shape %s)"
                         % (name, tuple(strides), tuple(shape)))
    return pitch, head


# -------------------------------------------------------------------------------- rotary positions

def rope_freqs(R, theta=10000.0, *, scaling=None, factor=1.0, original=4096, fast=32.0, slow=1.0):
    """Angles a position of R / 2 pairs, ``theta ** (-2 i / R)`` radians, and the factor on the turned values
    (1 but for "yarn"): (fp64 tensor [R / 2] on the host, magnitude), for rope_table and rope_fwd.

    scaling, for contexts `factor` times the `original` one: "linear" divides all angles by the factor; "ntk"
    takes the base ``theta * factor ** (R / (R - 2))``; "yarn" divides the angles of pairs that turn less than
    `slow` times within the original context, keeps those of pairs that turn more than `fast` times, goes
    from one to the other linearly in the pair's number, and has magnitude ``1 + 0.1 log(factor)``."""
    if not isinstance(R, int) or R < 2 or R % 2:
        raise ValueError("R must be a positive even number, got %r" % (R,))
    if not (theta > 1.0 and math.isfinite(theta)) or not (factor >= 1.0 and math.isfinite(factor)):
        raise ValueError("theta must be above 1 and factor at least 1, got %r and %r" % (theta, factor))
    i = torch.arange(R // 2, dtype=torch.float64)
    f = float(theta) ** (-2.0 * i / R)
    if scaling is None:
        return f, 1.0
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "ntk":
        return ((theta * factor ** (R / (R - 2))) ** (-2.0 * i / R) if R > 2 else f), 1.0
    if scaling == "yarn":
        if not (original > 0 and fast > slow > 0):
            raise ValueError("original, fast and slow must be positive and fast above slow")

        def pair(turns):  # the (fractional) pair that turns so often within the original context
            return R * math.log(original / (2.0 * math.pi * turns)) / (2.0 * math.log(theta))

        lo, hi = max(math.floor(pair(fast)), 0), min(math.ceil(pair(slow)), R - 1)
        share = ((i - lo) / max(hi - lo, 1e-3)).clamp(0.0, 1.0)  # of the divided angle
        return f * (1.0 - share) + f / factor * share, 1.0 + 0.1 * math.log(factor)
    raise ValueError('scaling must be None, "linear", "ntk" or "yarn", got %r' % (scaling,))


_TURN = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494")


def rope_table(freqs, device):
    """What rope_fwd takes: the angles a position `freqs` [R / 2] (radians) as int64 [R / 2] on the device,
    64-bit fractions of a turn.  (The angle of a position is then the low 64 bits of a product of integers:
    whole turns drop out, and far positions are as exact as near ones.)"""
    if not isinstance(freqs, torch.Tensor) or freqs.dim() != 1 or not freqs.is_floating_point() or not len(freqs):
        raise ValueError("freqs must be a floating-point tensor [R / 2]")
    if not bool(torch.isfinite(freqs).all()):
        raise ValueError("freqs must be finite")
    out = []
    for f in freqs.detach().to("cpu", torch.float64).tolist():
        n = round(Fraction(f) / _TURN * (1 << 64)) % (1 << 64)
        out.append(n - (1 << 64) if n >> 63 else n)
    return torch.tensor(out, dtype=torch.int64).to(device)


def _rope(name, what, x, positions, table, interleaved, magnitude):
    if not isinstance(x, torch.Tensor) or x.dim() < 2:
        raise ValueError("%s must be a tensor [.., H, D]" % what)
    dev, dt, code = _act(x, what, x.dim())
    shape = x.shape
    H, D = shape[-2:]
    T = x.numel() // max(H * D, 1)
    if T > _INT or H > _INT or D > _INT:
        _large(T, H, D)
    if not isinstance(table, torch.Tensor) or table.dim() != 1:
        raise ValueError("table must be a tensor [R / 2] (rope_table)")
    half = table.shape[0]
    if half > _INT // 2:
        _large(half)
    pitch, head = _heads(x, what, shape, dt, dev)
    pp = _need(positions, "positions", shape[:-2], I32, dev)
    tp = _need(table, "table", (half,), torch.int64, dev)
    y = _like(x)
    _call(name, dev, x.data_ptr(), pitch, head, pp, tp, magnitude, y.data_ptr(), T, H, D, 2 * half,
          1 if interleaved else 0, code)
    return y


def rope_fwd(x, positions, table, *, interleaved=False, magnitude=1.0):
    """Rotary positions: pair i of each head's first R columns, (u, w), becomes
    ``magnitude * (u cos a - w sin a, u sin a + w cos a)`` with a = position * freqs[i]; the columns behind pass.

    x [..,H,D] (fp32 or bf16; queries and keys together in one call, as the columns of a projection),
    positions [..] int32 (a position for each token), table [R/2] of rope_table(freqs).  Pairs are columns
    (i, i + R/2), or (2i, 2i + 1) with interleaved.  Returns y [..,H,D]."""
    return _rope("rope_fwd", "x", x, positions, table, interleaved, magnitude)


def rope_bwd(dy, positions, table, *, interleaved=False, magnitude=1.0):
    """Gradient of rope_fwd: dx [..,H,D] from dy [..,H,D]."""
    return _rope("rope_bwd", "dy", dy, positions, table, interleaved, magnitude)


# ------------------------------------------------------------------------------------------- cache

def _cache(k_cache, v_cache, k_scale, v_scale, dt, dev):
    """The cache's addresses and (pages, places, heads, columns, library dtype)."""
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4:
        raise ValueError("k_cache must be a tensor [pages, Hk, P, D]")
    shape = k_cache.shape
    pages, H, P, D = shape
    ct = k_cache.dtype
    if ct is not dt and ct is not E4M3:
        raise ValueError("the cache must be %s or torch.float8_e4m3fn, got %s" % (dt, ct))
    if pages > _INT or H > _INT or P > _INT or D > _INT:
        _large(pages, H, P, D)
    kp, vp = _need(k_cache, "k_cache", shape, ct, dev), _need(v_cache, "v_cache", shape, ct, dev)
    if v_cache is None:
        raise ValueError("v_cache is needed")
    ksp, vsp = _need(k_scale, "k_scale", shape[:3], F32, dev), _need(v_scale, "v_scale", shape[:3], F32, dev)
    return (kp, vp, ksp, vsp), (pages, P, H, D), _lib.DTYPE_E4M3 if ct is E4M3 else _DT[ct]


def kv_cache_write(k, v, k_cache, v_cache, slots, k_scale=None, v_scale=None):
    """Writes rows of keys and values into their places of a paged cache.

    k, v [..,H,D] (one type, fp32 or bf16), k_cache, v_cache [pages,H,P,D] of that type or
    torch.float8_e4m3fn with k_scale, v_scale [pages,H,P] fp32 (each row is then e4m3(x / scale) with
    ``scale = max(max |x|, 1e-12) / 448``), slots [..] int32: place slot % P of page slot / P.  A row whose slot is
    outside the cache (-1: a padded row) or is an earlier row's changes nothing."""
    if not isinstance(k, torch.Tensor) or k.dim() < 2:
        raise ValueError("k must be a tensor [.., H, D]")
    dev, dt, code = _act(k, "k", k.dim())
    ptrs, (pages, P, H, D), cc = _cache(k_cache, v_cache, k_scale, v_scale, dt, dev)
    shape = k.shape
    if shape[-2] != H or shape[-1] != D:
        raise ValueError("k has shape %s, expected [.., %d, %d]" % (tuple(shape), H, D))
    T = k.numel() // max(H * D, 1)
    if T > _INT:
        _large(T)
    kp, kh = _heads(k, "k", shape, dt, dev)
    vp, vh = _heads(v, "v", shape, dt, dev)
    sp = _need(slots, "slots", shape[:-2], I32, dev)
    _call("kv_cache_write", dev, k.data_ptr(), kp, kh, v.data_ptr(), vp, vh, sp, *ptrs, T, pages, P, H, D, code, cc)


def kv_cache_read(k_cache, v_cache, slots, k_scale=None, v_scale=None, *, dtype=None):
    """Reads rows of a paged cache back: k, v [..,H,D] at slots [..] (0 where a slot is outside the cache), in
    the cache's type, or in dtype (bf16 by default) from an 8-bit cache."""
    if not isinstance(k_cache, torch.Tensor):
        raise ValueError("k_cache must be a torch.Tensor")
    if dtype is None:
        dtype = torch.bfloat16 if k_cache.dtype is E4M3 else k_cache.dtype
    if dtype not in _DT:
        raise ValueError("dtype must be float32 or bfloat16, got %s" % dtype)
    dev = k_cache.device
    ptrs, (pages, P, H, D), cc = _cache(k_cache, v_cache, k_scale, v_scale, dtype, dev)
    if not isinstance(slots, torch.Tensor):
        raise ValueError("slots must be a torch.Tensor")
    sp = _need(slots, "slots", slots.shape, I32, dev)
    T = slots.numel()
    if T > _INT:
        _large(T)
    k, v = (torch.empty(*slots.shape, H, D, dtype=dtype, device=dev) for _ in range(2))
    _call("kv_cache_read", dev, *ptrs, sp, k.data_ptr(), v.data_ptr(), T, pages, P, H, D, _DT[dtype], cc)
    return {"k": k, "v": v}


# --------------------------------------------------------------------------------------- attention

def _window(n):
    """A window as the library's 32-bit integer: a larger one hides no more than the largest, nothing (ctypes would
    pass on its low bits)."""
    if n < 0:
        raise ValueError("window must not be negative, got %r" % (n,))
    return n if n <= _INT else _INT


def _attn_args(q, n, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, scale):
    """The arguments that the forms share: of n sequences, up to the scale; and the sizes."""
    dev, dt, code = _act(q, "q", q.dim())
    ptrs, (pages, P, Hk, D), cc = _cache(k_cache, v_cache, k_scale, v_scale, dt, dev)
    shape = q.shape
    Hq = shape[-2]
    if shape[-1] != D:
        raise ValueError("q has shape %s, the cache has %d columns" % (tuple(shape), D))
    if Hq > _INT:
        _large(Hq)
    pitch, head = _heads(q, "q", shape, dt, dev)
    if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2:
        raise ValueError("block_table must be a tensor [sequences, pages]")
    width = block_table.shape[1]
    if width > _INT:
        _large(width)
    if block_table.shape[0] != n or block_table.dtype is not I32 or block_table.device != dev:
        _refuse(block_table, "block_table", (n, width), I32, dev, None)
    row, one = block_table.stride()
    if (one != 1 and width > 1) or (row < width and n > 1):
        raise ValueError("block_table must have dense rows (strides %s)" % ((row, one),))
    lp = _need(seq_lens, "seq_lens", (n,), I32, dev)
    if lp is None:
        raise ValueError("seq_lens is needed")
    if scale is None:
        scale = D ** -0.5 if D else 1.0
    return dev, (q.data_ptr(), pitch, head, *ptrs, block_table.data_ptr(), row if n > 1 else width, width, lp), \
        scale, Hq, (Hq, Hk, D, pages, P, code, cc), (Hq, Hk, D, P, width, code, cc)


def paged_attn_fwd(q, k_cache, v_cache, block_table, seq_lens, k_scale=None, v_scale=None, *, scale=None, causal=True,
                   window=0, want_lse=False):
    """Attention of new tokens over a paged cache: ``o = softmax(scale q . k) v`` over the keys that a token
    sees.

    q [B,T,Hq,D] (fp32 or bf16; D 64, 128 or 256): T new tokens a sequence, whose keys and values are in the cache
    already (kv_cache_write); k_cache, v_cache [pages,Hk,P,D] with Hq a multiple of Hk, 8-bit ones with
    k_scale, v_scale [pages,Hk,P]; block_table [B,max_pages] int32: a sequence's pages in order; seq_lens [B]
    int32: its keys, the new tokens' included.  With causal, a sequence's token t is at position seq_len - T + t and
    sees the positions up to its own, with a window only the last `window` of them; without, all keys (cross
    attention to cached states).  A token that sees no key gets 0.  scale: 1 / sqrt(D) by default.  Returns
    o [B,T,Hq,D] and, when requested, lse [B,T,Hq] fp32: the log of the sum of exp(scores) (-inf without keys)."""
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        raise ValueError("q must be a tensor [B, T, Hq, D]")
    B, T = q.shape[:2]
    if B > _INT or T > _INT:
        _large(B, T)
    dev, args, scale, Hq, sizes, ws_sizes = _attn_args(q, B, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens,
                                                       scale)
    o = _like(q)
    lse = torch.empty(B, T, Hq, dtype=F32, device=dev) if want_lse else None
    n = _lib.load().paged_attn_workspace_bytes(B, T, *ws_sizes)
    ws = _workspace(n, dev)
    _call("paged_attn_fwd", dev, *args, scale, 1 if causal else 0, _window(window), o.data_ptr(),
          lse.data_ptr() if want_lse else None, B, T, *sizes, ws.data_ptr() if n else None, n)
    return {"o": o, "lse": lse} if want_lse else {"o": o}


def paged_attn_fwd_varlen(q, k_cache, v_cache, block_table, seq_lens, cu_seqlens, k_scale=None, v_scale=None, *,
                          scale=None, causal=True, window=0, want_lse=False, cu_seqlens_host=None):
    """paged_attn_fwd over packed sequences of new tokens: q, o [1,T,Hq,D], lse [1,T,Hq], block_table
    [N,max_pages], seq_lens [N]; cu_seqlens and cu_seqlens_host as in gdn_fwd_varlen."""
    if not isinstance(q, torch.Tensor) or q.dim() != 4 or q.shape[0] != 1:
        raise ValueError("q must be a packed tensor [1, T, Hq, D]")
    T = q.shape[1]
    if T > _INT:
        _large(T)
    if cu_seqlens is None:
        raise ValueError("a packed call needs cu_seqlens")
    if _int32(cu_seqlens, q.device) and _int32(cu_seqlens_host, _CPU) and cu_seqlens.shape == cu_seqlens_host.shape:
        cu, host = cu_seqlens, cu_seqlens_host  # as they are (what a serving loop passes)
    else:
        from . import _cu_pair

        cu, host = _cu_pair(cu_seqlens, cu_seqlens_host, q.device)
    if host.dim() != 1 or host.numel() < 2:
        raise ValueError("cu_seqlens must hold at least two offsets")
    N = host.numel() - 1
    dev, args, scale, Hq, sizes, ws_sizes = _attn_args(q, N, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens,
                                                       scale)
    o = _like(q)
    lse = torch.empty(1, T, Hq, dtype=F32, device=dev) if want_lse else None
    n = _lib.load().paged_attn_varlen_workspace_bytes(host.data_ptr(), N, *ws_sizes)
    ws = _workspace(n, dev)
    _call("paged_attn_fwd_varlen", dev, *args, cu.data_ptr(), host.data_ptr(), N, scale, 1 if causal else 0,
          _window(window), o.data_ptr(), lse.data_ptr() if want_lse else None, T, *sizes, ws.data_ptr() if n else None,
          n)
    return {"o": o, "lse": lse} if want_lse else {"o": o}


def paged_attn_step(q, k_cache, v_cache, block_table, seq_lens, k_scale=None, v_scale=None, *, scale=None, window=0):
    """paged_attn_fwd for one token a row: q [B,Hq,D], whose keys and values are in the cache already.  A row
    that pads the batch has seq_len 0 and gets 0.  Returns o [B,Hq,D]."""
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q must be a tensor [B, Hq, D]")
    B = q.shape[0]
    if B > _INT:
        _large(B)
    dev, args, scale, _, sizes, ws_sizes = _attn_args(q, B, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens,
                                                      scale)
    o = _like(q)
    n = _lib.load().paged_attn_workspace_bytes(B, 1, *ws_sizes)
    ws = _workspace(n, dev)
    _call("paged_attn_step", dev, *args, scale, _window(window), o.data_ptr(), B, *sizes, ws.data_ptr() if n else None,
          n)
    return o
