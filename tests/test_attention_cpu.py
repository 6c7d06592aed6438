"""Refusals of the full-attention layers' operators, by the library (status codes, before any launch) and by the
binding (ValueError), and what the binding computes on the host, on the CPU."""
import ctypes
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

FAKE = ctypes.c_void_p(0x1000)  # never dereferenced: every call below fails validation first
ODD = ctypes.c_void_p(0x1004)
E4M3 = torch.float8_e4m3fn


def _lib():
    from gated_delta_rule_29_amd import _lib as L

    return L, L.load()


def _cu(*v):
    a = np.asarray(v, np.int32)
    return a, a.ctypes.data_as(ctypes.c_void_p)


def test_rope_codes():
    L, lib = _lib()
    for name in ("rope_fwd", "rope_bwd"):
        def call(**kw):
            a = dict(x=FAKE, p=128, hp=64, pos=FAKE, table=FAKE, y=FAKE, T=2, H=2, D=64, R=64, dt=1)
            a.update(kw)
            return getattr(lib, name)(a["x"], a["p"], a["hp"], a["pos"], a["table"], 1.0, a["y"], a["T"], a["H"], a["D"],
                                      a["R"], 0, a["dt"], None)

        for bad in (dict(x=None), dict(pos=None), dict(table=None), dict(y=None), dict(T=0), dict(H=0), dict(D=0),
                    dict(T=-1), dict(T=(1 << 30) + 1), dict(R=0), dict(R=3), dict(R=66), dict(dt=2), dict(p=63),
                    dict(hp=63), dict(T=1 << 24, H=2)):
            assert call(**bad) == L.ERR_INVALID, bad
        for bad in (dict(D=1026, p=2052, hp=1026), dict(H=4097), dict(p=1 << 33), dict(hp=1 << 33)):
            assert call(**bad) == L.ERR_UNSUPPORTED, bad


def test_cache_codes():
    L, lib = _lib()

    def write(**kw):
        a = dict(k=FAKE, kp=128, kh=64, v=FAKE, vp=128, vh=64, slots=FAKE, kc=FAKE, vc=FAKE, ks=None, vs=None, T=3, pages=4,
                 P=16, H=2, D=64, dt=1, ct=1)
        a.update(kw)
        return lib.kv_cache_write(a["k"], a["kp"], a["kh"], a["v"], a["vp"], a["vh"], a["slots"], a["kc"], a["vc"], a["ks"],
                                  a["vs"], a["T"], a["pages"], a["P"], a["H"], a["D"], a["dt"], a["ct"], None)

    def read(**kw):
        a = dict(k=FAKE, v=FAKE, slots=FAKE, kc=FAKE, vc=FAKE, ks=None, vs=None, T=3, pages=4, P=16, H=2, D=64, dt=1, ct=1)
        a.update(kw)
        return lib.kv_cache_read(a["kc"], a["vc"], a["ks"], a["vs"], a["slots"], a["k"], a["v"], a["T"], a["pages"], a["P"],
                                 a["H"], a["D"], a["dt"], a["ct"], None)

    shared = [dict(k=None), dict(v=None), dict(slots=None), dict(kc=None), dict(vc=None), dict(T=0), dict(pages=0), dict(H=0),
              dict(D=0), dict(dt=2), dict(ct=0), dict(ct=3), dict(ct=2), dict(ct=2, ks=FAKE), dict(ks=FAKE, vs=FAKE),
              dict(pages=1 << 27), dict(T=1 << 23, H=2)]
    for bad in shared:
        assert write(**bad) == L.ERR_INVALID, bad
        assert read(**bad) == L.ERR_INVALID, bad
    for bad in (dict(kp=63), dict(kh=60), dict(vp=63), dict(vh=1)):
        assert write(**bad) == L.ERR_INVALID, bad
    for bad in (dict(P=8), dict(P=48), dict(P=2048), dict(P=0), dict(D=513, kp=1026, kh=513, vp=1026, vh=513)):
        assert write(**bad) == L.ERR_UNSUPPORTED, bad
        assert read(**{k: x for k, x in bad.items() if k in "PD"}) == L.ERR_UNSUPPORTED, bad


ATTN = dict(q=FAKE, qp=256, qh=64, kc=FAKE, vc=FAKE, ks=None, vs=None, table=FAKE, tp=4, width=4, lens=FAKE, scale=0.1,
            causal=1, window=0, o=FAKE, B=2, T=3, Hq=4, Hk=2, D=64, pages=9, P=16, dt=1, ct=1, ws=None, n=0)


def _fwd(lib, **kw):
    a = dict(ATTN, **kw)
    return lib.paged_attn_fwd(a["q"], a["qp"], a["qh"], a["kc"], a["vc"], a["ks"], a["vs"], a["table"], a["tp"], a["width"],
                              a["lens"], a["scale"], a["causal"], a["window"], a["o"], None, a["B"], a["T"], a["Hq"],
                              a["Hk"], a["D"], a["pages"], a["P"], a["dt"], a["ct"], a["ws"], a["n"], None)


def _step(lib, **kw):
    a = dict(ATTN, **kw)
    return lib.paged_attn_step(a["q"], a["qp"], a["qh"], a["kc"], a["vc"], a["ks"], a["vs"], a["table"], a["tp"], a["width"],
                               a["lens"], a["scale"], a["window"], a["o"], a["B"], a["Hq"], a["Hk"], a["D"], a["pages"],
                               a["P"], a["dt"], a["ct"], a["ws"], a["n"], None)


def _packed(lib, cu, T, cu_dev=FAKE, **kw):
    keep, p = _cu(*cu)
    a = dict(ATTN, **kw)
    return lib.paged_attn_fwd_varlen(a["q"], a["qp"], a["qh"], a["kc"], a["vc"], a["ks"], a["vs"], a["table"], a["tp"],
                                     a["width"], a["lens"], cu_dev, p, len(keep) - 1, a["scale"], a["causal"],
                                     a["window"], a["o"], None, T, a["Hq"], a["Hk"], a["D"], a["pages"], a["P"], a["dt"],
                                     a["ct"], a["ws"], a["n"], None)


def test_attention_codes():
    L, lib = _lib()
    bad_all = [dict(q=None), dict(kc=None), dict(vc=None), dict(table=None), dict(lens=None), dict(o=None), dict(qp=63),
               dict(qh=63), dict(tp=3), dict(width=0), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(window=-1), dict(Hq=0), dict(Hk=0), dict(Hq=3), dict(pages=0), dict(dt=2),
               dict(ct=0), dict(ct=2), dict(ks=FAKE, vs=FAKE), dict(kc=ODD), dict(vc=ODD), dict(o=ODD),
               dict(pages=1 << 27), dict(width=1 << 27, tp=1 << 27)]
    for bad in bad_all:
        assert _fwd(lib, **bad) == L.ERR_INVALID, bad
        assert _step(lib, **bad) == L.ERR_INVALID, bad
        assert _packed(lib, (0, 3, 6), 6, **bad) == L.ERR_INVALID, bad
    for bad in (dict(D=32), dict(D=96, qp=999, qh=96), dict(P=8), dict(P=24), dict(Hq=8192, qp=1 << 20), dict(qp=1 << 33),
                dict(tp=1 << 33)):
        assert _fwd(lib, **bad) == L.ERR_UNSUPPORTED, bad
        assert _step(lib, **bad) == L.ERR_UNSUPPORTED, bad
    for bad in (dict(B=0), dict(T=0), dict(B=1 << 16, T=1 << 16), dict(causal=0, window=4),
                dict(B=1 << 22, T=1, Hq=8, Hk=8, qp=512), dict(B=1, T=1 << 30)):
        assert _fwd(lib, **bad) == L.ERR_INVALID, bad
    for cu, T in (((0, 3, 3), 3), ((1, 3), 3), ((0, 3), 4), ((0, 5, 3), 3), ((0,), 1)):
        assert _packed(lib, cu, T) == L.ERR_INVALID, cu
    assert _packed(lib, (0, 3), 3, cu_dev=None) == L.ERR_INVALID


def test_attention_workspace():
    L, lib = _lib()
    # short tables are never cut; long ones need a workspace
    assert lib.paged_attn_workspace_bytes(2, 1, 4, 2, 64, 16, 4, 1, 1) == 0
    n = lib.paged_attn_workspace_bytes(2, 1, 4, 2, 64, 16, 400, 1, 1)
    assert n > 0
    assert _step(lib, width=400, tp=400) == L.ERR_WORKSPACE
    assert _step(lib, width=400, tp=400, ws=FAKE, n=n - 1) == L.ERR_WORKSPACE
    assert _step(lib, width=400, tp=400, ws=ctypes.c_void_p(0x1010), n=n) == L.ERR_INVALID  # misaligned
    assert lib.paged_attn_workspace_bytes(2, 1, 4, 3, 64, 16, 400, 1, 1) == 0  # what cannot be sized
    assert lib.paged_attn_workspace_bytes(2, 1, 4, 2, 65, 16, 400, 1, 1) == 0
    keep, p = _cu(0, 1, 2)
    assert lib.paged_attn_varlen_workspace_bytes(p, 2, 4, 2, 64, 16, 400, 1, 1) == n
    assert lib.paged_attn_varlen_workspace_bytes(None, 2, 4, 2, 64, 16, 400, 1, 1) == 0
    keep, p = _cu(0, 2, 1)
    assert lib.paged_attn_varlen_workspace_bytes(p, 2, 4, 2, 64, 16, 400, 1, 1) == 0


def test_binding_refusals():
    import gated_delta_rule_29_amd as g

    bf = torch.bfloat16
    x, pos, table = torch.zeros(2, 3, 8, dtype=bf), torch.zeros(2, dtype=torch.int32), torch.zeros(4, dtype=torch.int64)
    for f in (g.rope_fwd, g.rope_bwd):
        for args in ((x[0, 0], pos, table), (x.half(), pos, table), (x, pos.long(), table), (x, pos[:1], table),
                     (x, pos, table.double()), (x, pos, table[None]), (None, pos, table), (x.transpose(1, 2), pos, table),
                     (x, None, None), (x, pos, table)):  # (the last: not on a GPU)
            with pytest.raises(ValueError):
                f(*args)
    c, s, slots = torch.zeros(2, 3, 16, 8, dtype=bf), torch.zeros(2, 3, 16), torch.zeros(2, dtype=torch.int32)
    q8 = torch.zeros(2, 3, 16, 8).to(E4M3)
    for args in ((x, x, c[0], c, slots), (x, x[:1], c, c, slots), (x, x, c, c[:1], slots), (x, x, c, None, slots),
                 (x, x, c.float(), c.float(), slots), (x, x, q8, c, slots, s, s), (x, x, q8, q8, slots, s, s[:1]),
                 (x, x, c, c, slots.long()), (x, x, c, c, slots[:1]), (x[..., :4], x[..., :4], c, c, slots),
                 (x, x.float(), c, c, slots), (x, x, c.transpose(1, 2), c, slots), (x, x, c, c, slots)):
        with pytest.raises(ValueError):
            g.kv_cache_write(*args)
    for args, kw in (((c, c, None), {}), ((c, c, slots.long()), {}), ((c, c, slots), dict(dtype=torch.float32)),
                     ((q8, q8, slots, s, s), dict(dtype=torch.float16)), ((None, c, slots), {}), ((c, c, slots), {})):
        with pytest.raises(ValueError):
            g.kv_cache_read(*args, **kw)
    D = 64
    c, q8, s = torch.zeros(5, 2, 16, D, dtype=bf), torch.zeros(5, 2, 16, D).to(E4M3), torch.zeros(5, 2, 16)
    q, t, n = torch.zeros(3, 4, D, dtype=bf), torch.zeros(3, 4, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    bad = [(q[0], c, c, t, n), (q.float(), c, c, t, n), (q[..., :32], c, c, t, n), (q, c[0], c, t, n), (q, c, c, t[:2], n),
           (q, c, c, t.long(), n), (q, c, c, t[0], n), (q, c, c, t.t().contiguous().t(), n), (q, c, c, t, n[:2]),
           (q, c, c, t, n.long()), (q, c, c, t, None), (q, c, c, None, n), (None, c, c, t, n), (q, q8, q8, t, n, s, None),
           (q, c, c, t, n)]
    for a in bad:
        with pytest.raises((ValueError, AttributeError)) as e:
            g.paged_attn_step(*a)
        assert e.type is ValueError, a
    cu = torch.tensor([0, 1, 3], dtype=torch.int32)
    for a in ((q, c, c, t[:2], n[:2], cu), (q[None], c, c, t[:2], n[:2], None), (q[None], c, c, t, n, cu),
              (q[None], c, c, t[:2], n[:2], cu[:1]), (q[None].expand(2, -1, -1, -1), c, c, t[:2], n[:2], cu)):
        with pytest.raises(ValueError):
            g.paged_attn_fwd_varlen(*a)
    for a in ((q, c, c, t, n), (q[:, None], c, c, t[:2], n), (q[:, None], c, c, t, n)):
        with pytest.raises(ValueError):
            g.paged_attn_fwd(*a)


def test_pitches_of_views():
    from gated_delta_rule_29_amd.attention import _heads

    dev, bf = torch.device("cpu"), torch.bfloat16
    x = torch.zeros(6, 40, dtype=bf)
    v = x[:, 8:32].view(6, 3, 8)
    assert _heads(v, "x", v.shape, bf, dev) == (40, 8)
    h = torch.zeros(3, 6, 8, dtype=bf).transpose(0, 1)
    assert _heads(h, "x", h.shape, bf, dev) == (8, 48)
    b = torch.zeros(2, 5, 3, 16, dtype=bf)[..., :8]
    assert _heads(b, "x", b.shape, bf, dev) == (48, 16)
    one = torch.zeros(1, 3, 8, dtype=bf)[:, :1]
    assert _heads(one, "x", one.shape, bf, dev) == (8, 8)
    for bad in (torch.zeros(2, 5, 3, 8, dtype=bf)[:, :4], torch.zeros(6, 8, 3, dtype=bf).transpose(1, 2),
                torch.zeros(1, 3, 8, dtype=bf).expand(4, 3, 8)):
        with pytest.raises(ValueError):
            _heads(bad, "x", bad.shape, bf, dev)


def test_sizes_beyond_32_bits():
    import gated_delta_rule_29_amd as g

    big = torch.zeros(1, dtype=torch.bfloat16).expand(1 << 32, 1, 1)
    with pytest.raises(ValueError, match="32 bits"):
        g.rope_fwd(big, torch.zeros(1, dtype=torch.int32).expand(1 << 32), torch.zeros(1, dtype=torch.int64))
    wide = torch.zeros(1, dtype=torch.int32).expand(1, 1 << 32)
    c = torch.zeros(1, 1, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="32 bits"):
        g.paged_attn_step(torch.zeros(1, 1, 64, dtype=torch.bfloat16), c, c, wide, torch.zeros(1, dtype=torch.int32))


def test_rope_freqs():
    import gated_delta_rule_29_amd as g

    f, m = g.rope_freqs(8, 100.0)
    assert m == 1.0 and torch.allclose(f, torch.tensor([1.0, 100 ** -0.25, 0.1, 100 ** -0.75], dtype=torch.float64))
    assert torch.equal(g.rope_freqs(8, 100.0, scaling="linear", factor=4.0)[0], f / 4)
    n, _ = g.rope_freqs(8, 100.0, scaling="ntk", factor=4.0)  # the first pair stays, the last is divided by the factor
    assert n[0] == 1.0 and abs(n[-1] * 4 / f[-1] - 1) < 1e-14
    y, m = g.rope_freqs(128, 10000.0, scaling="yarn", factor=16.0, original=4096)
    f, _ = g.rope_freqs(128)
    assert abs(m - (1 + 0.1 * math.log(16.0))) < 1e-15
    turns = 4096 * f / (2 * math.pi)
    assert torch.equal(y[turns > 40], f[turns > 40]) and torch.equal(y[turns < 0.8], f[turns < 0.8] / 16)
    assert (y[:-1] > y[1:]).all() and (y <= f).all() and (y >= f / 16).all()
    assert torch.allclose(g.rope_freqs(128, scaling="yarn")[0], f, rtol=2.0 ** -51, atol=0)  # (three roundings)
    assert g.rope_freqs(2, scaling="ntk", factor=9.0)[0] == 1
    for kw in (dict(R=3), dict(R=0), dict(R=8, theta=1.0), dict(R=8, scaling="other"), dict(R=8, scaling="linear", factor=0.5),
               dict(R=8, scaling="yarn", fast=1.0, slow=2.0)):
        with pytest.raises(ValueError):
            g.rope_freqs(**kw)


def test_rope_table():
    import gated_delta_rule_29_amd as g

    pi = Fraction("3.14159265358979323846264338327950288419716939937510582097494")
    f = torch.tensor([1.0, 0.3, 1e-6, 6.5, -0.25], dtype=torch.float64)
    t = g.rope_table(f, "cpu")
    assert t.dtype == torch.int64 and t.shape == f.shape
    for a, n in zip(f.tolist(), t.tolist()):
        off = (Fraction(n, 1 << 64) - Fraction(a) / (2 * pi)) % 1
        assert min(off, 1 - off) <= Fraction(1, 1 << 65)
    for bad in (f[None], f.long(), f[:0], torch.tensor([1.0, float("nan")]), [1.0]):
        with pytest.raises(ValueError):
            g.rope_table(bad, "cpu")


@pytest.mark.parametrize("form", ["fwd", "varlen", "step"])
def test_windows_beyond_32_bits(form, monkeypatch):
    """A window that no 32-bit integer holds reaches the library as one that hides nothing, and not as its low bits."""
    import gated_delta_rule_29_amd as g
    from gated_delta_rule_29_amd import attention

    seen = []

    def call(name, dev, *args):
        # (the argument's place in the C signature, as the library would read it)
        at = {"paged_attn_fwd": 13, "paged_attn_fwd_varlen": 16, "paged_attn_step": 12}[name]
        seen.append(ctypes.c_int(args[at]).value)

    monkeypatch.setattr(attention, "_call", call)
    c = torch.zeros(5, 2, 16, 64, dtype=torch.bfloat16)
    q, t = torch.zeros(3, 4, 64, dtype=torch.bfloat16), torch.zeros(3, 4, dtype=torch.int32)
    n, cu = torch.ones(3, dtype=torch.int32), torch.arange(4, dtype=torch.int32)

    def run(window):
        if form == "step":
            return g.paged_attn_step(q, c, c, t, n, window=window)
        if form == "fwd":
            return g.paged_attn_fwd(q[:, None], c, c, t, n, window=window)
        return g.paged_attn_fwd_varlen(q[None], c, c, t, n, cu, window=window)

    most = 2 ** 31 - 1
    for window in (0, 1, 64, most, most + 1, 2 ** 32 - 1, 2 ** 32, 2 ** 32 + 64, 2 ** 70):
        run(window)
        assert seen[-1] == min(window, most), window
    for window in (-1, -2 ** 31 - 1, -2 ** 32, -2 ** 32 + 7, -2 ** 70):
        with pytest.raises(ValueError, match="window"):
            run(window)


@pytest.mark.parametrize("bad", [[0, 2 ** 32 + 1, 3], [0, 1, 2 ** 32 + 3], [-2 ** 32, 1, 3], [0, -2 ** 32 + 1, 3]])
def test_offsets_beyond_32_bits(bad):
    """Offsets whose low 32 bits would make a good call are refused, as the device's, the host's or both."""
    import gated_delta_rule_29_amd as g

    cpu = torch.device("cpu")
    good, wide = torch.tensor([0, 1, 3]), torch.tensor(bad)
    for args in ((wide, None), (wide, wide), (wide.to(torch.int32), wide), (good, bad)):
        with pytest.raises(ValueError, match="32 bits"):
            g._cu_pair(*args, cpu)
    for args in ((good, None), (good, good), (good.to(torch.int32), [0, 1, 3]), (good, good.numpy())):
        for t in g._cu_pair(*args, cpu):
            assert t.dtype == torch.int32 and t.tolist() == [0, 1, 3]
    c = torch.zeros(5, 2, 16, 64, dtype=torch.bfloat16)
    t, n = torch.zeros(2, 4, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="32 bits"):
        g.paged_attn_fwd_varlen(torch.zeros(1, 3, 4, 64, dtype=torch.bfloat16), c, c, t, n, wide)
