"""Refusals of the layer operators, by the library (status codes, before any launch) and by the binding
(ValueError), on the CPU."""
import ctypes

import numpy as np
import pytest
import torch

FAKE = ctypes.c_void_p(0x1000)  # never dereferenced: every call below fails validation first
ODD = ctypes.c_void_p(0x1004)


def _lib():
    from gated_delta_rule_29_amd import _lib as L

    return L, L.load()


def _cu(*v):
    a = np.asarray(v, np.int32)
    return a, a.ctypes.data_as(ctypes.c_void_p)


def test_chunk_constant():
    import gated_delta_rule_29_amd as g

    with open(g.layer.__file__.replace("gated_delta_rule_29_amd/layer.py", "include/gdn.h")) as f:
        line = next(s for s in f if s.startswith("#define GDN_SSM_CHUNK"))
    assert int(line.split()[2]) == g.SSM_CHUNK


def test_conv_codes():
    L, lib = _lib()

    def fwd(**kw):
        a = dict(x=FAKE, p=8, w=FAKE, y=FAKE, B=1, T=4, D=8, W=4, dt=1)
        a.update(kw)
        return lib.causal_conv_fwd(a["x"], a["p"], a["w"], None, None, a["y"], None, a["B"], a["T"], a["D"],
                                   a["W"], 1, a["dt"], None)

    for bad in (dict(x=None), dict(w=None), dict(y=None), dict(B=0), dict(T=0), dict(D=0), dict(dt=2), dict(p=7),
                dict(W=0), dict(B=1 << 16, T=1 << 16), dict(T=(1 << 30) + 1), dict(T=1 << 30, D=1 << 20, p=1 << 20)):
        assert fwd(**bad) == L.ERR_INVALID, bad
    assert fwd(W=1) == L.ERR_UNSUPPORTED and fwd(W=5) == L.ERR_UNSUPPORTED

    def packed(cu, T):
        keep, p = _cu(*cu)
        return lib.causal_conv_fwd_varlen(FAKE, 8, FAKE, None, FAKE, p, len(keep) - 1, None, FAKE, None, T, 8, 4, 1,
                                          1, None)

    for cu, T in (((0, 3, 3), 3), ((1, 3), 3), ((0, 3), 4), ((0, 5, 3), 3), ((0,), 1)):
        assert packed(cu, T) == L.ERR_INVALID, cu

    def bwd(ws=None, n=0, **kw):
        a = dict(dy=FAKE, dyp=8, dx=FAKE, dw=FAKE, W=4)
        a.update(kw)
        return lib.causal_conv_bwd(a["dy"], a["dyp"], FAKE, 8, FAKE, None, None, None, a["dx"], None, a["dw"], None,
                                   1, 4, 8, a["W"], 1, 1, ws, n, None)

    for bad in (dict(dy=None), dict(dx=None), dict(dw=None), dict(dyp=4)):
        assert bwd(**bad) == L.ERR_INVALID, bad
    n = lib.causal_conv_bwd_workspace_bytes(4, 8, 4)
    assert n >= 5 * 8 * 4 and lib.causal_conv_bwd_workspace_bytes(4, 8, 5) == 0
    assert bwd() == L.ERR_WORKSPACE and bwd(FAKE, n - 1) == L.ERR_WORKSPACE
    assert bwd(ctypes.c_void_p(0x1010), n) == L.ERR_INVALID  # misaligned

    def step(**kw):
        a = dict(x=FAKE, st=FAKE, y=FAKE, slots=None, B=2, S=2, W=4)
        a.update(kw)
        return lib.causal_conv_step(a["x"], 8, FAKE, None, a["st"], a["slots"], a["y"], a["B"], a["S"], 8, a["W"], 1,
                                    1, None)

    for bad in (dict(st=None), dict(y=None), dict(B=0), dict(S=0), dict(S=1)):
        assert step(**bad) == L.ERR_INVALID, bad
    assert step(W=7) == L.ERR_UNSUPPORTED
    assert step(B=1 << 24, S=1 << 24) == L.ERR_INVALID  # a workgroup a row: 2^32 threads


def _scan(lib, **kw):
    a = dict(x=FAKE, xp=8, dt=FAKE, dp=8, A=FAKE, B_=FAKE, bp=16, C_=FAKE, z=None, zp=0, h0=None, y=FAKE, ht=None, h=None,
             B=1, T=4, D=8, N=16, ty=1, ws=None, n=0)
    a.update(kw)
    return lib.ssm_scan_fwd(a["x"], a["xp"], a["dt"], a["dp"], a["A"], a["B_"], a["bp"], a["C_"], 64, None, a["z"],
                            a["zp"], None, a["h0"], a["y"], a["ht"], a["h"], a["B"], a["T"], a["D"], a["N"], 1,
                            a["ty"], a["ws"], a["n"], None)


def test_scan_codes():
    L, lib = _lib()
    for bad in (dict(x=None), dict(dt=None), dict(A=None), dict(B_=None), dict(C_=None), dict(y=None), dict(B=0),
                dict(T=0), dict(D=0), dict(N=0), dict(ty=3), dict(xp=7), dict(bp=15), dict(z=FAKE, zp=7),
                dict(A=ODD), dict(h0=ODD), dict(ht=ODD), dict(h=ODD), dict(B=1 << 16, T=1 << 16),
                dict(B=1 << 18, T=1, D=1 << 12, xp=1 << 12, dp=1 << 12)):  # (2^24 workgroups: 2^32 threads)
        assert _scan(lib, **bad) == L.ERR_INVALID, bad
    assert _scan(lib, N=65, bp=65) == L.ERR_UNSUPPORTED
    # a long sequence of few channels is cut and needs a workspace; a short or a wide one does not
    n = lib.ssm_scan_fwd_workspace_bytes(1, 4096, 8, 16)
    assert n > 0 and _scan(lib, T=4096) == L.ERR_WORKSPACE
    assert _scan(lib, T=4096, ws=FAKE, n=n - 1) == L.ERR_WORKSPACE
    assert lib.ssm_scan_fwd_workspace_bytes(1, 64, 8, 16) == 0
    assert lib.ssm_scan_fwd_workspace_bytes(1, 64, 8, 65) == 0
    keep, p = _cu(0, 64, 4160)
    assert lib.ssm_scan_fwd_varlen_workspace_bytes(p, 2, 8, 16) > 0
    keep, p = _cu(0, 1, 17, 50)
    assert lib.ssm_scan_num_chunks(p, 3) == 1 + 1 + 3
    keep, p = _cu(0, 64, 64)
    assert lib.ssm_scan_num_chunks(p, 2) == -1
    assert lib.ssm_scan_fwd_varlen_workspace_bytes(p, 2, 8, 16) == 0
    assert lib.ssm_scan_bwd_varlen_workspace_bytes(p, 2, 8, 16) == 0
    assert lib.ssm_scan_bwd_varlen_workspace_bytes(None, 2, 8, 16) == 0


def test_scan_bwd_codes():
    L, lib = _lib()

    def call(**kw):
        a = dict(dy=FAKE, dyp=8, h=FAKE, z=None, zp=0, dht=None, dx=FAKE, ddt=FAKE, dA=FAKE, dB=FAKE, dC=FAKE,
                 dz=None, dh0=None, N=16, ws=None, n=0)
        a.update(kw)
        return lib.ssm_scan_bwd(a["dy"], a["dyp"], a["h"], FAKE, 8, FAKE, 8, FAKE, FAKE, 64, FAKE, 64, None, a["z"],
                                a["zp"], None, a["dht"], a["dx"], a["ddt"], a["dA"], a["dB"], a["dC"], None, a["dz"],
                                None, a["dh0"], 1, 4, 8, a["N"], 1, 1, a["ws"], a["n"], None)

    for bad in (dict(dy=None), dict(dyp=7), dict(h=None), dict(h=ODD), dict(dht=ODD), dict(dh0=ODD), dict(dx=None),
                dict(ddt=None), dict(dA=None), dict(dB=None), dict(dC=None), dict(z=FAKE, zp=8), dict(dz=FAKE)):
        assert call(**bad) == L.ERR_INVALID, bad
    assert call(N=65) in (L.ERR_INVALID, L.ERR_UNSUPPORTED)
    n = lib.ssm_scan_bwd_workspace_bytes(1, 4, 8, 16)
    assert n >= 4 * 2 * 16 * 4 and call() == L.ERR_WORKSPACE and call(ws=FAKE, n=n - 1) == L.ERR_WORKSPACE


def test_step_and_norm_codes():
    L, lib = _lib()

    def step(**kw):
        a = dict(st=FAKE, y=FAKE, B=2, S=4, N=16)
        a.update(kw)
        return lib.ssm_step(FAKE, 8, FAKE, 8, FAKE, FAKE, 64, FAKE, 64, None, None, 0, None, a["st"], None, a["y"],
                            a["B"], a["S"], 8, a["N"], 1, 1, None)

    for bad in (dict(st=None), dict(st=ODD), dict(y=None), dict(B=0), dict(S=1), dict(B=1 << 24, S=1 << 24)):
        assert step(**bad) == L.ERR_INVALID, bad
    assert step(N=65) in (L.ERR_INVALID, L.ERR_UNSUPPORTED)

    def norm(**kw):
        a = dict(x=FAKE, xp=8, r=None, rp=0, w=FAKE, eps=1e-5, y=FAKE, s=None, M=2, D=8, dt=1, rt=1)
        a.update(kw)
        return lib.rms_norm_fwd(a["x"], a["xp"], a["r"], a["rp"], a["w"], a["eps"], a["y"], a["s"], None, a["M"],
                                a["D"], a["dt"], a["rt"], None)

    for bad in (dict(x=None), dict(w=None), dict(y=None), dict(xp=7), dict(r=FAKE, rp=7), dict(eps=0.0),
                dict(eps=float("nan")), dict(M=0), dict(M=(1 << 30) + 1), dict(D=0), dict(dt=2), dict(rt=2), dict(s=FAKE)):
        assert norm(**bad) == L.ERR_INVALID, bad
    assert norm(dt=0, rt=1) == L.ERR_UNSUPPORTED and norm(D=32769, xp=32769) == L.ERR_UNSUPPORTED

    def q8(**kw):
        a = dict(block=0, q=FAKE, sc=FAKE)
        a.update(kw)
        return lib.rms_norm_q8_fwd(FAKE, 8, None, 0, FAKE, 1e-5, a["block"], a["q"], a["sc"], None, 2, 8, 1, 1, None)

    assert q8(q=None) == L.ERR_INVALID and q8(sc=None) == L.ERR_INVALID and q8(block=64) == L.ERR_UNSUPPORTED

    def bwd(**kw):
        a = dict(dy=FAKE, s=FAKE, r=FAKE, ds=FAKE, dw=FAKE, sp=8, ws=None, n=0)
        a.update(kw)
        return lib.rms_norm_bwd(a["dy"], 8, a["s"], a["sp"], FAKE, a["r"], None, 0, a["ds"], None, a["dw"], 2, 8, 1,
                                1, a["ws"], a["n"], None)

    for bad in (dict(dy=None), dict(s=None), dict(r=None), dict(ds=None), dict(dw=None), dict(sp=7)):
        assert bwd(**bad) == L.ERR_INVALID, bad
    n = lib.rms_norm_bwd_workspace_bytes(2, 8)
    assert n >= 2 * 8 * 4 and bwd() == L.ERR_WORKSPACE and bwd(ws=FAKE, n=n - 1) == L.ERR_WORKSPACE


def test_binding_refusals():
    import gated_delta_rule_29_amd as g

    x, w = torch.zeros(2, 5, 8), torch.zeros(8, 4)
    for bad, why in ((lambda: g.causal_conv_fwd(x.half(), w), "float32 or bfloat16"),
                     (lambda: g.causal_conv_fwd(x[0], w), "dimensions"),
                     (lambda: g.causal_conv_fwd(x, w[:7]), "shape"),
                     (lambda: g.causal_conv_fwd(x, w.double()), "dtype"),
                     (lambda: g.causal_conv_fwd(x, w[0]), r"\[D, W\]"),
                     (lambda: g.causal_conv_fwd(x, w, init=torch.zeros(2, 4, 8)), "shape"),
                     (lambda: g.causal_conv_fwd(x.transpose(0, 1), w), "evenly spaced"),
                     (lambda: g.causal_conv_fwd(torch.zeros(2, 5, 16)[..., ::2], w), "dense rows"),
                     (lambda: g.causal_conv_fwd(torch.zeros(2, 1, 8).expand(2, 5, 8), w), "evenly|overlap"),
                     (lambda: g.causal_conv_fwd(x, w.t().contiguous().t()), "contiguous"),
                     (lambda: g.causal_conv_fwd(x, w), "GPU"),
                     (lambda: g.causal_conv_fwd_varlen(x, w, torch.tensor([0, 5])), "batch 1"),
                     (lambda: g.causal_conv_fwd_varlen(x[:1], w, torch.tensor([0], dtype=torch.int32)), "two offsets"),
                     (lambda: g.causal_conv_bwd(x[:1], x, w), "shape"),
                     (lambda: g.causal_conv_bwd(x, x, w, dfinal=torch.zeros(2, 3, 7)), "shape"),
                     (lambda: g.causal_conv_step(x[:, 0], w, torch.zeros(1, 3, 8)), "a slot a row"),
                     (lambda: g.causal_conv_step(x[:, 0], w, torch.zeros(3, 3, 8), slots=torch.zeros(2)), "dtype"),
                     (lambda: g.causal_conv_step(x[:, 0], w, torch.zeros(3, 2, 8)), "shape")):
        with pytest.raises(ValueError, match=why):
            bad()

    A, bc = torch.zeros(8, 16), torch.zeros(2, 5, 16)
    h, st = torch.zeros(2, 1, 8, 16), torch.zeros(2, 8, 16)
    for bad, why in ((lambda: g.ssm_scan_fwd(x, x, A[:7], bc, bc), "shape"),
                     (lambda: g.ssm_scan_fwd(x, x.bfloat16(), A, bc, bc), "dtype"),
                     (lambda: g.ssm_scan_fwd(x, x, A, bc[..., :15], bc), "shape"),
                     (lambda: g.ssm_scan_fwd(x, x, A, bc, bc, h0=st[:1]), "shape"),
                     (lambda: g.ssm_scan_fwd(x, x, A, bc, bc, z=bc), "shape"),
                     (lambda: g.ssm_scan_fwd(x, x, A, bc, bc), "GPU"),
                     (lambda: g.ssm_scan_bwd(x, None, x, x, A, bc, bc), "want_h"),
                     (lambda: g.ssm_scan_bwd(x, h[:1], x, x, A, bc, bc), "shape"),
                     (lambda: g.ssm_scan_bwd(x[:, :4], h, x, x, A, bc, bc), "shape"),
                     (lambda: g.ssm_step(x[:, 0], x[:, 0], A, bc[:, 0], bc[:, 0], st.double()), "dtype"),
                     (lambda: g.ssm_step(x[:, 0], x[:, 0], A, bc[:, 0], bc[:, 0], st[:1]), "a slot a row"),
                     (lambda: g.ssm_step(x[:, 0], x[:, 0], A, bc[:, 0], bc[:, 0], st[0]), "state")):
        with pytest.raises(ValueError, match=why):
            bad()

    v = torch.ones(8)
    for bad, why in ((lambda: g.rms_norm_fwd(x, v[:7]), "shape"),
                     (lambda: g.rms_norm_fwd(x, v, residual=x[:1]), "shape"),
                     (lambda: g.rms_norm_fwd(x, v, residual=x.half()), "residual"),
                     (lambda: g.rms_norm_fwd(x, v), "GPU"),
                     (lambda: g.rms_norm_bwd(x, x, v, None), "want_rstd"),
                     (lambda: g.rms_norm_bwd(x, x, v, torch.ones(2, 4)), "shape"),
                     (lambda: g.rms_norm_bwd(x, x, v, torch.ones(2, 5), dsum=x.bfloat16()), "dtype")):
        with pytest.raises(ValueError, match=why):
            bad()


def test_pitches_of_views():
    """Rows are found evenly spaced also where dimensions of one row have strides of their own."""
    from gated_delta_rule_29_amd.layer import _rows

    wide = torch.zeros(3, 4, 20)
    cpu = torch.device("cpu")
    assert _rows(wide[..., 2:10], "x", (3, 4, 8), torch.float32, cpu) == 20
    assert _rows(wide[:, :1, 2:10], "x", (3, 1, 8), torch.float32, cpu) == 80
    assert _rows(wide[1:2, 1:2, 2:10], "x", (1, 1, 8), torch.float32, cpu) == 8
    assert _rows(wide[:, 0, :8], "x", (3, 8), torch.float32, cpu) == 80
    assert _rows(wide[..., 5:6], "x", (3, 4, 1), torch.float32, cpu) == 20
    with pytest.raises(ValueError):
        _rows(wide[:, :3, 2:10], "x", (3, 3, 8), torch.float32, cpu)  # batches are further apart


def test_sizes_beyond_32_bits():
    """Refused before the library, which would see their low bits.  (Meta tensors: no memory.)"""
    import gated_delta_rule_29_amd as g

    big = (1 << 32) + 4
    t = lambda *s: torch.empty(s, device="meta")  # noqa: E731
    x, w, A, bc, v = t(1, big, 1), t(1, 4), t(1, 4), t(1, big, 4), t(1)
    for bad in (lambda: g.causal_conv_fwd(x, w), lambda: g.causal_conv_bwd(x, x, w),
                lambda: g.causal_conv_fwd(t(1 << 17, 1 << 16, 1), w),
                lambda: g.causal_conv_fwd_varlen(x, w, torch.tensor([0, 4], dtype=torch.int32)),
                lambda: g.causal_conv_fwd(t(1, 4, 1), t(1, big)), lambda: g.causal_conv_bwd(t(1, 4, 1), t(1, 4, 1), t(1, big)),
                lambda: g.causal_conv_step(x[0], w, t(4, 3, 1), slots=torch.empty(big, dtype=torch.int32, device="meta")),
                lambda: g.causal_conv_step(t(2, 1), w, t(big, 3, 1)),
                lambda: g.ssm_scan_fwd(x, x, A, bc, bc), lambda: g.ssm_scan_fwd(t(1, 4, 1), t(1, 4, 1), t(1, big), t(1, 4, big), t(1, 4, big)),
                lambda: g.ssm_scan_bwd(x, t(1, big // 16 + 1, 1, 4), x, x, A, bc, bc),
                lambda: g.ssm_step(t(2, 1), t(2, 1), A, t(2, 4), t(2, 4), t(big, 1, 4)),
                lambda: g.ssm_step(x[0], x[0], A, bc[0], bc[0], t(big, 1, 4)),
                lambda: g.rms_norm_fwd(x, v), lambda: g.rms_norm_q8_fwd(x, v), lambda: g.rms_norm_bwd(x, x, v, x[..., 0])):
        with pytest.raises(ValueError, match="32 bits"):
            bad()


def test_packed_calls_without_offsets():
    """None in the place of the offsets is refused, not taken for a dense batch."""
    import gated_delta_rule_29_amd as g

    x, w, A, bc = torch.zeros(1, 5, 8), torch.zeros(8, 4), torch.zeros(8, 16), torch.zeros(1, 5, 16)
    for bad in (lambda: g.causal_conv_fwd_varlen(x, w, None), lambda: g.causal_conv_bwd_varlen(x, x, w, None),
                lambda: g.causal_conv_fwd_varlen(x, w, None, cu_seqlens_host=torch.tensor([0, 5], dtype=torch.int32)),
                lambda: g.ssm_scan_fwd_varlen(x, x, A, bc, bc, None),
                lambda: g.ssm_scan_bwd_varlen(x, torch.zeros(1, 1, 8, 16), x, x, A, bc, bc, None)):
        with pytest.raises(ValueError, match="cu_seqlens"):
            bad()
