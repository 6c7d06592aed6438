"""GPU parity of the residual RMS norm, its 8-bit output and its gradient against the fp64 oracle."""
import numpy as np
import pytest
import torch

from oracle import layer as L
from tests.gpu_util import say
from tests.layer_util import DEV, TYPES, arr, check, gen, pitched, rn

pytestmark = pytest.mark.gpu
EPS = 1e-5

# rows, columns, (extra columns, offset)
CASES = [(1, 1, (0, 0)), (1, 4096, (0, 0)), (5, 64, (0, 0)), (9, 200, (3, 1)), (7, 512, (8, 8)), (3, 520, (0, 0)),
         (67, 2570, (0, 0)), (4, 4100, (5, 2)), (3, 6144, (16, 8)), (2, 16384, (0, 0)), (2, 17001, (0, 0)),
         (2, 32768, (0, 0)), (300, 136, (0, 0))]


def _inputs(M, D, pitch, dtype, rtype, seed):
    g = gen(seed)
    t, rt = TYPES[dtype], TYPES[rtype]
    c = dict(x=rn(g, M, D, dtype=t), residual=(3 * rn(g, M, D)).to(rt), w=1 + 0.2 * rn(g, D), dy=rn(g, M, D, dtype=t),
             dsum=rn(g, M, D, dtype=rt))
    d = {k: v.to(DEV) for k, v in c.items()}
    if pitch[0]:
        for k in ("x", "residual", "dy", "dsum"):
            d[k] = pitched(c[k], *pitch)
    return c, d


def _sum(c):
    """The stored sum: fp32 addition, rounded to the residual's type."""
    return (c["x"].float() + c["residual"].float()).to(c["residual"].dtype)


@pytest.mark.parametrize("dtype,rtype", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_forward_and_gradient(case, dtype, rtype):
    import gated_delta_rule_29_amd as g

    M, D, pitch = CASES[case]
    say("norm M %d D %d pitch %s %s residual %s" % (M, D, pitch, dtype, rtype))
    c, d = _inputs(M, D, pitch, dtype, rtype, case)
    out = g.rms_norm_fwd(d["x"], d["w"], residual=d["residual"], eps=EPS, want_rstd=True)
    s = _sum(c)
    assert torch.equal(out["sum"].cpu(), s)
    y, rstd = L.norm(arr(s), arr(c["w"]), EPS)
    check("y", out["y"], y)
    check("rstd", out["rstd"], rstd)
    alone = g.rms_norm_fwd(d["x"], d["w"], eps=EPS)
    assert set(alone) == {"y"}
    check("y alone", alone["y"], L.norm(arr(c["x"]), arr(c["w"]), EPS)[0])

    s_in = pitched(s, *pitch) if pitch[0] else out["sum"]
    gr = g.rms_norm_bwd(d["dy"], s_in, d["w"], out["rstd"], dsum=d["dsum"])
    ref = L.norm_bwd(arr(c["dy"]), arr(s), arr(c["w"]), EPS, arr(c["dsum"]))
    check("dx", gr["dx"], ref["ds"])
    check("dresidual", gr["dresidual"], ref["ds"])
    assert gr["dx"].dtype == TYPES[dtype] and gr["dresidual"].dtype == TYPES[rtype]
    check("dw", gr["dw"], ref["dw"])
    if D > 1:  # one column without eps cancels to rounding
        gr = g.rms_norm_bwd(d["dy"], s_in, d["w"], out["rstd"])
        check("dx without dsum", gr["dx"], L.norm_bwd(arr(c["dy"]), arr(s), arr(c["w"]), EPS)["ds"])


def _half_step_e4m3(v):
    """Half the distance between e4m3 values around |v| (below 2^-6 they are 2^-9 apart)."""
    e = np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -6)))
    return np.exp2(e - 4)


@pytest.mark.parametrize("block", [0, 128])
@pytest.mark.parametrize("dtype,rtype", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_eight_bits(case, dtype, rtype, block):
    import gated_delta_rule_29_amd as g

    M, D, pitch = CASES[case]
    say("norm q8 M %d D %d pitch %s %s residual %s block %d" % (M, D, pitch, dtype, rtype, block))
    c, d = _inputs(M, D, pitch, dtype, rtype, 100 + case)
    out = g.rms_norm_q8_fwd(d["x"], d["w"], residual=d["residual"], eps=EPS, block=block)
    s = _sum(c)
    assert torch.equal(out["sum"].cpu(), s)
    y, _ = L.norm(arr(s), arr(c["w"]), EPS)
    scale = L.norm_scales(y, block)
    check("scale", out["scale"], scale)
    v = y / np.repeat(scale, block or D, 1)[:, :D]  # exact quotients, at most 448
    q = arr(out["q"].float())
    assert np.abs(q).max() <= 448
    # nearest value, up to the fp32 roundings of y and the scale (16 u of the quotient)
    assert (np.abs(q - v) <= _half_step_e4m3(np.maximum(np.abs(q), np.abs(v))) + 16 * 2.0 ** -24 * np.abs(v)).all()


def test_eight_bits_of_zero_and_not_finite_rows():
    import gated_delta_rule_29_amd as g

    for D in (256, 1030):  # 16-byte vectors and single columns
        say("norm q8 special rows D %d" % D)
        x = torch.ones(4, D)
        x[0] = 0.0
        x[1, 5] = float("nan")
        x[2, :128] = 0.0
        for block in (0, 128):
            o = g.rms_norm_q8_fwd(x.to(DEV), torch.ones(D, device=DEV), block=block)
            q, sc = o["q"].float().cpu(), o["scale"].cpu()
            assert not q[0].any() and (sc[0] == torch.tensor(1e-12) / 448).all()
            assert q[1].isnan().all() and sc[1].isnan().all()
            assert (q[3] == 448).all() and torch.isfinite(q[2]).all()
            assert not q[2, :128].any() and (q[2, 128:] == 448).all()


def test_gradient_over_many_rows_is_deterministic():
    import gated_delta_rule_29_amd as g

    say("norm gradient of many rows")
    c, d = _inputs(5000, 96, (0, 0), "f32", "f32", 8)
    o = g.rms_norm_fwd(d["x"], d["w"], residual=d["residual"], want_rstd=True)
    a = g.rms_norm_bwd(d["dy"], o["sum"], d["w"], o["rstd"])
    b = g.rms_norm_bwd(d["dy"], o["sum"], d["w"], o["rstd"])
    ref = L.norm_bwd(arr(c["dy"]), arr(_sum(c)), arr(c["w"]), EPS)
    check("dw", a["dw"], ref["dw"])
    check("dx", a["dx"], ref["ds"])
    assert torch.equal(a["dw"], b["dw"])


@pytest.mark.parametrize("D,seam", [(513, 1 << 20), (8, 1 << 24)])
def test_more_rows_than_one_launch_takes(D, seam):
    """The rows around the seam between two launches are those of a call on them alone, bit for bit."""
    import gated_delta_rule_29_amd as g

    say("norm rows around %d, D %d" % (seam, D))
    M, part = seam + 5, slice(seam - 3, seam + 5)
    x = torch.randn(M, D, device=DEV, dtype=torch.bfloat16)
    w = torch.rand(D, device=DEV) + 0.5
    for call, kw in ((g.rms_norm_fwd, dict(want_rstd=True)), (g.rms_norm_q8_fwd, {}), (g.rms_norm_q8_fwd, dict(block=128))):
        full, alone = call(x, w, residual=x, **kw), call(x[part], w, residual=x[part], **kw)
        for k in alone:
            a, b = full[k][part], alone[k]
            if k == "q":
                a, b = a.view(torch.uint8), b.view(torch.uint8)
            assert torch.equal(a, b), (call.__name__, k)


def _e4m3_midpoints():
    """Every value half way between two neighbouring e4m3 values (0 .. 448)."""
    v = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    return (v[1:] + v[:-1]) / 2


@pytest.mark.parametrize("block", [0, 128])
@pytest.mark.parametrize("D", [256, 250, 1030])  # 16-byte vectors, single columns in one wave and in many
def test_eight_bits_round_the_quotient(D, block):
    """Values whose quotient by the scale is half way between two e4m3 values, or next to it: q is e4m3 of the
    fp32 quotient y / scale, bit for bit.  (Rows of ones with an eps that adds nothing: y is w.)"""
    import gated_delta_rule_29_amd as g

    say("norm q8 of midpoints D %d block %d" % (D, block))
    mid, r = _e4m3_midpoints(), gen(D + block)
    for _ in range(8):
        largest = 1 + torch.rand(1, generator=r)
        s = largest / 448  # fp32, as the scale is formed
        w = (mid[torch.randint(mid.numel(), (D,), generator=r)] * s.double()).float()
        w *= torch.randint(0, 2, (D,), generator=r) * 2 - 1
        w[::128] = largest
        o = g.rms_norm_q8_fwd(torch.ones(2, D, device=DEV), w.to(DEV), eps=1e-30, block=block)
        assert (o["scale"].cpu() == s).all()
        assert torch.equal(o["q"].cpu().view(torch.uint8), (w / s).to(torch.float8_e4m3fn).view(torch.uint8).expand(2, D))


@pytest.mark.parametrize("D,M", [(16, 1 << 24), (15, 1 << 24), (520, 1 << 22)])
def test_weight_gradient_of_many_equal_terms(D, M):
    """4096 rows a worker, all alike: dw's terms have one sign, and a running fp32 sum of 4096 of them loses
    up to 2048 u.  Here 64 terms meet in a register and 64 of their sums after that, (64 + 64) / 2 u; the
    workers' shares are added in 64 bits, and rstd and a term are off by 4 u."""
    import gated_delta_rule_29_amd as g

    say("norm: sums of equal terms, %d rows of %d" % (M, D))
    dy = 1 + torch.rand(D, generator=gen(D))
    s = torch.ones(M, D, device=DEV)
    rstd = g.rms_norm_fwd(s, torch.ones(D, device=DEV), want_rstd=True)["rstd"]
    o = g.rms_norm_bwd(dy.to(DEV).expand(M, D).contiguous(), s, torch.ones(D, device=DEV), rstd)
    ref = M * dy.double() / (1 + EPS) ** 0.5
    err = float(((o["dw"].cpu().double() - ref).abs() / ref).max()) * 2 ** 24
    say("  error %.1f u" % err)
    assert err <= 68
