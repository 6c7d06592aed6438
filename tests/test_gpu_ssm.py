"""GPU parity of the selective scan, its gradient and its single-token form against the fp64 oracle."""
import numpy as np
import pytest
import torch

from oracle import layer as L
from tests.gpu_util import say
from tests.layer_util import DEV, TYPES, arr, check, flat, gen, pitched, rn, rows

pytestmark = pytest.mark.gpu

# lengths, dense, channels, states, (extra columns, offset) of the rows, everything given
CASES = [
    ([1], True, 1, 1, (0, 0), True),
    ([1, 1], True, 16, 16, (0, 0), False),
    ([31, 32, 33, 1, 64], False, 70, 16, (0, 0), True),       # chunk borders
    ([40, 40, 40], True, 65, 3, (7, 5), True),                # nothing aligned
    ([100, 5], False, 33, 17, (0, 0), True),
    ([70], True, 20, 32, (8, 8), False),
    ([65, 2, 30], False, 18, 40, (1, 1), True),
    ([90, 90], True, 9, 64, (0, 0), True),
    ([700, 3, 129, 260], False, 64, 16, (16, 0), True),       # cut into segments
    ([1500], True, 24, 5, (0, 0), True),                      # cut, one sequence
    ([333, 333], True, 12, 33, (0, 0), False),                # cut, 16 lanes a channel
    ([200], True, 1030, 16, (0, 0), True),
]


def _inputs(lens, dense, D, N, pitch, dtype, seed):
    g = gen(seed)
    lead, cu = rows(lens, dense)
    t, n = TYPES[dtype], len(lens)
    A = -torch.arange(1, N + 1).float() * torch.exp(0.3 * rn(g, D, N))
    c = dict(x=rn(g, *lead, D, dtype=t), dt=(rn(g, *lead, D) - 1.0).to(t), A=A, Bm=rn(g, *lead, N, dtype=t),
             Cm=rn(g, *lead, N, dtype=t), skip=rn(g, D), z=rn(g, *lead, D, dtype=t), dt_bias=0.5 * rn(g, D),
             h0=rn(g, n, D, N), dy=rn(g, *lead, D, dtype=t), dht=rn(g, n, D, N))
    d = {k: v.to(DEV) for k, v in c.items()}
    if pitch[0]:
        for k in ("x", "dt", "z", "Bm", "Cm", "dy"):
            d[k] = pitched(c[k], *pitch)
    return c, d, cu


def _ref(c, full):
    k = dict(x=flat(c["x"]), dt=flat(c["dt"]), A=arr(c["A"]), Bm=flat(c["Bm"]), Cm=flat(c["Cm"]))
    if full:
        k.update(skip=arr(c["skip"]), z=flat(c["z"]), dt_bias=arr(c["dt_bias"]), h0=arr(c["h0"]))
    return k


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_forward_and_gradient(case, dtype):
    import gated_delta_rule_29_amd as g

    lens, dense, D, N, pitch, full = CASES[case]
    say("scan %s dense %s D %d N %d pitch %s %s" % (lens, dense, D, N, pitch, dtype))
    c, d, cu = _inputs(lens, dense, D, N, pitch, dtype, case)
    at = () if dense else (cu,)
    fwd, bwd = (g.ssm_scan_fwd, g.ssm_scan_bwd) if dense else (g.ssm_scan_fwd_varlen, g.ssm_scan_bwd_varlen)
    args = (d["x"], d["dt"], d["A"], d["Bm"], d["Cm"], *at)
    opt = dict(D=d["skip"], z=d["z"], dt_bias=d["dt_bias"]) if full else {}
    out = fwd(*args, h0=d["h0"] if full else None, want_h=True, **opt)
    y, ht, h = L.scan(lens, chunk=g.SSM_CHUNK, **_ref(c, full))
    check("y", out["y"].reshape(-1, D), y)
    check("ht", out["ht"], ht)
    check("h", out["h"].reshape(h.shape), h) if h.any() else None
    lone = fwd(*args, h0=d["h0"] if full else None, want_ht=False, **opt)
    assert set(lone) == {"y"} and torch.equal(lone["y"], out["y"])  # saving changes no result

    say("gradient")
    gr = bwd(d["dy"], out["h"], *args, dht=d["dht"] if full else None, want_dh0=True, **opt)
    ref = L.scan_bwd(lens, flat(c["dy"]), dht=arr(c["dht"]) if full else None, **_ref(c, full))
    assert set(gr) == {"dx", "ddt", "dA", "dB", "dC", "dh0"} | ({"dD", "dz", "ddt_bias"} if full else set())
    for k in gr:
        check(k, gr[k].reshape(ref[k].shape), ref[k])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_plain_step_sizes(dtype):
    """softplus off: step sizes as they are, none (0) among them."""
    import gated_delta_rule_29_amd as g

    say("scan without softplus %s" % dtype)
    c, d, _ = _inputs([50, 50], True, 34, 16, (0, 0), dtype, 77)
    for k in (c, d):
        k["dt"] = torch.clamp(k["dt"], min=0.0)
    args = (d["x"], d["dt"], d["A"], d["Bm"], d["Cm"])
    out = g.ssm_scan_fwd(*args, softplus=False, want_h=True)
    ref = _ref(c, False)
    y, ht, _ = L.scan([50, 50], use_softplus=False, **ref)
    check("y", out["y"].reshape(-1, 34), y)
    check("ht", out["ht"], ht)
    gr = g.ssm_scan_bwd(d["dy"], out["h"], *args, softplus=False)
    rg = L.scan_bwd([50, 50], flat(c["dy"]), use_softplus=False, **ref)
    for k in gr:
        check(k, gr[k].reshape(rg[k].shape), rg[k])


def test_extreme_step_sizes():
    """Steps that keep everything (softplus of -inf and of very negative values) and steps that forget
    everything, in turn: no overflow, and the tokens that keep everything leave the state bit for bit."""
    import gated_delta_rule_29_amd as g

    say("scan with extreme step sizes")
    c, d, _ = _inputs([48], True, 16, 16, (0, 0), "f32", 3)
    for k in (c, d):
        k["dt"][0, ::3] = 300.0
        k["dt"][0, 1::3] = -200.0
        k["dt"][0, 2::6] = -float("inf")
    out = g.ssm_scan_fwd(d["x"], d["dt"], d["A"], d["Bm"], d["Cm"], want_h=True)
    y, ht, _ = L.scan([48], **_ref(c, False))
    check("y", out["y"].reshape(-1, 16), y)
    keep = torch.full_like(d["dt"], -float("inf"))
    out = g.ssm_scan_fwd(d["x"], keep, d["A"], d["Bm"], d["Cm"], h0=d["h0"])
    assert torch.equal(out["ht"], d["h0"])
    c["dt"] = torch.full_like(c["dt"], -200.0)
    d["dt"] = c["dt"].to(DEV)
    o = g.ssm_scan_fwd(d["x"], d["dt"], d["A"], d["Bm"], d["Cm"], h0=d["h0"], want_h=True)
    gr = g.ssm_scan_bwd(d["dy"], o["h"], d["x"], d["dt"], d["A"], d["Bm"], d["Cm"], dht=d["dht"], want_dh0=True)
    assert all(torch.isfinite(v).all() for v in gr.values())
    ref = dict(_ref(c, False), h0=arr(c["h0"]))
    rg = L.scan_bwd([48], flat(c["dy"]), dht=arr(c["dht"]), **ref)
    check("dh0", gr["dh0"], rg["dh0"])
    check("dC", gr["dC"].reshape(-1, 16), rg["dC"])


def test_gradient_against_differences():
    """Directional derivatives of the GPU forward itself (fp32): for a direction v the change of the loss
    over 2 eps is sum grad . v up to eps^2 and the forward's rounding, about 1e-6 |y| |dy| / eps."""
    import gated_delta_rule_29_amd as g

    say("scan gradient against differences")
    c, d, _ = _inputs([70, 70], True, 40, 16, (0, 0), "f32", 9)
    names = ("x", "dt", "A", "Bm", "Cm", "skip", "z", "dt_bias", "h0")

    def loss(**k):
        o = g.ssm_scan_fwd(k["x"], k["dt"], k["A"], k["Bm"], k["Cm"], D=k["skip"], z=k["z"], dt_bias=k["dt_bias"],
                           h0=k["h0"])
        return float((o["y"].double() * d["dy"].double()).sum() + (o["ht"].double() * d["dht"].double()).sum())

    k = {n: d[n] for n in names}
    o = g.ssm_scan_fwd(k["x"], k["dt"], k["A"], k["Bm"], k["Cm"], D=k["skip"], z=k["z"], dt_bias=k["dt_bias"],
                       h0=k["h0"], want_h=True)
    gr = g.ssm_scan_bwd(d["dy"], o["h"], k["x"], k["dt"], k["A"], k["Bm"], k["Cm"], D=k["skip"], z=k["z"],
                        dt_bias=k["dt_bias"], dht=d["dht"], want_dh0=True)
    of = dict(x="dx", dt="ddt", A="dA", Bm="dB", Cm="dC", skip="dD", z="dz", dt_bias="ddt_bias", h0="dh0")
    eps = 2e-3
    for n in names:
        v = torch.sign(gr[of[n]])  # every entry pushes the loss the same way: no cancellation
        num = (loss(**{**k, n: k[n] + eps * v}) - loss(**{**k, n: k[n] - eps * v})) / (2 * eps)
        ana = float((gr[of[n]].double() * v.double()).sum())
        say("  %-8s %.6e %.6e" % (n, num, ana))
        assert abs(num - ana) <= 1e-2 * abs(ana), n


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,N,pitch,full", [(64, 16, (0, 0), True), (70, 5, (3, 1), True), (9, 64, (0, 0), False),
                                            (1000, 24, (8, 8), True), (1, 1, (0, 0), True)])
def test_step(D, N, pitch, full, dtype):
    """Rows in slots of any order, padded rows, a slot named twice, a slot outside the cache."""
    import gated_delta_rule_29_amd as g

    say("scan step D %d N %d pitch %s %s" % (D, N, pitch, dtype))
    slots = [3, -1, 0, 3, 7, 9, 5, -7, 0]
    S, B, live = 9, 9, [0, 2, 4, 6]
    c, d, _ = _inputs([1] * B, True, D, N, pitch, dtype, D + N)
    st = rn(gen(N), S, D, N)
    state = st.to(DEV)
    row = {k: d[k][:, 0] for k in ("x", "dt", "Bm", "Cm", "z")}
    opt = dict(D=d["skip"], z=row["z"], dt_bias=d["dt_bias"]) if full else {}
    args = (row["x"], row["dt"], d["A"], row["Bm"], row["Cm"])
    y = g.ssm_step(*args, state, slots=torch.tensor(slots, dtype=torch.int32, device=DEV), **opt)
    want, ref_y = arr(st), np.zeros((B, D))
    for b in live:
        one = {k: flat(c[k][b]) for k in ("x", "dt", "Bm", "Cm")}
        if full:
            one.update(skip=arr(c["skip"]), z=flat(c["z"][b]), dt_bias=arr(c["dt_bias"]))
        o, ht, _ = L.scan([1], A=arr(c["A"]), h0=arr(st[slots[b]])[None], **one)
        ref_y[b], want[slots[b]] = o[0], ht[0]
    check("state", state, want)
    others = [s for s in range(S) if s not in (3, 0, 7, 5)]
    assert torch.equal(state.cpu()[others], st[others])
    check("y", y, ref_y)
    assert not y[[1, 3, 5, 7, 8]].any()


def test_split_sequences_agree_with_whole_ones():
    """The same tokens as one long sequence (cut into segments by the library) and as calls that are
    each too short to be cut: equal up to fp32 rounding."""
    import gated_delta_rule_29_amd as g

    say("scan: cut and uncut")
    c, d, _ = _inputs([1024], True, 32, 16, (0, 0), "f32", 4)
    whole = g.ssm_scan_fwd(d["x"], d["dt"], d["A"], d["Bm"], d["Cm"], h0=d["h0"])
    h, ys = d["h0"], []
    for t in range(0, 1024, 64):
        o = g.ssm_scan_fwd(*(d[k][:, t:t + 64].contiguous() if k != "A" else d[k] for k in ("x", "dt", "A", "Bm", "Cm")),
                           h0=h)
        ys.append(o["y"])
        h = o["ht"]
    check("y", whole["y"][0], arr(torch.cat(ys, 1)[0]))
    check("ht", whole["ht"], arr(h))
