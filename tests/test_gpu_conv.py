"""GPU parity of the short causal convolution, its gradient and its single-token form against the fp64
oracle."""
import pytest
import torch

from oracle import layer as L
from tests.gpu_util import say
from tests.layer_util import DEV, TYPES, arr, check, flat, gen, pitched, rn, rows

pytestmark = pytest.mark.gpu

# lengths, dense, D, W, (extra columns, offset) of the rows
CASES = [
    ([1], True, 8, 4, (0, 0)),
    ([1, 1, 1], True, 1, 2, (0, 0)),
    ([2, 1, 3, 64, 65, 5], False, 40, 4, (0, 0)),       # shorter than the window, across tiles
    ([130, 130], True, 72, 3, (8, 8)),                  # aligned columns of a wider tensor
    ([33, 200, 1], False, 70, 4, (5, 3)),               # nothing aligned
    ([16, 48, 63, 1, 1, 1, 1, 129], False, 264, 2, (264, 264)),
    ([300], True, 513, 4, (1, 0)),
    ([1000, 24], False, 2056, 4, (0, 0)),
    ([1, 2] * 600, False, 12, 3, (0, 0)),               # more sequences than are looked up in LDS
]


def _inputs(lens, dense, D, W, pitch, dtype, seed):
    g = gen(seed)
    lead, cu = rows(lens, dense)
    t = TYPES[dtype]
    c = dict(x=rn(g, *lead, D, dtype=t), w=rn(g, D, W), bias=rn(g, D), init=rn(g, len(lens), W - 1, D, dtype=t),
             dy=rn(g, *lead, D, dtype=t), dl=rn(g, len(lens), W - 1, D, dtype=t))
    d = {k: v.to(DEV) for k, v in c.items()}
    if pitch[0]:
        d["x"], d["dy"] = pitched(c["x"], *pitch), pitched(c["dy"], *pitch)
    return c, d, cu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_forward_and_gradient(case, dtype):
    import gated_delta_rule_29_amd as g

    lens, dense, D, W, pitch = CASES[case]
    say("conv %s dense %s D %d W %d pitch %s %s" % (lens, dense, D, W, pitch, dtype))
    c, d, cu = _inputs(lens, dense, D, W, pitch, dtype, case)
    at = () if dense else (cu,)
    fwd, bwd = (g.causal_conv_fwd, g.causal_conv_bwd) if dense else (g.causal_conv_fwd_varlen, g.causal_conv_bwd_varlen)
    for silu, full in ((True, True), (False, False)):
        opt = dict(bias=d["bias"], init=d["init"]) if full else {}
        ref = dict(bias=arr(c["bias"]), init=arr(c["init"])) if full else {}
        out = fwd(d["x"], d["w"], *at, silu=silu, **opt)
        y, last = L.conv(lens, flat(c["x"]), arr(c["w"]), silu=silu, **ref)
        check("y", out["y"].reshape(-1, D), y)
        assert torch.equal(out["final"].cpu().double(), torch.from_numpy(last))
        gr = bwd(d["dy"], d["x"], d["w"], *at, silu=silu, dfinal=d["dl"] if full else None, **opt)
        rg = L.conv_bwd(lens, flat(c["dy"]), flat(c["x"]), arr(c["w"]), silu=silu,
                        dlast=arr(c["dl"]) if full else None, **ref)
        check("dx", gr["dx"].reshape(-1, D), rg["dx"])
        check("dw", gr["dw"], rg["dw"])
        assert set(gr) == ({"dx", "dw", "dbias", "dinit"} if full else {"dx", "dw"})
        if full:
            check("dbias", gr["dbias"], rg["dbias"])
            check("dinit", gr["dinit"], rg["dinit"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_tiles_of_one_filter(dtype):
    """Weight gradients over many tiles; dense and packed agree bit for bit."""
    import gated_delta_rule_29_amd as g

    say("conv many tiles %s" % dtype)
    lens = [700] * 3
    c, d, _ = _inputs(lens, True, 24, 4, (0, 0), dtype, 5)
    out = g.causal_conv_bwd(d["dy"], d["x"], d["w"], bias=d["bias"], init=d["init"])
    ref = L.conv_bwd(lens, flat(c["dy"]), flat(c["x"]), arr(c["w"]), arr(c["bias"]), arr(c["init"]))
    for k in out:
        check(k, out[k].reshape(ref[k].shape), ref[k])
    cu = torch.arange(0, 2101, 700, dtype=torch.int32)
    one = {k: d[k].reshape(1, -1, 24) for k in ("x", "dy")}
    packed = g.causal_conv_bwd_varlen(one["dy"], one["x"], d["w"], cu, bias=d["bias"], init=d["init"])
    for k in out:
        assert torch.equal(out[k].reshape(-1), packed[k].reshape(-1)), k


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,W,pitch", [(64, 4, (0, 0)), (70, 3, (3, 1)), (2064, 2, (2064, 0)), (1, 4, (0, 0))])
def test_step(D, W, pitch, dtype):
    """Rows in slots of any order, padded rows, a slot named twice, a slot outside the cache."""
    import gated_delta_rule_29_amd as g

    say("conv step D %d W %d pitch %s %s" % (D, W, pitch, dtype))
    r, t = gen(D + W), TYPES[dtype]
    slots = [3, -1, 0, 3, 7, 9, 5, -7, 0]
    S, B = 9, len(slots)
    x, w, bias, st = rn(r, B, D, dtype=t), rn(r, D, W), rn(r, D), rn(r, S, W - 1, D, dtype=t)
    xd = pitched(x, *pitch) if pitch[0] else x.to(DEV)
    state = st.to(DEV)
    y = g.causal_conv_step(xd, w.to(DEV), state, bias.to(DEV), slots=torch.tensor(slots, dtype=torch.int32, device=DEV))
    want, ref_y, live = st.clone(), torch.zeros(B, D, dtype=torch.float64), [0, 2, 4, 6]
    for b in live:
        o, last = L.conv([1], flat(x[b:b + 1]), arr(w), arr(bias), arr(st[slots[b]])[None])
        ref_y[b], want[slots[b]] = torch.from_numpy(o[0]), torch.from_numpy(last[0]).to(t)
    assert torch.equal(state.cpu(), want)
    check("y", y, ref_y.numpy())
    assert not y[[1, 3, 5, 7, 8]].any()
    # without slots: row b has slot b; slots behind the last row stay as they are
    state = st.to(DEV)
    g.causal_conv_step(xd[:2], w.to(DEV), state)
    assert torch.equal(state.cpu()[2:], st[2:]) and torch.equal(state.cpu()[1, -1], x[1])


def test_weight_sums_of_many_equal_terms():
    """2^24 tokens of one value a channel: a running fp32 sum of that many equal terms loses up to 2^13 u
    (u = 2^-24: each addition is off by half a unit of the sum so far).  A tile's 64 terms of 16 bits
    add up exactly and the tiles' shares are added in 64 bits, so the result is off by its own rounding."""
    import gated_delta_rule_29_amd as g

    say("conv: sums of 2^24 equal terms")
    T, D, r = 1 << 24, 16, gen(41)
    x, dy = ((1 + torch.rand(D, generator=r)).bfloat16() for _ in range(2))
    o = g.causal_conv_bwd(dy.to(DEV).expand(1, T, D).contiguous(), x.to(DEV).expand(1, T, D).contiguous(),
                          torch.zeros(D, 4, device=DEV), bias=torch.zeros(D, device=DEV), silu=False)
    terms = T - 3 + torch.arange(4.0, dtype=torch.float64)  # (the first tokens' windows begin with zeros)
    for k, ref in (("dbias", T * dy.double()), ("dw", (x.double() * dy.double())[:, None] * terms)):
        err = float(((o[k].cpu().double() - ref).abs() / ref).max()) * 2 ** 24
        say("  %s error %.1f u" % (k, err))
        assert err <= 2
