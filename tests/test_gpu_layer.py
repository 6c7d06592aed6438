"""The layer operators run together as a recurrent layer uses them: a prompt in one piece, in pieces and
token by token on the caches; a training step's gradients; captured graphs and other streams."""
import pytest
import torch

from oracle import layer as L
from tests.gpu_util import say
from tests.layer_util import DEV, TYPES, arr, check, flat, gen, rn

pytestmark = pytest.mark.gpu


class Layer:
    """norm(+residual) -> in-projection -> convolution -> projection of dt, B, C -> gated scan."""

    def __init__(self, H, C, N, dtype, seed):
        g = gen(seed)
        self.t, self.H, self.C, self.N, self.R = TYPES[dtype], H, C, N, 5
        self.norm_w = (1 + 0.1 * rn(g, H)).to(DEV)
        self.w_in = (rn(g, H, 2 * C) / H ** 0.5).to(self.t).to(DEV)
        self.w_conv, self.b_conv = rn(g, C, 4).to(DEV), (0.1 * rn(g, C)).to(DEV)
        self.w_bc = (rn(g, C, self.R + 2 * N) / C ** 0.5).to(self.t).to(DEV)
        self.w_dt = (rn(g, self.R, C) / self.R ** 0.5).to(self.t).to(DEV)
        self.A = -torch.arange(1, N + 1).float().repeat(C, 1).to(DEV)
        self.D, self.dt_bias = torch.ones(C, device=DEV), (rn(g, C) - 2).to(DEV)

    def project(self, g, x, residual):
        n = g.rms_norm_fwd(x, self.norm_w, residual=residual)
        xz = n["y"] @ self.w_in
        return xz[..., :self.C], xz[..., self.C:]  # columns of one tensor, read in place

    def steps(self, u):
        p = u @ self.w_bc
        R, N = self.R, self.N
        return p[..., :R] @ self.w_dt, p[..., R:R + N], p[..., R + N:]

    def prompt(self, g, x, residual, init=None, h0=None):
        xc, z = self.project(g, x, residual)
        c = g.causal_conv_fwd(xc, self.w_conv, self.b_conv, init)
        dt, Bm, Cm = self.steps(c["y"])
        o = g.ssm_scan_fwd(c["y"], dt, self.A, Bm, Cm, D=self.D, z=z, dt_bias=self.dt_bias, h0=h0)
        return o["y"], c["final"], o["ht"]

    def token(self, g, x, residual, conv_state, ssm_state, slots):
        xc, z = self.project(g, x, residual)
        u = g.causal_conv_step(xc, self.w_conv, conv_state, self.b_conv, slots=slots)
        dt, Bm, Cm = self.steps(u)
        return g.ssm_step(u, dt, self.A, Bm, Cm, ssm_state, D=self.D, z=z, dt_bias=self.dt_bias, slots=slots)


def test_prompt_pieces_and_tokens():
    """fp32: the whole prompt, the prompt in two pieces, and its last tokens one by one from the caches
    agree.  The projections' products may be summed in another order for other row counts, which is
    within the tolerance's count of roundings."""
    import gated_delta_rule_29_amd as g

    say("layer: prompt, pieces, tokens")
    ly, r = Layer(48, 80, 16, "f32", 1), gen(2)
    B, T, cut = 3, 45, 33
    x, res = rn(r, B, T, 48).to(DEV), rn(r, B, T, 48).to(DEV)
    y, conv, state = ly.prompt(g, x, res)
    a, ca, sa = ly.prompt(g, x[:, :cut].contiguous(), res[:, :cut].contiguous())
    b, cb, sb = ly.prompt(g, x[:, cut:].contiguous(), res[:, cut:].contiguous(), ca, sa)
    check("pieces", torch.cat([a, b], 1), arr(y))
    check("state", sb, arr(state))
    check("window", cb, arr(conv))
    # caches of more slots than rows; the rows' slots in another order
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device=DEV)
    cc, ss = torch.full((6, 3, 80), 7.0, device=DEV), torch.full((6, 80, 16), 7.0, device=DEV)
    cc[slots.long()], ss[slots.long()] = ca, sa
    for t in range(cut, T):
        yt = ly.token(g, x[:, t], res[:, t], cc, ss, slots)
        check("token %d" % t, yt, arr(y[:, t]))
    check("state", ss[slots.long()], arr(state))
    check("window", cc[slots.long()], arr(conv))
    assert (cc[[1, 3, 5]] == 7).all() and (ss[[1, 3, 5]] == 7).all()


def test_training_step():
    """fp32: the layer's gradients, operator by operator backwards, against the oracle's chained the
    same way in fp64, with the projections left out (the conv feeds the scan's x directly)."""
    import gated_delta_rule_29_amd as g

    say("layer: training step")
    r, lens, C, N = gen(3), [50, 50], 40, 16
    x, w, b, nw = rn(r, 2, 50, C), rn(r, C, 4), rn(r, C), 1 + 0.1 * rn(r, C)
    res, dy = rn(r, 2, 50, C), rn(r, 2, 50, C)
    dt, Bm, Cm, A = rn(r, 2, 50, C) - 2, rn(r, 2, 50, N), rn(r, 2, 50, N), -torch.arange(1, N + 1).float().repeat(C, 1)
    d = lambda t: t.to(DEV)  # noqa: E731
    n = g.rms_norm_fwd(d(x), d(nw), residual=d(res), want_rstd=True)
    c = g.causal_conv_fwd(n["y"], d(w), d(b))
    o = g.ssm_scan_fwd(c["y"], d(dt), d(A), d(Bm), d(Cm), z=n["y"], want_h=True)
    gs = g.ssm_scan_bwd(d(dy), o["h"], c["y"], d(dt), d(A), d(Bm), d(Cm), z=n["y"])
    gc = g.causal_conv_bwd(gs["dx"], n["y"], d(w), d(b))
    gn = g.rms_norm_bwd(gc["dx"] + gs["dz"], n["sum"], d(nw), n["rstd"])

    s = (x + res).reshape(-1, C).double().numpy()
    y0, _ = L.norm(s, arr(nw), 1e-5)
    u, _ = L.conv(lens, y0, arr(w), arr(b))
    k = dict(x=u, dt=flat(dt), A=arr(A), Bm=flat(Bm), Cm=flat(Cm), z=y0)
    check("y", o["y"].reshape(-1, C), L.scan(lens, **k)[0])
    rs = L.scan_bwd(lens, flat(dy), **k)
    rc = L.conv_bwd(lens, rs["dx"], y0, arr(w), arr(b))
    rn_ = L.norm_bwd(rc["dx"] + rs["dz"], s, arr(nw), 1e-5)
    # three operators in a row: three times one operator's tolerance
    for name, got, ref in (("dA", gs["dA"], rs["dA"]), ("dw", gc["dw"], rc["dw"]), ("dx", gn["dx"], rn_["ds"]),
                           ("dnorm", gn["dw"], rn_["dw"])):
        check(name, got.reshape(ref.shape), ref, 6e-5)


def _all(g, seed):
    """Every operator once, as a list of (name, call); steps work on copies of their caches."""
    r = gen(seed)
    C, N, t = 72, 16, torch.bfloat16
    d = lambda *s: rn(r, *s).to(t).to(DEV)  # noqa: E731
    x, z, dt, Bm, Cm = d(1, 600, C), d(1, 600, C), d(1, 600, C), d(1, 600, N), d(1, 600, N)
    A = -torch.arange(1, N + 1).float().repeat(C, 1).to(DEV)
    w, nw = rn(r, C, 4).to(DEV), torch.ones(C, device=DEV)
    cu_h = torch.tensor([0, 7, 500, 600], dtype=torch.int32)
    cu = cu_h.to(DEV)
    slots = torch.tensor([2, -1, 0], dtype=torch.int32, device=DEV)
    cs, ss = d(4, 3, C), rn(r, 4, C, N).to(DEV)
    h = g.ssm_scan_fwd_varlen(x, dt, A, Bm, Cm, cu, z=z, want_h=True, cu_seqlens_host=cu_h)["h"]
    rstd = g.rms_norm_fwd(x, nw, want_rstd=True)["rstd"]

    def conv_step():
        st = cs.clone()
        return {"y": g.causal_conv_step(x[0, :3], w, st, slots=slots), "state": st}

    def ssm_step():
        st = ss.clone()
        return {"y": g.ssm_step(x[0, :3], dt[0, :3], A, Bm[0, :3], Cm[0, :3], st, z=z[0, :3], slots=slots), "state": st}

    return [("conv", lambda: g.causal_conv_fwd_varlen(x, w, cu, cu_seqlens_host=cu_h)),
            ("conv gradient", lambda: g.causal_conv_bwd_varlen(z, x, w, cu, cu_seqlens_host=cu_h)),
            ("conv step", conv_step), ("scan step", ssm_step),
            ("scan", lambda: g.ssm_scan_fwd_varlen(x, dt, A, Bm, Cm, cu, z=z, want_h=True, cu_seqlens_host=cu_h)),
            ("scan gradient", lambda: g.ssm_scan_bwd_varlen(z, h, x, dt, A, Bm, Cm, cu, z=z, cu_seqlens_host=cu_h)),
            ("norm", lambda: g.rms_norm_fwd(x, nw, residual=z)),
            ("norm 8 bits", lambda: g.rms_norm_q8_fwd(x, nw, residual=z, block=128)),
            ("norm gradient", lambda: g.rms_norm_bwd(z, x, nw, rstd))]


def _same(a, b):
    for k in a:
        u, v = (t[k].view(torch.uint8) if t[k].dtype == torch.float8_e4m3fn else t[k] for t in (a, b))
        assert torch.equal(u, v), k


def test_captured_calls():
    """Every operator captured; two graphs replayed in turn with eager work between, several times."""
    import gated_delta_rule_29_amd as g

    for (name, call), (_, other) in zip(_all(g, 4), _all(g, 5)):
        say("captured: " + name)
        want, want2 = call(), other()
        want, want2 = ({k: v.clone() for k, v in o.items()} for o in (want, want2))
        torch.cuda.synchronize()
        graphs = []
        for f in (call, other):
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr):
                out = f()
            graphs.append((gr, out))
        for _ in range(3):
            for (gr, out), ref in zip(graphs, (want, want2)):
                gr.replay()
                torch.cuda.synchronize()
                _same(out, ref)
            _same(other(), want2)
            torch.cuda.synchronize()


def test_two_streams_at_once():
    """Calls on two streams at once have workspaces of their own."""
    import gated_delta_rule_29_amd as g

    a, b = _all(g, 6), _all(g, 7)
    want = [[{k: v.clone() for k, v in f().items()} for _, f in c] for c in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    say("two streams")
    got = [[], []]
    for i in range(len(a)):
        for k, c in enumerate((a, b)):
            with torch.cuda.stream(streams[k]):
                got[k].append(c[i][1]())
    torch.cuda.synchronize()
    for k in range(2):
        for o, ref in zip(got[k], want[k]):
            _same(o, ref)
