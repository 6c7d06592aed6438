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


def test_nothing_outside_the_rows():
    """Through the C ABI: input rows behind the last sequence hold NaN and are not read, output rows behind
    it are left as they were.  (37 tokens of 64 rows; the last chunk and tile end inside.)"""
    import gated_delta_rule_29_amd as g
    from gated_delta_rule_29_amd import _lib

    say("guard rows")
    lib, r, C, N, T, R = _lib.load(), gen(8), 72, 16, 37, 64
    st = torch.cuda.current_stream().cuda_stream

    def rows(width):
        t = torch.full((R, width), float("nan"))
        t[:T] = rn(r, T, width)
        return t.to(DEV)

    def out(*shape, dtype=torch.float32):
        return torch.full(shape, 7.0, device=DEV).to(dtype)

    x, z, dt, dy, Bm, Cm = rows(C), rows(C), rows(C), rows(C), rows(N), rows(N)
    A, w = -torch.arange(1, N + 1).float().repeat(C, 1).to(DEV), rn(r, C, 4).to(DEV)
    cu_h = torch.tensor([0, 20, T], dtype=torch.int32)
    cu = cu_h.to(DEV)
    p = lambda t: t.data_ptr()  # noqa: E731
    y, last = out(R, C), out(3, 3, C)
    assert lib.causal_conv_fwd_varlen(p(x), C, p(w), None, p(cu), p(cu_h), 2, None, p(y), p(last), T, C, 4, 1, 0, st) == 0
    dx, dw = out(R, C), out(C, 4)
    n = lib.causal_conv_bwd_workspace_bytes(T, C, 4)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    assert lib.causal_conv_bwd_varlen(p(dy), C, p(x), C, p(w), None, p(cu), p(cu_h), 2, None, None, p(dx), None, p(dw),
                                      None, T, C, 4, 1, 0, p(ws), n, st) == 0
    ys, ht, h = out(R, C), out(3, C, N), out(5, C, N)  # 2 + 2 chunks
    assert lib.ssm_scan_fwd_varlen(p(x), C, p(dt), C, p(A), p(Bm), N, p(Cm), N, p(cu), p(cu_h), 2, None, p(z), C, None,
                                   None, p(ys), p(ht), p(h), T, C, N, 1, 0, None, 0, st) == 0
    g5 = [out(R, C) for _ in range(3)] + [out(R, N), out(R, N), out(C, N)]
    n = lib.ssm_scan_bwd_varlen_workspace_bytes(p(cu_h), 2, C, N)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    assert lib.ssm_scan_bwd_varlen(p(dy), C, p(h), p(x), C, p(dt), C, p(A), p(Bm), N, p(Cm), N, p(cu), p(cu_h), 2, None,
                                   p(z), C, None, None, p(g5[0]), p(g5[1]), p(g5[5]), p(g5[3]), p(g5[4]), None, p(g5[2]),
                                   None, None, T, C, N, 1, 0, p(ws), n, st) == 0
    yn, sm, dn = out(R, C), out(R, C), out(R, C)
    nw, rstd, dnw = torch.ones(C, device=DEV), out(R), out(C)
    assert lib.rms_norm_fwd(p(x), C, p(z), C, p(nw), 1e-5, p(yn), p(sm), p(rstd), T, C, 0, 0, st) == 0
    n = lib.rms_norm_bwd_workspace_bytes(T, C)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    assert lib.rms_norm_bwd(p(dy), C, p(sm), C, p(nw), p(rstd), None, 0, p(dn), None, p(dnw), T, C, 0, 0, p(ws), n, st) == 0
    torch.cuda.synchronize()
    for t in (y, dx, ys, *g5[:5], yn, sm, dn, rstd):
        assert torch.isfinite(t[:T]).all() and (t[T:] == 7).all()
    for t, k in ((last, 2), (ht, 2), (h, 4)):
        assert torch.isfinite(t[:k]).all() and (t[k:] == 7).all()
    assert torch.isfinite(dw).all() and torch.isfinite(g5[5]).all() and torch.isfinite(dnw).all()
    # and the same through the binding
    one = lambda t: t[None, :T]  # noqa: E731
    o = g.ssm_scan_fwd_varlen(one(x), one(dt), A, one(Bm), one(Cm), cu, z=one(z), cu_seqlens_host=cu_h)
    assert torch.equal(o["y"][0], ys[:T])


def test_offsets_past_32_bits():
    """Rows 2^20 elements apart: more than 2^31 elements, and more than 2^32 bytes, from first to last; a
    cache of more than 2^32 bytes.  Equal to the same rows side by side."""
    import gated_delta_rule_29_amd as g

    say("offsets past 32 bits")
    T, C, N, t = 2200, 64, 16, torch.bfloat16
    r = gen(12)
    wide = torch.empty(T, 1 << 20, dtype=t, device=DEV)

    def place(at, width):
        v = wide[None, :, at:at + width]
        v.copy_(rn(r, 1, T, width).to(t))
        return v, v.contiguous()

    (x, xc), (dt, dc), (z, zc), (Bm, bc), (Cm, cc), (dy, yc) = (place(0, C), place(128, C), place(304, C), place(400, N),
                                                               place(500, N), place(600, C))
    A, w = -torch.arange(1, N + 1).float().repeat(C, 1).to(DEV), rn(r, C, 4).to(DEV)
    _same(g.causal_conv_fwd(x, w), g.causal_conv_fwd(xc, w))
    _same(g.causal_conv_bwd(dy, x, w), g.causal_conv_bwd(yc, xc, w))
    a = g.ssm_scan_fwd(x, dt, A, Bm, Cm, z=z, want_h=True)
    _same(a, g.ssm_scan_fwd(xc, dc, A, bc, cc, z=zc, want_h=True))
    _same(g.ssm_scan_bwd(dy, a["h"], x, dt, A, Bm, Cm, z=z), g.ssm_scan_bwd(yc, a["h"], xc, dc, A, bc, cc, z=zc))
    nw = torch.ones(C, device=DEV)
    n = g.rms_norm_fwd(x, nw, residual=z, want_rstd=True)
    _same(n, g.rms_norm_fwd(xc, nw, residual=zc, want_rstd=True))
    _same(g.rms_norm_q8_fwd(x, nw, residual=z), g.rms_norm_q8_fwd(xc, nw, residual=zc))
    _same(g.rms_norm_bwd(dy, x, nw, n["rstd"], dsum=z), g.rms_norm_bwd(yc, xc, nw, n["rstd"], dsum=zc))
    del wide, x, dt, z, Bm, Cm, dy
    S = (1 << 32) // (C * N * 4) + 5
    state, small = torch.zeros(S, C, N, device=DEV), rn(r, 2, C, N).to(DEV)
    slots = torch.tensor([S - 1, 1], dtype=torch.int32, device=DEV)
    state[slots.long()] = small
    row = [v[0, :2] for v in (xc, dc)]
    y0 = g.ssm_step(*row, A, bc[0, :2], cc[0, :2], small)
    y1 = g.ssm_step(*row, A, bc[0, :2], cc[0, :2], state, slots=slots)
    assert torch.equal(y0, y1) and torch.equal(state[slots.long()], small)


def test_device_offsets_that_are_not_the_hosts():
    """Against the contract: offsets on the device that give other pieces than the host's.  Results are then
    not defined, but what the call was sized for is not left (rows behind the outputs stay)."""
    from gated_delta_rule_29_amd import _lib

    say("device offsets differ from the host's")
    lib, r, C, N, T = _lib.load(), gen(9), 32, 16, 600
    st, p = torch.cuda.current_stream().cuda_stream, lambda t: t.data_ptr()  # noqa: E731
    x, bc = rn(r, T, C).to(DEV), rn(r, T, N).to(DEV)
    A, w = -torch.ones(C, N, device=DEV), rn(r, C, 4).to(DEV)
    host = torch.tensor([0, 300, 596, 600], dtype=torch.int32)
    for bad in ([0, 1, 2, 600], [0, 17, 18, 600], [-5, 900, 10, 2000], [300, 200, 100, 0], [0, 0, 0, 600]):
        cu = torch.tensor(bad, dtype=torch.int32, device=DEV)
        chunks = lib.ssm_scan_num_chunks(p(host), 3)
        full = lambda *s: torch.full(s, 7.0, device=DEV)  # noqa: E731
        y, ht, h, last = full(T + 16, C), full(3 + 1, C, N), full(chunks + 4, C, N), full(4, 3, C)
        n = lib.ssm_scan_fwd_varlen_workspace_bytes(p(host), 3, C, N)
        ws = full(n // 4 + 4096)
        assert lib.ssm_scan_fwd_varlen(p(x), C, p(x), C, p(A), p(bc), N, p(bc), N, p(cu), p(host), 3, None, None, 0, None,
                                       None, p(y), p(ht), p(h), T, C, N, 1, 0, p(ws), n, st) == 0
        torch.cuda.synchronize()
        assert (ws[n // 4:] == 7).all() and (h[chunks:] == 7).all()
        n = lib.ssm_scan_bwd_varlen_workspace_bytes(p(host), 3, C, N)
        ws = full(n // 4 + 4096)
        o = [full(T + 16, C), full(T + 16, C), full(T + 16, N), full(T + 16, N)]
        dA, h2 = full(C, N), torch.zeros(chunks, C, N, device=DEV)
        assert lib.ssm_scan_bwd_varlen(p(x), C, p(h2), p(x), C, p(x), C, p(A), p(bc), N, p(bc), N, p(cu), p(host), 3, None,
                                       None, 0, None, None, p(o[0]), p(o[1]), p(dA), p(o[2]), p(o[3]), None, None, None,
                                       None, T, C, N, 1, 0, p(ws), n, st) == 0
        torch.cuda.synchronize()
        assert (ws[n // 4:] == 7).all()
        assert lib.causal_conv_fwd_varlen(p(x), C, p(w), None, p(cu), p(host), 3, None, p(y), p(last), T, C, 4, 1, 0, st) == 0
        torch.cuda.synchronize()
        for t, k in ((y, T), (ht, 3), (last, 3), *((t, T) for t in o)):
            assert (t[k:] == 7).all()
