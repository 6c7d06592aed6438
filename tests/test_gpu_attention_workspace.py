"""Attention whose keys are cut, so that partial results go through the workspace: captured and replayed with other
lengths, two graphs and two streams at once, repeated, and with guards around everything that a call writes."""
import ctypes

import pytest
import torch

from tests.attention_util import DEV, TYPES, Cache, reference, within

pytestmark = pytest.mark.gpu

HQ, HK, P, WIDTH = 8, 2, 16, 600  # a table of 9600 keys

# (new tokens, keys of each sequence) of calls with the same sizes: many pieces of some sequences, two of others, one
# of all, none; rows of both kinds (8 and 4 rows beside 160 and 1200)
STEPS = [[1, 9000, 4000], [9600, 1, 700], [1200, 800, 0], [5, 600, 300]]
NEW = [2, 40, 1, 300]
CHUNKS = [[3000, 9600, 1, 5000], [700, 40, 8000, 2600], [2, 1700, 900, 300], [1, 39, 0, 9000]]
KINDS = [("bf16", "same"), ("bf16", "e4m3"), ("f32", "same")]


def lib():
    import gated_delta_rule_29_amd as g

    return g


class Call:
    """Inputs of a call in buffers that stay; `run` makes the call."""

    def __init__(self, seed, form, dtype="bf16", kind="same", D=64):
        g = torch.Generator().manual_seed(seed)
        t = TYPES[dtype]
        self.form, self.new = form, [1, 1, 1] if form == "step" else NEW
        self.lens_list = STEPS if form == "step" else CHUNKS
        n = len(self.new)
        self.cache = Cache(g, 700, HK, P, D, kind, t)
        # (sequences share pages: what is in them does not change)
        self.table_host = torch.stack([torch.randperm(700, generator=g)[:WIDTH] for _ in range(n)]).to(torch.int32)
        self.table = self.table_host.to(DEV)
        self.q = torch.randn(sum(self.new), HQ, D, generator=g).to(t).to(DEV)
        self.lens = torch.zeros(n, dtype=torch.int32, device=DEV)
        self.cu_host = torch.tensor([0] + self.new).cumsum(0).to(torch.int32)
        self.cu = self.cu_host.to(DEV)
        self.set(0)

    def set(self, i):
        self.lens.copy_(torch.tensor(self.lens_list[i], dtype=torch.int32))

    def run(self):
        if self.form == "step":
            return lib().paged_attn_step(self.q, *self.cache.args(), self.table, self.lens, **self.cache.scales())
        r = lib().paged_attn_fwd_varlen(self.q[None], *self.cache.args(), self.table, self.lens, self.cu,
                                        want_lse=self.form == "lse", cu_seqlens_host=self.cu_host, **self.cache.scales())
        return torch.cat([r["o"][0].float(), r["lse"][0][..., None]], -1) if self.form == "lse" else r["o"]


def test_calls_are_cut():
    """What the tests below rest on: the calls have a workspace, and their keys make several pieces."""
    for new in ([1, 1, 1], NEW):
        cu = torch.tensor([0] + new, dtype=torch.int32).cumsum(0).to(torch.int32)
        n = lib()._lib.load().paged_attn_varlen_workspace_bytes(cu.data_ptr(), len(new), HQ, HK, 64, P, WIDTH, 1, 1)
        assert n > 0
    # (a piece of few rows has 512 keys at the least, one of many 1024, and half as many more before a unit is cut)
    assert any(1536 <= L for i in STEPS for L in i) and any(L < 768 for i in STEPS for L in i)


@pytest.mark.parametrize("form", ["step", "varlen", "lse"])
@pytest.mark.parametrize("dtype,kind", KINDS)
def test_captured_calls_with_other_lengths(form, dtype, kind):
    """One graph, replayed with lengths of many pieces, two, one and none, with eager calls between the replays; the
    first lengths against the oracle."""
    c = Call(1, form, dtype, kind)
    want = []
    for i in range(4):
        c.set(i)
        want.append(c.run().clone())
    if form != "lse":
        o, _, bound, _ = reference(c.q, c.cache, c.table_host, STEPS[2] if form == "step" else CHUNKS[2], c.new, 64 ** -0.5)
        within("o", want[2].view(o.shape), o, bound)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        c.run()
    torch.cuda.current_stream().wait_stream(stream)
    c.set(0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = c.run()
    for i in (0, 3, 1, 2, 1, 0, 3, 2):
        c.set(i)
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i]), i
        assert torch.equal(c.run(), want[i]), i
        torch.cuda.synchronize()


@pytest.mark.parametrize("form", ["step", "varlen"])
@pytest.mark.parametrize("dtype,kind", KINDS)
def test_two_graphs_and_two_streams_with_workspaces(form, dtype, kind):
    """Two captured calls whose keys are cut, replayed on two streams at once; then both eagerly."""
    calls = [Call(2, form, dtype, kind), Call(3, form, dtype, kind)]
    calls[1].set(1)
    want = [c.run().clone() for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    graphs, outs = [], []
    for c, st in zip(calls, streams):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=st):
            outs.append([c.run() for _ in range(4)])  # (several, so that the two overlap)
        graphs.append(gr)
    for _ in range(4):
        for gr, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert all(torch.equal(x, w) for x in o)
            for x in o:
                x.fill_(7.0)
        torch.cuda.synchronize()
    for _ in range(4):
        got = [[], []]
        for _ in range(3):
            for r, c, st in zip(got, calls, streams):
                with torch.cuda.stream(st):
                    r.append(c.run())
        torch.cuda.synchronize()
        for r, w in zip(got, want):
            assert all(torch.equal(x, w) for x in r)


@pytest.mark.parametrize("form", ["step", "varlen", "lse"])
@pytest.mark.parametrize("dtype,kind", KINDS)
def test_cut_results_repeat(form, dtype, kind):
    c = Call(4, form, dtype, kind, 128)
    first = c.run()
    for _ in range(5):
        assert torch.equal(first, c.run())


PAD = 4096  # bytes of guard


class Guarded:
    """n bytes between two guards, all of them 0x5a."""

    def __init__(self, n):
        self.n = n
        self.all = torch.full((PAD + -(-n // 256) * 256 + PAD,), 0x5a, dtype=torch.uint8, device=DEV)
        self.ptr = ctypes.c_void_p(self.all.data_ptr() + PAD)

    def view(self, dtype):
        return self.all[PAD:PAD + self.n].view(dtype)

    def check(self, name):
        a = self.all
        assert bool((a[:PAD] == 0x5a).all()) and bool((a[PAD + self.n:] == 0x5a).all()), name


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype,kind", KINDS)
def test_nothing_is_written_outside(D, dtype, kind):
    """Outputs, lse and workspace between guards, through the C entry: with the host's offsets, and with offsets and
    lengths on the device that are not (whose results mean nothing, but stay inside)."""
    g = torch.Generator().manual_seed(5)
    t = TYPES[dtype]
    width, host = 200, [0, 2, 60, 63]  # 8 and 12 rows, and 232
    cache = Cache(g, 220, 1, P, D, kind, t)
    T, Hq, N = host[-1], 4, len(host) - 1
    table = torch.stack([torch.randperm(220, generator=g)[:width] for _ in range(N)]).to(torch.int32).to(DEV)
    q = torch.randn(T, Hq, D, generator=g).to(t).to(DEV)
    L = lib()._lib
    fn = L.load()
    cu_host = torch.tensor(host, dtype=torch.int32)
    code, ccode = (L.DTYPE_BF16 if dtype == "bf16" else L.DTYPE_F32), L.DTYPE_E4M3
    if kind != "e4m3":
        ccode = code
    n = fn.paged_attn_varlen_workspace_bytes(cu_host.data_ptr(), N, Hq, 1, D, P, width, code, ccode)
    assert n > 0
    ks, vs = (cache.s[x].data_ptr() if kind == "e4m3" else None for x in "kv")

    def call(cu, lens):
        dev = torch.tensor(cu, dtype=torch.int32, device=DEV)
        dl = torch.tensor(lens, dtype=torch.int32, device=DEV)
        o, lse, ws = Guarded(T * Hq * D * t.itemsize), Guarded(T * Hq * 4), Guarded(n)
        print("  case", D, dtype, kind, cu, lens, flush=True)
        rc = fn.paged_attn_fwd_varlen(q.data_ptr(), Hq * D, D, cache.t["k"].data_ptr(), cache.t["v"].data_ptr(), ks, vs,
                                      table.data_ptr(), width, width, dl.data_ptr(), dev.data_ptr(), cu_host.data_ptr(), N,
                                      D ** -0.5, 1, 0, o.ptr, lse.ptr, T, Hq, 1, D, 220, P, code, ccode, ws.ptr, n,
                                      torch.cuda.current_stream().cuda_stream)
        assert rc == L.OK
        torch.cuda.synchronize()
        for name, x in (("o", o), ("lse", lse), ("workspace", ws)):
            x.check(name)
        return o.view(t), lse.view(torch.float32)

    whole = [3200, 3000, 2900]
    good, good_lse = call(host, whole)
    ref = lib().paged_attn_fwd_varlen(q[None], *cache.args(), table, torch.tensor(whole, dtype=torch.int32, device=DEV),
                                      cu_host.to(DEV), want_lse=True, cu_seqlens_host=cu_host, **cache.scales())
    assert torch.equal(good, ref["o"].view(-1)) and torch.equal(good_lse, ref["lse"].view(-1))
    for cu in ([0, 58, 60, 63], [0, 60, 2, 63], [5, -3, 10 ** 6, -1], [0, 0, 63, 63], [0, 63, 0, 63], [0, 21, 42, 63]):
        for lens in (whole, [0, 10 ** 9, -7]):
            call(cu, lens)
    again, again_lse = call(host, whole)
    assert torch.equal(again, good) and torch.equal(again_lse, good_lse)
