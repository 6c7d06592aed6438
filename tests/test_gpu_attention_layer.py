"""The full-attention layer's operators together, as a serving loop and a training step use them; streams,
captured graphs, and what stays untouched."""
import numpy as np
import pytest
import torch

from oracle import attention as O
from tests.attention_util import DEV, E4M3, U, f64, quantised, within

pytestmark = pytest.mark.gpu


def lib():
    import gated_delta_rule_29_amd as g

    return g


def bf(t):
    return t.to(torch.bfloat16)


class Server:
    """Sequences that share a paged cache: the loop keeps the lengths and gives pages out."""

    def __init__(self, n, pages, Hq, Hk, D, P, R, q8):
        self.Hq, self.Hk, self.D, self.P = Hq, Hk, D, P
        ty = E4M3 if q8 else torch.bfloat16
        self.k, self.v = (torch.zeros(pages, Hk, P, D, device=DEV).to(ty) for _ in "kv")
        self.scales = {x: torch.zeros(pages, Hk, P, device=DEV) for x in ("k_scale", "v_scale")} if q8 else {}
        freqs, self.mag = lib().rope_freqs(R, scaling="yarn", factor=8.0)
        self.freqs, self.rope = freqs.tolist(), lib().rope_table(freqs, DEV)
        self.table = torch.full((n, pages), -1, dtype=torch.int32)
        self.free = list(range(pages - 1, -1, -1))
        self.len = [0] * n

    def places(self, i, m):
        """Slots of sequence i's next m tokens."""
        out = []
        for p in range(self.len[i], self.len[i] + m):
            if p % self.P == 0:
                self.table[i, p // self.P] = self.free.pop(len(self.free) // 2)
            out.append(int(self.table[i, p // self.P]) * self.P + p % self.P)
        self.len[i] += m
        return out

    def run(self, qkv, new, form):
        """qkv [T, (Hq + 2 Hk) D]: the projection's output for the new tokens of each sequence."""
        Hq, Hk, D = self.Hq, self.Hk, self.D
        pos = torch.tensor([p for i, m in enumerate(new) for p in range(self.len[i], self.len[i] + m)], dtype=torch.int32)
        slots = torch.tensor([s for i, m in enumerate(new) for s in self.places(i, m)], dtype=torch.int32)
        T = len(pos)
        qk = lib().rope_fwd(qkv[:, :(Hq + Hk) * D].view(T, Hq + Hk, D), pos.to(DEV), self.rope, magnitude=self.mag)
        lib().kv_cache_write(qk[:, Hq:], qkv[:, (Hq + Hk) * D:].view(T, Hk, D), self.k, self.v, slots.to(DEV), **self.scales)
        n = torch.tensor(self.len, dtype=torch.int32, device=DEV)
        table = self.table.to(DEV)
        if form == "step":
            return lib().paged_attn_step(qk[:, :Hq], self.k, self.v, table, n, **self.scales)
        cu = torch.tensor([0] + list(new)).cumsum(0).to(torch.int32)
        return lib().paged_attn_fwd_varlen(qk[None, :, :Hq], self.k, self.v, table, n, cu.to(DEV), cu_seqlens_host=cu,
                                           **self.scales)["o"][0]


@pytest.mark.parametrize("q8", [False, True])
def test_prompts_then_tokens(q8):
    """Prompts, a chunk beside single tokens, then single tokens, against the oracle of the whole sequences.

    Bounds: rotated queries and keys are bf16 (2^-8 each) of what the oracle turns in fp64, so a score is off
    by 2 * 2^-8 of its terms' size (and 2^-8 squared); 8-bit rows are compared with the oracle's on the rows that
    were stored, which the test reads back."""
    Hq, Hk, D, P, R, n = 4, 2, 64, 16, 32, 3
    s = Server(n, 40, Hq, Hk, D, P, R, q8)
    g = torch.Generator().manual_seed(1)
    calls = [([20, 1, 70], "varlen"), ([1, 45, 1], "varlen"), ([1, 1, 1], "step"), ([1, 1, 1], "step")]
    for new, form in calls:
        before = list(s.len)
        qkv = bf(torch.randn(sum(new), (Hq + 2 * Hk) * D, generator=g)).to(DEV)
        o = s.run(qkv, new, form)
        t0 = 0
        for i, m in enumerate(new):
            L = s.len[i]
            slots = torch.tensor([int(s.table[i, p // P]) * P + p % P for p in range(L)], dtype=torch.int32, device=DEV)
            rows = lib().kv_cache_read(s.k, s.v, slots, dtype=torch.float32, **s.scales) if q8 else \
                lib().kv_cache_read(s.k, s.v, slots)
            pos = list(range(before[i], L))
            q = O.rope(f64(qkv[t0:t0 + m, :Hq * D].view(m, Hq, D)), pos, s.freqs, magnitude=s.mag)
            k = O.rope(f64(qkv[t0:t0 + m, Hq * D:(Hq + Hk) * D].view(m, Hk, D)), pos, s.freqs, magnitude=s.mag)
            kr, vr = f64(rows["k"]), f64(rows["v"])
            # what was written: the new rows, to the cache's precision (e4m3: 2^-4 of a value, or of the least
            # normal one, 2^-6, times the scale)
            half = 2.0 ** -4 if q8 else 2.0 ** -8
            floor = half * 2.0 ** -6 * 2 * np.abs(k).max(-1, keepdims=True) / 448 if q8 else 0.0
            assert (np.abs(kr[before[i]:] - k) <= 1.02 * ((half + 2.0 ** -8) * np.abs(k) + floor) + 20 * U * np.abs(k).max()).all()
            want, _, mean, size = O.attention(q, kr, vr, m, D ** -0.5)
            d = (2.0 ** -8 + (D + 4) * U) * size + (4 + 2 * L) * U  # the query's rounding, and the sums'
            within("o", o[t0:t0 + m], want, (2 * d[..., None] * np.exp(d[..., None]) + 2.0 ** -8) * mean)
            t0 += m


def test_training_step_of_positions():
    """rope_fwd and rope_bwd as an autograd function around queries and keys: gradients against autograd of the
    formula in fp64."""
    class Rope(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, pos, table):
            ctx.save_for_backward(pos, table)
            return lib().rope_fwd(x, pos, table)

        @staticmethod
        def backward(ctx, dy):
            return lib().rope_bwd(dy, *ctx.saved_tensors), None, None

    g = torch.Generator().manual_seed(2)
    x0, w = torch.randn(2, 10, 3, 32, generator=g), torch.randn(2, 10, 3, 32, generator=g)
    pos = torch.arange(10, dtype=torch.int32).expand(2, 10).contiguous()
    freqs, _ = lib().rope_freqs(16)
    x = x0.to(DEV).requires_grad_()
    (Rope.apply(x, pos.to(DEV), lib().rope_table(freqs, DEV)) * w.to(DEV)).sum().backward()
    y = x0.double().requires_grad_()
    a = (pos.double()[..., None] * freqs)[:, :, None]
    u, v = y[..., :8], y[..., 8:16]
    z = torch.cat([u * a.cos() - v * a.sin(), u * a.sin() + v * a.cos(), y[..., 16:]], -1)
    (z * w.double()).sum().backward()
    assert (x.grad.cpu().double() - y.grad).abs().max() <= 8 * U * 2 * w.abs().max()


def _layer(seed, B=3):
    g = torch.Generator().manual_seed(seed)
    Hq, Hk, D, P, pages = 8, 2, 128, 16, 200
    lens = [1, 700, 333][:B]
    s = {"qkv": bf(torch.randn(B, (Hq + 2 * Hk) * D, generator=g)).to(DEV), "pos": torch.tensor([n - 1 for n in lens])}
    for x in "kv":
        q, sc = quantised(torch.randn(pages, Hk, P, D, generator=g))
        s[x], s[x + "s"] = q.to(DEV), sc.to(DEV)
    need = [-(-n // P) for n in lens]
    order = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.full((B, 50), -1, dtype=torch.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    slots = torch.tensor([int(table[i, (n - 1) // P]) * P + (n - 1) % P for i, n in enumerate(lens)], dtype=torch.int32)
    s.update(table=table.to(DEV), slots=slots.to(DEV), lens=torch.tensor(lens, dtype=torch.int32, device=DEV),
             pos=s["pos"].to(torch.int32).to(DEV), rope=lib().rope_table(lib().rope_freqs(64)[0], DEV))
    return s


def _token(s):
    Hq, Hk, D = 8, 2, 128
    B = s["qkv"].shape[0]
    qk = lib().rope_fwd(s["qkv"][:, :(Hq + Hk) * D].view(B, Hq + Hk, D), s["pos"], s["rope"])
    kw = dict(k_scale=s["ks"], v_scale=s["vs"])
    lib().kv_cache_write(qk[:, Hq:], s["qkv"][:, (Hq + Hk) * D:].view(B, Hk, D), s["k"], s["v"], s["slots"], **kw)
    return lib().paged_attn_step(qk[:, :Hq], s["k"], s["v"], s["table"], s["lens"], **kw)


def test_captured_token():
    """One token's layer captured once, replayed with other inputs and lengths in the same buffers."""
    s = _layer(3)
    fresh = _layer(4)
    want = _token(s)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        _token(s)
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _token(s)
    for i in range(4):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), i
        # other inputs; fewer keys than when it was captured, then more
        s["qkv"].copy_(fresh["qkv"])
        s["lens"].copy_(torch.tensor([[1, 600, 0], [1, 700, 333], [1, 300, 17], [1, 700, 20]][i], dtype=torch.int32))
        want = _token(s)  # eager, between the replays
        torch.cuda.synchronize()


def test_two_graphs_and_two_streams():
    """Two captured layers with workspaces of their own, replayed on two streams at once."""
    states = [_layer(5), _layer(6)]
    want = [_token(s) for s in states]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in states]
    graphs, outs = [], []
    for s, st in zip(states, streams):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=st):
            outs.append(_token(s))
        graphs.append(gr)
    for _ in range(5):
        for gr, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w)
    for _ in range(5):
        got = []
        for s, st in zip(states, streams):
            with torch.cuda.stream(st):
                got.append(_token(s))
        torch.cuda.synchronize()
        for o, w in zip(got, want):
            assert torch.equal(o, w)


def test_device_offsets_that_are_not_the_hosts():
    """Offsets on the device are held to what the host sized: nothing outside the outputs is written."""
    g = torch.Generator().manual_seed(7)
    Hq, Hk, D, P = 4, 1, 64, 16
    k, v = (bf(torch.randn(80, Hk, P, D, generator=g)).to(DEV) for _ in "kv")
    table = torch.arange(80, dtype=torch.int32).view(2, 40).to(DEV)
    lens = torch.tensor([600, 500], dtype=torch.int32, device=DEV)
    q = bf(torch.randn(1, 60, Hq, D, generator=g)).to(DEV)
    host = torch.tensor([0, 2, 60], dtype=torch.int32)
    good = lib().paged_attn_fwd_varlen(q, k, v, table, lens, host.to(DEV), cu_seqlens_host=host)["o"]
    guard = torch.zeros(1 << 22, device=DEV)
    for other in ([0, 58, 60], [0, 60, 2], [5, -3, 10 ** 6], [0, 0, 60]):
        dev = torch.tensor(other, dtype=torch.int32, device=DEV)
        lib().paged_attn_fwd_varlen(q, k, v, table, lens, dev, cu_seqlens_host=host)
        torch.cuda.synchronize()
    assert (guard == 0).all()
    assert torch.equal(good, lib().paged_attn_fwd_varlen(q, k, v, table, lens, host.to(DEV), cu_seqlens_host=host)["o"])


def test_nothing_outside_the_rows():
    """Outputs are whole and the caches' other rows stay as they are."""
    s = _layer(8)
    k, v, ks, vs = (s[x].clone() for x in ("k", "v", "ks", "vs"))
    _token(s)
    Hk, P = 2, 16
    hit = torch.zeros(200 * P, dtype=torch.bool, device=DEV)
    hit[s["slots"].long()] = True
    keep = ~hit.view(200, 1, P).expand(200, Hk, P)
    for a, b in ((k, s["k"]), (v, s["v"])):
        assert torch.equal(a.view(torch.uint8)[keep], b.view(torch.uint8)[keep])
    assert torch.equal(ks[keep], s["ks"][keep]) and torch.equal(vs[keep], s["vs"][keep])
