"""Attention over a paged cache against the fp64 oracle: single tokens, chunks, cross attention."""
import pytest
import torch

from tests.attention_util import (DEV, TYPES, Cache, pages_of, reference, within)

pytestmark = pytest.mark.gpu


def lib():
    import gated_delta_rule_29_amd as g

    return g


def queries(g, n, Hq, D, dtype, how="dense"):
    q = torch.randn(n, Hq, D, generator=g).to(dtype)
    if how == "dense":
        return q.to(DEV)
    if how == "columns":  # of a wider projection, whose other columns hold NaN
        wide = torch.full((n, Hq * D + 64), float("nan"), dtype=dtype, device=DEV)
        out = wide[:, 32:32 + Hq * D].view(n, Hq, D)
    elif how == "odd":  # nothing aligned
        wide = torch.full((n, Hq, D + 3), float("nan"), dtype=dtype, device=DEV)
        out = wide[:, :, 1:1 + D]
    else:  # heads first
        out = torch.empty(Hq, n, D, dtype=dtype, device=DEV).transpose(0, 1)
    out.copy_(q)
    return out


def check(seed, new, ctx, Hq, Hk, D, P, kind="same", dtype="bf16", causal=True, window=0, how="dense", extra=0,
          form="varlen", spare=3, scale=None, change=None):
    """One call against the oracle.  ctx: keys before the new tokens (of a causal call), or all keys."""
    g = torch.Generator().manual_seed(seed)
    t = TYPES[dtype]
    lens = [c + n for c, n in zip(ctx, new)] if causal else list(ctx)
    pages = sum(-(-n // P) for n in lens) + spare
    cache = Cache(g, pages, Hk, P, D, "e4m3" if kind == "e4m3" else "same", t)
    table = pages_of(g, pages, lens, P, extra)
    if change:
        change(cache, table, lens)
    # what no token sees holds NaN: places behind the lengths, pages of no sequence
    used = torch.zeros(pages, P, dtype=torch.bool)
    for i, n in enumerate(lens):
        for j in range(n):
            if 0 <= table[i, j // P] < pages:
                used[table[i, j // P], j % P] = True
    hidden = (~used)[:, None, :].expand(pages, Hk, P).to(DEV)
    for n in "kv":
        if cache.kind == "e4m3":
            cache.t[n].view(torch.uint8)[hidden] = 0x7f
            cache.s[n][hidden] = float("nan")
        else:
            cache.t[n][hidden] = float("nan")
    q = queries(g, sum(new), Hq, D, t, how)
    o, lse, bound, lbound = reference(q, cache, table, lens, new, scale or D ** -0.5, causal, window)
    dt, dl = table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)
    kw = dict(cache.scales(), scale=scale, window=window)
    print("  case", seed, new, lens, Hq, Hk, D, P, kind, dtype, causal, window, how, form, flush=True)
    if form == "step":
        got = {"o": lib().paged_attn_step(q, *cache.args(), dt, dl, **kw)}
    elif form == "dense":
        r = lib().paged_attn_fwd(q.view(len(new), new[0], Hq, D), *cache.args(), dt, dl, causal=causal, want_lse=True, **kw)
        got = {"o": r["o"].view(-1, Hq, D), "lse": r["lse"].view(-1, Hq)}
    else:
        cu = torch.tensor([0] + new).cumsum(0).to(torch.int32)
        r = lib().paged_attn_fwd_varlen(q[None], *cache.args(), dt, dl, cu.to(DEV), causal=causal, want_lse=True,
                                        cu_seqlens_host=cu, **kw)
        got = {"o": r["o"][0], "lse": r["lse"][0]}
    torch.cuda.synchronize()
    within("o", got["o"], o, bound)
    if "lse" in got:
        within("lse", got["lse"], lse, lbound)


KINDS = [("bf16", "same"), ("bf16", "e4m3"), ("f32", "same"), ("f32", "e4m3")]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype,kind", KINDS)
def test_single_tokens(D, dtype, kind):
    """Lengths around tiles and pages, a row without keys, one key; several heads a key head."""
    check(1, [1] * 9, [0, -1, 15, 16, 31, 62, 63, 64, 200], 6, 2, D, 16, kind, dtype, form="step")
    check(2, [1] * 3, [700, 5, 300], 17, 1, D, 64, kind, dtype, form="step")  # 17 rows: a second tile
    check(3, [1], [40], 1, 1, D, 1024, kind, dtype, form="step", how="odd")


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype,kind", KINDS)
def test_chunks(D, dtype, kind):
    """Chunks of all lengths in one packed call, so that both classes of sequences run."""
    check(4, [1, 5, 70, 2, 33], [100, 0, 61, 17, 3], 4, 2, D, 16, kind, dtype)
    check(5, [150, 1], [0, 129], 3, 1, D, 32, kind, dtype, how="columns")


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype,kind", KINDS)
def test_cross_attention(D, dtype, kind):
    check(6, [40, 3, 65], [1, 77, 130], 2, 2, D, 16, kind, dtype, causal=False)
    check(7, [20, 20], [0, 33], 4, 4, D, 16, kind, dtype, causal=False, form="dense", how="heads")


@pytest.mark.parametrize("window", [1, 7, 64, 100, 5000])
@pytest.mark.parametrize("dtype,kind", [("bf16", "same"), ("bf16", "e4m3"), ("f32", "same")])
def test_windows(window, dtype, kind):
    check(8, [100, 1, 3], [50, 300, 130], 4, 2, 64, 16, kind, dtype, window=window)
    check(9, [1, 1], [1500, 2], 8, 1, 128, 16, kind, dtype, window=window, form="step", extra=200)


@pytest.mark.parametrize("P", [16, 32, 64, 128, 256, 512, 1024])
@pytest.mark.parametrize("kind", ["same", "e4m3"])
def test_pages(P, kind):
    check(10, [1, 40, 1], [P - 1, 2 * P - 20, 3 * P], 4, 1, 128, P, kind)


@pytest.mark.parametrize("dtype,kind", KINDS)
def test_cut_keys(dtype, kind):
    """Long contexts of few rows are cut into pieces and joined; beside them short ones and one without keys."""
    check(11, [1, 1, 1, 1], [4000, 3, 900, -1], 4, 2, 64, 16, kind, dtype, form="step")
    check(12, [2, 1, 40], [2500, 0, 1800], 4, 1, 128, 64, kind, dtype, extra=70)


def test_cut_keys_of_wide_heads():
    check(13, [1, 20, 3], [2100, 900, 10], 8, 2, 256, 64)
    check(14, [1, 20, 3], [2100, 900, 10], 8, 2, 256, 64, "e4m3")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_fewer_keys_than_new_tokens(dtype):
    """A sequence whose length leaves its first tokens without keys."""
    g = torch.Generator().manual_seed(15)
    t = TYPES[dtype]
    new, lens, Hq, Hk, D, P = [5, 80, 3], [2, 30, 0], 4, 2, 64, 16
    cache = Cache(g, 8, Hk, P, D, "same", t)
    table = pages_of(g, 8, lens, P)
    q = queries(g, sum(new), Hq, D, t)
    o, lse, bound, lbound = reference(q, cache, table, lens, new, 0.2)
    cu = torch.tensor([0] + new).cumsum(0).to(torch.int32)
    r = lib().paged_attn_fwd_varlen(q[None], *cache.args(), table.to(DEV), torch.tensor(lens, dtype=torch.int32).to(DEV),
                                    cu.to(DEV), scale=0.2, want_lse=True)
    assert (o[:3] == 0).all() and (r["o"][0, :3] == 0).all() and torch.isneginf(r["lse"][0, :3]).all()
    within("o", r["o"][0], o, bound)
    within("lse", r["lse"][0], lse, lbound)


@pytest.mark.parametrize("dtype,kind", KINDS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_not_finite_values_that_a_token_does_not_see(dtype, kind, bad):
    """NaN and infinities in keys and values of later tokens of the chunk (and, with a window, of places
    before it) leave a token's result as it is; tokens that see them get what the formula gives."""
    if kind == "e4m3" and bad == bad:
        bad = float("nan")  # e4m3 has no infinities
    for new, ctx, window in (([90], [20], 0), ([6], [70], 5)):
        g = torch.Generator().manual_seed(16)
        t = TYPES[dtype]
        L, Hq, Hk, D, P = new[0] + ctx[0], 4, 2, 64, 16
        at = L - new[0] // 2  # the place, in the middle of the chunk
        cache = Cache(g, 10, Hk, P, D, kind, t)
        table = pages_of(g, 10, [L], P)
        q = queries(g, new[0], Hq, D, t)
        o, lse, bound, lbound = reference(q, cache, table, [L], new, D ** -0.5, window=window)
        page, place = int(table[0, at // P]), at % P
        d = 5  # one column
        if kind == "e4m3":
            cache.t["v"].view(torch.uint8)[page, 1, place, d] = 0x7f
            cache.s["k"][page, 0, place] = bad
        else:
            cache.t["v"][page, 1, place, d] = bad
            cache.t["k"][page, 0, place, d] = bad
        cu = torch.tensor([0] + new, dtype=torch.int32)
        r = lib().paged_attn_fwd_varlen(q[None], *cache.args(), table.to(DEV),
                                        torch.tensor([L], dtype=torch.int32).to(DEV), cu.to(DEV), window=window,
                                        want_lse=True, **cache.scales())
        first = at - ctx[0]  # the first token that sees it
        got, gl = r["o"][0], r["lse"][0]
        before = slice(0, first)
        within("o", got[before], o[before], bound[before])
        within("lse", gl[before], lse[before], lbound[before])
        end = min(new[0], first + window) if window else new[0]
        if end < new[0]:
            within("o", got[end:], o[end:], bound[end:])
        # head 1's values: that column is not finite, the others are as they were
        hit = got[first:end, 2:, d].float()
        assert (torch.isnan(hit) if bad != bad else hit == bad).all()
        rest = [c for c in range(D) if c != d]
        within("rest", got[first:end, 2:][..., rest], o[first:end, 2:][..., rest], bound[first:end, 2:][..., rest])
        if bad != bad or kind == "e4m3":
            assert torch.isnan(got[first:end, :2].float()).all()


def test_scores_that_are_large():
    """Scores of hundreds: the running maximum moves, and the weights of most keys vanish."""
    check(17, [70, 1], [60, 400], 4, 2, 128, 16, scale=8.0)
    check(17, [70, 1], [60, 400], 4, 2, 128, 16, scale=8.0, dtype="f32")


def test_pages_that_the_cache_does_not_have():
    """A page outside the cache reads as keys and values of 0."""
    for kind in ("same", "e4m3"):
        def change(cache, table, lens):
            table[0, 1] = -1
            table[1, 0] = 10 ** 6
            table[1, 2] = -2 ** 31

        check(18, [1, 50], [100, 60], 4, 1, 64, 16, kind, change=change)


def test_lengths_outside_the_table():
    """A length is taken as the nearest one that the table holds."""
    g = torch.Generator().manual_seed(19)
    cache = Cache(g, 4, 1, 16, 64, "same", torch.bfloat16)
    table = torch.tensor([[2, 0], [3, 1]], dtype=torch.int32, device=DEV)
    q = queries(g, 2, 2, 64, torch.bfloat16)
    a = lib().paged_attn_step(q, *cache.args(), table, torch.tensor([33, -5], dtype=torch.int32, device=DEV))
    b = lib().paged_attn_step(q, *cache.args(), table, torch.tensor([32, 0], dtype=torch.int32, device=DEV))
    assert torch.equal(a, b) and (a[1] == 0).all()


def test_table_rows_of_a_wider_table():
    g = torch.Generator().manual_seed(20)
    cache = Cache(g, 12, 2, 16, 64, "same", torch.bfloat16)
    lens = torch.tensor([30, 17, 60], dtype=torch.int32, device=DEV)
    table = pages_of(g, 12, lens.tolist(), 16)
    wide = torch.full((3, 11), 99, dtype=torch.int32, device=DEV)
    wide[:, 2:2 + table.shape[1]] = table.to(DEV)
    q = queries(g, 3, 4, 64, torch.bfloat16)
    a = lib().paged_attn_step(q, *cache.args(), table.to(DEV), lens)
    b = lib().paged_attn_step(q, *cache.args(), wide[:, 2:2 + table.shape[1]], lens)
    assert torch.equal(a, b)


def test_forms_agree():
    """A batch of single tokens through all three entry points, and a chunk against its tokens."""
    g = torch.Generator().manual_seed(21)
    cache = Cache(g, 40, 2, 16, 128, "same", torch.bfloat16)
    lens = [130, 1, 77, 200]
    table = pages_of(g, 40, lens, 16).to(DEV)
    dl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    q = queries(g, 4, 8, 128, torch.bfloat16)
    a = lib().paged_attn_step(q, *cache.args(), table, dl)
    b = lib().paged_attn_fwd(q[:, None], *cache.args(), table, dl)["o"][:, 0]
    cu = torch.arange(5, dtype=torch.int32)
    c = lib().paged_attn_fwd_varlen(q[None], *cache.args(), table, dl, cu.to(DEV))["o"][0]
    assert torch.equal(a, b) and torch.equal(a, c)


def test_many_sequences():
    g = torch.Generator().manual_seed(22)
    n = 300  # several waves' worth of sequences
    ctx = torch.randint(0, 90, (n,), generator=g).tolist()
    new = [1 if i % 7 else 9 for i in range(n)]
    check(23, new, ctx, 4, 2, 64, 16)
    check(24, [1] * n, ctx, 4, 2, 64, 16, "e4m3", form="step")


def test_results_repeat():
    g = torch.Generator().manual_seed(25)
    cache = Cache(g, 300, 2, 16, 128, "same", torch.bfloat16)
    lens = [3500, 700]
    table = pages_of(g, 300, lens, 16).to(DEV)
    dl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    q = queries(g, 2, 8, 128, torch.bfloat16)
    first = lib().paged_attn_step(q, *cache.args(), table, dl)
    for _ in range(5):
        assert torch.equal(first, lib().paged_attn_step(q, *cache.args(), table, dl))


@pytest.mark.parametrize("D,kind", [(64, "same"), (64, "e4m3"), (128, "same"), (128, "e4m3"), (256, "same"),
                                    (256, "e4m3")])
def test_cut_chunks(D, kind):
    """Chunks of several tiles over contexts that are cut into pieces: the first tiles of a chunk have fewer of them
    than the last ones, and long chunks stand beside level ones and single tokens."""
    check(26, [300, 1, 70, 3], [2900, 40, 4500, 10], 8, 2, D, 64, kind)
    check(27, [700, 130], [0, 2200], 4, 1, D, 16, kind, how="odd", extra=100)
    check(28, [90, 90], [3500, 3500], 4, 1, D, 32, kind, form="dense")
    check(29, [40, 600], [5000, 1], 4, 2, D, 128, kind, causal=False)


@pytest.mark.parametrize("window", [1, 33, 600, 4000])
@pytest.mark.parametrize("D,kind", [(64, "same"), (128, "same"), (128, "e4m3"), (256, "same"), (256, "e4m3")])
def test_windows_of_long_chunks(window, D, kind):
    check(30, [400, 2, 50], [1500, 900, 5000], 8, 2, D, 32, kind, window=window)


def test_fp32_chunks_that_are_cut():
    check(31, [100, 1, 20], [2500, 700, 0], 4, 2, 128, 16, dtype="f32")
    check(31, [100, 1, 20], [2500, 700, 0], 4, 2, 64, 16, "e4m3", dtype="f32", window=1800)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kind", ["same", "e4m3"])
def test_single_tokens_of_many_heads(D, kind):
    """More query heads a key head than a tile of few rows has."""
    check(32, [1, 1, 1], [1200, 0, 77], 66, 2, D, 16, kind, form="step")


def test_many_long_sequences():
    """More sequences than a wave has lanes, of both classes and both orders, cut."""
    g = torch.Generator().manual_seed(33)
    ctx = torch.randint(0, 400, (150,), generator=g).tolist()
    new = [1 if i % 3 else 20 + i for i in range(150)]
    ctx[3], ctx[77], ctx[148] = 3000, 4000, 5000
    check(34, new, ctx, 4, 2, 64, 16)


@pytest.mark.parametrize("D,kind", [(64, "same"), (128, "same"), (128, "e4m3"), (256, "same"), (256, "e4m3")])
def test_not_finite_values_in_long_chunks(D, kind):
    """NaN in values at many places of a long chunk, cut or not: each token's result has those that it sees, and
    no other."""
    g = torch.Generator().manual_seed(35)
    new, L, Hq, Hk, P = 300, 2700, 4, 2, 32
    for window in (0, 700):
        cache = Cache(g, 90, Hk, P, D, kind)
        table = pages_of(g, 90, [L], P)
        q = queries(g, new, Hq, D, torch.bfloat16)
        o, _, bound, _ = reference(q, cache, table, [L], [new], D ** -0.5, window=window)
        # (column, place): before the window of all, of some, in the chunk, its last token's
        places = [(0, 100), (1, L - new - 650), (2, L - new), (3, L - new + 63), (4, L - 130), (5, L - 1)]
        for d, at in places:
            page, place = int(table[0, at // P]), at % P
            if kind == "e4m3":
                cache.t["v"].view(torch.uint8)[page, :, place, d] = 0x7f
            else:
                cache.t["v"][page, :, place, d] = float("nan")
        cu = torch.tensor([0, new], dtype=torch.int32)
        got = lib().paged_attn_fwd_varlen(q[None], *cache.args(), table.to(DEV),
                                          torch.tensor([L], dtype=torch.int32).to(DEV), cu.to(DEV), window=window,
                                          **cache.scales())["o"][0].clone()
        for d, at in places:
            last = torch.arange(L - new, L)
            sees = (last >= at) & ((last - at < window) if window else True)
            bad = torch.isnan(got[:, :, d].float()).all(1).cpu()
            none = torch.isnan(got[:, :, d].float()).any(1).cpu()
            assert torch.equal(bad, sees) and torch.equal(none, sees), (d, at, window)
            hit = sees.to(DEV)
            got[hit, :, d] = 0
            o[sees.numpy(), :, d] = 0
        within("o", got, o, bound)


@pytest.mark.parametrize("kind", ["same", "e4m3"])
def test_pages_past_32_bits(kind):
    """Pages whose elements lie past 2^32 of the cache."""
    g = torch.Generator().manual_seed(36)
    H, P, D, pages = 4, 64, 128, (1 << 32) // (4 * 64 * 128) + 80
    lens, new = [1500, 300], [40, 1]
    small = Cache(g, 40, H, P, D, kind)
    table = pages_of(g, 40, lens, P)
    big = {n: torch.empty(pages, H, P, D, dtype=small.t[n].dtype, device=DEV) for n in "kv"}
    scales = {}
    for n in "kv":
        big[n][-40:] = small.t[n]
        if kind == "e4m3":
            scales[n + "_scale"] = torch.empty(pages, H, P, device=DEV)
            scales[n + "_scale"][-40:] = small.s[n]
    far = torch.where(table >= 0, table + pages - 40, table)
    q = queries(g, 41, 8, D, torch.bfloat16)
    dl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, 40, 41], dtype=torch.int32)
    a = lib().paged_attn_fwd_varlen(q[None], *small.args(), table.to(DEV), dl, cu.to(DEV), **small.scales())["o"]
    b = lib().paged_attn_fwd_varlen(q[None], big["k"], big["v"], far.to(DEV), dl, cu.to(DEV), **scales)["o"]
    assert torch.equal(a, b)
    o, _, bound, _ = reference(q, small, table, lens, new, D ** -0.5)
    within("o", a[0], o, bound)


@pytest.mark.parametrize("kind", ["same", "e4m3"])
def test_pages_that_sequences_share(kind):
    """Sequences with a common beginning name the same pages; one names a page twice."""
    def change(cache, table, lens):
        table[1, :3] = table[0, :3]
        table[2, 1] = table[2, 0]

    check(37, [40, 1, 9], [50, 60, 30], 4, 2, 64, 16, kind, change=change)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_largest_window(dtype):
    """A window of 2^31 - 1 hides nothing, also where a sequence's first tokens have no keys."""
    g = torch.Generator().manual_seed(38)
    t = TYPES[dtype]
    new, lens = [1000, 5, 3], [100, 300, 1]
    cache = Cache(g, 30, 2, 16, 64, "same", t)
    table = pages_of(g, 30, lens, 16)
    q = queries(g, sum(new), 4, 64, t)
    cu = torch.tensor([0] + new).cumsum(0).to(torch.int32).to(DEV)
    dl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    whole = lib().paged_attn_fwd_varlen(q[None], *cache.args(), table.to(DEV), dl, cu)["o"]
    for window in (2 ** 31 - 1, 2 ** 30, 304, 303):
        r = lib().paged_attn_fwd_varlen(q[None], *cache.args(), table.to(DEV), dl, cu, window=window)["o"]
        assert torch.equal(r, whole), window
    o, _, bound, _ = reference(q, cache, table, lens, new, 64 ** -0.5)
    within("o", whole[0], o, bound)


@pytest.mark.parametrize("kind", ["same", "e4m3"])
def test_more_heads_of_a_key_head_than_a_tile_has_rows(kind):
    check(39, [1, 3], [70, 1100], 300, 1, 64, 16, kind)
    check(39, [1, 1], [70, 1100], 300, 1, 256, 16, kind, form="step")
