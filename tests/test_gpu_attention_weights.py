"""Weights of the attention over a paged cache where their rounding, the running maximum and values that are not finite
show: against the fp64 oracle, with the bounds of attention_util but for the weights' term, which is said at each test."""
import numpy as np
import pytest
import torch

from tests.attention_util import DEV, TYPES, U, Cache, pages_of, reference, within
from tests.test_gpu_attention import KINDS, check, lib

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scale", [1.4e-45, 1e-39, 1.5e-38, 3e-38])
@pytest.mark.parametrize("dtype,kind", KINDS)
def test_scales_that_are_tiny(scale, dtype, kind):
    """Scales down to the least number of fp32: all keys count alike, in tiles, pieces and their join."""
    check(50, [150, 1, 40], [60, 70, 2500], 4, 2, 64, 16, kind, dtype, scale=scale)
    check(51, [40], [100], 2, 1, 256, 16, kind, dtype, scale=scale, causal=False)


def _call(q, cache, table, lens, new, window=0, scale=None):
    cu = torch.tensor([0] + new).cumsum(0).to(torch.int32)
    return lib().paged_attn_fwd_varlen(q[None], *cache.args(), table.to(DEV), torch.tensor(lens, dtype=torch.int32).to(DEV),
                                       cu.to(DEV), window=window, scale=scale, want_lse=True, cu_seqlens_host=cu,
                                       **cache.scales())


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_infinite_values_that_tokens_see(D, dtype):
    """Every key has an infinite value in one of the first D / 2 columns, of the column's sign: a token's result is that
    infinity where it sees one, whichever tile, wave or piece the key falls to and whatever its weight (the largest one
    of a row is 1); the other columns are as they were.  (Weights here are e^-12 at the least.)"""
    for seed, new, ctx, window in ((60, [1, 4, 1], [99, 30, 700], 0), (61, [100], [70], 0), (62, [90], [130], 0),
                                   (63, [70, 1], [200, 2600], 0), (64, [40], [2300], 0), (65, [90, 3], [150, 200], 77)):
        g = torch.Generator().manual_seed(seed)
        Hq, Hk, P = 4, 2, 16
        lens = [n + c for n, c in zip(new, ctx)]
        pages = sum(-(-n // P) for n in lens) + 2
        cache = Cache(g, pages, Hk, P, D, "same", TYPES[dtype])
        table = pages_of(g, pages, lens, P)
        q = torch.randn(sum(new), Hq, D, generator=g).to(TYPES[dtype]).to(DEV)
        o, lse, bound, lbound = reference(q, cache, table, lens, new, D ** -0.5, window=window)
        half, t0 = D // 2, 0
        for i, L in enumerate(lens):
            for j in range(L):
                cache.t["v"][int(table[i, j // P]), :, j % P, j % half] = float("inf") * (1 if j % half % 2 else -1)
            for t in range(new[i]):
                at = L - new[i] + t
                first = max(0, at - window + 1) if window else 0
                hit = np.array(sorted({j % half for j in range(first, at + 1)}))
                o[t0 + t][:, hit] = np.inf * np.where(hit % 2, 1, -1)
            t0 += new[i]
        print("  case", new, ctx, window, D, dtype, flush=True)
        r = _call(q, cache, table, lens, new, window)
        within("o", r["o"][0], o, bound)
        within("lse", r["lse"][0], lse, lbound)


def _cancelling(seed, kind, D, Hq, Hk, lens, new, dtype="bf16"):
    """Every other key has weight 1 and values of 1, the others weight e^-a and values of about -e^c, with a of the token
    and head and c of the column: results are small beside the sum of their terms' sizes, so that a relative error of the
    weights e^-a, which a rounding to bf16 takes no two of alike, shows in them as it is."""
    g = torch.Generator().manual_seed(seed)
    P = 16
    pages = sum(-(-n // P) for n in lens) + 1
    cache = Cache(g, pages, Hk, P, D, kind, TYPES[dtype])
    k, v = torch.zeros(pages, Hk, P, D), torch.ones(pages, Hk, P, D)
    k[:, :, 1::2, 0] = -1.0
    v[:, :, 1::2] = -torch.exp(3 * torch.rand(D, generator=g))
    cache.put("k", k, TYPES[dtype])
    cache.put("v", v, TYPES[dtype])
    q = torch.zeros(sum(new), Hq, D)
    q[:, :, 0] = 0.05 + 2.95 * torch.rand(sum(new), Hq, generator=g)
    return q.to(TYPES[dtype]).to(DEV), cache, pages_of(g, pages, lens, P)


def _two_bf16(q, cache, table, lens, new):
    """The oracle and its bound where weights enter as two bf16: the first is off by less than 2^-7 of the weight's power
    of two, the second rounds that to 2^-9 of it, so a weight is off by 2^-16 of itself at most; the sums as in
    attention_util, and two roundings more for weights times 8-bit rows' scales."""
    o, lse, bound, lbound = reference(q, cache, table, lens, new, 1.0)
    # (|v| is 1 or more in every place, so that the weighted mean of |v| is taken from the oracle on |v|)
    size = {n: np.abs(x) if n == "v" else x for n, x in cache.values.items()}
    keep, cache.values = cache.values, size
    mean = reference(q, cache, table, lens, new, 1.0)[0]
    cache.values = keep
    L, D = max(lens), q.shape[-1]
    d = (D + 4) * U * 3.0 + (8 + 2 * L) * U  # (scores are 3 at most)
    return o, lse, (2 * d + 2.0 ** -16) * mean, lbound


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kind", ["same", "e4m3"])
def test_weights_are_two_bf16(D, kind):
    """Few rows, cut or not, and tiles of many rows whose keys some rows see in part (all of them here)."""
    for seed, Hq, Hk, new, lens in ((70, 6, 2, [1, 1, 1], [100, 33, 1]), (71, 4, 1, [4, 8, 1], [64, 300, 3000]),
                                    (72, 2, 2, [60, 40], [60, 50]), (73, 8, 2, [40, 1], [63, 5])):
        q, cache, table = _cancelling(seed, kind, D, Hq, Hk, lens, new)
        o, lse, bound, lbound = _two_bf16(q, cache, table, lens, new)
        print("  case", new, lens, Hq, Hk, D, kind, flush=True)
        r = _call(q, cache, table, lens, new, scale=1.0)
        within("o", r["o"][0], o, bound)
        within("lse", r["lse"][0], lse, lbound)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kind", ["same", "e4m3"])
def test_weights_beside_values_that_are_not_finite(D, kind):
    """NaN in a place that only a chunk's last token sees: the others' weights enter as exactly as without it."""
    for seed, Hq, Hk, new, lens in ((80, 2, 2, [60], [60]), (81, 8, 2, [40], [63]), (82, 4, 1, [6], [40])):
        q, cache, table = _cancelling(seed, kind, D, Hq, Hk, lens, new)
        o, lse, bound, lbound = _two_bf16(q, cache, table, lens, new)
        last, d = lens[0] - 1, D - 3
        page, place = int(table[0, last // 16]), last % 16
        if kind == "e4m3":
            cache.t["v"].view(torch.uint8)[page, :, place, d] = 0x7f
        else:
            cache.t["v"][page, :, place, d] = float("nan")
        o[-1, :, d] = np.nan
        print("  case", new, lens, Hq, Hk, D, kind, flush=True)
        r = _call(q, cache, table, lens, new, scale=1.0)
        within("o", r["o"][0], o, bound)
        within("lse", r["lse"][0], lse, lbound)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("want_lse", [False, True])
def test_rows_that_one_key_dominates(D, want_lse):
    """A key in a tile that all rows see has e^3 to e^5.4 of the weight of the row's first maximum, all others next to
    nothing.  Weights w_j (1 + d_j), |d_j| <= 2^-8, in products and sum alike move a result by
    sum w_j d_j (v_j - o) / sum w_j (1 + d_j): by 2^-8 / (1 - 2^-8) of the weighted mean of |v_j - o| at most, which is
    small where one key has nearly all of the weight.  (Not so of 8-bit rows, whose weights enter with their scale.)"""
    g = torch.Generator().manual_seed(90)
    Hq, Hk, P = 4, 2, 16
    for new, lens in (([40, 1], [1100, 700]), ([64], [5000])):
        pages = sum(-(-n // P) for n in lens) + 1
        cache = Cache(g, pages, Hk, P, D, "same")
        table = pages_of(g, pages, lens, P)
        k = torch.zeros(pages, Hk, P, D)
        k[..., 0] = -16.0
        for i in range(len(lens)):
            k[int(table[i, 0]), :, 3] = 0.0
            k[int(table[i, 200 // P]), :, 200 % P, 0] = 1.0
        cache.put("k", k, torch.bfloat16)
        q = torch.zeros(sum(new), Hq, D)
        q[:, :, 0] = 3 + 2.4 * torch.rand(sum(new), Hq, generator=g)
        q = q.to(torch.bfloat16).to(DEV)
        o, lse, _, lbound = reference(q, cache, table, lens, new, 1.0)
        a = q[:, :, :1].double().cpu().numpy()
        bound, t0 = np.zeros_like(o), 0
        for i, n in enumerate(new):
            first, main = (np.repeat(cache.values["v"][int(table[i, at // P]), :, at % P], Hq // Hk, 0) for at in (3, 200))
            x = a[t0:t0 + n]
            r = o[t0:t0 + n]
            spread = (np.exp(x) * np.abs(main - r) + np.abs(first - r)) / (np.exp(x) + 1)
            mean = (np.exp(x) * np.abs(main) + np.abs(first)) / (np.exp(x) + 1)
            # (the two keys' scores are below 6, and the others' weights, e^-48 each, within the sums' roundings)
            bound[t0:t0 + n] = 2.0 ** -8 / (1 - 2.0 ** -8) * spread + 2 * ((D + 4) * U * 6 + (4 + 2 * lens[i]) * U) * mean
            t0 += n
        cu = torch.tensor([0] + new).cumsum(0).to(torch.int32)
        print("  case", new, lens, D, want_lse, flush=True)
        r = lib().paged_attn_fwd_varlen(q[None], *cache.args(), table.to(DEV), torch.tensor(lens, dtype=torch.int32).to(DEV),
                                        cu.to(DEV), scale=1.0, want_lse=want_lse, cu_seqlens_host=cu)
        within("o", r["o"][0], o, bound)
        if want_lse:
            within("lse", r["lse"][0], lse, lbound)
