"""Weights of the attention over a paged cache where their rounding, the running maximum and values that are not finite
show: against the fp64 oracle, with the bounds of attention_util but for the weights' term, which is said at each test."""
import numpy as np
import pytest
import torch

from tests.attention_util import DEV, TYPES, Cache, pages_of, reference, within
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
