"""The paged cache: rows written (in their type or in 8 bits) and read back, against the definition's steps in
torch on the CPU, bit for bit."""
import pytest
import torch

from tests.attention_util import DEV, E4M3, TYPES, quantised

pytestmark = pytest.mark.gpu


def lib():
    import gated_delta_rule_29_amd as g

    return g


def bits(t):
    t = t.detach().cpu().contiguous()
    return t.view(torch.uint8 if t.element_size() == 1 else (torch.int16 if t.element_size() == 2 else torch.int32))


def new_cache(pages, H, P, D, kind, dtype):
    """A cache of poison (every byte 0x55) and its copy on the CPU."""
    ty = E4M3 if kind == "e4m3" else TYPES[dtype]
    out = {}
    for n in "kv":
        out[n] = torch.full((pages, H, P, D * (1 if kind == "e4m3" else ty.itemsize)), 0x55, dtype=torch.uint8).view(ty)
        if kind == "e4m3":
            out[n + "s"] = torch.full((pages, H, P), -3.0)
    return out


def on_gpu(c):
    return {n: t.to(DEV) for n, t in c.items()}


def scales(c):
    return {"k_scale": c["ks"], "v_scale": c["vs"]} if "ks" in c else {}


def write(c, k, v, slots, P):
    """The definition: the first row of a slot counts; slots outside the cache change nothing."""
    done = set()
    limit = c["k"].shape[0] * P
    for t, s in enumerate(slots.tolist()):
        if not 0 <= s < limit or s in done:
            continue
        done.add(s)
        for n, x in (("k", k), ("v", v)):
            if "ks" in c:
                q, scale = quantised(x[t])
                c[n].view(torch.uint8)[s // P, :, s % P] = q.view(torch.uint8)
                c[n + "s"][s // P, :, s % P] = scale
            else:
                c[n][s // P, :, s % P] = x[t]


def read(c, slots, P, dtype):
    out = {}
    limit = c["k"].shape[0] * P
    for n in "kv":
        rows = torch.zeros(len(slots), c[n].shape[1], c[n].shape[3], dtype=dtype)
        for t, s in enumerate(slots.tolist()):
            if 0 <= s < limit:
                x = c[n][s // P, :, s % P]
                rows[t] = (x.float() * c[n + "s"][s // P, :, s % P, None]).to(dtype) if "ks" in c else x
        out[n] = rows
    return out


def same(a, b):
    for n in a:
        assert torch.equal(bits(a[n]), bits(b[n])), n


KINDS = [("bf16", "same"), ("bf16", "e4m3"), ("f32", "same"), ("f32", "e4m3")]


@pytest.mark.parametrize("D", [1, 7, 64, 72, 100, 128, 200, 256, 509, 512])
@pytest.mark.parametrize("dtype,kind", KINDS)
def test_write_and_read(D, dtype, kind):
    for T, H, P, pages, how in ((1, 1, 16, 1, "dense"), (5, 3, 16, 4, "columns"), (70, 2, 64, 3, "odd"),
                                (40, 5, 1024, 1, "heads")):
        print("  case", T, H, P, pages, D, dtype, kind, how, flush=True)
        g = torch.Generator().manual_seed(T + D)
        k, v = (torch.randn(T, H, D, generator=g).to(TYPES[dtype]) for _ in range(2))
        slots = torch.randperm(pages * P, generator=g)[:T].to(torch.int32)
        if T > 3:
            slots[1], slots[3], slots[2] = -1, pages * P, slots[0]  # padded rows, and a slot named twice
        if how == "columns":
            wide = torch.full((T, 3 * H * D), float("nan"), dtype=k.dtype, device=DEV)
            dk, dv = wide[:, :H * D].view(T, H, D), wide[:, 2 * H * D:].view(T, H, D)
        elif how == "odd":
            dk, dv = (torch.full((T, H, D + 3), float("nan"), dtype=k.dtype, device=DEV)[..., 1:1 + D] for _ in "kv")
        elif how == "heads":
            dk, dv = (torch.empty(H, T, D, dtype=k.dtype, device=DEV).transpose(0, 1) for _ in "kv")
        else:
            dk, dv = (torch.empty(T, H, D, dtype=k.dtype, device=DEV) for _ in "kv")
        dk.copy_(k)
        dv.copy_(v)
        ref = new_cache(pages, H, P, D, kind, dtype)
        got = on_gpu(ref)
        lib().kv_cache_write(dk, dv, got["k"], got["v"], slots.to(DEV), **scales(got))
        write(ref, k, v, slots, P)
        same(got, ref)
        for dt in (TYPES[dtype],) if kind == "same" else (torch.bfloat16, torch.float32):
            back = lib().kv_cache_read(got["k"], got["v"], slots.to(DEV), dtype=dt, **scales(got))
            same(back, read(ref, slots, P, dt))


@pytest.mark.parametrize("T", [300, 2500, 20000])
def test_slots_named_twice(T):
    """Repeated slots anywhere in long calls: the first row of each counts."""
    g = torch.Generator().manual_seed(T)
    H, P, D = 1, 64, 8
    pages = T // P + 2
    slots = torch.randint(-5, pages * P, (T,), generator=g).to(torch.int32)
    slots[T // 2:T // 2 + 70] = slots[0] if slots[0] >= 0 else 3
    k, v = (torch.randn(T, H, D, generator=g).to(torch.bfloat16) for _ in range(2))
    ref = new_cache(pages, H, P, D, "e4m3", "bf16")
    got = on_gpu(ref)
    lib().kv_cache_write(k.to(DEV), v.to(DEV), got["k"], got["v"], slots.to(DEV), **scales(got))
    write(ref, k, v, slots, P)
    same(got, ref)


def test_rows_of_zero_and_not_finite_rows():
    H, P, D = 2, 16, 128
    k = torch.randn(4, H, D, generator=torch.Generator().manual_seed(3))
    k[0] = 0
    k[1, 0, 5] = float("nan")
    k[2, 1, 7] = float("inf")
    k[3, 0] *= 1e-30
    c = on_gpu(new_cache(1, H, P, D, "e4m3", "f32"))
    slots = torch.arange(4, dtype=torch.int32, device=DEV)
    lib().kv_cache_write(k.to(DEV), k.to(DEV), c["k"], c["v"], slots, **scales(c))
    q, s = c["k"][0].float().cpu(), c["ks"][0].cpu()
    assert (q[:, 0] == 0).all() and torch.equal(s[:, 0], torch.full((H,), 1e-12) / 448)
    assert torch.isnan(s[0, 1]) and torch.isnan(q[0, 1]).all() and torch.isfinite(q[1, 1]).all()
    assert torch.isinf(s[1, 2]) and torch.isnan(q[1, 2, 7]) and (q[1, 2, :7] == 0).all()
    want, ws = quantised(k[3])
    assert torch.equal(s[:, 3], ws) and torch.equal(q[:, 3], want.float())


def test_places_past_32_bits():
    """A cache of more than 2^32 bytes (and elements, with 8 bits): its first and last places."""
    H, P, D = 8, 128, 128
    for kind, n in (("same", 17000), ("e4m3", 34000)):
        ty = E4M3 if kind == "e4m3" else torch.bfloat16
        pages = n
        c = {x: torch.empty(pages, H, P, D, dtype=ty, device=DEV) for x in "kv"}
        if kind == "e4m3":
            c.update({x + "s": torch.empty(pages, H, P, device=DEV) for x in "kv"})
        assert c["k"].numel() * c["k"].element_size() > 1 << 32
        slots = torch.tensor([0, pages * P - 1, pages * P // 2 + 5], dtype=torch.int32, device=DEV)
        k, v = (torch.randn(3, H, D, generator=torch.Generator().manual_seed(i)).to(torch.bfloat16) for i in (1, 2))
        lib().kv_cache_write(k.to(DEV), v.to(DEV), c["k"], c["v"], slots, **scales(c))
        back = lib().kv_cache_read(c["k"], c["v"], slots, **scales(c))
        for x, t in (("k", k), ("v", v)):
            if kind == "e4m3":
                q, s = quantised(t)
                t = (q.float() * s[..., None]).to(torch.bfloat16)
            assert torch.equal(back[x].cpu(), t)
        # attention over pages at both ends (each row its own page, one key): the key's value
        table = torch.tensor([[0], [pages - 1]], dtype=torch.int32, device=DEV)
        first = torch.tensor([0, (pages - 1) * P], dtype=torch.int32, device=DEV)
        lib().kv_cache_write(k[:2].to(DEV), v[:2].to(DEV), c["k"], c["v"], first, **scales(c))
        q = torch.randn(2, H, D, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16).to(DEV)
        o = lib().paged_attn_step(q, c["k"], c["v"], table, torch.ones(2, dtype=torch.int32, device=DEV), **scales(c))
        want = lib().kv_cache_read(c["k"], c["v"], first, **scales(c))["v"]
        if kind == "same":
            assert torch.equal(o, want)
        else:
            # the weight 1 times the row's scale is rounded to bf16, (1 + a) scale, then its product with the e4m3
            # value, (1 + b); the row that is read back is (1 + c) scale value; |a|, |b|, |c| <= 2^-8, so the two
            # differ by at most 3 * 2^-8 of the value, and (2^-8)^2 terms: below 3.05 * 2^-8
            o, want = o.double(), want.double()
            assert ((o - want).abs() <= 3.05 * 2.0 ** -8 * want.abs()).all()
