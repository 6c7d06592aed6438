"""Rotary positions and their gradient against the fp64 oracle (angles reduced in exact arithmetic)."""
import numpy as np
import pytest
import torch

from oracle import attention as O
from tests.attention_util import DEV, HALF, TYPES, U, f64

pytestmark = pytest.mark.gpu

# (tokens, heads, columns, turned columns)
SIZES = [(1, 1, 2, 2), (1, 40, 128, 128), (7, 3, 64, 16), (33, 2, 80, 40), (5, 4, 256, 64), (3, 2, 33, 6), (4, 1, 31, 30),
         (2, 50, 192, 96), (130, 5, 16, 8), (1, 3, 1024, 1024), (9, 2, 24, 12)]


def lib():
    import gated_delta_rule_29_amd as g

    return g


def turned(x, positions, freqs, inter, magnitude, back):
    """(result, bound): the bound on every element is 8 u m (|u| + |w|), 0 for columns that pass."""
    xn = f64(x)
    half = len(freqs)
    ref = O.rope(xn, positions, freqs, inter, magnitude, back)
    bound = np.zeros_like(xn)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if inter else (i, i + half)
        bound[..., a] = bound[..., b] = 8 * U * magnitude * (np.abs(xn[..., a]) + np.abs(xn[..., b]))
    return ref, bound


def close(name, got, ref, bound):
    g = f64(got).reshape(ref.shape)
    err = np.abs(g - ref)
    limit = bound + np.where(bound > 0, HALF[got.dtype] * (np.abs(ref) + bound), 0.0)  # columns that pass: equal
    worst = (err[bound > 0] / limit[bound > 0]).max()
    print("  %s error at most %.3f of its bound" % (name, worst), flush=True)
    assert (err <= limit).all(), (name, worst)


def layout(x, how):
    """x [T, H, D] on the GPU: dense, as columns of a wider projection, heads first, or with nothing aligned."""
    T, H, D = x.shape
    if how == "columns":
        wide = torch.full((T, H * D + 32), float("nan"), dtype=x.dtype, device=DEV)
        out = wide[:, 16:16 + H * D].view(T, H, D)
    elif how == "heads":
        out = torch.empty(H, T, D, dtype=x.dtype, device=DEV).transpose(0, 1)
    elif how == "odd":
        out = torch.full((T, H, D + 5), float("nan"), dtype=x.dtype, device=DEV)[..., 3:3 + D]
    else:
        out = torch.empty(T, H, D, dtype=x.dtype, device=DEV)
    return out.copy_(x)


@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_forward_and_gradient(size, inter, dtype):
    T, H, D, R = size
    g = torch.Generator().manual_seed(T * 1000 + D)
    x, dy = (torch.randn(T, H, D, generator=g).to(TYPES[dtype]) for _ in range(2))
    pos = torch.randint(-50, 100000, (T,), generator=g).to(torch.int32)
    freqs, _ = lib().rope_freqs(R)
    table = lib().rope_table(freqs, DEV)
    print("  case", size, inter, dtype, flush=True)
    for how in ("dense", "columns", "heads", "odd"):
        y = lib().rope_fwd(layout(x, how), pos.to(DEV), table, interleaved=inter)
        dx = lib().rope_bwd(layout(dy, how), pos.to(DEV), table, interleaved=inter)
        assert y.is_contiguous() and y.shape == x.shape
        if how == "dense":
            first = y, dx
            close("y", y, *turned(x, pos.tolist(), freqs.tolist(), inter, 1.0, False))
            close("dx", dx, *turned(dy, pos.tolist(), freqs.tolist(), inter, 1.0, True))
        else:
            assert torch.equal(y, first[0]) and torch.equal(dx, first[1]), how


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_any_position(dtype):
    """The ends of 32 bits are as exact as the beginning; angles of quarter turns; large frequencies."""
    pos = torch.tensor([0, 1, -1, 2 ** 20 + 1, 2 ** 31 - 1, -2 ** 31, 123456789], dtype=torch.int32)
    freqs = torch.tensor([1.0, np.pi / 2, 1e-9, 0.25, 7.3, 2.0 ** -40, -0.5, 0.0], dtype=torch.float64)
    x = torch.randn(7, 3, 20, generator=torch.Generator().manual_seed(1)).to(TYPES[dtype])
    table = lib().rope_table(freqs, DEV)
    for inter in (False, True):
        y = lib().rope_fwd(x.to(DEV), pos.to(DEV), table, interleaved=inter, magnitude=1.25)
        close("y", y, *turned(x, pos.tolist(), freqs.tolist(), inter, 1.25, False))
        dx = lib().rope_bwd(x.to(DEV), pos.to(DEV), table, interleaved=inter, magnitude=1.25)
        close("dx", dx, *turned(x, pos.tolist(), freqs.tolist(), inter, 1.25, True))


def test_gradient_is_the_difference():
    """The map is linear, so a difference along any direction is the gradient's product with it: both sides are
    sums of n products of N(0, 1) values, each off by 16 u of its size."""
    g = torch.Generator().manual_seed(2)
    x, e, dy = (torch.randn(2, 9, 4, 64, generator=g).to(DEV) for _ in range(3))
    pos = torch.randint(0, 5000, (2, 9), generator=g).to(torch.int32).to(DEV)
    freqs, m = lib().rope_freqs(32, scaling="yarn", factor=4.0)
    table = lib().rope_table(freqs, DEV)
    kw = dict(magnitude=m, interleaved=True)
    d = (lib().rope_fwd(x + e, pos, table, **kw).double() - lib().rope_fwd(x, pos, table, **kw).double()) * dy.double()
    p = lib().rope_bwd(dy, pos, table, **kw).double() * e.double()
    size = (d.abs().sum() + p.abs().sum() + 2 * (x.abs().double() * dy.abs().double()).sum() * m).item()
    assert abs(d.sum().item() - p.sum().item()) <= 16 * U * 2 * size


def test_leading_dimensions_and_many_tokens():
    g = torch.Generator().manual_seed(3)
    x = torch.randn(3, 1500, 6, 64, generator=g).to(torch.bfloat16).to(DEV)
    pos = torch.arange(1500, dtype=torch.int32).expand(3, 1500).contiguous().to(DEV)
    table = lib().rope_table(lib().rope_freqs(64)[0], DEV)
    y = lib().rope_fwd(x, pos, table)
    flat = lib().rope_fwd(x.view(-1, 6, 64), pos.view(-1), table)
    assert y.shape == x.shape and torch.equal(y.view(-1, 6, 64), flat)
    some = [0, 1, 1499, 1500, 4499]
    close("y", flat[some], *turned(x.view(-1, 6, 64)[some], pos.view(-1)[some].tolist(),
                                   lib().rope_freqs(64)[0].tolist(), False, 1.0, False))


def test_rows_past_32_bits():
    """Tokens 2^31 elements and more behind the first."""
    T, H, D = 3, 2, 64
    pitch = (1 << 30) + 64
    buf = torch.empty((T - 1) * pitch + H * D, dtype=torch.bfloat16, device=DEV)
    x = buf.as_strided((T, H, D), (pitch, D, 1))
    v = torch.randn(T, H, D, generator=torch.Generator().manual_seed(4)).to(torch.bfloat16).to(DEV)
    x.copy_(v)
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    table = lib().rope_table(lib().rope_freqs(64)[0], DEV)
    assert torch.equal(lib().rope_fwd(x, pos, table), lib().rope_fwd(v, pos, table))
