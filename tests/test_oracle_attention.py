"""The oracle of the full-attention layers' operators, pinned to library routines and closed forms."""
import math

import numpy as np
import torch

from oracle import attention as O


def rng(seed):
    return np.random.default_rng(seed)


def test_cos_sin_of_far_positions():
    # 2^31 - 1 and -2^31 positions at one radian: reduced by hand with 60 digits of pi
    for p in (0, 1, 7, -3, 1000):
        c, s = O.cos_sin(p, 0.37)
        assert abs(c - math.cos(0.37 * p)) < 1e-12 and abs(s - math.sin(0.37 * p)) < 1e-12
    big = 2 ** 31 - 1
    c, s = O.cos_sin(big, 1.0)
    assert abs(c * c + s * s - 1) < 1e-15
    c1, s1 = O.cos_sin(big - 1, 1.0)
    d, e = O.cos_sin(1, 1.0)  # addition theorem
    assert abs(c1 * d - s1 * e - c) < 1e-14 and abs(s1 * d + c1 * e - s) < 1e-14


def test_rope_is_a_rotation_and_its_gradient_the_transpose():
    g = rng(0)
    x, dy = g.standard_normal((5, 2, 12)), g.standard_normal((5, 2, 12))
    pos, freqs = np.array([0, 3, -2, 100, 7]), np.array([1.0, 0.3, 0.01, 0.2])
    for inter in (False, True):
        y = O.rope(x, pos, freqs, inter)
        assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1), rtol=1e-14)
        assert np.array_equal(y[..., 8:], x[..., 8:]) and np.array_equal(y[0], x[0])
        dx = O.rope(dy, pos, freqs, inter, back=True)
        assert np.allclose(O.rope(y, pos, freqs, inter, back=True), x, atol=1e-14)
        # linear: the difference along any direction is the gradient's product with it
        e = g.standard_normal(x.shape)
        diff = ((O.rope(x + e, pos, freqs, inter, 1.5) - O.rope(x, pos, freqs, inter, 1.5)) * dy).sum()
        assert abs(diff - (O.rope(dy, pos, freqs, inter, 1.5, back=True) * e).sum()) < 1e-11
    z = torch.view_as_complex(torch.tensor(x[..., :8]).unflatten(-1, (4, 2)))
    a = torch.outer(torch.tensor(pos, dtype=torch.float64), torch.tensor(freqs))
    want = torch.view_as_real(z * torch.polar(torch.ones_like(a), a)[:, None]).flatten(-2)
    assert np.allclose(O.rope(x, pos, freqs, True)[..., :8], want.numpy(), atol=1e-12)


def test_attention_is_the_librarys():
    g = rng(1)
    for n, L, causal, window in ((3, 3, True, 0), (2, 9, True, 0), (4, 9, True, 3), (5, 2, False, 0), (1, 1, True, 0)):
        q, k, v = g.standard_normal((n, 4, 8)), g.standard_normal((L, 2, 8)), g.standard_normal((L, 2, 8))
        at = torch.arange(L - n, L)[:, None] - torch.arange(L)
        mask = (at >= 0) & ((at < window) if window else True) if causal else torch.ones(n, L, dtype=torch.bool)
        want = torch.nn.functional.scaled_dot_product_attention(
            torch.tensor(q).transpose(0, 1), torch.tensor(k).repeat_interleave(2, 1).transpose(0, 1),
            torch.tensor(v).repeat_interleave(2, 1).transpose(0, 1), attn_mask=mask, scale=0.4).transpose(0, 1)
        o, lse, mean, _ = O.attention(q, k, v, n, 0.4, causal, window)
        assert np.allclose(o, want.numpy(), atol=1e-13)
        assert (mean >= np.abs(o) - 1e-13).all()
        one = O.attention(q, k, np.ones_like(v), n, 0.4, causal, window)[0]
        assert np.allclose(one, 1.0)


def test_attention_without_keys():
    g = rng(2)
    q, k = g.standard_normal((3, 2, 4)), g.standard_normal((1, 1, 4))
    o, lse, _, _ = O.attention(q, k, k, 3, 1.0)
    assert (o[:2] == 0).all() and np.isneginf(lse[:2]).all() and np.allclose(o[2], k[0])  # one key: its value
    o, lse, _, _ = O.attention(q, k[:0], k[:0], 3, 1.0, causal=False)
    assert (o == 0).all() and np.isneginf(lse).all()


def test_rows_of():
    c = np.arange(2 * 1 * 2 * 1, dtype=np.float64).reshape(2, 1, 2, 1)
    assert O.rows_of(c, [1, 0, 7], 5)[:, 0, 0].tolist() == [2, 3, 0, 1, 0]
