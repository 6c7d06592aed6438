"""Pins of the layer operators' fp64 oracle: closed forms, library routines, split and resumed
sequences, and central differences for every gradient."""
import numpy as np
import pytest
import torch

from oracle import layer as L

RNG = np.random.default_rng(11)


def _rn(*shape):
    return RNG.standard_normal(shape)


def test_conv_is_torch_conv1d():
    x, w, b, init = _rn(9, 5), _rn(5, 4), _rn(5), _rn(1, 3, 5)
    y, last = L.conv([9], x, w, b, init, silu=False)
    line = torch.tensor(np.concatenate([init[0], x])).T[None]
    ref = torch.nn.functional.conv1d(line, torch.tensor(w)[:, None], torch.tensor(b), groups=5)[0].T
    assert np.allclose(y, ref.numpy(), atol=1e-13)
    assert np.array_equal(last[0], x[-3:])
    ys, _ = L.conv([9], x, w, b, init)
    assert np.allclose(ys, torch.nn.functional.silu(ref).numpy(), atol=1e-13)


@pytest.mark.parametrize("W", [2, 3, 4])
def test_conv_resumes(W):
    x, w, init = _rn(8, 3), _rn(3, W), _rn(1, W - 1, 3)
    y, last = L.conv([8], x, w, None, init)
    a, mid = L.conv([1], x[:1], w, None, init)  # shorter than the window
    b, end = L.conv([7], x[1:], w, None, mid)
    assert np.allclose(np.concatenate([a, b]), y) and np.allclose(end, last)


def test_scan_closed_forms():
    """No decay and unit steps: the state is the sum of B x; a decay to nothing: y = B.C de x."""
    x, B, C = _rn(6, 2), _rn(6, 3), _rn(6, 3)
    one = np.ones((6, 2))
    y, ht, _ = L.scan([6], x, one, np.zeros((2, 3)), B, C, use_softplus=False)
    assert np.allclose(ht[0], np.einsum("td,tn->dn", x, B))
    assert np.allclose(y, np.einsum("tn,sn,sd,ts->td", C, B, x, np.tril(np.ones((6, 6)))))
    y, _, _ = L.scan([6], x, one, np.full((2, 3), -800.0), B, C, h0=_rn(1, 2, 3), use_softplus=False)
    assert np.allclose(y, x * (B * C).sum(1)[:, None])


def test_scan_resumes_and_packs():
    x, dt, A, B, C, h0 = _rn(7, 2), _rn(7, 2), -np.abs(_rn(2, 3)), _rn(7, 3), _rn(7, 3), _rn(2, 2, 3)
    y, ht, h = L.scan([3, 4], x, dt, A, B, C, h0=h0, chunk=2)
    y0, e0, _ = L.scan([3], x[:3], dt[:3], A, B[:3], C[:3], h0=h0[:1])
    assert np.allclose(y[:3], y0) and np.allclose(ht[0], e0[0])
    assert h.shape == (4, 2, 3) and np.allclose(h[0], h0[0]) and np.allclose(h[2], h0[1])
    y1, e1, _ = L.scan([2], x[5:], dt[5:], A, B[5:], C[5:], h0=h[3:])
    assert np.allclose(y[5:], y1) and np.allclose(ht[1], e1[0])


def _check_grads(loss, args, grads, eps=1e-6):
    """Central differences of loss(**args) by every entry of the arrays named in grads.  Their error is
    about eps^2 times a third derivative and 1e-16 |loss| / eps of cancellation: below 1e-7 of
    values of order one."""
    for name, g in grads.items():
        base = args[name]
        for at in np.ndindex(base.shape):
            keep = base[at]
            base[at] = keep + eps
            hi = loss(**args)
            base[at] = keep - eps
            lo = loss(**args)
            base[at] = keep
            assert abs((hi - lo) / (2 * eps) - g[at]) <= 1e-7 * max(1.0, np.abs(g).max()), (name, at)


@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("W", [2, 4])
def test_conv_gradient(W, silu):
    lens = [1, 4, 2]
    a = dict(x=_rn(7, 2), w=_rn(2, W), bias=_rn(2), init=_rn(3, W - 1, 2))
    dy, dl = _rn(7, 2), _rn(3, W - 1, 2)

    def loss(x, w, bias, init):
        y, last = L.conv(lens, x, w, bias, init, silu)
        return (y * dy).sum() + (last * dl).sum()

    g = L.conv_bwd(lens, dy, a["x"], a["w"], a["bias"], a["init"], dl, silu)
    _check_grads(loss, a, dict(x=g["dx"], w=g["dw"], bias=g["dbias"], init=g["dinit"]))


@pytest.mark.parametrize("use_softplus", [True, False])
def test_scan_gradient(use_softplus):
    lens = [1, 4]
    a = dict(x=_rn(5, 2), dt=0.3 * _rn(5, 2), A=-np.abs(_rn(2, 3)), Bm=_rn(5, 3), Cm=_rn(5, 3), skip=_rn(2),
             z=_rn(5, 2), dt_bias=0.3 * _rn(2), h0=_rn(2, 2, 3))
    dy, dh = _rn(5, 2), _rn(2, 2, 3)

    def loss(**k):
        y, ht, _ = L.scan(lens, use_softplus=use_softplus, **k)
        return (y * dy).sum() + (ht * dh).sum()

    g = L.scan_bwd(lens, dy, dht=dh, use_softplus=use_softplus, **a)
    _check_grads(loss, a, dict(x=g["dx"], dt=g["ddt"], A=g["dA"], Bm=g["dB"], Cm=g["dC"], skip=g["dD"], z=g["dz"],
                               dt_bias=g["ddt_bias"], h0=g["dh0"]))


def test_norm_is_torch_rms_norm_and_its_gradient():
    s, w = _rn(3, 6), _rn(6)
    y, _ = L.norm(s, w, 1e-5)
    ref = torch.nn.functional.rms_norm(torch.tensor(s), (6,), torch.tensor(w), 1e-5)
    assert np.allclose(y, ref.numpy(), atol=1e-13)
    dy, ds = _rn(3, 6), _rn(3, 6)
    g = L.norm_bwd(dy, s, w, 1e-5, ds)
    _check_grads(lambda s, w: (L.norm(s, w, 1e-5)[0] * dy).sum() + (s * ds).sum(), dict(s=s, w=w),
                 dict(s=g["ds"], w=g["dw"]))


def test_scales():
    y = np.zeros((2, 200))
    y[0, 3], y[0, 150], y[1, 199] = -4.48, 8.96, 448.0
    assert np.allclose(L.norm_scales(y, 0), [[0.02], [1.0]])
    assert np.allclose(L.norm_scales(y, 128), [[0.01, 0.02], [1e-12 / 448, 1.0]])
