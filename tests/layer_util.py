"""Inputs and the comparison rule of the layer operators' GPU tests.

Tolerance: max over elements of the error over the RMS of the oracle's values, at most 2e-5, for
every output; the storage rounding of bf16 outputs is not counted (tests/gpu_util.py).  A result goes
through at most about 40 fp32 roundings in a row (the step size's exponential, reciprocal and eight
series terms; the decay's argument, where an error of u |arg| is worth u |arg| e^{-|arg|} < u / 2; the
recurrence, whose older roundings decay with the state; the output's products), each at most
u = 2^-24 relative, and the largest element is at most 8 RMS: 40 * 8 u = 1.9e-5.  Sums over
channels or tokens of terms of either sign gain no more: their errors add up as the terms do.
"""
import torch

from tests.gpu_util import assert_close

TOL32 = 2e-5
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
DEV = "cuda:0"


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g).to(dtype)


def pitched(t, extra, offset):
    """The values of t [.., C] on the GPU as columns of a wider tensor: `offset` elements in, rows C +
    extra apart; the columns around them hold NaN."""
    wide = torch.full((*t.shape[:-1], t.shape[-1] + extra), float("nan"), dtype=t.dtype, device=DEV)
    out = wide[..., offset:offset + t.shape[-1]]
    out.copy_(t)
    return out


def check(name, got, ref, tol=TOL32):
    assert torch.isfinite(got.float()).all(), "%s has values that are not finite" % name
    assert_close(name, got, ref, tol)


def rows(lens, dense):
    """(leading shape, cu) of a dense batch (all lens equal) or a packed one."""
    if dense:
        return (len(lens), lens[0]), None
    cu = torch.zeros(len(lens) + 1, dtype=torch.int32)
    cu[1:] = torch.tensor(lens).cumsum(0)
    return (1, sum(lens)), cu


def flat(t):
    return None if t is None else t.detach().cpu().double().reshape(-1, t.shape[-1]).numpy()


def arr(t):
    return None if t is None else t.detach().cpu().double().numpy()
