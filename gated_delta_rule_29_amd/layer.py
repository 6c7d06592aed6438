"""Layer operators around the recurrent scans: the short causal convolution, the selective state space
scan and the residual RMS norm, each with its gradient, and for single tokens on a cache.

As everywhere in the binding, arguments are marshalled and shapes checked here; every step of the
method runs in the library.  Row inputs (activations) may be columns of a wider tensor: the last
dimension has to be dense and the rows evenly spaced.  Everything else is contiguous.  Calls run on the
inputs' device, on its current stream.
"""
from __future__ import annotations

import torch

from . import _lib

__all__ = ["causal_conv_fwd", "causal_conv_fwd_varlen", "causal_conv_bwd", "causal_conv_bwd_varlen",
           "causal_conv_step", "ssm_scan_fwd", "ssm_scan_fwd_varlen", "ssm_scan_bwd", "ssm_scan_bwd_varlen",
           "ssm_step", "rms_norm_fwd", "rms_norm_q8_fwd", "rms_norm_bwd", "SSM_CHUNK"]

SSM_CHUNK = 16
F32 = torch.float32
_DT = {torch.float32: _lib.DTYPE_F32, torch.bfloat16: _lib.DTYPE_BF16}


def _ptr(t):
    return None if t is None else t.data_ptr()


def _refuse(t, name, shape, dtype, dev, why):
    """Says what is wrong with a tensor that failed a check: why, unless it is its kind or shape."""
    if not isinstance(t, torch.Tensor):
        why = "%s must be a torch.Tensor" % name
    elif t.shape != shape:
        why = "%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape))
    elif t.dtype != dtype:
        why = "%s has dtype %s, expected %s" % (name, t.dtype, dtype)
    elif t.device != dev:
        why = "%s is on %s, expected %s" % (name, t.device, dev)
    raise ValueError(why)


# The checks are written out: single-token calls are bound by the time that they take on the host.

def _need(t, name, shape, dtype, dev):
    """Address of a contiguous tensor, or None for None where the caller allows that."""
    if t is None:
        return None
    if not (isinstance(t, torch.Tensor) and t.shape == shape and t.dtype is dtype and t.device == dev
            and t.is_contiguous()):
        _refuse(t, name, shape, dtype, dev, "%s must be contiguous" % name)
    return t.data_ptr()


def _rows(t, name, shape, dtype, dev):
    """The pitch of a row tensor [.., C]: elements from one row to the next, over all its rows."""
    if not (isinstance(t, torch.Tensor) and t.shape == shape and t.dtype is dtype and t.device == dev):
        _refuse(t, name, shape, dtype, dev, None)
    if t.is_contiguous():
        return shape[-1]
    strides = t.stride()
    pitch, span = None, None  # of the innermost dimension with more than one row; rows so far
    for n, s in zip(reversed(shape[:-1]), reversed(strides[:-1])):
        if n == 1:
            continue
        if pitch is None:
            pitch, span = s, n
        elif s != pitch * span:
            raise ValueError("%s must have evenly spaced rows (strides %s of shape %s)"
                             % (name, tuple(strides), tuple(shape)))
        else:
            span *= n
    if pitch is None:
        pitch = shape[-1]
    if (strides[-1] != 1 and shape[-1] != 1) or pitch < shape[-1]:
        raise ValueError("%s must have dense rows that do not overlap (strides %s of shape %s)"
                         % (name, tuple(strides), tuple(shape)))
    return pitch


def _act(x, name, dims):
    """(device, dtype, library dtype) of the activations."""
    if not isinstance(x, torch.Tensor):
        raise ValueError("%s must be a torch.Tensor" % name)
    if x.dim() != dims:
        raise ValueError("%s must have %d dimensions, got shape %s" % (name, dims, tuple(x.shape)))
    if x.dtype not in _DT:
        raise ValueError("%s must be float32 or bfloat16, got %s" % (name, x.dtype))
    return x.device, x.dtype, _DT[x.dtype]


def _call(name, dev, *args):
    """The library's entry point on the device's current stream."""
    if dev.type != "cuda":
        raise ValueError("%s needs tensors on a GPU, got %s" % (name, dev))
    fn = getattr(_lib.load(), name)
    # the current stream's handle without a Stream object around it: 0.1 us against 1.9 us
    if torch.cuda.current_device() == dev.index:
        rc = fn(*args, torch._C._cuda_getCurrentRawStream(dev.index))
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, torch._C._cuda_getCurrentRawStream(dev.index))
    if rc:
        _lib.check(rc, name)


_INT = 0x7fffffff  # the library's sizes are 32-bit integers: ctypes would pass on the low bits of larger ones


def _large(*sizes):
    raise ValueError("sizes beyond 32 bits: %s" % (sizes,))


_CPU = torch.device("cpu")


def _int32(t, dev):
    return isinstance(t, torch.Tensor) and t.dtype == torch.int32 and t.device == dev and t.is_contiguous()


def _like(x):
    """A new contiguous tensor of x's shape, type and device."""
    return torch.empty_like(x, memory_format=torch.contiguous_format)


def _workspace(nbytes, dev):
    return torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None


_DENSE = object()  # in the place of a dense call's offsets


class _Seqs:
    """The sequences of a call: a dense batch, or the offsets of a packed one."""

    def __init__(self, x, cu_seqlens=_DENSE, cu_seqlens_host=None):
        if x.shape[0] * x.shape[1] > _INT or x.shape[2] > _INT:
            _large(x.shape[0] * x.shape[1], x.shape[2])
        self.packed = cu_seqlens is not _DENSE
        if self.packed:
            if cu_seqlens is None:
                raise ValueError("a packed call needs cu_seqlens")
            if x.shape[0] != 1:
                raise ValueError("packed input must have batch 1, got %d" % x.shape[0])
            if _int32(cu_seqlens, x.device) and _int32(cu_seqlens_host, _CPU) \
                    and cu_seqlens.shape == cu_seqlens_host.shape:
                self.cu, self.host = cu_seqlens, cu_seqlens_host  # as they are (what a serving loop passes)
            else:
                from . import _cu_pair

                self.cu, self.host = _cu_pair(cu_seqlens, cu_seqlens_host, x.device)
            if self.host.dim() != 1 or self.host.numel() < 2:
                raise ValueError("cu_seqlens must hold at least two offsets")
            self.n = self.host.numel() - 1
        else:
            self.n = x.shape[0]

    def name(self, base):
        return base + "_varlen" if self.packed else base

    def offsets(self):
        return (self.cu.data_ptr(), self.host.data_ptr(), self.n) if self.packed else ()

    def sizes(self, x):
        return (x.shape[1],) if self.packed else (x.shape[0], x.shape[1])

    def chunks(self, x):
        """(leading dimension, chunks) of the saved states."""
        if not self.packed:
            return x.shape[0], (x.shape[1] + SSM_CHUNK - 1) // SSM_CHUNK
        n = _lib.load().ssm_scan_num_chunks(self.host.data_ptr(), self.n)
        if n < 0:
            raise ValueError("malformed cu_seqlens: %s" % self.host.tolist()[:16])
        return 1, n


# ----------------------------------------------------------------------------------- convolution

def _conv_fwd(x, w, bias, init, silu, want_last, cu=_DENSE, cu_host=None):
    dev, dt, code = _act(x, "x", 3)
    seqs = _Seqs(x, cu, cu_host)
    D = x.shape[2]
    if not isinstance(w, torch.Tensor) or w.dim() != 2:
        raise ValueError("w must be a [D, W] tensor")
    W = w.shape[1]
    if W > _INT:
        _large(W)
    pitch = _rows(x, "x", x.shape, dt, dev)
    wp, bp = _need(w, "w", (D, W), F32, dev), _need(bias, "bias", (D,), F32, dev)
    edge = (seqs.n, max(W - 1, 0), D)
    ip = _need(init, "init", edge, dt, dev)
    y = _like(x)
    last = torch.empty(edge, dtype=dt, device=dev) if want_last else None
    _call(seqs.name("causal_conv_fwd"), dev, x.data_ptr(), pitch, wp, bp, *seqs.offsets(),
          ip, y.data_ptr(), _ptr(last), *seqs.sizes(x), D, W, 1 if silu else 0, code)
    return {"y": y, "final": last} if want_last else {"y": y}


def causal_conv_fwd(x, w, bias=None, init=None, *, silu=True, want_final=True):
    """Short causal convolution, one filter of W (2..4) taps a channel:
    ``u_t = bias + sum_i w[:, i] x_{t-(W-1)+i}``, ``y = u * sigmoid(u)`` (or u).

    x [B,T,D] (fp32 or bf16; rows may be pitched), w [D,W], bias [D] fp32, init [B,W-1,D]: the tokens
    before the first one, oldest first (zero by default).  Returns y [B,T,D] and, unless want_final is
    off, final [B,W-1,D]: the last W-1 tokens, the init of the call that goes on."""
    return _conv_fwd(x, w, bias, init, silu, want_final)


def causal_conv_fwd_varlen(x, w, cu_seqlens, bias=None, init=None, *, silu=True, want_final=True,
                           cu_seqlens_host=None):
    """causal_conv_fwd over packed sequences: x [1,T,D], init and final [N,W-1,D]; cu_seqlens and
    cu_seqlens_host as in gdn_fwd_varlen."""
    return _conv_fwd(x, w, bias, init, silu, want_final, cu_seqlens, cu_seqlens_host)


def _conv_bwd(dy, x, w, bias, init, dfinal, silu, cu=_DENSE, cu_host=None):
    dev, dt, code = _act(x, "x", 3)
    seqs = _Seqs(x, cu, cu_host)
    D = x.shape[2]
    if not isinstance(w, torch.Tensor) or w.dim() != 2:
        raise ValueError("w must be a [D, W] tensor")
    W = w.shape[1]
    if W > _INT:
        _large(W)
    pitch, dy_pitch = _rows(x, "x", x.shape, dt, dev), _rows(dy, "dy", x.shape, dt, dev)
    _need(w, "w", (D, W), F32, dev)
    _need(bias, "bias", (D,), F32, dev)
    edge = (seqs.n, max(W - 1, 0), D)
    _need(init, "init", edge, dt, dev)
    _need(dfinal, "dfinal", edge, dt, dev)
    out = {"dx": _like(x), "dw": torch.empty_like(w)}
    if bias is not None:
        out["dbias"] = torch.empty_like(bias)
    if init is not None:
        out["dinit"] = torch.empty_like(init)
    n = _lib.load().causal_conv_bwd_workspace_bytes(x.shape[0] * x.shape[1], D, W)
    ws = _workspace(n, dev)
    _call(seqs.name("causal_conv_bwd"), dev, _ptr(dy), dy_pitch, _ptr(x), pitch, _ptr(w), _ptr(bias),
          *seqs.offsets(), _ptr(init), _ptr(dfinal), _ptr(out["dx"]), _ptr(out.get("dinit")),
          _ptr(out["dw"]), _ptr(out.get("dbias")), *seqs.sizes(x), D, W, 1 if silu else 0, code,
          _ptr(ws), n)
    return out


def causal_conv_bwd(dy, x, w, bias=None, init=None, dfinal=None, *, silu=True):
    """Gradient of causal_conv_fwd from its inputs, dy [B,T,D] and dfinal [B,W-1,D] (zero by default).
    Returns dx, dw [D,W] fp32, and dbias / dinit where bias / init are given."""
    return _conv_bwd(dy, x, w, bias, init, dfinal, silu)


def causal_conv_bwd_varlen(dy, x, w, cu_seqlens, bias=None, init=None, dfinal=None, *, silu=True,
                           cu_seqlens_host=None):
    """Gradient of causal_conv_fwd_varlen."""
    return _conv_bwd(dy, x, w, bias, init, dfinal, silu, cu_seqlens, cu_seqlens_host)


def _slots(state, slots, B, dev):
    """Address of the slots."""
    if slots is None and state.shape[0] < B:
        raise ValueError("without slots the cache needs a slot a row: %d rows, %d slots" % (B, state.shape[0]))
    return _need(slots, "slots", (B,), torch.int32, dev)


def causal_conv_step(x, w, state, bias=None, *, slots=None, silu=True):
    """causal_conv_fwd for one token a row on a cache, which moves on by one token in place.

    x [B,D], w [D,W], state [S,W-1,D] (x's type), slots [B] int32: the slot of each row (row b uses
    slot b by default).  A row whose slot is outside the cache (-1: a padded row) or is an earlier
    row's changes nothing and gives 0.  Returns y [B,D]."""
    dev, dt, code = _act(x, "x", 2)
    B, D = x.shape
    if not isinstance(w, torch.Tensor) or w.dim() != 2 or not isinstance(state, torch.Tensor) or state.dim() != 3:
        raise ValueError("w must be a [D, W] and state a [S, W-1, D] tensor")
    W, S = w.shape[1], state.shape[0]
    if B > _INT or S > _INT or D > _INT or W > _INT:
        _large(B, S, D, W)
    pitch = _rows(x, "x", x.shape, dt, dev)
    wp, bp = _need(w, "w", (D, W), F32, dev), _need(bias, "bias", (D,), F32, dev)
    sp = _need(state, "state", (S, max(W - 1, 0), D), dt, dev)
    lp = _slots(state, slots, B, dev)
    y = _like(x)
    _call("causal_conv_step", dev, x.data_ptr(), pitch, wp, bp, sp, lp, y.data_ptr(), B, S, D, W, 1 if silu else 0,
          code)
    return y


# ------------------------------------------------------------------------------------------ scan

def _scan_args(x, dt_, A, Bm, Cm, skip, z, dt_bias, dev, dt):
    """The scan's inputs as the library takes them, up to Cm, and from skip to dt_bias."""
    *lead, D = x.shape
    if not isinstance(A, torch.Tensor) or A.dim() != 2:
        raise ValueError("A must be a [D, N] tensor")
    N = A.shape[1]
    if D > _INT or N > _INT:
        _large(D, N)
    shape, per_n = x.shape, (*lead, N)
    px, pd = _rows(x, "x", shape, dt, dev), _rows(dt_, "dt", shape, dt, dev)
    ap = _need(A, "A", (D, N), F32, dev)
    pb, pc = _rows(Bm, "Bm", per_n, dt, dev), _rows(Cm, "Cm", per_n, dt, dev)
    kp, tp = _need(skip, "D", (D,), F32, dev), _need(dt_bias, "dt_bias", (D,), F32, dev)
    zp, pz = (z.data_ptr(), _rows(z, "z", shape, dt, dev)) if z is not None else (None, 0)
    return N, (x.data_ptr(), px, dt_.data_ptr(), pd, ap, Bm.data_ptr(), pb, Cm.data_ptr(), pc), (kp, zp, pz, tp)


def _scan_workspace(which, seqs, x, N):
    lib, D = _lib.load(), x.shape[2]
    if seqs.packed:
        return getattr(lib, "ssm_scan_%s_varlen_workspace_bytes" % which)(seqs.host.data_ptr(), seqs.n, D, N)
    return getattr(lib, "ssm_scan_%s_workspace_bytes" % which)(x.shape[0], x.shape[1], D, N)


def _scan_fwd(x, dt, A, Bm, Cm, skip, z, dt_bias, h0, softplus, want_ht, want_h, cu=_DENSE, cu_host=None):
    dev, ty, code = _act(x, "x", 3)
    seqs = _Seqs(x, cu, cu_host)
    N, ins, opts = _scan_args(x, dt, A, Bm, Cm, skip, z, dt_bias, dev, ty)
    D = x.shape[2]
    _need(h0, "h0", (seqs.n, D, N), F32, dev)
    y = _like(x)
    ht = torch.empty(seqs.n, D, N, dtype=F32, device=dev) if want_ht else None
    h = torch.empty(*seqs.chunks(x), D, N, dtype=F32, device=dev) if want_h else None
    n = _scan_workspace("fwd", seqs, x, N)
    ws = _workspace(n, dev)
    _call(seqs.name("ssm_scan_fwd"), dev, *ins, *seqs.offsets(), *opts, _ptr(h0), _ptr(y), _ptr(ht), _ptr(h),
          *seqs.sizes(x), D, N, 1 if softplus else 0, code, _ptr(ws), n)
    out = {"y": y}
    if want_ht:
        out["ht"] = ht
    if want_h:
        out["h"] = h
    return out


def ssm_scan_fwd(x, dt, A, Bm, Cm, D=None, z=None, dt_bias=None, h0=None, *, softplus=True, want_ht=True,
                 want_h=False):
    """Selective state space scan, N (1..64) states a channel:
    ``de = softplus(dt + dt_bias)`` (or dt + dt_bias), ``h_t = exp(de_t A) h_{t-1} + de_t x_t B_t``,
    ``y_t = (h_t . C_t + D x_t) * (z * sigmoid(z) where z is given)``.

    x, dt, z [B,T,C] and Bm, Cm [B,T,N] (one type, fp32 or bf16; rows may be pitched), A [C,N], D and
    dt_bias [C], h0 [B,C,N] fp32.  Returns y [B,T,C] and, when requested, ht [B,C,N] fp32 and h
    [B,NC,C,N] fp32: the states entering each chunk of SSM_CHUNK tokens, which ssm_scan_bwd needs."""
    return _scan_fwd(x, dt, A, Bm, Cm, D, z, dt_bias, h0, softplus, want_ht, want_h)


def ssm_scan_fwd_varlen(x, dt, A, Bm, Cm, cu_seqlens, D=None, z=None, dt_bias=None, h0=None, *, softplus=True,
                        want_ht=True, want_h=False, cu_seqlens_host=None):
    """ssm_scan_fwd over packed sequences: tokens [1,T,.], h0 and ht [N_seq,C,N], h [1,NC_total,C,N] with
    the sequences' chunks in order; cu_seqlens and cu_seqlens_host as in gdn_fwd_varlen."""
    return _scan_fwd(x, dt, A, Bm, Cm, D, z, dt_bias, h0, softplus, want_ht, want_h, cu_seqlens, cu_seqlens_host)


def _scan_bwd(dy, h, x, dt, A, Bm, Cm, skip, z, dt_bias, dht, softplus, want_dh0, cu=_DENSE, cu_host=None):
    dev, ty, code = _act(x, "x", 3)
    seqs = _Seqs(x, cu, cu_host)
    N, ins, opts = _scan_args(x, dt, A, Bm, Cm, skip, z, dt_bias, dev, ty)
    D = x.shape[2]
    dy_pitch = _rows(dy, "dy", x.shape, ty, dev)
    if h is None:
        raise ValueError("h is needed: the states that the forward saves with want_h")
    _need(h, "h", (*seqs.chunks(x), D, N), F32, dev)
    _need(dht, "dht", (seqs.n, D, N), F32, dev)

    def rows(width):
        return torch.empty(*x.shape[:2], width, dtype=ty, device=dev)

    out = {"dx": _like(x), "ddt": _like(x), "dA": torch.empty_like(A), "dB": rows(N), "dC": rows(N)}
    if skip is not None:
        out["dD"] = torch.empty_like(skip)
    if z is not None:
        out["dz"] = _like(x)
    if dt_bias is not None:
        out["ddt_bias"] = torch.empty_like(dt_bias)
    if want_dh0:
        out["dh0"] = torch.empty(seqs.n, D, N, dtype=F32, device=dev)
    n = _scan_workspace("bwd", seqs, x, N)
    ws = _workspace(n, dev)
    g = out.get
    _call(seqs.name("ssm_scan_bwd"), dev, _ptr(dy), dy_pitch, _ptr(h), *ins, *seqs.offsets(), *opts, _ptr(dht),
          _ptr(g("dx")), _ptr(g("ddt")), _ptr(g("dA")), _ptr(g("dB")), _ptr(g("dC")), _ptr(g("dD")),
          _ptr(g("dz")), _ptr(g("ddt_bias")), _ptr(g("dh0")), *seqs.sizes(x), D, N, 1 if softplus else 0, code,
          _ptr(ws), n)
    return out


def ssm_scan_bwd(dy, h, x, dt, A, Bm, Cm, D=None, z=None, dt_bias=None, dht=None, *, softplus=True,
                 want_dh0=False):
    """Gradient of ssm_scan_fwd from its inputs, the states h that it saved, dy [B,T,C] and dht [B,C,N]
    (zero by default).  Returns dx, ddt [B,T,C], dA [C,N], dB, dC [B,T,N], and dD, dz, ddt_bias where
    those inputs are given, dh0 [B,C,N] when requested."""
    return _scan_bwd(dy, h, x, dt, A, Bm, Cm, D, z, dt_bias, dht, softplus, want_dh0)


def ssm_scan_bwd_varlen(dy, h, x, dt, A, Bm, Cm, cu_seqlens, D=None, z=None, dt_bias=None, dht=None, *,
                        softplus=True, want_dh0=False, cu_seqlens_host=None):
    """Gradient of ssm_scan_fwd_varlen."""
    return _scan_bwd(dy, h, x, dt, A, Bm, Cm, D, z, dt_bias, dht, softplus, want_dh0, cu_seqlens, cu_seqlens_host)


def ssm_step(x, dt, A, Bm, Cm, state, D=None, z=None, dt_bias=None, *, slots=None, softplus=True):
    """ssm_scan_fwd for one token a row on a cache of states, updated in place.

    x, dt, z [B,C], Bm, Cm [B,N], state [S,C,N] fp32, slots [B] int32 as in causal_conv_step.
    Returns y [B,C]."""
    dev, ty, code = _act(x, "x", 2)
    B, C = x.shape
    if not isinstance(state, torch.Tensor) or state.dim() != 3:
        raise ValueError("state must be a [S, C, N] tensor")
    N, ins, opts = _scan_args(x, dt, A, Bm, Cm, D, z, dt_bias, dev, ty)
    S = state.shape[0]
    if B > _INT or S > _INT:
        _large(B, S)
    sp = _need(state, "state", (S, C, N), F32, dev)
    lp = _slots(state, slots, B, dev)
    y = _like(x)
    _call("ssm_step", dev, *ins, *opts, sp, lp, y.data_ptr(), B, S, C, N, 1 if softplus else 0, code)
    return y


# ------------------------------------------------------------------------------------------ norm

def _norm_args(x, w, residual):
    if not isinstance(x, torch.Tensor) or x.dim() < 1:
        raise ValueError("x must be a tensor [.., D]")
    dev, dt, code = _act(x, "x", x.dim())
    shape = x.shape
    D = shape[-1]
    M = x.numel() // max(D, 1)
    if M > _INT or D > _INT:
        _large(M, D)
    pitch = _rows(x, "x", shape, dt, dev)
    wp = _need(w, "w", (D,), F32, dev)
    rcode, rpitch, rp = code, 0, None
    if residual is not None:
        if not isinstance(residual, torch.Tensor) or residual.dtype not in _DT:
            raise ValueError("residual must be a float32 or bfloat16 tensor")
        rcode = _DT[residual.dtype]
        rp, rpitch = residual.data_ptr(), _rows(residual, "residual", shape, residual.dtype, dev)
    return dev, code, rcode, D, M, (x.data_ptr(), pitch, rp, rpitch, wp)


def rms_norm_fwd(x, w, residual=None, eps=1e-5, *, want_rstd=False):
    """Root-mean-square norm over the last dimension, with the residual's addition:
    ``sum = x + residual`` in the residual's type, ``y = sum * rsqrt(mean(sum^2) + eps) * w`` in x's.

    x [..,D] (fp32 or bf16; rows may be pitched), w [D] fp32, residual [..,D] of x's type or fp32.
    Returns y, sum where a residual is given, and rstd [..] fp32 (for rms_norm_bwd) when requested."""
    dev, code, rcode, D, M, ins = _norm_args(x, w, residual)
    y = _like(x)
    out = {"y": y}
    sp = rp = None
    if residual is not None:
        out["sum"] = s = _like(residual)
        sp = s.data_ptr()
    if want_rstd:
        out["rstd"] = r = torch.empty(x.shape[:-1], dtype=F32, device=dev)
        rp = r.data_ptr()
    _call("rms_norm_fwd", dev, *ins, eps, y.data_ptr(), sp, rp, M, D, code, rcode)
    return out


def rms_norm_q8_fwd(x, w, residual=None, eps=1e-5, *, block=0):
    """rms_norm_fwd with y in 8 bits: q [..,D] float8_e4m3fn and scale fp32 with y = q * scale.

    block 0: one scale a row, scale [..,1]; block 128: one for each 128 columns, scale
    [..,ceil(D/128)].  ``scale = max(max |y|, 1e-12) / 448``.  Returns q, scale, and sum where a
    residual is given."""
    dev, code, rcode, D, M, ins = _norm_args(x, w, residual)
    out = {"q": torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=dev),
           "scale": torch.empty(*x.shape[:-1], (D + 127) // 128 if block else 1, dtype=F32, device=dev)}
    if residual is not None:
        out["sum"] = _like(residual)
    _call("rms_norm_q8_fwd", dev, *ins, eps, int(block), _ptr(out["q"]), _ptr(out["scale"]), _ptr(out.get("sum")),
          M, D, code, rcode)
    return out


def rms_norm_bwd(dy, s, w, rstd, dsum=None):
    """Gradient of rms_norm_fwd from the normalised values s (its sum; x where there was no residual)
    and rstd.  dsum: gradient of the sum itself (zero by default), s's type.

    Returns dx in dy's type, dresidual in s's (the same tensor where the types agree), dw [D] fp32."""
    if not isinstance(dy, torch.Tensor) or dy.dim() < 1:
        raise ValueError("dy must be a tensor [.., D]")
    dev, dt, code = _act(dy, "dy", dy.dim())
    D = dy.shape[-1]
    M = dy.numel() // max(D, 1)
    if M > _INT or D > _INT:
        _large(M, D)
    if not isinstance(s, torch.Tensor) or s.dtype not in _DT:
        raise ValueError("s must be a float32 or bfloat16 tensor")
    pitch, s_pitch = _rows(dy, "dy", dy.shape, dt, dev), _rows(s, "s", dy.shape, s.dtype, dev)
    d_pitch = _rows(dsum, "dsum", dy.shape, s.dtype, dev) if dsum is not None else 0
    _need(w, "w", (D,), F32, dev)
    if rstd is None:
        raise ValueError("rstd is needed: rms_norm_fwd gives it with want_rstd")
    _need(rstd, "rstd", dy.shape[:-1], F32, dev)
    ds = _like(s)
    dx = ds if s.dtype == dt else _like(dy)
    dw = torch.empty_like(w)
    n = _lib.load().rms_norm_bwd_workspace_bytes(M, D)
    ws = _workspace(n, dev)
    _call("rms_norm_bwd", dev, _ptr(dy), pitch, _ptr(s), s_pitch, _ptr(w), _ptr(rstd), _ptr(dsum), d_pitch, _ptr(ds),
          None if dx is ds else _ptr(dx), _ptr(dw), M, D, code, _DT[s.dtype], _ptr(ws), n)
    return {"dx": dx, "dresidual": ds, "dw": dw}
