"""ctypes loader for libgdn.so (the C ABI declared in include/gdn.h).

The library is built in-tree by ``gated_delta_rule_29_amd.build``.  Loading fails loudly if
it is missing: there is no fallback implementation of any entry point.
"""
from __future__ import annotations

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libgdn.so")

OK, ERR_INVALID, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_HIP = 0, 1, 2, 3, 4
DTYPE_F32, DTYPE_BF16, DTYPE_E4M3 = 0, 1, 2
FWD_PER_KEY, FWD_SAVES = 1, 2
BWD_ACCUMULATE = 2
BWD_REUSE_STATS = 4

P = ctypes.c_void_p
I = ctypes.c_int
U = ctypes.c_uint
F = ctypes.c_float
L = ctypes.c_int64
SZ = ctypes.c_size_t

# name -> (restype, argtypes), mirroring include/gdn.h
SIGNATURES = {
    "gdn_abi_version": (I, []),
    "gdn_last_error": (ctypes.c_char_p, []),
    "gdn_fwd_workspace_bytes": (SZ, [I, I, I, I, I, I, U]),
    "gdn_fwd": (I, [P, P, P, P, P, P, F, P, P, P, P, P, I, I, I, I, I, I, P, SZ, P]),
    "gdn_varlen_num_chunks": (I, [P, I]),
    "gdn_fwd_varlen_workspace_bytes": (SZ, [I, I, I, I, I, I, I, U]),
    "gdn_fwd_varlen": (I, [P, P, P, P, P, P, F, P, P, I, P, P, P, P, P, P, P, I, I, I, I, I, P,
                           SZ, P]),
    "gdn_fwd_varlen_noalloc": (I, [P, P, P, P, P, P, F, P, P, I, P, P, P, P, P, P, P, I, I, I, I,
                                   I, P]),
    "gdn_prep": (I, [P, P, P, P, P, F, F, P, P, P, P, P, P, P, I, I, I, I, P]),
    "gdn_state_summary_workspace_bytes": (SZ, [I, I, I, I, I, I, U]),
    "gdn_state_summary": (I, [P, P, P, P, P, P, P, I, I, I, I, I, I, P, SZ, P]),
    "gdn_state_apply": (I, [P, P, P, P, I, I, I, P]),
    "bigdn_fwd_workspace_bytes": (SZ, [I, I, I, I, I]),
    "bigdn_fwd": (I, [P, P, P, P, P, P, P, F, F, P, P, I, I, I, I, I, P, SZ, P]),
    "bigdn_fwd_merged_workspace_bytes": (SZ, [I, I, I, I, I, I]),
    "bigdn_fwd_merged": (I, [P, P, P, P, P, P, P, P, P, P, F, F, P, F, P, P, P, I, I, I, I, I, P,
                             SZ, P]),
    "cam_prep_workspace_bytes": (SZ, [I, I]),
    "cam_prep": (I, [P, P, P, P, P, P, P, P, P, F, F, P, P, P, P, I, I, I, I, P, SZ, P]),
    "cam_scan_workspace_bytes": (SZ, [I, I, I, I]),
    "cam_scan": (I, [P, P, P, P, P, I, P, P, P, I, I, I, I, I, P, SZ, P]),
    "cam_scan_bidi_workspace_bytes": (SZ, [I, I, I, I]),
    "cam_scan_bidi": (I, [P, P, P, P, P, P, P, P, P, P, I, I, I, I, I, P, SZ, P]),
    "cam_scan_bwd_workspace_bytes": (SZ, [I, I, I, I]),
    "cam_scan_bwd": (I, [P, P, P, P, P, P, I, P, P, P, P, P, I, I, I, I, I, P, SZ, P]),
    "bigdn_dir_bwd_workspace_bytes": (SZ, [I, I, I, I]),
    "bigdn_dir_bwd": (I, [P] * 9 + [I] + [P] * 7 + [I, I, I, I, I, P, SZ, P]),
    "bigdn_merge_bwd": (I, [P, P, P, P, F, P, P, P, I, I, I, I, P]),
    "gdn_prep_bwd_workspace_bytes": (SZ, [I, I, I, I]),
    "gdn_prep_bwd": (I, [P, P, P, P, P, F, F, I] + [P] * 8 + [I, I, I, I, P, SZ, P]),
    "cam_prep_bwd_workspace_bytes": (SZ, [I, I, I, I]),
    "cam_prep_bwd": (I, [P] * 8 + [F, F, I] + [P] * 9 + [I, I, I, I, P, SZ, P]),
    "gdn_bwd_prep": (I, [P, P, P, P, P, P, F, P, P, I, I, I, I, I, I, P]),
    "gdn_state_grad_summary_workspace_bytes": (SZ, [I, I, I, I, I]),
    "gdn_state_grad_summary": (I, [P, P, P, P, P, P, P, F, P, I, I, I, I, I, I, P, SZ, P]),
    "gdn_state_grad_apply": (I, [P, P, P, P, I, I, I, P]),
    "gdn_bwd_dhu": (I, [P, P, P, P, P, P, P, P, F, P, P, P, I, I, I, I, I, I, P]),
    "gdn_bwd_dhu_varlen_workspace_bytes": (SZ, [I, I]),
    "gdn_bwd_dhu_varlen": (I, [P, P, P, P, P, P, P, P, F, P, P, I, P, P, P, I, I, I, I, I, P,
                               SZ, P]),
    # layer operators
    "causal_conv_fwd": (I, [P, L, P, P, P, P, P, I, I, I, I, I, I, P]),
    "causal_conv_fwd_varlen": (I, [P, L, P, P, P, P, I, P, P, P, I, I, I, I, I, P]),
    "causal_conv_bwd_workspace_bytes": (SZ, [I, I, I]),
    "causal_conv_bwd": (I, [P, L, P, L, P, P, P, P, P, P, P, P, I, I, I, I, I, I, P, SZ, P]),
    "causal_conv_bwd_varlen": (I, [P, L, P, L, P, P, P, P, I, P, P, P, P, P, P, I, I, I, I, I, P, SZ,
                                   P]),
    "causal_conv_step": (I, [P, L, P, P, P, P, P, I, I, I, I, I, I, P]),
    "ssm_scan_fwd_workspace_bytes": (SZ, [I, I, I, I]),
    "ssm_scan_fwd": (I, [P, L, P, L, P, P, L, P, L, P, P, L, P, P, P, P, P, I, I, I, I, I, I, P, SZ,
                         P]),
    "ssm_scan_fwd_varlen_workspace_bytes": (SZ, [P, I, I, I]),
    "ssm_scan_fwd_varlen": (I, [P, L, P, L, P, P, L, P, L, P, P, I, P, P, L, P, P, P, P, P, I, I, I, I,
                                I, P, SZ, P]),
    "ssm_scan_bwd_workspace_bytes": (SZ, [I, I, I, I]),
    "ssm_scan_bwd": (I, [P, L, P, P, L, P, L, P, P, L, P, L, P, P, L, P, P] + [P] * 9
                     + [I, I, I, I, I, I, P, SZ, P]),
    "ssm_scan_bwd_varlen_workspace_bytes": (SZ, [P, I, I, I]),
    "ssm_scan_bwd_varlen": (I, [P, L, P, P, L, P, L, P, P, L, P, L, P, P, I, P, P, L, P, P] + [P] * 9
                            + [I, I, I, I, I, P, SZ, P]),
    "ssm_scan_num_chunks": (I, [P, I]),
    "ssm_step": (I, [P, L, P, L, P, P, L, P, L, P, P, L, P, P, P, P, I, I, I, I, I, I, P]),
    "rms_norm_fwd": (I, [P, L, P, L, P, F, P, P, P, I, I, I, I, P]),
    "rms_norm_q8_fwd": (I, [P, L, P, L, P, F, I, P, P, P, I, I, I, I, P]),
    "rms_norm_bwd_workspace_bytes": (SZ, [I, I]),
    "rms_norm_bwd": (I, [P, L, P, L, P, P, P, L, P, P, P, I, I, I, I, P, SZ, P]),
    # full-attention layers
    "rope_fwd": (I, [P, L, L, P, P, F, P, I, I, I, I, I, I, P]),
    "rope_bwd": (I, [P, L, L, P, P, F, P, I, I, I, I, I, I, P]),
    "kv_cache_write": (I, [P, L, L, P, L, L, P, P, P, P, P, I, I, I, I, I, I, I, P]),
    "kv_cache_read": (I, [P, P, P, P, P, P, P, I, I, I, I, I, I, I, P]),
    "paged_attn_workspace_bytes": (SZ, [I] * 9),
    "paged_attn_varlen_workspace_bytes": (SZ, [P] + [I] * 8),
    "paged_attn_fwd": (I, [P, L, L, P, P, P, P, P, L, I, P, F, I, I, P, P] + [I] * 9 + [P, SZ, P]),
    "paged_attn_fwd_varlen": (I, [P, L, L, P, P, P, P, P, L, I, P, P, P, I, F, I, I, P, P] + [I] * 8
                              + [P, SZ, P]),
    "paged_attn_step": (I, [P, L, L, P, P, P, P, P, L, I, P, F, I, P] + [I] * 8 + [P, SZ, P]),
}

_lib = None


def load():
    """Load libgdn.so once; raise if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                "libgdn.so is not built; run `python -m gated_delta_rule_29_amd.build` "
                "(there is no non-HIP fallback)")
        lib = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def last_error() -> str:
    return load().gdn_last_error().decode("utf-8", "replace")


def check(rc: int, what: str) -> None:
    """Map a status code to the exception class the pages' wrappers use for it."""
    if rc == OK:
        return
    msg = "%s: %s" % (what, last_error())
    if rc == ERR_INVALID or rc == ERR_WORKSPACE:
        raise ValueError(msg)
    if rc == ERR_UNSUPPORTED:
        raise NotImplementedError(msg)
    raise RuntimeError(msg)
