"""ctypes view of the C ABI declared in include/kda.h and include/mixer.h (argument marshalling only)."""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libkda.so")

KDA_OK = 0
KDA_ERR_INVALID_ARG = -1
KDA_ERR_UNSUPPORTED = -2
KDA_ERR_WORKSPACE = -3
KDA_ERR_CUDA = -4
KDA_ERR_TIMEOUT = -5
KDA_ERR_RANGE = -6

KDA_BF16 = 0
KDA_F32 = 1

KDA_GATE_NONE = 0
KDA_GATE_SCALAR = 1
KDA_GATE_CHANNEL = 2

KDA_FLAG_BETA_SCALES_V = 1

# Every symbol include/kda.h declares.
EXPORTS = ("kda_chunk_fwd_workspace", "kda_chunk_fwd", "kda_chunk_fwd_noalloc", "kda_status_read",
           "kda_status_string", "kda_chunk_bwd_workspace", "kda_chunk_bwd", "dplr_chunk_fwd_workspace",
           "dplr_chunk_fwd", "dplr_factor_norms", "dplr_chunk_bwd_workspace", "dplr_chunk_bwd")

DPLR_FLAG_CLIP_GATE = 1


class KdaFwdArgs(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int), ("T", ctypes.c_int), ("H", ctypes.c_int),
        ("dk", ctypes.c_int), ("dv", ctypes.c_int), ("chunk", ctypes.c_int),
        ("dtype", ctypes.c_int), ("gate_kind", ctypes.c_int), ("g_dtype", ctypes.c_int),
        ("flags", ctypes.c_uint),
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("g", ctypes.c_void_p), ("beta", ctypes.c_void_p), ("h0", ctypes.c_void_p),
        ("o", ctypes.c_void_p), ("ht", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
        ("cu_seqlens", ctypes.c_void_p),
    ]


class KdaBwdArgs(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int), ("T", ctypes.c_int), ("H", ctypes.c_int),
        ("dk", ctypes.c_int), ("dv", ctypes.c_int), ("chunk", ctypes.c_int),
        ("dtype", ctypes.c_int), ("gate_kind", ctypes.c_int), ("g_dtype", ctypes.c_int),
        ("flags", ctypes.c_uint),
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("g", ctypes.c_void_p), ("beta", ctypes.c_void_p), ("h0", ctypes.c_void_p),
        ("grad_o", ctypes.c_void_p), ("grad_ht", ctypes.c_void_p),
        ("grad_q", ctypes.c_void_p), ("grad_k", ctypes.c_void_p), ("grad_v", ctypes.c_void_p),
        ("grad_g", ctypes.c_void_p), ("grad_beta", ctypes.c_void_p), ("grad_h0", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
        ("cu_seqlens", ctypes.c_void_p),
    ]


class DplrFwdArgs(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int), ("T", ctypes.c_int), ("H", ctypes.c_int),
        ("dk", ctypes.c_int), ("dv", ctypes.c_int), ("chunk", ctypes.c_int),
        ("dtype", ctypes.c_int), ("gate_kind", ctypes.c_int), ("g_dtype", ctypes.c_int),
        ("flags", ctypes.c_uint),
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("a", ctypes.c_void_p), ("b", ctypes.c_void_p), ("g", ctypes.c_void_p),
        ("h0", ctypes.c_void_p), ("o", ctypes.c_void_p), ("ht", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
        ("cu_seqlens", ctypes.c_void_p),
    ]


class DplrBwdArgs(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int), ("T", ctypes.c_int), ("H", ctypes.c_int),
        ("dk", ctypes.c_int), ("dv", ctypes.c_int), ("chunk", ctypes.c_int),
        ("dtype", ctypes.c_int), ("gate_kind", ctypes.c_int), ("g_dtype", ctypes.c_int),
        ("flags", ctypes.c_uint),
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("a", ctypes.c_void_p), ("b", ctypes.c_void_p), ("g", ctypes.c_void_p),
        ("h0", ctypes.c_void_p), ("grad_o", ctypes.c_void_p), ("grad_ht", ctypes.c_void_p),
        ("grad_q", ctypes.c_void_p), ("grad_k", ctypes.c_void_p), ("grad_v", ctypes.c_void_p),
        ("grad_a", ctypes.c_void_p), ("grad_b", ctypes.c_void_p), ("grad_g", ctypes.c_void_p),
        ("grad_h0", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
        ("cu_seqlens", ctypes.c_void_p),
    ]


# ------------------------------------------------------------ include/mixer.h
SHORT_CONV_FLAG_SILU = 1
SSM_FLAG_DELTA_SOFTPLUS = 1

_I, _L, _U, _F, _Z, _P = (ctypes.c_int, ctypes.c_longlong, ctypes.c_uint, ctypes.c_float, ctypes.c_size_t,
                          ctypes.c_void_p)


class LayerNormFwdArgs(ctypes.Structure):
    _fields_ = [("rows", _L), ("D", _I), ("dtype", _I), ("w_dtype", _I), ("eps", _F), ("x", _P), ("ld_x", _L),
                ("weight", _P), ("bias", _P), ("y", _P), ("ld_y", _L), ("mean", _P), ("rstd", _P)]


class LayerNormBwdArgs(ctypes.Structure):
    _fields_ = [("rows", _L), ("D", _I), ("dtype", _I), ("w_dtype", _I), ("dy", _P), ("ld_dy", _L), ("x", _P),
                ("ld_x", _L), ("weight", _P), ("mean", _P), ("rstd", _P), ("dx", _P), ("ld_dx", _L), ("dweight", _P),
                ("dbias", _P), ("workspace", _P), ("workspace_bytes", _Z)]


class ShortConvFwdArgs(ctypes.Structure):
    _fields_ = [("B", _I), ("T", _I), ("D", _I), ("W", _I), ("dtype", _I), ("w_dtype", _I), ("flags", _U), ("x", _P),
                ("ld_x", _L), ("weight", _P), ("bias", _P), ("h0", _P), ("y", _P), ("ld_y", _L), ("ht", _P),
                ("cu_seqlens", _P)]


class ShortConvBwdArgs(ctypes.Structure):
    _fields_ = [("B", _I), ("T", _I), ("D", _I), ("W", _I), ("dtype", _I), ("w_dtype", _I), ("flags", _U), ("x", _P),
                ("ld_x", _L), ("weight", _P), ("bias", _P), ("h0", _P), ("dy", _P), ("ld_dy", _L), ("dht", _P),
                ("dx", _P), ("ld_dx", _L), ("dh0", _P), ("dweight", _P), ("dbias", _P), ("workspace", _P),
                ("workspace_bytes", _Z), ("cu_seqlens", _P)]


class ShortConvStepArgs(ctypes.Structure):
    _fields_ = [("B", _I), ("D", _I), ("W", _I), ("slots", _I), ("dtype", _I), ("w_dtype", _I), ("flags", _U),
                ("x", _P), ("ld_x", _L), ("weight", _P), ("bias", _P), ("state", _P), ("slot", _P), ("y", _P),
                ("ld_y", _L)]


class SsmScanFwdArgs(ctypes.Structure):
    _fields_ = [("B", _I), ("T", _I), ("D", _I), ("N", _I), ("dtype", _I), ("flags", _U), ("x", _P), ("ld_x", _L),
                ("delta", _P), ("ld_delta", _L), ("Bm", _P), ("ld_B", _L), ("Cm", _P), ("ld_C", _L), ("z", _P),
                ("ld_z", _L), ("A", _P), ("Dskip", _P), ("delta_bias", _P), ("h0", _P), ("y", _P), ("ld_y", _L),
                ("ht", _P), ("workspace", _P), ("workspace_bytes", _Z), ("cu_seqlens", _P)]


class SsmScanBwdArgs(ctypes.Structure):
    _fields_ = [("B", _I), ("T", _I), ("D", _I), ("N", _I), ("dtype", _I), ("flags", _U), ("x", _P), ("ld_x", _L),
                ("delta", _P), ("ld_delta", _L), ("Bm", _P), ("ld_B", _L), ("Cm", _P), ("ld_C", _L), ("z", _P),
                ("ld_z", _L), ("A", _P), ("Dskip", _P), ("delta_bias", _P), ("h0", _P), ("dy", _P), ("ld_dy", _L),
                ("dht", _P), ("dx", _P), ("ld_dx", _L), ("ddelta", _P), ("ld_ddelta", _L), ("dBm", _P),
                ("ld_dB", _L), ("dCm", _P), ("ld_dC", _L), ("dz", _P), ("ld_dz", _L), ("dA", _P), ("dDskip", _P),
                ("ddelta_bias", _P), ("dh0", _P), ("workspace", _P), ("workspace_bytes", _Z), ("cu_seqlens", _P)]


class SsmScanStepArgs(ctypes.Structure):
    _fields_ = [("B", _I), ("D", _I), ("N", _I), ("slots", _I), ("dtype", _I), ("flags", _U), ("x", _P),
                ("ld_x", _L), ("delta", _P), ("ld_delta", _L), ("Bm", _P), ("ld_B", _L), ("Cm", _P), ("ld_C", _L),
                ("z", _P), ("ld_z", _L), ("A", _P), ("Dskip", _P), ("delta_bias", _P), ("state", _P), ("slot", _P),
                ("y", _P), ("ld_y", _L)]


GATED_SCAN_STATE_ROWS = 8
GROUP_NORM_FLAG_CENTER = 1
GROUP_NORM_FLAG_SHARED = 2
GLU_FLAG_GELU = 1


class GatedScanFwdArgs(ctypes.Structure):
    _fields_ = [("B", _I), ("T", _I), ("D", _I), ("dtype", _I), ("scale", _F), ("x", _P), ("ld_x", _L), ("decay", _P),
                ("ld_decay", _L), ("gate", _P), ("ld_gate", _L), ("rate", _P), ("h0", _P), ("y", _P), ("ld_y", _L),
                ("ht", _P), ("states", _P), ("workspace", _P), ("workspace_bytes", _Z), ("cu_seqlens", _P)]


class GatedScanBwdArgs(ctypes.Structure):
    _fields_ = [("B", _I), ("T", _I), ("D", _I), ("dtype", _I), ("scale", _F), ("x", _P), ("ld_x", _L), ("decay", _P),
                ("ld_decay", _L), ("gate", _P), ("ld_gate", _L), ("rate", _P), ("h0", _P), ("dy", _P), ("ld_dy", _L),
                ("dht", _P), ("states", _P), ("dx", _P), ("ld_dx", _L), ("ddecay", _P), ("ld_ddecay", _L),
                ("dgate", _P), ("ld_dgate", _L), ("drate", _P), ("dh0", _P), ("workspace", _P),
                ("workspace_bytes", _Z), ("cu_seqlens", _P)]


class GatedScanStepArgs(ctypes.Structure):
    _fields_ = [("B", _I), ("D", _I), ("slots", _I), ("dtype", _I), ("scale", _F), ("x", _P), ("ld_x", _L),
                ("decay", _P), ("ld_decay", _L), ("gate", _P), ("ld_gate", _L), ("rate", _P), ("state", _P),
                ("slot", _P), ("y", _P), ("ld_y", _L)]


class GroupNormFwdArgs(ctypes.Structure):
    _fields_ = [("rows", _L), ("groups", _I), ("C", _I), ("dtype", _I), ("w_dtype", _I), ("flags", _U), ("eps", _F),
                ("x", _P), ("ld_x", _L), ("gate", _P), ("ld_gate", _L), ("weight", _P), ("bias", _P), ("y", _P),
                ("ld_y", _L), ("mean", _P), ("rstd", _P)]


class GroupNormBwdArgs(ctypes.Structure):
    _fields_ = [("rows", _L), ("groups", _I), ("C", _I), ("dtype", _I), ("w_dtype", _I), ("flags", _U), ("dy", _P),
                ("ld_dy", _L), ("x", _P), ("ld_x", _L), ("gate", _P), ("ld_gate", _L), ("weight", _P), ("bias", _P),
                ("mean", _P), ("rstd", _P), ("dx", _P), ("ld_dx", _L), ("dgate", _P), ("ld_dgate", _L),
                ("dweight", _P), ("dbias", _P), ("workspace", _P), ("workspace_bytes", _Z)]


class GluFwdArgs(ctypes.Structure):
    _fields_ = [("rows", _L), ("D", _I), ("F", _I), ("dtype", _I), ("flags", _U), ("x", _P), ("ld_x", _L),
                ("w_gate", _P), ("ld_w_gate", _L), ("w_up", _P), ("ld_w_up", _L), ("h", _P), ("ld_h", _L), ("g", _P),
                ("u", _P), ("workspace", _P), ("workspace_bytes", _Z), ("status", _P)]


class GluBwdArgs(ctypes.Structure):
    _fields_ = [("rows", _L), ("D", _I), ("F", _I), ("dtype", _I), ("flags", _U), ("x", _P), ("ld_x", _L),
                ("w_gate", _P), ("ld_w_gate", _L), ("w_up", _P), ("ld_w_up", _L), ("dh", _P), ("ld_dh", _L),
                ("g", _P), ("u", _P), ("dx", _P), ("ld_dx", _L), ("dw_gate", _P), ("ld_dw_gate", _L), ("dw_up", _P),
                ("ld_dw_up", _L), ("workspace", _P), ("workspace_bytes", _Z), ("status", _P)]


# Every symbol include/mixer.h declares, with its argument block and whether it takes a stream
# (launches) or answers a size (workspace queries).
MIXER_EXPORTS = {
    "layer_norm_fwd": (LayerNormFwdArgs, True),
    "layer_norm_bwd_workspace": (LayerNormBwdArgs, False),
    "layer_norm_bwd": (LayerNormBwdArgs, True),
    "short_conv_fwd": (ShortConvFwdArgs, True),
    "short_conv_bwd_workspace": (ShortConvBwdArgs, False),
    "short_conv_bwd": (ShortConvBwdArgs, True),
    "short_conv_step": (ShortConvStepArgs, True),
    "ssm_scan_fwd_workspace": (SsmScanFwdArgs, False),
    "ssm_scan_fwd": (SsmScanFwdArgs, True),
    "ssm_scan_bwd_workspace": (SsmScanBwdArgs, False),
    "ssm_scan_bwd": (SsmScanBwdArgs, True),
    "ssm_scan_step": (SsmScanStepArgs, True),
    "gated_scan_fwd_workspace": (GatedScanFwdArgs, False),
    "gated_scan_fwd": (GatedScanFwdArgs, True),
    "gated_scan_bwd_workspace": (GatedScanBwdArgs, False),
    "gated_scan_bwd": (GatedScanBwdArgs, True),
    "gated_scan_step": (GatedScanStepArgs, True),
    "group_norm_fwd": (GroupNormFwdArgs, True),
    "group_norm_bwd_workspace": (GroupNormBwdArgs, False),
    "group_norm_bwd": (GroupNormBwdArgs, True),
    "glu_fwd_workspace": (GluFwdArgs, False),
    "glu_fwd": (GluFwdArgs, True),
    "glu_bwd_workspace": (GluBwdArgs, False),
    "glu_bwd": (GluBwdArgs, True),
}


class KdaError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {status_string(code)} ({code})")
        self.code = code


_lib = None


def load() -> ctypes.CDLL:
    """Load libkda.so.  Raises if it has not been built: there is no fallback."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(
                f"{LIB_PATH} is missing: build the CUDA library first "
                "(python -c 'import __graft_entry__ as g; g.build()')")
        lib = ctypes.CDLL(LIB_PATH)
        lib.kda_chunk_fwd_workspace.restype = ctypes.c_size_t
        lib.kda_chunk_fwd_workspace.argtypes = [ctypes.POINTER(KdaFwdArgs)]
        lib.kda_chunk_fwd.restype = ctypes.c_int
        lib.kda_chunk_fwd.argtypes = [ctypes.POINTER(KdaFwdArgs), ctypes.c_void_p]
        lib.kda_chunk_fwd_noalloc.restype = ctypes.c_int
        lib.kda_chunk_fwd_noalloc.argtypes = [ctypes.POINTER(KdaFwdArgs), ctypes.c_void_p]
        lib.kda_chunk_bwd_workspace.restype = ctypes.c_size_t
        lib.kda_chunk_bwd_workspace.argtypes = [ctypes.POINTER(KdaBwdArgs)]
        lib.kda_chunk_bwd.restype = ctypes.c_int
        lib.kda_chunk_bwd.argtypes = [ctypes.POINTER(KdaBwdArgs), ctypes.c_void_p]
        lib.dplr_chunk_fwd_workspace.restype = ctypes.c_size_t
        lib.dplr_chunk_fwd_workspace.argtypes = [ctypes.POINTER(DplrFwdArgs)]
        lib.dplr_chunk_fwd.restype = ctypes.c_int
        lib.dplr_chunk_fwd.argtypes = [ctypes.POINTER(DplrFwdArgs), ctypes.c_void_p]
        lib.dplr_factor_norms.restype = ctypes.c_int
        lib.dplr_factor_norms.argtypes = [ctypes.POINTER(DplrFwdArgs), ctypes.c_void_p, ctypes.c_void_p,
                                          ctypes.c_void_p, ctypes.c_void_p]
        lib.dplr_chunk_bwd_workspace.restype = ctypes.c_size_t
        lib.dplr_chunk_bwd_workspace.argtypes = [ctypes.POINTER(DplrBwdArgs)]
        lib.dplr_chunk_bwd.restype = ctypes.c_int
        lib.dplr_chunk_bwd.argtypes = [ctypes.POINTER(DplrBwdArgs), ctypes.c_void_p]
        lib.kda_status_read.restype = ctypes.c_int
        lib.kda_status_read.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
        lib.kda_status_string.restype = ctypes.c_char_p
        lib.kda_status_string.argtypes = [ctypes.c_int]
        for name, (args, launches) in MIXER_EXPORTS.items():
            fn = getattr(lib, name)
            fn.restype = ctypes.c_int if launches else ctypes.c_size_t
            fn.argtypes = [ctypes.POINTER(args)] + ([ctypes.c_void_p] if launches else [])
        _lib = lib
    return _lib


def status_string(code: int) -> str:
    return load().kda_status_string(code).decode()
