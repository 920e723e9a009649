"""ctypes view of the C ABI declared in include/gdn.h and include/gdn_block.h (argument marshalling only)."""
from __future__ import annotations

import ctypes
import os
import threading

from . import build as _build

GDN_BF16, GDN_FP32 = 0, 1
GDN_OK, GDN_ERR_INVALID_ARG, GDN_ERR_UNSUPPORTED, GDN_ERR_WORKSPACE, GDN_ERR_CUDA = 0, 1, 2, 3, 4
GDN_ERR_TIMEOUT, GDN_ERR_NUMERIC = 5, 6
GDN_L2NORM_QK, GDN_SP_OFF, GDN_WINDOW_OFF, GDN_SP_SINGLE_LAUNCH = 1, 2, 4, 8
GDN_DEBUG_WAIT_TIMEOUT = 0x80000000
GDN_DEBUG_PEER_TIMEOUT = 0x40000000
GDN_STATIC_SCRATCH_BYTES = 16 << 20

# every symbol include/gdn.h declares
EXPORTS = ("gdn_fwd_workspace_size", "gdn_bwd_workspace_size", "gdn_chunk_fwd", "gdn_chunk_fwd_static",
           "gdn_chunk_bwd", "gdn_saved_size", "gdn_bwd_saved_workspace_size", "gdn_chunk_fwd_save",
           "gdn_chunk_bwd_saved", "gdn_recurrent_fwd",
           "gdn_get_device_status", "gdn_device_status_code", "gdn_plan_query", "gdn_plan_estimate", "gdn_profile_enable", "gdn_profile_report", "gdn_profile_only",
           "gdn_status_string", "gdn_last_error_string")


# every symbol include/gdn_block.h declares
BLOCK_EXPORTS = ("gdn_paged_attn_workspace_size", "gdn_paged_attn_fwd", "gdn_paged_attn_status",
                 "gdn_rotary_table", "gdn_rotary",
                 "gdn_rotary_append", "gdn_slots_copy", "gdn_pages_workspace_size", "gdn_pages_extend", "gdn_pages_fork",
                 "gdn_pages_free", "gdn_pages_compact", "gdn_rmsnorm_fwd", "gdn_rmsnorm_bwd_workspace_size",
                 "gdn_rmsnorm_bwd", "gdn_paged_attn_sinks_fwd", "gdn_prefix_attn_workspace_size", "gdn_prefix_attn_fwd",
                 "gdn_prefix_attn_status", "gdn_norm_rotary", "gdn_norm_rotary_bwd_workspace_size", "gdn_norm_rotary_bwd",
                 "gdn_norm_rotary_append", "gdn_scan_states_rows", "gdn_scan_fwd", "gdn_scan_bwd", "gdn_scan_step")


class GdnShape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("H", ctypes.c_int),
                ("Dk", ctypes.c_int), ("Dv", ctypes.c_int),
                ("cu_seqlens", ctypes.c_void_p), ("num_seqs", ctypes.c_int),
                ("dtype", ctypes.c_int), ("scale", ctypes.c_float), ("flags", ctypes.c_uint),
                ("seg_chunks", ctypes.c_int), ("seg_first", ctypes.c_int),
                ("reserved", ctypes.c_int * 2)]


_I, _L, _F = ctypes.c_int, ctypes.c_int64, ctypes.c_float


class GdnPagedShape(ctypes.Structure):
    _fields_ = [(n, _I) for n in ("num_seqs", "total_q", "num_heads", "num_kv_heads", "head_dim", "page_size", "num_pages",
                                  "max_pages", "dtype", "max_q", "window")] + [("scale", _F)] + \
               [(n, _L) for n in ("table_stride", "q_tok", "q_head", "k_page", "k_tok", "k_head", "v_page", "v_tok", "v_head",
                                  "o_tok", "o_head", "kn_tok", "kn_head", "vn_tok", "vn_head")] + \
               [(n, _I) for n in ("rot", "interleaved", "table_rows", "reserved")]


class GdnRotaryShape(ctypes.Structure):
    _fields_ = [(n, _I) for n in ("tokens", "q_heads", "k_heads", "head_dim", "rot", "interleaved", "inverse", "table_rows",
                                  "dtype", "reserved")] + \
               [(n, _L) for n in ("q_tok", "q_head", "k_tok", "k_head", "qo_tok", "qo_head", "ko_tok", "ko_head")]


class GdnPagesShape(ctypes.Structure):
    _fields_ = [("num_seqs", _I), ("max_pages", _I), ("num_pages", _I), ("page_size", _I), ("table_stride", _L),
                ("reserved", _I * 2)]


class GdnSlotPool(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("stride", _L), ("bytes", _L), ("slots", _L)]


class GdnNormShape(ctypes.Structure):
    _fields_ = [("rows", _L), ("dim", _I), ("dtype", _I), ("fp8", _I), ("group", _I), ("eps", _F), ("weight_offset", _F),
                ("x_row", _L), ("r_row", _L), ("h_row", _L), ("y_row", _L), ("reserved", _I * 2)]


class GdnScanShape(ctypes.Structure):
    _fields_ = [("num_seqs", _I), ("tokens", _I), ("dim", _I), ("dtype", _I), ("gate_dtype", _I), ("reserved", _I),
                ("x_row", _L), ("g_row", _L), ("y_row", _L), ("dy_row", _L), ("dg_row", _L), ("state_row", _L),
                ("zero_rest", _I), ("reserved1", _I)]


_lock = threading.Lock()
_lib = None


def library_path() -> str:
    return _build.LIB


def load():
    """Load libgdn.so.  Raises if it has not been built: there is no fallback."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = _build.LIB
        if not os.path.exists(path):
            raise ImportError(f"{path} is missing: build the CUDA library first "
                              "(gated_deltanet_linear_15_gb300.build.build() or __graft_entry__.build())")
        lib = ctypes.CDLL(path)
        P, S = ctypes.c_void_p, ctypes.POINTER(GdnShape)
        lib.gdn_fwd_workspace_size.argtypes = [S]
        lib.gdn_fwd_workspace_size.restype = ctypes.c_size_t
        lib.gdn_bwd_workspace_size.argtypes = [S]
        lib.gdn_bwd_workspace_size.restype = ctypes.c_size_t
        lib.gdn_chunk_fwd.argtypes = [S, P, P, P, P, P, P, P, P, P, ctypes.c_size_t, P]
        lib.gdn_chunk_fwd.restype = ctypes.c_int
        lib.gdn_chunk_fwd_static.argtypes = [S, P, P, P, P, P, P, P, P, P]
        lib.gdn_chunk_fwd_static.restype = ctypes.c_int
        lib.gdn_chunk_bwd.argtypes = [S, P, P, P, P, P, P, P, P, P, P, P, P, P, P, P, ctypes.c_size_t, P]
        lib.gdn_chunk_bwd.restype = ctypes.c_int
        lib.gdn_saved_size.argtypes = [S]
        lib.gdn_saved_size.restype = ctypes.c_size_t
        lib.gdn_bwd_saved_workspace_size.argtypes = [S]
        lib.gdn_bwd_saved_workspace_size.restype = ctypes.c_size_t
        lib.gdn_chunk_fwd_save.argtypes = [S, P, P, P, P, P, P, P, P, P, ctypes.c_size_t, P, ctypes.c_size_t, P]
        lib.gdn_chunk_fwd_save.restype = ctypes.c_int
        lib.gdn_chunk_bwd_saved.argtypes = [S, P, P, P, P, P, P, P, P, P, P, P, P, P, P, P, ctypes.c_size_t, P,
                                            ctypes.c_size_t, P]
        lib.gdn_chunk_bwd_saved.restype = ctypes.c_int
        lib.gdn_recurrent_fwd.argtypes = [S, P, P, P, P, P, P, P, P, P]
        lib.gdn_recurrent_fwd.restype = ctypes.c_int
        lib.gdn_get_device_status.argtypes = [S, P, P]
        lib.gdn_get_device_status.restype = ctypes.c_int
        lib.gdn_device_status_code.argtypes = [ctypes.c_int]
        lib.gdn_device_status_code.restype = ctypes.c_int
        lib.gdn_plan_query.argtypes = [S, ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int),
                                       ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int)]
        lib.gdn_plan_query.restype = ctypes.c_int
        lib.gdn_plan_estimate.argtypes = [S, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_double)]
        lib.gdn_plan_estimate.restype = ctypes.c_int
        lib.gdn_profile_enable.argtypes = [ctypes.c_int]
        lib.gdn_profile_enable.restype = ctypes.c_int
        lib.gdn_profile_report.argtypes = [ctypes.c_char_p, ctypes.c_size_t, ctypes.c_int]
        lib.gdn_profile_report.restype = ctypes.c_int
        lib.gdn_profile_only.argtypes = [ctypes.c_char_p]
        lib.gdn_profile_only.restype = ctypes.c_int
        lib.gdn_status_string.argtypes = [ctypes.c_int]
        lib.gdn_status_string.restype = ctypes.c_char_p
        lib.gdn_last_error_string.argtypes = []
        lib.gdn_last_error_string.restype = ctypes.c_char_p
        Z, D = ctypes.c_size_t, ctypes.c_double
        for name, args in {
                "gdn_paged_attn_fwd": [P] * 10 + [Z, P],
                "gdn_paged_attn_status": [P, P, P],
                "gdn_paged_attn_sinks_fwd": [P, _I] + [P] * 9 + [Z, P],
                "gdn_prefix_attn_fwd": [P, _I, _I] + [P] * 11 + [Z, P],
                "gdn_prefix_attn_status": [P, _I, _I, P, P],
                "gdn_rotary_table": [P, _I, _I, D, P, P],
                "gdn_rotary": [P] * 8,
                "gdn_rotary_append": [P] * 12,
                "gdn_norm_rotary": [P, _F, _F] + [P] * 9,
                "gdn_norm_rotary_bwd": [P, _F, _F] + [P] * 13 + [Z, P],
                "gdn_norm_rotary_append": [P, _F, _F] + [P] * 13,
                "gdn_slots_copy": [P, _I, P, P, _I, P],
                "gdn_pages_extend": [P] * 6 + [_I, P, P, Z, P],
                "gdn_pages_fork": [P] * 6 + [_I, P, _I, P, _I, P, P, Z, P],
                "gdn_pages_free": [P] * 5 + [_I, P],
                "gdn_pages_compact": [P] * 6 + [_I, P, P, Z, P],
                "gdn_rmsnorm_fwd": [P] * 9,
                "gdn_rmsnorm_bwd": [P] * 9 + [Z, P],
                "gdn_scan_fwd": [P] * 9,
                "gdn_scan_bwd": [P] * 12,
                "gdn_scan_step": [P] * 6}.items():
            getattr(lib, name).argtypes = args
            getattr(lib, name).restype = ctypes.c_int
        for name, args in {"gdn_paged_attn_workspace_size": [P], "gdn_pages_workspace_size": [P, _I],
                           "gdn_rmsnorm_bwd_workspace_size": [P], "gdn_norm_rotary_bwd_workspace_size": [P],
                           "gdn_prefix_attn_workspace_size": [P, _I, _I]}.items():
            getattr(lib, name).argtypes = args
            getattr(lib, name).restype = Z
        lib.gdn_scan_states_rows.argtypes, lib.gdn_scan_states_rows.restype = [P], _L
        _lib = lib
        return lib


# the C entry points that csrc/block_py.cpp calls, in the order of its table
_PY_CALLS = ("gdn_paged_attn_workspace_size", "gdn_paged_attn_fwd", "gdn_paged_attn_status", "gdn_rotary", "gdn_rotary_append",
             "gdn_slots_copy", "gdn_pages_workspace_size", "gdn_pages_extend", "gdn_pages_fork", "gdn_pages_free",
             "gdn_pages_compact", "gdn_rmsnorm_fwd", "gdn_rmsnorm_bwd_workspace_size", "gdn_rmsnorm_bwd", "gdn_scan_states_rows",
             "gdn_scan_fwd", "gdn_scan_bwd", "gdn_scan_step", "gdn_norm_rotary", "gdn_norm_rotary_bwd_workspace_size", "gdn_norm_rotary_bwd",
             "gdn_norm_rotary_append", "gdn_paged_attn_sinks_fwd", "gdn_prefix_attn_workspace_size", "gdn_prefix_attn_fwd",
             "gdn_prefix_attn_status", "gdn_status_string", "gdn_last_error_string")
_py = None


def load_py():
    """Load the Python extension of the operators in block.py and connect it to libgdn.so.  Raises if either is missing."""
    global _py
    if _py is not None:
        return _py
    lib = load()
    with _lock:
        if _py is None:
            import importlib.machinery
            import importlib.util
            if not os.path.exists(_build.PY_LIB):
                raise ImportError(f"{_build.PY_LIB} is missing: build the library first, with this torch and Python "
                                  "(gated_deltanet_linear_15_gb300.build.build(), which says why where it cannot)")
            loader = importlib.machinery.ExtensionFileLoader("gdn_block_py", _build.PY_LIB)
            mod = importlib.util.module_from_spec(importlib.util.spec_from_file_location("gdn_block_py", _build.PY_LIB, loader=loader))
            loader.exec_module(mod)
            mod.connect(*(ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in _PY_CALLS))
            _py = mod
    return _py


def last_error() -> str:
    return load().gdn_last_error_string().decode()
