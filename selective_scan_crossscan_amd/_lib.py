"""libss2d.so (ctypes): loading, argument types, status codes."""
from __future__ import annotations

import ctypes
import os
import threading

SS2D_F32 = 0
SS2D_BF16 = 1

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libss2d.so")
_lock = threading.Lock()
_lib = None


class SS2DError(RuntimeError):
    def __init__(self, code: int, message: str):
        super().__init__(f"libss2d call failed ({code}): {message}")
        self.code = code


def library_path() -> str:
    return _LIB_PATH


class Peaks(ctypes.Structure):
    """ss2d_peaks: rates measured on the device by ss2d_measure_peaks."""
    _fields_ = [("exp_per_s", ctypes.c_double), ("fma_per_s", ctypes.c_double),
                ("update_mix_per_s", ctypes.c_double), ("hbm_read_Bps", ctypes.c_double),
                ("hbm_copy_Bps", ctypes.c_double), ("lds_read_Bps", ctypes.c_double),
                ("compute_units", ctypes.c_int), ("state_loop_per_s", ctypes.c_double)]


def lib():
    """The loaded libss2d.so (ctypes), with argument types declared."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(_LIB_PATH):
                raise ImportError(f"{_LIB_PATH} is not built; run __graft_entry__.build() or "
                                  "python -m selective_scan_crossscan_amd._build")
            L = ctypes.CDLL(_LIB_PATH)
            vp, i64 = ctypes.c_void_p, ctypes.c_int64
            L.ss2d_forward.argtypes = [vp] * 8 + [i64] * 5 + [ctypes.c_int, vp]
            L.ss2d_forward.restype = ctypes.c_int
            L.ss2d_status_string.argtypes = [ctypes.c_int]
            L.ss2d_status_string.restype = ctypes.c_char_p
            L.ss2d_last_hip_error.argtypes = []
            L.ss2d_last_hip_error.restype = ctypes.c_char_p
            L.ss2d_version.argtypes = []
            L.ss2d_version.restype = ctypes.c_int
            L.ss2d_describe.argtypes = [i64] * 5 + [ctypes.c_int, ctypes.c_char_p, i64]
            L.ss2d_describe.restype = ctypes.c_int
            L.ss2d_describe_lanes.argtypes = [i64] * 5 + [ctypes.c_int, ctypes.c_int, ctypes.c_char_p, i64]
            L.ss2d_describe_lanes.restype = ctypes.c_int
            L.ss2d_forward_lanes.argtypes = [vp] * 8 + [i64] * 5 + [ctypes.c_int, ctypes.c_int, vp]
            L.ss2d_forward_lanes.restype = ctypes.c_int
            L.ss2d_bidir_forward.argtypes = [vp] * 8 + [i64] * 4 + [ctypes.c_int, vp]
            L.ss2d_bidir_forward.restype = ctypes.c_int
            L.ss2d_forward_noalloc.argtypes = [vp] * 8 + [i64] * 5 + [ctypes.c_int, vp]
            L.ss2d_forward_noalloc.restype = ctypes.c_int
            L.ss2d_trim_memory.argtypes = []
            L.ss2d_trim_memory.restype = ctypes.c_int
            L.ss2d_project.argtypes = [vp] * 6 + [i64] * 6 + [ctypes.c_int, vp]
            L.ss2d_project.restype = ctypes.c_int
            L.ss2d_forward_from_x.argtypes = [vp] * 7 + [i64] * 6 + [ctypes.c_int, vp]
            L.ss2d_forward_from_x.restype = ctypes.c_int
            L.ss2d_channel_last.argtypes = [vp, vp, vp, ctypes.c_float, ctypes.c_int, vp] + [i64] * 4 + [
                ctypes.c_int, vp]
            L.ss2d_channel_last.restype = ctypes.c_int
            L.ss2d_backward.argtypes = [vp] * 15 + [i64] * 5 + [ctypes.c_int, vp]
            L.ss2d_backward.restype = ctypes.c_int
            L.ss2d_bidir_backward.argtypes = [vp] * 15 + [i64] * 4 + [ctypes.c_int, vp]
            L.ss2d_bidir_backward.restype = ctypes.c_int
            L.ss2d_measure_peaks.argtypes = [ctypes.POINTER(Peaks), i64, vp]
            L.ss2d_measure_peaks.restype = ctypes.c_int
            sizes = ctypes.POINTER(i64)
            f32, ci = ctypes.c_float, ctypes.c_int
            L.ss2d_linear_attention.argtypes = [vp] * 8 + [sizes, f32, ci, vp, i64, vp]
            L.ss2d_linear_attention.restype = ci
            L.ss2d_linear_attention_workspace.argtypes = [sizes, ci, ci]
            L.ss2d_linear_attention_workspace.restype = i64
            L.ss2d_linear_attention_backward.argtypes = [vp] * 13 + [sizes, f32, ci, vp, i64, vp]
            L.ss2d_linear_attention_backward.restype = ci
            L.ss2d_linear_attention_backward_workspace.argtypes = [sizes, ci, ci]
            L.ss2d_linear_attention_backward_workspace.restype = i64
            L.ss2d_linear_attention_step.argtypes = [vp] * 7 + [i64] * 9 + [f32, ci, vp]
            L.ss2d_linear_attention_step.restype = ci
            L.ss2d_matmul_fp8.argtypes = [vp] * 5 + [i64] * 3 + [ci, vp]
            L.ss2d_matmul_fp8.restype = ci
            L.ss2d_rms_norm.argtypes = [vp] * 3 + [f32] + [vp] * 3 + [i64] * 2 + [ci, vp]
            L.ss2d_rms_norm.restype = ci
            L.ss2d_rms_norm_backward.argtypes = [vp] * 4 + [f32] + [vp] * 2 + [i64] * 2 + [ci, vp, i64, vp]
            L.ss2d_rms_norm_backward.restype = ci
            L.ss2d_rms_norm_backward_workspace.argtypes = [i64, i64, ci]
            L.ss2d_rms_norm_backward_workspace.restype = i64
            L.ss2d_delta_rule.argtypes = [vp] * 9 + [sizes, f32, ci, vp, i64, vp]
            L.ss2d_delta_rule.restype = ci
            L.ss2d_delta_rule_workspace.argtypes = [sizes, ci, ci]
            L.ss2d_delta_rule_workspace.restype = i64
            L.ss2d_delta_rule_backward.argtypes = [vp] * 15 + [sizes, f32, ci, vp, i64, vp]
            L.ss2d_delta_rule_backward.restype = ci
            L.ss2d_delta_rule_backward_workspace.argtypes = [sizes, ci, ci]
            L.ss2d_delta_rule_backward_workspace.restype = i64
            L.ss2d_delta_rule_step.argtypes = [vp] * 8 + [i64] * 9 + [f32, ci, vp]
            L.ss2d_delta_rule_step.restype = ci
            L.ss2d_qk_norm.argtypes = [vp] * 8 + [sizes, f32, ci, ci, vp]
            L.ss2d_qk_norm.restype = ci
            L.ss2d_qk_norm_backward.argtypes = [vp] * 12 + [sizes, f32, ci, ci, vp, i64, vp]
            L.ss2d_qk_norm_backward.restype = ci
            L.ss2d_qk_norm_backward_workspace.argtypes = [sizes, ci]
            L.ss2d_qk_norm_backward_workspace.restype = i64
            _lib = L
    return _lib


def status_string(code: int) -> str:
    return lib().ss2d_status_string(int(code)).decode()


def check(rc: int) -> None:
    """Raises the error of a status code other than 0."""
    msg = status_string(rc)
    if rc == -8:
        msg += ": " + lib().ss2d_last_hip_error().decode()
    raise SS2DError(rc, msg)
