"""ctypes binding of libqstate.so (include/qstate.h): argument marshalling only.

Every step of the decode path runs in the library's HIP kernels; this module
turns torch tensors into device pointers and torch streams into hipStream_t.
It raises if the library is missing: there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libqstate.so")

ABI_VERSION = 2

QS_OK, QS_EINVAL, QS_EUNSUPPORTED, QS_ENOMEM, QS_EHIP = 0, -1, -2, -3, -4
KIND = {"additive": 0, "delta": 1}
DECAY = {"head": 0, "key": 1}
DTYPE = {"fp32": 0, "bf16": 1, "fp16": 2}
MAP = {"none": 0, "head": 1, "key": 2}
ROUNDING = {"nearest": 0, "stochastic": 1}
AXIS = {"value": 0, "key": 1, "head": 2}
NORM = {"none": 0, "l2": 1, "rms": 2}
MAX_EXTRA = 6      # extra per-slot buffers of a slot copy

EXPORTS = (
    "qstate_plan", "qstate_init", "qstate_quantize", "qstate_decode_step", "qstate_decode_step_batch",
    "qstate_dequantize", "qstate_build_map", "qstate_destroy", "qstate_strerror",
    "qstate_last_error", "qstate_kernel_name",
    "qstate_causal_conv", "qstate_causal_conv_step", "qstate_qk_norm_rotate", "qstate_scan_workspace", "qstate_scan",
    "qstate_copy_slots", "qstate_compact_slots",
)


class Config(ctypes.Structure):
    _fields_ = [
        ("abi_version", ctypes.c_uint32),
        ("kind", ctypes.c_int32), ("decay_mode", ctypes.c_int32),
        ("B", ctypes.c_int32), ("H", ctypes.c_int32), ("dk", ctypes.c_int32), ("dv", ctypes.c_int32),
        ("qbits", ctypes.c_int32), ("hp_dtype", ctypes.c_int32), ("map_mode", ctypes.c_int32),
        ("map", ctypes.POINTER(ctypes.c_uint8)), ("in_dtype", ctypes.c_int32),
        ("rounding", ctypes.c_int32), ("sr_bits", ctypes.c_int32),
        ("bdr", ctypes.c_int32), ("bdr_bound", ctypes.c_float),
        ("lrb_rank", ctypes.c_int32), ("lrb_period", ctypes.c_int32), ("lrb_theta", ctypes.c_float),
        ("seed", ctypes.c_uint64), ("scale_dtype", ctypes.c_int32), ("lrb_dtype", ctypes.c_int32),
        ("scale_axis", ctypes.c_int32),
    ]


class Sizes(ctypes.Structure):
    _fields_ = [(n, ctypes.c_uint64) for n in ("codes", "scales", "hp", "lrb_W", "lrb_U", "lrb_n")]


TENSORS = ("codes", "scales", "hp", "lrb_W", "lrb_U", "lrb_n")


class Tensors(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("hp", ctypes.c_void_p),
                ("lrb_W", ctypes.c_void_p), ("lrb_U", ctypes.c_void_p), ("lrb_n", ctypes.c_void_p)]


class Inputs(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("decay", ctypes.c_void_p), ("beta", ctypes.c_void_p)]


_VP, _I32, _I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64


class Conv(ctypes.Structure):
    _fields_ = [("x", _VP), ("out", _VP), ("weight", _VP), ("bias", _VP), ("window", _VP), ("slot", _VP),
                ("offsets", _VP), ("x_stride", _I64), ("out_stride", _I64), ("dtype", _I32), ("tokens", _I32),
                ("channels", _I32), ("width", _I32), ("n", _I32), ("slots", _I32), ("silu", _I32)]


class Qk(ctypes.Structure):
    _fields_ = [("q", _VP), ("k", _VP), ("q_out", _VP), ("k_out", _VP), ("q_weight", _VP), ("k_weight", _VP),
                ("position", _VP), ("frequency", _VP), ("q_stride", _I64), ("k_stride", _I64),
                ("q_out_stride", _I64), ("k_out_stride", _I64), ("dtype", _I32), ("tokens", _I32),
                ("q_heads", _I32), ("k_heads", _I32), ("dim", _I32), ("rot", _I32), ("norm", _I32),
                ("interleaved", _I32), ("eps", ctypes.c_float), ("q_scale", ctypes.c_float)]


class Scan(ctypes.Structure):
    _fields_ = [("q", _VP), ("k", _VP), ("v", _VP), ("decay", _VP), ("beta", _VP), ("skip", _VP), ("initial", _VP),
                ("final", _VP), ("out", _VP), ("offsets", _VP), ("q_stride", _I64), ("k_stride", _I64),
                ("v_stride", _I64), ("decay_stride", _I64), ("beta_stride", _I64), ("out_stride", _I64),
                ("tokens", _I32), ("n", _I32), ("k_heads", _I32)]


class SlotBuffer(ctypes.Structure):
    _fields_ = [("src", _VP), ("dst", _VP), ("bytes", ctypes.c_uint64)]


class QStateError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str):
        super().__init__(f"{where}: status {status} ({detail})")
        self.status = status


_LIB = None


def lib() -> ctypes.CDLL:
    """Load libqstate.so (built in-tree by build()); raises if it is missing."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"libqstate.so not found at {LIB_PATH}; build it with "
                "`python -m quantized_recurrent_state_qstate_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        P = ctypes.POINTER
        vp = ctypes.c_void_p
        L.qstate_plan.argtypes = [P(Config), P(Sizes)]
        L.qstate_init.argtypes = [P(Config), P(vp), P(Sizes)]
        L.qstate_quantize.argtypes = [vp, vp, P(Tensors), ctypes.c_uint64, vp]
        L.qstate_decode_step.argtypes = [vp, P(Tensors), P(Inputs), vp, ctypes.c_uint64, vp]
        L.qstate_decode_step_batch.argtypes = [vp, P(Tensors), P(Inputs), vp, ctypes.c_int32, vp, vp, vp]
        L.qstate_dequantize.argtypes = [vp, P(Tensors), vp, vp]
        L.qstate_build_map.argtypes = [vp, ctypes.c_int32, ctypes.c_int32, ctypes.c_float, vp]
        L.qstate_causal_conv.argtypes = [P(Conv), vp]
        L.qstate_causal_conv_step.argtypes = [P(Conv), vp]
        L.qstate_qk_norm_rotate.argtypes = [P(Qk), vp]
        L.qstate_scan_workspace.argtypes = [vp, P(Scan), P(ctypes.c_uint64)]
        L.qstate_scan.argtypes = [vp, P(Scan), vp, ctypes.c_uint64, vp]
        L.qstate_copy_slots.argtypes = [vp, P(Tensors), P(Tensors), _I32, _I32, vp, vp, P(SlotBuffer), _I32, vp]
        L.qstate_compact_slots.argtypes = [vp, P(Tensors), vp, vp, P(SlotBuffer), _I32, vp]
        for f in ("qstate_causal_conv", "qstate_causal_conv_step", "qstate_qk_norm_rotate", "qstate_scan_workspace",
                  "qstate_scan", "qstate_copy_slots", "qstate_compact_slots"):
            getattr(L, f).restype = ctypes.c_int
        for f in ("qstate_plan", "qstate_init", "qstate_quantize", "qstate_decode_step",
                  "qstate_decode_step_batch", "qstate_dequantize", "qstate_build_map"):
            getattr(L, f).restype = ctypes.c_int
        L.qstate_destroy.argtypes = [vp]
        L.qstate_destroy.restype = None
        L.qstate_strerror.argtypes = [ctypes.c_int]
        L.qstate_strerror.restype = ctypes.c_char_p
        L.qstate_last_error.argtypes = []
        L.qstate_last_error.restype = ctypes.c_char_p
        L.qstate_kernel_name.argtypes = [vp]
        L.qstate_kernel_name.restype = ctypes.c_char_p
        _LIB = L
    return _LIB


def check(status: int, where: str) -> None:
    if status != QS_OK:
        L = lib()
        detail = L.qstate_last_error().decode() or L.qstate_strerror(status).decode()
        raise QStateError(status, where, detail)
