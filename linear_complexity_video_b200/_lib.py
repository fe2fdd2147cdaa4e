"""ctypes declarations of libmate.so (the C ABI in include/mate.h).

Argument marshalling only. Loading fails loudly when the library has not
been built: there is no fallback implementation of any kernel.
"""
from __future__ import annotations

import ctypes
import os
import struct

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmate.so")

MATE_OK = 0
MATE_ERR_INVALID_ARG = -1
MATE_ERR_UNSUPPORTED = -2
MATE_ERR_CUDA = -3
MATE_ERR_TIMEOUT = -4
MATE_ERR_WORKSPACE = -5

MATE_F32 = 0
MATE_BF16 = 1
MATE_I8 = 2

MATE_NORM_NONE, MATE_NORM_RMS, MATE_NORM_LAYER = 0, 1, 2

MATE_DIR_FWD, MATE_DIR_BWD, MATE_DIR_BI = 1, 2, 3

# every symbol include/mate.h declares
EXPORTS = (
    "mate_bissd_workspace_bytes",
    "mate_bissd_fwd",
    "tesa_fwd",
    "mate_debug_rms_map",
    "mate_debug_tesa_map",
    "mate_debug_fastdiv",
    "mate_last_error",
    "mate_status_string",
    "mate_version",
    "mate_set_phase_hook",
    "mate_kernel_launches",
    "mate_bissd_fwd_noalloc",
    "mate_compose_fwd",
    "mate_frontend_workspace_bytes",
    "mate_frontend_fwd",
    "mate_gate_norm_fwd",
    "mate_quant_rows_fwd",
    "mate_linear_i8_fwd",
    "mate_gate_norm_i8_fwd",
    "mate_block_norm_fwd",
    "mate_frontend_i8_fwd",
)

NOALLOC_SCRATCH_BYTES = 32 << 20

PHASES = {1: "review_pool", 2: "review_scan", 3: "chunk_state", 4: "state_pass", 5: "chunk_out", 6: "tesa",
          7: "compose", 8: "front_proj", 9: "front_conv", 10: "front_dt", 11: "gate_norm",
          12: "quant_rows", 13: "linear_i8", 14: "block_norm"}
PHASE_HOOK = ctypes.CFUNCTYPE(None, ctypes.c_int, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p)


_INT_MIN, _INT_MAX = -2 ** 31, 2 ** 31 - 1


class Int:
    """Argument type of the C entry points' ints. ctypes.c_int keeps the low 32 bits of a larger
    value without a word; this refuses it."""

    @classmethod
    def from_param(cls, v):
        if isinstance(v, ctypes.c_int):
            return v
        if not _INT_MIN <= v <= _INT_MAX:
            raise ValueError(f"{v} does not fit the library's 32-bit integers")
        return ctypes.c_int(v)


class Dims(ctypes.Structure):
    """Base of the mate_*_dims structures: refuses values that their fields cannot hold, which
    ctypes would cut to the field's low bits without a word."""
    _CODES = {ctypes.c_int: "i", ctypes.c_int64: "q", ctypes.c_float: "f"}

    def __init_subclass__(cls, **kw):
        super().__init_subclass__(**kw)
        cls._names = [n for n, _ in cls._fields_]
        cls._pack = struct.Struct("@" + "".join(Dims._CODES[t] for _, t in cls._fields_)).pack

    def __init__(self, *args, **kw):
        super().__init__(*args, **kw)
        self.of(*args, *(kw.get(n, 0) for n in self._names[len(args):]))

    @classmethod
    def of(cls, *values):
        """cls(*values), every field given, for the calls whose host time counts."""
        try:
            return cls.from_buffer_copy(cls._pack(*values))
        except struct.error:
            raise ValueError(f"{cls.__name__}{values}: a value does not fit the library's integers") from None


class mate_ssd_dims(Dims):
    _fields_ = [("batch", ctypes.c_int), ("nheads", ctypes.c_int), ("headdim", ctypes.c_int),
                ("dstate", ctypes.c_int), ("ngroups", ctypes.c_int), ("chunk", ctypes.c_int),
                ("dtype", ctypes.c_int), ("directions", ctypes.c_int)]


class mate_attn_dims(Dims):
    _fields_ = [("batch", ctypes.c_int), ("nheads", ctypes.c_int), ("headdim", ctypes.c_int),
                ("dtype", ctypes.c_int)]


class mate_compose_dims(Dims):
    _fields_ = [("tokens", ctypes.c_int), ("k_ma", ctypes.c_int), ("k_te", ctypes.c_int), ("d_model", ctypes.c_int),
                ("dtype", ctypes.c_int)]


class mate_gate_norm_dims(Dims):
    _fields_ = [("tokens", ctypes.c_int), ("channels", ctypes.c_int), ("group", ctypes.c_int), ("dtype", ctypes.c_int)]


class mate_frontend_dims(Dims):
    _fields_ = [("batch", ctypes.c_int), ("d_model", ctypes.c_int), ("nheads", ctypes.c_int), ("headdim", ctypes.c_int),
                ("ngroups", ctypes.c_int), ("dstate", ctypes.c_int), ("dtype", ctypes.c_int)]


class mate_quant_dims(Dims):
    _fields_ = [("rows", ctypes.c_int), ("k", ctypes.c_int), ("dtype", ctypes.c_int)]


class mate_linear_i8_dims(Dims):
    _fields_ = [("tokens", ctypes.c_int), ("k", ctypes.c_int), ("n", ctypes.c_int), ("out_dtype", ctypes.c_int)]


class mate_block_norm_dims(Dims):
    _fields_ = [("batch", ctypes.c_int), ("tokens", ctypes.c_int), ("channels", ctypes.c_int),
                ("post_norm", ctypes.c_int), ("pre_norm", ctypes.c_int), ("x_dtype", ctypes.c_int),
                ("h_dtype", ctypes.c_int), ("gate_stride", ctypes.c_int64), ("scale_stride", ctypes.c_int64),
                ("shift_stride", ctypes.c_int64), ("residual_scale", ctypes.c_float), ("eps", ctypes.c_float)]


class MateError(RuntimeError):
    def __init__(self, fn: str, code: int, text: str):
        super().__init__(f"{fn} returned {code} ({text})")
        self.code = code


_vp = ctypes.c_void_p
_ip = ctypes.POINTER(ctypes.c_int)
_lib = None


def load() -> ctypes.CDLL:
    """Load libmate.so once; raise if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libmate.so not built at {LIB_PATH}; run python -m linear_complexity_video_b200.build")
    L = ctypes.CDLL(LIB_PATH)
    L.mate_bissd_workspace_bytes.argtypes = [Int] * 3 + [_ip, ctypes.POINTER(mate_ssd_dims)]
    L.mate_bissd_workspace_bytes.restype = ctypes.c_size_t
    L.mate_bissd_fwd.argtypes = [_vp] * 6 + [Int] * 4 + [_ip, _vp, ctypes.POINTER(mate_ssd_dims), _vp,
                                                                    ctypes.c_size_t, _vp]
    L.mate_bissd_fwd.restype = ctypes.c_int
    L.tesa_fwd.argtypes = [_vp] * 3 + [Int] * 5 + [_ip, _vp, ctypes.POINTER(mate_attn_dims), _vp]
    L.tesa_fwd.restype = ctypes.c_int
    L.mate_debug_rms_map.argtypes = [Int] * 5 + [_vp, _vp]
    L.mate_debug_rms_map.restype = ctypes.c_int
    L.mate_debug_tesa_map.argtypes = [Int] * 5 + [_ip, _vp, _vp]
    L.mate_debug_tesa_map.restype = ctypes.c_int
    L.mate_last_error.argtypes = [_vp]
    L.mate_last_error.restype = ctypes.c_int
    L.mate_status_string.argtypes = [Int]
    L.mate_status_string.restype = ctypes.c_char_p
    L.mate_debug_fastdiv.argtypes = [_vp, _vp, ctypes.c_size_t, ctypes.c_uint32]
    L.mate_debug_fastdiv.restype = ctypes.c_int
    L.mate_compose_fwd.argtypes = [_vp] * 5 + [ctypes.POINTER(mate_compose_dims), _vp]
    L.mate_compose_fwd.restype = ctypes.c_int
    L.mate_gate_norm_fwd.argtypes = [_vp] * 3 + [ctypes.c_float, _vp, ctypes.POINTER(mate_gate_norm_dims), _vp]
    L.mate_gate_norm_fwd.restype = ctypes.c_int
    L.mate_frontend_workspace_bytes.argtypes = [Int] * 3 + [ctypes.POINTER(mate_frontend_dims)]
    L.mate_frontend_workspace_bytes.restype = ctypes.c_size_t
    L.mate_frontend_fwd.argtypes = [_vp] * 5 + [Int] * 4 + [_vp] * 5 + [ctypes.POINTER(mate_frontend_dims),
                                                                            _vp, ctypes.c_size_t, _vp]
    L.mate_frontend_fwd.restype = ctypes.c_int
    L.mate_frontend_i8_fwd.argtypes = [_vp] * 7 + [Int] * 4 + [_vp] * 5 + [ctypes.POINTER(mate_frontend_dims),
                                                                               _vp, ctypes.c_size_t, _vp]
    L.mate_frontend_i8_fwd.restype = ctypes.c_int
    L.mate_quant_rows_fwd.argtypes = [_vp] * 3 + [ctypes.POINTER(mate_quant_dims), _vp]
    L.mate_quant_rows_fwd.restype = ctypes.c_int
    L.mate_linear_i8_fwd.argtypes = [_vp] * 7 + [ctypes.POINTER(mate_linear_i8_dims), _vp]
    L.mate_linear_i8_fwd.restype = ctypes.c_int
    L.mate_gate_norm_i8_fwd.argtypes = [_vp] * 3 + [ctypes.c_float, _vp, _vp, ctypes.POINTER(mate_gate_norm_dims), _vp]
    L.mate_gate_norm_i8_fwd.restype = ctypes.c_int
    L.mate_block_norm_fwd.argtypes = [_vp] * 10 + [ctypes.POINTER(mate_block_norm_dims), _vp]
    L.mate_block_norm_fwd.restype = ctypes.c_int
    L.mate_version.argtypes = []
    L.mate_version.restype = ctypes.c_int
    L.mate_set_phase_hook.argtypes = [PHASE_HOOK, ctypes.c_void_p]
    L.mate_set_phase_hook.restype = None
    L.mate_bissd_fwd_noalloc.argtypes = [_vp] * 6 + [Int] * 4 + [_ip, _vp, ctypes.POINTER(mate_ssd_dims),
                                                                            _vp]
    L.mate_bissd_fwd_noalloc.restype = ctypes.c_int
    L.mate_kernel_launches.argtypes = []
    L.mate_kernel_launches.restype = ctypes.c_uint64
    _lib = L
    return L


def check(fn: str, code: int) -> None:
    if code != MATE_OK:
        raise MateError(fn, code, load().mate_status_string(code).decode())
