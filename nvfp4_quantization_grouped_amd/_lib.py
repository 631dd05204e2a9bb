"""ctypes loader for libmxq.so, the HIP library behind this package.

Loads the in-tree ``libmxq.so`` and declares the C signatures of
``include/mxq.h``, ``include/mxq_moe.h`` and ``include/mxq_pages.h``.  There is no fallback: if the library is missing or cannot
be loaded, using any op raises.
"""

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmxq.so")

# mxq_dtype / mxq_format codes (include/mxq.h)
MXQ_F32, MXQ_BF16, MXQ_F16 = 0, 1, 2
MXQ_FMT_FP8, MXQ_FMT_MXFP4, MXQ_FMT_NVFP4 = 0, 1, 2
MXQ_ERR_OFFS = -9

EXPORTS = (
    "quantize_mxfp4", "dequantize_mxfp4", "quantize_cache", "quantize_cache_bwd", "quantize_nvfp4", "dequantize_nvfp4",
    "quantize_cache_packed", "dequantize_cache_packed", "quantize_nvfp4_mse",
    "mxfp4_grouped_mm_fwd", "mxfp4_grouped_mm_bwd_x", "mxfp4_grouped_mm_fwd_w4a4", "mxfp4_grouped_mm_fwd_w4a8",
    "mxq_validate_offs", "mxq_status_string",
)

# include/mxq_moe.h
MOE_EXPORTS = (
    "moe_route", "moe_route_bwd", "moe_plan_workspace", "moe_plan", "moe_dispatch", "moe_dispatch_bwd",
    "moe_dispatch_quantized", "moe_combine", "moe_combine_bwd", "swiglu_fwd", "swiglu_bwd", "swiglu_quantized",
)

# include/mxq_pages.h
CACHE_EXPORTS = (
    "cache_append", "cache_attention_workspace", "cache_attention", "cache_fork", "cache_reserve_workspace",
    "cache_reserve", "cache_accept", "cache_compact_workspace", "cache_compact",
)

_lib = None
_moe_declared = None
_cache_declared = None

_vp, _i64, _i32, _int = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_int
_f64 = ctypes.c_double
_SIGS = {
    "quantize_mxfp4": ([_vp, _int, _i64, _i64, _vp, _vp, _vp], _int),
    "dequantize_mxfp4": ([_vp, _vp, _i64, _i64, _vp, _int, _vp], _int),
    "quantize_cache": ([_vp, _vp, _int, _i64, _i64, _int, _i32, _vp], _int),
    "quantize_cache_bwd": ([_vp, _vp, _int, _i64, _vp], _int),
    "quantize_nvfp4": ([_vp, _int, _i64, _i64, _vp, _vp, _vp, _vp], _int),
    "dequantize_nvfp4": ([_vp, _vp, _vp, _i64, _i64, _vp, _int, _vp], _int),
    "quantize_nvfp4_mse": ([_vp, _int, _i64, _i64, _vp, _vp, _vp, _vp], _int),
    "quantize_cache_packed": ([_vp, _int, _i64, _i64, _int, _i32, _vp, _vp, _vp], _int),
    "dequantize_cache_packed": ([_vp, _vp, _i64, _i64, _int, _i32, _vp, _int, _vp], _int),
    "mxfp4_grouped_mm_fwd": ([_vp, _i64, _i64, _vp, _vp, _i64, _i64, _vp, _vp, _vp], _int),
    "mxfp4_grouped_mm_bwd_x": ([_vp, _i64, _i64, _vp, _vp, _i64, _i64, _vp, _vp, _vp], _int),
    "mxfp4_grouped_mm_fwd_w4a4": ([_vp, _vp, _i64, _i64, _vp, _vp, _i64, _i64, _vp, _vp, _vp], _int),
    "mxfp4_grouped_mm_fwd_w4a8": ([_vp, _vp, _i64, _i64, _vp, _vp, _i64, _i64, _vp, _vp, _vp], _int),
    "mxq_validate_offs": ([_vp, _i64, _i64, _vp, _vp], _int),
    "mxq_status_string": ([_int], ctypes.c_char_p),
}
_MOE_SIGS = {
    "moe_route": ([_vp, _int, _i64, _i64, _i64, _int, _vp, _i64, _i64, _int, _int, _f64, _vp, _vp, _vp, _vp], _int),
    "moe_route_bwd": ([_vp, _int, _i64, _i64, _i64, _int, _int, _f64, _vp, _vp, _vp, _vp], _int),
    "moe_plan_workspace": ([_i64, _i64, _i64], _i64),
    "moe_plan": ([_vp, _i64, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _i64, _vp], _int),
    "moe_dispatch": ([_vp, _int, _i64, _i64, _i64, _vp, _vp, _vp], _int),
    "moe_dispatch_bwd": ([_vp, _int, _i64, _i64, _i64, _vp, _vp, _vp], _int),
    "moe_dispatch_quantized": ([_vp, _int, _i64, _i64, _i64, _vp, _int, _vp, _vp, _vp], _int),
    "moe_combine": ([_vp, _int, _i64, _i64, _i64, _vp, _vp, _vp, _vp], _int),
    "moe_combine_bwd": ([_vp, _vp, _int, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp], _int),
    "swiglu_fwd": ([_vp, _int, _i64, _i64, _vp, _i64, _vp, _vp, _vp, _vp], _int),
    "swiglu_bwd": ([_vp, _vp, _vp, _vp, _int, _i64, _i64, _vp, _i64, _vp, _vp], _int),
    "swiglu_quantized": ([_vp, _int, _i64, _i64, _vp, _i64, _int, _vp, _vp, _vp], _int),
}


class Cache(ctypes.Structure):
    """``mxq_cache`` of ``include/mxq_pages.h``."""
    _fields_ = [("pages", _i64), ("page_size", _i64), ("kv_heads", _i64), ("head_dim", _i64), ("fmt", _i32),
                ("block", _i32), ("k_codes", _vp), ("k_scales", _vp), ("v_codes", _vp), ("v_scales", _vp)]


_cp = ctypes.POINTER(Cache)
_CACHE_SIGS = {
    "cache_append": ([_cp, _vp, _i64, _i64, _vp, _vp, _vp, _vp, _int, _i64, _vp, _vp], _int),
    "cache_attention_workspace": ([_cp, _i64, _i64, _int, _i64, _i64], _i64),
    "cache_attention": ([_cp, _vp, _i64, _i64, _vp, _vp, _int, _i64, _i64, _vp, _int, _vp, _f64, _vp, _vp, _vp, _i64,
                         _vp], _int),
    "cache_fork": ([_vp, _i64, _i64, _vp, _vp, _i64, _i64, _vp, _i64, _vp, _int, _vp, _vp, _vp, _vp], _int),
    "cache_reserve_workspace": ([_i64, _i64, _i64], _i64),
    "cache_reserve": ([_cp, _vp, _i64, _i64, _vp, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _i64, _vp], _int),
    "cache_accept": ([_cp, _vp, _i64, _i64, _vp, _vp, _vp, _i64, _vp, _vp], _int),
    "cache_compact_workspace": ([_i64], _i64),
    "cache_compact": ([_cp, _vp, _i64, _i64, _vp, _vp, _vp, _vp, _i64, _vp], _int),
}


class MxqError(RuntimeError):
    """A libmxq entry point returned a non-zero status."""


def lib():
    """The loaded library (loads it on first use; raises if it is not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is not built; run `python -m nvfp4_quantization_grouped_amd.build` "
                "(hipcc for gfx950).  There is no fallback implementation.")
        l = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in _SIGS.items():
            f = getattr(l, name)
            f.argtypes = args
            f.restype = res
        _lib = l
    return _lib


def moe_lib():
    """The loaded library with the entry points of ``include/mxq_moe.h`` declared too."""
    global _moe_declared
    if _moe_declared is None:
        l = lib()
        for name, (args, res) in _MOE_SIGS.items():
            f = getattr(l, name)
            f.argtypes = args
            f.restype = res
        _moe_declared = l
    return _moe_declared


def cache_lib():
    """The loaded library with the entry points of ``include/mxq_pages.h`` declared too."""
    global _cache_declared
    if _cache_declared is None:
        l = lib()
        for name, (args, res) in _CACHE_SIGS.items():
            f = getattr(l, name)
            f.argtypes = args
            f.restype = res
        _cache_declared = l
    return _cache_declared


def check(status, fn):
    if status != 0:
        msg = lib().mxq_status_string(status).decode()
        raise MxqError(f"{fn}: status {status} ({msg})")
