"""ctypes loader for the in-tree CUDA library ``libdiffattn.so``.

Loading fails loudly when the library has not been built: there is no other
implementation behind these calls.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdiffattn.so")
# the bounds-checked build (same entry points; kernels record DIFFATTN_ERR_BOUNDS)
DEBUG_LIB_PATH = os.path.join(_HERE, "libdiffattn_debug.so")

_handles = {}
_active = LIB_PATH
_marshal = None  # the compiled marshalling module, bound to the active library; False: it was not built

# name -> (restype, argtypes); mirrors include/diffattn.h
_c_int, _c_float, _c_size, _vp, _c_ll = ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_longlong
SIGNATURES = {
    "diffattn_lambda": (_c_int, [_vp, _vp, _vp, _vp, _c_int, _c_float, _vp, _vp]),
    "diffattn_fwd": (_c_int, [_vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int, _c_int, _c_int,
                              _vp, _c_float, _vp, _c_float, _vp]),
    "diffattn_fwd_mode": (_c_int, [_vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int, _c_int, _c_int,
                                   _vp, _c_float, _vp, _c_float, _c_int, _vp]),
    "diffattn_quantize_qk": (_c_int, [_vp, _c_int, _c_int, _c_int, _c_int, _vp, _vp, _vp]),
    "diffattn_fwd_qk8": (_c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int, _c_int,
                                  _vp, _c_float, _vp, _c_float, _c_int, _vp]),
    "diffattn_quantize_qk4": (_c_int, [_vp, _c_int, _c_int, _c_int, _c_int, _vp, _vp, _vp]),
    "diffattn_fwd_qk4": (_c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int, _c_int,
                                  _vp, _c_float, _vp, _c_float, _c_int, _vp]),
    "diffattn_bwd_workspace_size": (_c_size, [_c_int, _c_int, _c_int, _c_int]),
    "diffattn_bwd": (_c_int, [_vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int, _c_int, _c_int, _vp, _c_float,
                              _vp, _c_float, _c_int, _vp, _vp, _vp, _vp, _vp, _vp, _c_size, _vp]),
    "diffattn_bwd_tc_workspace_size": (_c_size, [_c_int, _c_int, _c_int, _c_int]),
    "diffattn_bwd_tc": (_c_int, [_vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int, _c_int, _vp, _c_float,
                                 _vp, _c_float, _c_int, _vp, _vp, _vp, _vp, _vp, _vp, _c_size, _vp]),
    "diffattn_fwd_train": (_c_int, [_vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int, _c_int, _vp, _c_float, _vp,
                                    _c_float, _c_int, _vp, _c_size, _vp]),
    "diffattn_bwd_tc_saved": (_c_int, [_vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int, _c_int, _vp, _c_float,
                                       _vp, _c_float, _c_int, _vp, _vp, _vp, _vp, _vp, _vp, _c_size, _vp]),
    "diffattn_rope_table": (_c_int, [_c_int, _c_int, ctypes.c_double, _vp, _vp]),
    "diffattn_qkv_proj": (_c_int, [_vp, _vp, _c_int, _c_int, _c_int, _c_int, _c_int, _vp, _vp, _vp, _vp, _vp]),
    "diffattn_out_proj": (_c_int, [_vp, _vp, _c_int, _c_int, _c_int, _vp, _vp]),
    "diffattn_lambda_bwd": (_c_int, [_vp, _vp, _vp, _vp, _c_int, _vp, _vp, _vp, _vp, _vp, _vp]),
    "diffattn_decode_workspace_size": (_c_size, [_c_int, _c_int, _c_int, _c_int]),
    "diffattn_decode": (_c_int, [_vp, _vp, _vp, _vp, _c_int, _vp, _c_int, _c_int, _c_int, _vp, _c_float,
                                 _vp, _c_float, _vp, _c_size, _vp]),
    "diffattn_decode_mode": (_c_int, [_vp, _vp, _vp, _vp, _c_int, _vp, _c_int, _c_int, _c_int, _vp, _c_float,
                                      _vp, _c_float, _c_int, _vp, _c_size, _vp]),
    "diffattn_decode_noalloc": (_c_int, [_vp, _vp, _vp, _vp, _c_int, _vp, _c_int, _c_int, _c_int, _vp,
                                         _c_float, _vp, _c_float, _vp]),
    "diffattn_paged_step": (_c_int, [_vp, _vp, _c_int, _vp, _c_int, _vp, _c_int, _vp, _vp, _c_int, _c_int,
                                     _vp, _vp, _vp, _vp, _vp, _vp]),
    "diffattn_rope_table_scaled": (_c_int, [_c_int, _c_int, ctypes.c_double, _c_int, ctypes.c_double, _c_int,
                                            ctypes.c_double, ctypes.c_double, _vp, _vp]),
    "diffattn_rope": (_c_int, [_vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int, _c_int, _c_int, _c_int, _c_int,
                               _c_int, _vp, _vp, _vp]),
    "diffattn_kv_append": (_c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int, _c_int, _c_int,
                                    _c_int, _c_int, _c_int, _vp, _vp, _vp, _vp]),
    "diffattn_extend_plan_size": (_c_size, [_c_int] * 6),
    "diffattn_extend_plan": (_c_int, [_vp, _vp, _c_int, _c_int, _c_int, _c_int, _c_int, _c_int, _c_int, _vp, _c_size,
                                      _vp]),
    "diffattn_extend_workspace_size": (_c_size, [_c_int] * 6),
    "diffattn_extend": (_c_int, [_vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _vp, _c_size, _c_int, _c_int, _c_int,
                                 _c_int, _c_int, _c_int, _vp, _c_float, _vp, _c_float, _c_int, _vp, _vp, _c_size,
                                 _vp]),
    "diffattn_device_status": (_c_int, [ctypes.POINTER(_c_int)]),
    "diffattn_set_wait_limit_ns": (_c_int, [_c_ll]),
    "diffattn_status_string": (ctypes.c_char_p, [_c_int]),
    "diffattn_version": (_c_int, []),
}


def _load(path: str) -> ctypes.CDLL:
    if path not in _handles:
        if not os.path.exists(path):
            raise RuntimeError(
                f"{path} is missing: build it with `python -m differential_attention_04_b200.build`"
                + (" --debug" if path == DEBUG_LIB_PATH else ""))
        handle = ctypes.CDLL(path)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _handles[path] = handle
    return _handles[path]


def _bind_marshal(handle: ctypes.CDLL) -> None:
    """Point the marshalling module (if it was built) at a library's entry points."""
    global _marshal
    try:
        from . import _marshal as m
    except ImportError:  # the Python binding marshals every call then
        _marshal = False
        return
    m.bind(*(ctypes.cast(getattr(handle, "diffattn_" + n), ctypes.c_void_p).value
             for n in ("paged_step", "rope", "kv_append", "extend")))
    _marshal = m


def marshal():
    """The marshalling module of the active library, or False where it was not built."""
    if _marshal is None:
        lib()
    return _marshal


def lib() -> ctypes.CDLL:
    """Load (once) and return the active library with typed entry points."""
    handle = _load(_active)
    if _marshal is None:
        _bind_marshal(handle)
    return handle


def use_debug_library(on: bool = True) -> None:
    """Route every binding call to the bounds-checked build (on) or back to the release one.

    The two are separate libraries, each with its own device status word."""
    global _active
    _active = DEBUG_LIB_PATH if on else LIB_PATH
    _bind_marshal(_load(_active))
