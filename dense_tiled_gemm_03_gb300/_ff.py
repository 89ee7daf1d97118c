"""Binding of a feed-forward block's operators (the C ABI in
``include/feed_forward.h``): the gated projection ``mm_tn_gated``, its backward
pass (``gated_grad``, ``mm_nt``), and products in 8-bit floating point with a
scale for each block of 128 (``quantize_e4m3``, ``mm_tn_e4m3``). These five are
an extension module's (``csrc/feed_forward_py.cpp``), loaded at their first use.

Argument marshalling only, as in ``_native``: every step runs in the library's
CUDA kernels, on the current CUDA stream of the operands' device.
"""
from __future__ import annotations

import ctypes

from . import _native
from ._native import GemmTnError, library

GEMM_TN_ACT_SILU = 3
GEMM_TN_ELEM_F16, GEMM_TN_ELEM_BF16, GEMM_TN_ELEM_F32 = 0, 1, 2

_i64 = ctypes.c_int64
_int = ctypes.c_int
_ptr = ctypes.c_void_p

_native._SIGNATURES.update({
    "gemm_tn_gated": (_int, [_int, _i64, _i64, _i64, _ptr, _i64, _ptr, _i64, _ptr, _i64, _ptr, _i64, _int, _ptr, _ptr]),
    "gated_grad": (_int, [_int, _i64, _i64, _ptr, _i64, _ptr, _i64, _ptr, _i64, _int, _ptr]),
    "gemm_nt": (_int, [_int, _i64, _i64, _i64, _ptr, _i64, _ptr, _i64, _ptr, _i64, _int, _int, _ptr, _ptr]),
    "quantize_e4m3": (_int, [_int, _i64, _i64, _ptr, _i64, _ptr, _i64, _ptr, _i64, _i64, _int, _int, _ptr]),
    "gemm_tn_e4m3": (_int, [_i64, _i64, _i64, _ptr, _i64, _ptr, _i64, _i64, _ptr, _i64, _ptr, _i64, _i64, _int, _ptr, _i64,
                            _int, _int, _ptr, _ptr]),
})

#: what the extension module defines (csrc/feed_forward_py.cpp)
BOUND = ("mm_tn_gated", "gated_grad", "mm_nt", "quantize_e4m3", "mm_tn_e4m3")


def binding():
    """The extension module, bound to the loaded library; raises if either has not been built, or the module against
    another torch (whose objects it reads in place)."""
    import torch  # loads the libraries that the module is linked to
    lib = library()
    try:
        from . import _feed_forward
        if _feed_forward.built_against != torch.__version__:
            raise ImportError(f"built against torch {_feed_forward.built_against}, not {torch.__version__}")
    except ImportError as e:
        raise RuntimeError("the feed-forward operators' binding is missing or does not fit the installed torch: build it with "
                           "`python -m dense_tiled_gemm_03_gb300.build --force`") from e
    _feed_forward.bind(GemmTnError, *(ctypes.cast(getattr(lib, name), ctypes.c_void_p).value for name in
                                      ("gemm_tn_gated", "gated_grad", "gemm_nt", "quantize_e4m3", "gemm_tn_e4m3")))
    return _feed_forward


def __getattr__(name):
    """BOUND's names, from their first use on."""
    if name not in BOUND:
        raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
    module = binding()
    globals().update({n: getattr(module, n) for n in BOUND})
    return globals()[name]
