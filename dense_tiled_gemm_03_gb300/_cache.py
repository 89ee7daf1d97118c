"""Binding of the paged key/value cache (the C ABI in ``include/kv_cache.h``):
``KVCache`` describes a cache the caller owns, ``tree_attn``, ``cache_append``,
``cache_weigh`` and ``cache_evict`` run on it. These five are an extension
module's (``csrc/kv_cache_py.cpp``: a small call's time would be mostly the
reading of its tensors' attributes from Python), loaded at their first use.

Argument marshalling only, as in ``_native``: every step runs in the library's
CUDA kernels, on the current CUDA stream of the cache's device.
"""
from __future__ import annotations

import ctypes

from . import _native
from ._native import GemmTnError, library

_i64 = ctypes.c_int64
_int = ctypes.c_int
_ptr = ctypes.c_void_p


class KvCacheStruct(ctypes.Structure):
    """struct kv_cache of include/kv_cache.h."""
    _fields_ = [("k", _ptr), ("v", _ptr), ("num_pages", _i64), ("page_size", _i64), ("kv_heads", _i64),
                ("head_dim", _i64), ("page_stride", _i64), ("slot_stride", _i64), ("head_stride", _i64),
                ("page_table", _ptr), ("table_stride", _i64), ("max_pages", _i64), ("lens", _ptr), ("weight", _ptr),
                ("pos", _ptr), ("seen", _ptr)]


class KvRows(ctypes.Structure):
    """struct kv_rows of include/kv_cache.h."""
    _fields_ = [("data", _ptr), ("batch_stride", _i64), ("token_stride", _i64), ("head_stride", _i64)]


_native._SIGNATURES.update({
    "tree_attn_fwd": (_int, [_int, _i64, _i64, _i64, _ptr, _ptr, _ptr, _ptr, _ptr, _ptr, _ptr, _ptr, ctypes.c_float, _ptr,
                             _ptr]),
    "kv_cache_append": (_int, [_int, _i64, _i64, _ptr, _ptr, _ptr, _ptr, _ptr, _i64, _ptr, _ptr, _ptr, _ptr]),
    "kv_cache_weigh": (_int, [_int, _i64, _i64, _i64, _ptr, _ptr, _ptr, _ptr, _ptr, _i64, _int, ctypes.c_float, _ptr, _ptr,
                              _ptr]),
    "kv_cache_evict": (_int, [_int, _i64, _ptr, _i64, _i64, _ptr, _ptr, _ptr, _ptr, _ptr]),
})

#: what the extension module defines (csrc/kv_cache_py.cpp)
BOUND = ("KVCache", "tree_attn", "cache_append", "cache_weigh", "cache_evict")


def binding():
    """The extension module, bound to the loaded library; raises if either has not been built, or the module against
    another torch (whose objects it reads in place)."""
    import torch  # loads the libraries that the module is linked to
    lib = library()
    try:
        from . import _kv_cache
        if _kv_cache.built_against != torch.__version__:
            raise ImportError(f"built against torch {_kv_cache.built_against}, not {torch.__version__}")
    except ImportError as e:
        raise RuntimeError("the paged cache's binding is missing or does not fit the installed torch: build it with "
                           "`python -m dense_tiled_gemm_03_gb300.build --force`") from e
    _kv_cache.bind(GemmTnError, *(ctypes.cast(getattr(lib, name), ctypes.c_void_p).value for name in
                                  ("tree_attn_fwd", "kv_cache_append", "kv_cache_weigh", "kv_cache_evict")))
    return _kv_cache


def __getattr__(name):
    """BOUND's names, from their first use on."""
    if name not in BOUND:
        raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
    module = binding()
    globals().update({n: getattr(module, n) for n in BOUND})
    return globals()[name]


def tree_mask(parents):
    """Mask words of drafted trees for ``tree_attn``. parents: integer tensor
    [batch, tokens]; parents[b][i] < i is the token that i was drafted after, -1
    for one drafted right after the cached ones. Token i sees itself and its
    ancestors. Returns int64 [batch, tokens, ceil(tokens / 64)] on parents'
    device (bit j % 64 of word j / 64: i sees j). Host code, a loop over the tokens:
    it waits for a CUDA tensor and cannot be captured, so make the mask of a tree
    shape once and reuse it."""
    import torch
    if parents.dim() != 2 or parents.is_floating_point() or parents.dtype == torch.bool:
        raise ValueError("parents must be an integer [batch, tokens] tensor")
    par = parents.to(device="cpu", dtype=torch.int64)
    batch, tokens = par.shape
    if bool(((par < -1) | (par >= torch.arange(tokens))).any()):
        raise ValueError("parents[b][i] must be -1 or an earlier token of b")
    words = (tokens + 63) // 64
    # row tokens: the empty set, which -1 picks
    out = torch.zeros((batch, tokens + 1, words), dtype=torch.int64)
    at = torch.arange(batch)
    for i in range(tokens):
        out[:, i] = out[at, par[:, i]]
        bit = 1 << (i % 64)
        out[:, i, i // 64] |= bit - (1 << 64) if bit >> 63 else bit
    return out[:, :tokens].contiguous().to(parents.device)
