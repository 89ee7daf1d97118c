"""ctypes binding of the paged key/value cache (the C ABI in
``include/kv_cache.h``): ``KVCache`` describes a cache the caller owns,
``tree_attn``, ``cache_append``, ``cache_weigh`` and ``cache_evict`` run on it.

Argument marshalling only, as in ``_native``: every step runs in the library's
CUDA kernels, on the current CUDA stream of the cache's device.
"""
from __future__ import annotations

import ctypes
import struct

from . import _native
from ._native import GEMM_TN_BF16, GEMM_TN_F16, GemmTnError, library

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


# struct kv_cache* and struct kv_rows* are passed as c_void_p: a ctypes.byref, or
# the bytes that struct.pack makes (a small call's time is mostly the
# binding's, and packing takes a fraction of filling a ctypes.Structure)
_native._SIGNATURES.update({
    "tree_attn_fwd": (_int, [_int, _i64, _i64, _i64, _ptr, _ptr, _ptr, _ptr, _ptr, _ptr, _ptr, _ptr, ctypes.c_float, _ptr,
                             _ptr]),
    "kv_cache_append": (_int, [_int, _i64, _i64, _ptr, _ptr, _ptr, _ptr, _ptr, _i64, _ptr, _ptr, _ptr, _ptr]),
    "kv_cache_weigh": (_int, [_int, _i64, _i64, _i64, _ptr, _ptr, _ptr, _ptr, _ptr, _i64, _int, ctypes.c_float, _ptr, _ptr,
                              _ptr]),
    "kv_cache_evict": (_int, [_int, _i64, _ptr, _i64, _i64, _ptr, _ptr, _ptr, _ptr, _ptr]),
})
_pack_cache = struct.Struct("16q").pack
_pack_rows = struct.Struct("4q").pack


# What the functions below use of torch and of the library, bound when the first
# cache is made: looking them up costs a fifth of a small call.
_int32 = _int64 = _float32 = _codes = _get_device = _set_device = _get_stream = None
_tree_attn_fwd = _kv_cache_append = _kv_cache_weigh = _kv_cache_evict = None


def _bind():
    global _int32, _int64, _float32, _codes, _get_device, _set_device, _get_stream
    global _tree_attn_fwd, _kv_cache_append, _kv_cache_weigh, _kv_cache_evict
    import torch
    lib = library()
    _tree_attn_fwd, _kv_cache_append = lib.tree_attn_fwd, lib.kv_cache_append
    _kv_cache_weigh, _kv_cache_evict = lib.kv_cache_weigh, lib.kv_cache_evict
    _int64, _float32 = torch.int64, torch.float32
    _codes = {torch.float16: GEMM_TN_F16, torch.bfloat16: GEMM_TN_BF16}
    _get_device, _set_device = torch._C._cuda_getDevice, torch._C._cuda_setDevice
    _get_stream = torch._C._cuda_getCurrentRawStream
    _int32 = torch.int32


def _call(fn, name: str, index: int, *args):
    """One call of the library on device `index` and its current stream."""
    current = _get_device()
    if current == index:
        rc = fn(*args, _get_stream(index))
    else:
        _set_device(index)
        try:
            rc = fn(*args, _get_stream(index))
        finally:
            _set_device(current)
    if rc:
        raise GemmTnError(rc, name)


class KVCache:
    """A paged key/value cache in the caller's tensors (nothing is copied; the
    tensors are kept alive).

    k, v: [num_pages, page_size, kv_heads, head_dim] CUDA fp16/bf16 views with
    unit stride along head_dim and the same strides; permute a
    [num_pages, kv_heads, page_size, head_dim] pool into this order. page_size 8,
    16, 32, 64 or a multiple of 128; head_dim 64 or 128. page_table: int32
    [batch, max_pages]; lens: int32 [batch], slots in use. Where an operator
    needs them: weight, fp32 [batch, kv_heads, capacity], the accumulated
    attention weight of each slot; pos, int32 of that shape, the position of
    the token in it; seen, int32 [batch], the next token's position
    (capacity = max_pages * page_size).
    """

    __slots__ = ("k", "v", "page_table", "lens", "weight", "pos", "seen", "batch", "capacity", "index", "dtype",
                 "kv_heads", "head_dim", "_code", "_struct")

    def __init__(self, k, v, page_table, lens, weight=None, pos=None, seen=None):
        if _int32 is None:
            _bind()
        index = k.get_device()
        if index < 0 or v.get_device() != index or page_table.get_device() != index or lens.get_device() != index:
            raise ValueError("the cache's tensors must be CUDA tensors on one device")
        dtype = k.dtype
        if v.dtype is not dtype:
            raise TypeError("k and v must have the same dtype")
        code = _codes.get(dtype)
        if code is None:
            raise TypeError(f"unsupported dtype {dtype}: expected float16 or bfloat16")
        shape, strides = k.shape, k.stride()
        if len(shape) != 4 or v.shape != shape or v.stride() != strides:
            raise ValueError("k and v must be [num_pages, page_size, kv_heads, head_dim] with the same strides")
        pages, page_size, heads, dim = shape
        page_stride, slot_stride, head_stride, unit = strides
        if unit != 1:
            raise ValueError("k and v must have unit stride along head_dim")
        int32 = _int32
        if page_table.dtype is not int32 or lens.dtype is not int32:
            raise TypeError("page_table and lens must be int32")
        if page_table.dim() != 2:
            raise ValueError("page_table must be [batch, max_pages]")
        batch, max_pages = page_table.shape
        table_stride, unit = page_table.stride()
        if unit != 1 and max_pages > 1:
            raise ValueError("page_table must have unit stride along max_pages")
        if lens.shape != (batch,) or not lens.is_contiguous():
            raise ValueError("lens must be a contiguous [batch] tensor")
        self.index, self.batch, self.kv_heads = index, batch, heads
        self.capacity = capacity = max_pages * page_size
        w = p = s = 0
        if weight is not None:
            w = _floats(weight, self, "weight", (batch, heads, capacity))
        if pos is not None:
            p = _ints(pos, self, "pos", (batch, heads, capacity))
        if seen is not None:
            s = _ints(seen, self, "seen", (batch,))
        self.k, self.v, self.page_table, self.lens = k, v, page_table, lens
        self.weight, self.pos, self.seen = weight, pos, seen
        self.dtype, self.head_dim, self._code = dtype, dim, code
        self._struct = _pack_cache(
            k.data_ptr(), v.data_ptr(), pages, page_size, heads, dim, page_stride, slot_stride,
            head_stride if heads > 1 else dim, page_table.data_ptr(), table_stride if batch > 1 else max_pages,
            max_pages, lens.data_ptr(), w, p, s)


def _rows(t, cache: KVCache, what: str, shape):
    """struct kv_rows of a [batch, tokens, heads, head_dim] tensor of that shape."""
    if t.get_device() != cache.index:
        raise ValueError(f"{what} must be on the cache's device")
    if t.dtype is not cache.dtype:
        raise TypeError(f"{what} must have the cache's dtype")
    if t.shape != shape:
        raise ValueError(f"{what} must be [batch, tokens, heads, head_dim] = {tuple(shape)}")
    sb, st, sh, unit = t.stride()
    if unit != 1:
        raise ValueError(f"{what} must have unit stride along head_dim")
    return _pack_rows(t.data_ptr(), sb, st, sh)


def _ints(t, cache: KVCache, what: str, shape):
    """Device pointer of a contiguous int32 tensor of that shape, or None."""
    if t is None:
        return None
    if t.get_device() != cache.index or t.dtype is not _int32 or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous int32 {tuple(shape)} tensor on the cache's device")
    return t.data_ptr()


def _floats(t, cache: KVCache, what: str, shape):
    if t.get_device() != cache.index or t.dtype is not _float32 or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous float32 {tuple(shape)} tensor on the cache's device")
    return t.data_ptr()


def _status(t, cache: KVCache):
    """Device pointer of the optional status word."""
    if t is None:
        return None
    if t.get_device() != cache.index or t.dtype is not _int32 or t.numel() < 1 or not t.is_contiguous():
        raise ValueError("status must be a contiguous int32 tensor of at least one element on the cache's device")
    return t.data_ptr()


def _factor(scale):
    scale = float(scale)
    if scale == 0.0:   # the C ABI's word for the default
        raise ValueError("scale must be positive")
    return scale


def _queries(q, cache: KVCache):
    """q's shape and struct."""
    shape = q.shape
    if len(shape) != 4 or shape[0] != cache.batch or shape[3] != cache.head_dim:
        raise ValueError("q must be [batch, tokens, heads, head_dim] with the cache's batch size and head_dim")
    return shape, _rows(q, cache, "q", shape)


def tree_attn(q, cache: KVCache, k_new=None, v_new=None, mask=None, token_lens=None, scale=None, out=None, lse=None,
              status=None):
    """Attention of new (drafted) tokens over a paged cache and over one
    another through tree_attn_fwd. q: [batch, tokens, heads, head_dim], k_new,
    v_new: [batch, tokens, kv_heads, head_dim] (both None: the cache only),
    CUDA tensors of the cache's dtype with unit stride along head_dim; heads a
    multiple of kv_heads. mask: int64 [batch, tokens, ceil(tokens / 64)] words
    (``tree_mask``), None for the causal chain; token_lens: int32 [batch], new
    tokens of each sequence (None: all); scale: the factor on q.k (None:
    1/sqrt(head_dim)); out: optional contiguous tensor of q's shape and dtype,
    whose rows from token_lens on are left as they are (without it they come
    back as zeros); lse: optional contiguous fp32 [batch, tokens, heads] that
    receives the log of each row's sum of exponentials; status: optional
    one-element int32 CUDA tensor for device-side errors. Returns out."""
    shape, rq = _queries(q, cache)
    batch, tokens, heads, dim = shape
    rk = rv = d_mask = None
    if k_new is not None:
        if v_new is None:
            raise ValueError("k_new and v_new come together")
        new_shape = (batch, tokens, cache.kv_heads, dim)
        rk, rv = _rows(k_new, cache, "k_new", new_shape), _rows(v_new, cache, "v_new", new_shape)
    elif v_new is not None:
        raise ValueError("k_new and v_new come together")
    if mask is not None:
        if mask.get_device() != cache.index or mask.dtype is not _int64 or \
                mask.shape != (batch, tokens, (tokens + 63) // 64) or not mask.is_contiguous():
            raise ValueError("mask must be a contiguous int64 [batch, tokens, ceil(tokens / 64)] tensor on the cache's device")
        d_mask = mask.data_ptr()
    if out is None:
        out = q.new_empty(shape) if token_lens is None else q.new_zeros(shape)
    elif out.shape != shape or out.dtype is not cache.dtype or out.get_device() != cache.index or not out.is_contiguous():
        raise ValueError("out must be a contiguous tensor with q's shape, dtype and device")
    _call(_tree_attn_fwd, "tree_attn_fwd", cache.index, cache._code, batch, tokens, heads, cache._struct, rq, rk, rv, d_mask,
          _ints(token_lens, cache, "token_lens", (batch,)), out.data_ptr(),
          None if lse is None else _floats(lse, cache, "lse", (batch, tokens, heads)), 0.0 if scale is None else _factor(scale),
          _status(status, cache))
    return out


def _counted(cache: KVCache, rows, counts, batch: int, tokens: int):
    """(pointer of rows, pointer of counts, max_rows)"""
    if rows is None:
        return None, _ints(counts, cache, "counts", (batch,)), tokens
    if rows.dim() != 2:
        raise ValueError("rows must be [batch, max_rows]")
    max_rows = rows.shape[1]
    return _ints(rows, cache, "rows", (batch, max_rows)), _ints(counts, cache, "counts", (batch,)), max_rows


def cache_append(cache: KVCache, k_new, v_new, counts=None, rows=None, lens_out=None, seen_out=None, status=None):
    """Puts new tokens' keys and values into the cache through kv_cache_append.
    k_new, v_new: [batch, tokens, kv_heads, head_dim] with unit stride along
    head_dim. rows: int32 [batch, max_rows], which tokens, in order (None: the
    first ones); counts: int32 [batch], how many (None: all). weight becomes 0
    and pos the token's position where the cache has them. lens_out, seen_out:
    int32 [batch] that receive the new lengths (None: the cache's own lens and
    seen are advanced)."""
    shape = k_new.shape
    batch = cache.batch
    if len(shape) != 4 or shape[0] != batch or shape[2] != cache.kv_heads or shape[3] != cache.head_dim:
        raise ValueError("k_new must be [batch, tokens, kv_heads, head_dim] with the cache's sizes")
    tokens = shape[1]
    if seen_out is not None and cache.seen is None:
        raise ValueError("seen_out needs a cache with seen")
    d_rows, d_counts, max_rows = _counted(cache, rows, counts, batch, tokens)
    _call(_kv_cache_append, "kv_cache_append", cache.index, cache._code, batch, tokens, cache._struct, _rows(k_new, cache, "k_new", shape),
          _rows(v_new, cache, "v_new", shape), d_rows, d_counts, max_rows,
          _ints(cache.lens if lens_out is None else lens_out, cache, "lens_out", (batch,)),
          _ints(cache.seen if seen_out is None else seen_out, cache, "seen_out", (batch,)), _status(status, cache))


def cache_weigh(cache: KVCache, q, lse, counts=None, rows=None, causal=True, scale=None, out=None, status=None):
    """Adds to each cached key's weight the attention that counted queries gave
    it, through kv_cache_weigh. q: [batch, tokens, heads, head_dim], lse: fp32
    [batch, tokens, heads] as ``tree_attn`` fills it; rows, counts: the counted
    tokens as in ``cache_append``. causal: the counted tokens are the newest
    slots' queries and see the slots up to their own; False: every one sees
    every slot. out: fp32 tensor of weight's shape that receives the sums
    (None: the cache's weight, in place). Returns out."""
    shape, rq = _queries(q, cache)
    batch, tokens, heads, _ = shape
    if cache.weight is None:
        raise ValueError("the cache has no weight")
    if out is None:
        out = cache.weight
    d_rows, d_counts, max_rows = _counted(cache, rows, counts, batch, tokens)
    _call(_kv_cache_weigh, "kv_cache_weigh", cache.index, cache._code, batch, tokens, heads, cache._struct, rq,
          _floats(lse, cache, "lse", (batch, tokens, heads)), d_rows, d_counts, max_rows, 1 if causal else 0,
          0.0 if scale is None else _factor(scale), _floats(out, cache, "out", (batch, cache.kv_heads, cache.capacity)),
          _status(status, cache))
    return out


def cache_evict(cache: KVCache, keep: int, recent: int = 0, weight_out=None, pos_out=None, lens_out=None, status=None):
    """Cuts sequences longer than `keep` slots down to the newest `recent` ones
    and the heaviest others, for each KV head by its own weights, through
    kv_cache_evict. weight_out, pos_out, lens_out: tensors like the cache's
    that receive the results (None: the cache's own, in place)."""
    if cache.weight is None:
        raise ValueError("the cache has no weight")
    if pos_out is not None and cache.pos is None:
        raise ValueError("pos_out needs a cache with pos")
    batch = cache.batch
    shape = (batch, cache.kv_heads, cache.capacity)
    _call(_kv_cache_evict, "kv_cache_evict", cache.index, cache._code, batch, cache._struct, int(keep), int(recent),
          _floats(cache.weight if weight_out is None else weight_out, cache, "weight_out", shape),
          _ints(cache.pos if pos_out is None else pos_out, cache, "pos_out", shape),
          _ints(cache.lens if lens_out is None else lens_out, cache, "lens_out", (batch,)), _status(status, cache))


def _torch():
    import torch
    return torch


def tree_mask(parents):
    """Mask words of drafted trees for ``tree_attn``. parents: integer tensor
    [batch, tokens]; parents[b][i] < i is the token that i was drafted after, -1
    for one drafted right after the cached ones. Token i sees itself and its
    ancestors. Returns int64 [batch, tokens, ceil(tokens / 64)] on parents'
    device (bit j % 64 of word j / 64: i sees j). Plain torch operations; a tree
    shape is made once and reused."""
    torch = _torch()
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
