"""ctypes binding of the paged key/value cache (the C ABI in
``include/kv_cache.h``): ``KVCache`` describes a cache the caller owns,
``tree_attn``, ``cache_append``, ``cache_weigh`` and ``cache_evict`` run on it.

Argument marshalling only, as in ``_native``: every step runs in the library's
CUDA kernels, on the current CUDA stream of the cache's device.
"""
from __future__ import annotations

import ctypes

from . import _native
from ._native import GEMM_TN_OK, GemmTnError, _dtype_code, _on_device, _status_ptr, library

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


_cache_ptr = ctypes.POINTER(KvCacheStruct)
_rows_ptr = ctypes.POINTER(KvRows)

_native._SIGNATURES.update({
    "tree_attn_fwd": (_int, [_int, _i64, _i64, _i64, _cache_ptr, _rows_ptr, _rows_ptr, _rows_ptr, _ptr, _ptr, _ptr, _ptr,
                             ctypes.c_float, _ptr, _ptr]),
    "kv_cache_append": (_int, [_int, _i64, _i64, _cache_ptr, _rows_ptr, _rows_ptr, _ptr, _ptr, _i64, _ptr, _ptr, _ptr,
                               _ptr]),
    "kv_cache_weigh": (_int, [_int, _i64, _i64, _i64, _cache_ptr, _rows_ptr, _ptr, _ptr, _ptr, _i64, _int,
                              ctypes.c_float, _ptr, _ptr, _ptr]),
    "kv_cache_evict": (_int, [_int, _i64, _cache_ptr, _i64, _i64, _ptr, _ptr, _ptr, _ptr, _ptr]),
})


def _torch():
    import torch
    return torch


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

    __slots__ = ("k", "v", "page_table", "lens", "weight", "pos", "seen", "batch", "capacity", "device", "dtype",
                 "kv_heads", "head_dim", "struct", "_code", "_ref")

    def __init__(self, k, v, page_table, lens, weight=None, pos=None, seen=None):
        torch = _torch()
        dev = k.device
        if dev.type != "cuda" or v.device != dev or page_table.device != dev or lens.device != dev:
            raise ValueError("the cache's tensors must be CUDA tensors on one device")
        if v.dtype != k.dtype:
            raise TypeError("k and v must have the same dtype")
        self._code = _dtype_code(k)
        if k.dim() != 4 or v.shape != k.shape or k.stride() != v.stride():
            raise ValueError("k and v must be [num_pages, page_size, kv_heads, head_dim] with the same strides")
        pages, page_size, heads, dim = k.shape
        page_stride, slot_stride, head_stride, unit = k.stride()
        if unit != 1:
            raise ValueError("k and v must have unit stride along head_dim")
        if page_table.dtype != torch.int32 or lens.dtype != torch.int32:
            raise TypeError("page_table and lens must be int32")
        if page_table.dim() != 2 or (page_table.shape[1] > 1 and page_table.stride(1) != 1):
            raise ValueError("page_table must be [batch, max_pages] with unit stride along max_pages")
        batch, max_pages = page_table.shape
        if lens.shape != (batch,) or not lens.is_contiguous():
            raise ValueError("lens must be a contiguous [batch] tensor")
        capacity = max_pages * page_size
        for name, t, dt in (("weight", weight, torch.float32), ("pos", pos, torch.int32)):
            if t is not None and (t.dtype != dt or t.shape != (batch, heads, capacity) or t.device != dev or
                                  not t.is_contiguous()):
                raise ValueError(f"{name} must be a contiguous {dt} [batch, kv_heads, max_pages * page_size] tensor on {dev}")
        if seen is not None and (seen.dtype != torch.int32 or seen.shape != (batch,) or seen.device != dev or
                                 not seen.is_contiguous()):
            raise ValueError(f"seen must be a contiguous int32 [batch] tensor on {dev}")
        self.k, self.v, self.page_table, self.lens = k, v, page_table, lens
        self.weight, self.pos, self.seen = weight, pos, seen
        self.batch, self.capacity, self.device, self.dtype = batch, capacity, dev, k.dtype
        self.kv_heads, self.head_dim = heads, dim
        self.struct = KvCacheStruct(
            k.data_ptr(), v.data_ptr(), pages, page_size, heads, dim, page_stride, slot_stride,
            head_stride if heads > 1 else dim, page_table.data_ptr(),
            page_table.stride(0) if batch > 1 else max_pages, max_pages, lens.data_ptr(),
            weight.data_ptr() if weight is not None else None, pos.data_ptr() if pos is not None else None,
            seen.data_ptr() if seen is not None else None)
        self._ref = ctypes.byref(self.struct)


def _rows(t, cache: KVCache, what: str, batch: int, tokens: int, heads: int):
    """struct kv_rows of a [batch, tokens, heads, head_dim] tensor."""
    if t.device != cache.device:
        raise ValueError(f"{what} must be on the cache's device")
    if t.dtype != cache.dtype:
        raise TypeError(f"{what} must have the cache's dtype")
    if t.shape != (batch, tokens, heads, cache.head_dim):
        raise ValueError(f"{what} must be [batch, tokens, heads, head_dim] = {(batch, tokens, heads, cache.head_dim)}")
    sb, st, sh, unit = t.stride()
    if unit != 1:
        raise ValueError(f"{what} must have unit stride along head_dim")
    return KvRows(t.data_ptr(), sb, st, sh)


def _ints(t, cache: KVCache, what: str, shape):
    """Device pointer of a contiguous int32 tensor of that shape, or None."""
    if t is None:
        return None
    if t.device != cache.device or t.dtype != _torch().int32 or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous int32 {tuple(shape)} tensor on {cache.device}")
    return t.data_ptr()


def _floats(t, cache: KVCache, what: str, shape):
    if t.device != cache.device or t.dtype != _torch().float32 or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous float32 {tuple(shape)} tensor on {cache.device}")
    return t.data_ptr()


def _new_tokens(cache: KVCache, q):
    if q.dim() != 4:
        raise ValueError("q must be [batch, tokens, heads, head_dim]")
    batch, tokens, heads, _ = q.shape
    if batch != cache.batch:
        raise ValueError("q must have the cache's batch size")
    return batch, tokens, heads


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
    receives the log of each row's sum of exponentials. Returns out."""
    torch = _torch()
    batch, tokens, heads = _new_tokens(cache, q)
    rq = _rows(q, cache, "q", batch, tokens, heads)
    rk = rv = None
    if (k_new is None) != (v_new is None):
        raise ValueError("k_new and v_new come together")
    if k_new is not None:
        rk = ctypes.byref(_rows(k_new, cache, "k_new", batch, tokens, cache.kv_heads))
        rv = ctypes.byref(_rows(v_new, cache, "v_new", batch, tokens, cache.kv_heads))
    d_mask = None
    if mask is not None:
        if mask.device != cache.device or mask.dtype != torch.int64 or not mask.is_contiguous() or \
                mask.shape != (batch, tokens, (tokens + 63) // 64):
            raise ValueError("mask must be a contiguous int64 [batch, tokens, ceil(tokens / 64)] tensor on the cache's device")
        d_mask = mask.data_ptr()
    if out is None:
        shape = (batch, tokens, heads, cache.head_dim)
        out = (torch.empty if token_lens is None else torch.zeros)(shape, dtype=q.dtype, device=q.device)
    elif out.shape != q.shape or out.dtype != q.dtype or out.device != q.device or not out.is_contiguous():
        raise ValueError("out must be a contiguous tensor with q's shape, dtype and device")
    d_lse = _floats(lse, cache, "lse", (batch, tokens, heads)) if lse is not None else None
    d_lens = _ints(token_lens, cache, "token_lens", (batch,))
    d_status = _status_ptr(status, cache.device)
    with _on_device(cache.device) as stream:
        rc = library().tree_attn_fwd(cache._code, batch, tokens, heads, cache._ref, ctypes.byref(rq), rk, rv, d_mask, d_lens,
                                     out.data_ptr(), d_lse, 0.0 if scale is None else float(scale), d_status, stream)
    if rc != GEMM_TN_OK:
        raise GemmTnError(rc, "tree_attn_fwd")
    return out


def _counted(cache: KVCache, rows, counts, batch: int, tokens: int):
    """(pointer of rows, pointer of counts, max_rows)"""
    if rows is None:
        max_rows = tokens
    else:
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
    if k_new.dim() != 4 or k_new.shape[0] != cache.batch:
        raise ValueError("k_new must be [batch, tokens, kv_heads, head_dim] with the cache's batch size")
    batch, tokens = k_new.shape[:2]
    rk = _rows(k_new, cache, "k_new", batch, tokens, cache.kv_heads)
    rv = _rows(v_new, cache, "v_new", batch, tokens, cache.kv_heads)
    d_rows, d_counts, max_rows = _counted(cache, rows, counts, batch, tokens)
    d_lens = _ints(cache.lens if lens_out is None else lens_out, cache, "lens_out", (batch,))
    if seen_out is not None and cache.seen is None:
        raise ValueError("seen_out needs a cache with seen")
    d_seen = _ints(cache.seen if seen_out is None else seen_out, cache, "seen_out", (batch,))
    d_status = _status_ptr(status, cache.device)
    with _on_device(cache.device) as stream:
        rc = library().kv_cache_append(cache._code, batch, tokens, cache._ref, ctypes.byref(rk), ctypes.byref(rv), d_rows,
                                       d_counts, max_rows, d_lens, d_seen, d_status, stream)
    if rc != GEMM_TN_OK:
        raise GemmTnError(rc, "kv_cache_append")


def cache_weigh(cache: KVCache, q, lse, counts=None, rows=None, causal=True, scale=None, out=None, status=None):
    """Adds to each cached key's weight the attention that counted queries gave
    it, through kv_cache_weigh. q: [batch, tokens, heads, head_dim], lse: fp32
    [batch, tokens, heads] as ``tree_attn`` fills it; rows, counts: the counted
    tokens as in ``cache_append``. causal: the counted tokens are the newest
    slots' queries and see the slots up to their own; False: every one sees
    every slot. out: fp32 tensor of weight's shape that receives the sums
    (None: the cache's weight, in place). Returns out."""
    batch, tokens, heads = _new_tokens(cache, q)
    if cache.weight is None:
        raise ValueError("the cache has no weight")
    rq = _rows(q, cache, "q", batch, tokens, heads)
    d_lse = _floats(lse, cache, "lse", (batch, tokens, heads))
    d_rows, d_counts, max_rows = _counted(cache, rows, counts, batch, tokens)
    if out is None:
        out = cache.weight
    d_out = _floats(out, cache, "out", cache.weight.shape)
    d_status = _status_ptr(status, cache.device)
    with _on_device(cache.device) as stream:
        rc = library().kv_cache_weigh(cache._code, batch, tokens, heads, cache._ref, ctypes.byref(rq), d_lse, d_rows, d_counts,
                                      max_rows, 1 if causal else 0, 0.0 if scale is None else float(scale), d_out,
                                      d_status, stream)
    if rc != GEMM_TN_OK:
        raise GemmTnError(rc, "kv_cache_weigh")
    return out


def cache_evict(cache: KVCache, keep: int, recent: int = 0, weight_out=None, pos_out=None, lens_out=None, status=None):
    """Cuts sequences longer than `keep` slots down to the newest `recent` ones
    and the heaviest others, for each KV head by its own weights, through
    kv_cache_evict. weight_out, pos_out, lens_out: tensors like the cache's
    that receive the results (None: the cache's own, in place)."""
    if cache.weight is None:
        raise ValueError("the cache has no weight")
    d_weight = _floats(cache.weight if weight_out is None else weight_out, cache, "weight_out", cache.weight.shape)
    if pos_out is not None and cache.pos is None:
        raise ValueError("pos_out needs a cache with pos")
    d_pos = _ints(cache.pos if pos_out is None else pos_out, cache, "pos_out", cache.weight.shape)
    d_lens = _ints(cache.lens if lens_out is None else lens_out, cache, "lens_out", (cache.batch,))
    d_status = _status_ptr(status, cache.device)
    with _on_device(cache.device) as stream:
        rc = library().kv_cache_evict(cache._code, cache.batch, cache._ref, int(keep), int(recent), d_weight, d_pos, d_lens,
                                      d_status, stream)
    if rc != GEMM_TN_OK:
        raise GemmTnError(rc, "kv_cache_evict")


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
