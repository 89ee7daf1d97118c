"""Binding of a feed-forward block's operators (the C ABI in
``include/feed_forward.h``): the gated projection ``mm_tn_gated``, its backward
pass (``gated_grad``, ``mm_nt``), and products in 8-bit floating point with a
scale for each block of 128 (``quantize_e4m3``, ``mm_tn_e4m3``).

Argument marshalling only, as in ``_native``: every step runs in the library's
CUDA kernels, on the current CUDA stream of the operands' device.
"""
from __future__ import annotations

import ctypes

from . import _native
from ._native import (
    _ACTIVATIONS,
    _dtype_code,
    _on_device,
    _row_pitch,
    _status_ptr,
    GEMM_TN_OK,
    GEMM_TN_OUT_F32,
    GEMM_TN_OUT_INPUT,
    GemmTnError,
    library,
)

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

_GATES = {"relu": _ACTIVATIONS["relu"], "gelu": _ACTIVATIONS["gelu"], "silu": GEMM_TN_ACT_SILU}


def _element(dtype, what: str) -> int:
    import torch
    codes = {torch.float16: GEMM_TN_ELEM_F16, torch.bfloat16: GEMM_TN_ELEM_BF16, torch.float32: GEMM_TN_ELEM_F32}
    if dtype not in codes:
        raise TypeError(f"unsupported {what} {dtype}: expected float16, bfloat16 or float32")
    return codes[dtype]


def _gate(activation) -> int:
    if activation not in _GATES:
        raise ValueError(f"activation must be one of {', '.join(_GATES)}, not {activation!r}")
    return _GATES[activation]


def _on_one_device(**tensors):
    first = None
    for name, t in tensors.items():
        if t is None:
            continue
        if t.device.type != "cuda" or (first is not None and t.device != first):
            raise ValueError(f"{', '.join(n for n, x in tensors.items() if x is not None)} must be CUDA tensors on one device")
        first = t.device
    return first


def _matrix(t, name: str, shape, dtype, device) -> int:
    """Checks a given output or operand; its pitch."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}")
    if tuple(t.shape) != tuple(shape) or t.device != device:
        raise ValueError(f"{name} must be {list(shape)} on {device}")
    return _row_pitch(t, shape[1])


def _operand(t) -> int:
    """The pitch of a matrix of any shape."""
    return _row_pitch(t, t.shape[-1] if t.dim() > 0 else 0)


def _check(rc: int, where: str):
    if rc != GEMM_TN_OK:
        raise GemmTnError(rc, where)


def mm_tn_gated(a, b, out=None, pre=None, activation="silu", status=None):
    """act(A Bg^T) * (A Bu^T) through gemm_tn_gated. a: [M, K]; b: [2N, K], the
    gate's rows Bg then the other projection's Bu, CUDA fp16/bf16 with unit
    stride along K; out: optional [M, N]; pre: optional [M, 2N] that receives
    both projections side by side, for gated_grad; activation: "silu", "gelu"
    (erf form) or "relu"; status: optional one-element int32 CUDA tensor for the
    device watchdog."""
    import torch
    dev = _on_one_device(a=a, b=b, out=out, pre=pre)
    if a.dtype != b.dtype:
        raise TypeError("a and b must have the same dtype")
    lda, ldb = _operand(a), _operand(b)
    m, k = a.shape
    if b.shape[0] % 2 != 0 or b.shape[1] != k:
        raise ValueError(f"b must be [2N, {k}], the two projections' rows: not {tuple(b.shape)}")
    n = b.shape[0] // 2
    if out is None:
        out = torch.empty((m, n), dtype=a.dtype, device=dev)
    ldh = _matrix(out, "out", (m, n), a.dtype, dev)
    ldp = _matrix(pre, "pre", (m, 2 * n), a.dtype, dev) if pre is not None else 0
    act, d_status, code = _gate(activation), _status_ptr(status, dev), _dtype_code(a)
    with _on_device(dev) as stream:
        rc = library().gemm_tn_gated(code, m, n, k, a.data_ptr(), lda, b.data_ptr(), ldb, out.data_ptr(), ldh,
                                     pre.data_ptr() if pre is not None else None, ldp, act, d_status, stream)
    _check(rc, "gemm_tn_gated")
    return out


def gated_grad(grad, pre, out=None, activation="silu"):
    """The gradient of act(G) * U through gated_grad. grad: [M, N], of the
    output; pre: [M, 2N], G and U side by side (mm_tn_gated's); out: optional
    [M, 2N], dG and dU side by side (may be pre itself). With mm_tn_gated's a
    and b, the gradients are mm_nn(out, b) and mm_nt(out, a)."""
    import torch
    dev = _on_one_device(grad=grad, pre=pre, out=out)
    ldg = _operand(grad)
    m, n = grad.shape
    ldp = _matrix(pre, "pre", (m, 2 * n), grad.dtype, dev)
    if out is None:
        # rows a multiple of 16 bytes apart: the products read them in place
        out = torch.empty((m, (2 * n + 7) // 8 * 8), dtype=grad.dtype, device=dev)[:, :2 * n]
    ldo = _matrix(out, "out", (m, 2 * n), grad.dtype, dev)
    act, code = _gate(activation), _dtype_code(grad)
    with _on_device(dev) as stream:
        rc = library().gated_grad(code, m, n, grad.data_ptr(), ldg, pre.data_ptr(), ldp, out.data_ptr(), ldo, act, stream)
    _check(rc, "gated_grad")
    return out


def mm_nt(a, b, out=None, out_dtype=None, accumulate=False, status=None):
    """C = A^T B through gemm_nt. a: [K, M], b: [K, N] CUDA tensors of one
    fp16/bf16 dtype with unit stride along their last dimension; out: optional
    [M, N] of out_dtype (None: out's, or a's; or torch.float32). accumulate: the
    product is added to out, which is fp32."""
    import torch
    dev = _on_one_device(a=a, b=b, out=out)
    if a.dtype != b.dtype:
        raise TypeError("a and b must have the same dtype")
    lda, ldb = _operand(a), _operand(b)
    (k, m), (kb, n) = a.shape, b.shape
    if kb != k:
        raise ValueError(f"outer dimensions differ: {tuple(a.shape)}^T x {tuple(b.shape)}")
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else a.dtype
    if out_dtype not in (a.dtype, torch.float32):
        raise TypeError(f"unsupported output dtype {out_dtype}")
    if accumulate and (out is None or out_dtype != torch.float32):
        raise ValueError("accumulate needs an fp32 out")
    if out is None:
        out = torch.empty((m, n), dtype=out_dtype, device=dev)
    ldc = _matrix(out, "out", (m, n), out_dtype, dev)
    d_status, code = _status_ptr(status, dev), _dtype_code(a)
    with _on_device(dev) as stream:
        rc = library().gemm_nt(code, m, n, k, a.data_ptr(), lda, b.data_ptr(), ldb, out.data_ptr(), ldc,
                               GEMM_TN_OUT_F32 if out_dtype == torch.float32 else GEMM_TN_OUT_INPUT,
                               1 if accumulate else 0, d_status, stream)
    _check(rc, "gemm_nt")
    return out


def quantize_e4m3(x, block_rows=1, transpose=False, out=None, scale=None):
    """x [M, K] (CUDA fp16, bf16 or fp32, unit stride along K) as (q, scale)
    through quantize_e4m3: q float8_e4m3fn [M, K], or x's transpose [K, M]; a
    power of two for each block of block_rows (1 or 128) rows and 128 columns of
    q. Without out and scale, q's rows lie a multiple of 16 bytes apart, as
    mm_tn_e4m3 takes them, and a single row's scales (block_rows 1) side by
    side with the other rows' (scale.stride(0) is 1)."""
    import torch
    dev = _on_one_device(x=x, out=out, scale=scale)
    source = _element(x.dtype, "dtype")
    if block_rows not in (1, 128):
        raise ValueError("block_rows must be 1 or 128")
    ldx = _operand(x)
    rows, cols = x.shape
    lines, along = (cols, rows) if transpose else (rows, cols)
    shape = ((lines + block_rows - 1) // block_rows, (along + 127) // 128)
    if out is None:
        out = torch.empty((lines, (along + 15) // 16 * 16), dtype=torch.float8_e4m3fn, device=dev)[:, :along]
    if scale is None:
        scale = torch.empty((shape[1], shape[0]), dtype=torch.float32, device=dev).t() if block_rows == 1 else \
            torch.empty(shape, dtype=torch.float32, device=dev)
    elif scale.dtype != torch.float32:
        raise TypeError("scale must be float32")
    elif tuple(scale.shape) != shape:
        raise ValueError(f"scale must be {list(shape)}")
    ldq = _matrix(out, "out", (lines, along), torch.float8_e4m3fn, dev)
    with _on_device(dev) as stream:
        rc = library().quantize_e4m3(source, rows, cols, x.data_ptr(), ldx, out.data_ptr(), ldq,
                                     scale.data_ptr(), scale.stride(0), scale.stride(1), block_rows,
                                     1 if transpose else 0, stream)
    _check(rc, "quantize_e4m3")
    return out, scale


def mm_tn_e4m3(a, a_scale, b, b_scale, out=None, out_dtype=None, accumulate=False, status=None):
    """The product of two matrices quantised in blocks of 128 through
    gemm_tn_e4m3. a: [M, K], b: [N, K] CUDA float8_e4m3fn, rows a multiple of 16
    bytes apart (quantize_e4m3's are); a_scale: fp32 [M, ceil(K / 128)]; b_scale:
    [N, ceil(K / 128)], or [ceil(N / 128), ceil(K / 128)] where 128 rows share
    theirs; any strides. out: optional [M, N] of out_dtype: fp16, bf16 or fp32
    (None: out's, or bf16). accumulate: the product is added to out, which is
    fp32."""
    import torch
    dev = _on_one_device(a=a, a_scale=a_scale, b=b, b_scale=b_scale, out=out)
    if a.dtype != torch.float8_e4m3fn or b.dtype != torch.float8_e4m3fn:
        raise TypeError("a and b must be float8_e4m3fn")
    if a_scale.dtype != torch.float32 or b_scale.dtype != torch.float32:
        raise TypeError("a_scale and b_scale must be float32")
    lda, ldb = _operand(a), _operand(b)
    (m, k), (n, kb) = a.shape, b.shape
    if kb != k:
        raise ValueError(f"inner dimensions differ: {tuple(a.shape)} x {tuple(b.shape)}^T")
    blocks = (k + 127) // 128
    if tuple(a_scale.shape) != (m, blocks):
        raise ValueError(f"a_scale must be {[m, blocks]}")
    if tuple(b_scale.shape) not in ((n, blocks), ((n + 127) // 128, blocks)):
        raise ValueError(f"b_scale must be {[n, blocks]} or {[(n + 127) // 128, blocks]}")
    block_rows = 1 if b_scale.shape[0] == n else 128
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else torch.bfloat16
    out_type = _element(out_dtype, "output dtype")
    if accumulate and (out is None or out_dtype != torch.float32):
        raise ValueError("accumulate needs an fp32 out")
    if out is None:
        out = torch.empty((m, n), dtype=out_dtype, device=dev)
    ldc = _matrix(out, "out", (m, n), out_dtype, dev)
    # one row: its pitch is never stepped over, and a view's may be anything
    lda, ldb = lda if m > 1 else (k + 15) // 16 * 16, ldb if n > 1 else (k + 15) // 16 * 16
    d_status = _status_ptr(status, dev)
    with _on_device(dev) as stream:
        rc = library().gemm_tn_e4m3(m, n, k, a.data_ptr(), lda, a_scale.data_ptr(), a_scale.stride(0), a_scale.stride(1),
                                    b.data_ptr(), ldb, b_scale.data_ptr(), b_scale.stride(0), b_scale.stride(1), block_rows,
                                    out.data_ptr(), ldc, out_type, 1 if accumulate else 0, d_status, stream)
    _check(rc, "gemm_tn_e4m3")
    return out
