"""Operands and outputs of the feed-forward products in layouts that a user's
views have: rows at odd addresses whose last element is the last of the storage,
of every width around the copies' pieces (``_ff_ref``: the tolerances)."""
from __future__ import annotations

import math

import pytest
import torch

import dense_tiled_gemm_03_gb300 as gt

import _ff_ref as ref
from _parity import env_var, require_gpu

pytestmark = pytest.mark.gpu

#: widths on both sides of every multiple of 8, below, around and above 64
WIDTHS = sorted({w for q in range(8, 136, 8) for w in (q - 1, q, q + 1)} | {1, 2, 20, 100})


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    from dense_tiled_gemm_03_gb300 import build as native_build
    native_build.build()


def normal(gen, *shape, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=gen) * scale).to(dtype)


def at_the_end(x, before=9):
    """x on the GPU as the last columns of wider rows: its last element is the storage's last. NaN before it."""
    rows, cols = x.shape
    whole = torch.full((rows, before + cols), math.nan, dtype=x.dtype, device="cuda")
    whole[:, before:] = x.cuda()
    view = whole[:, before:]
    assert view.storage_offset() + (rows - 1) * view.stride(0) + cols == view.untyped_storage().nbytes() // x.element_size()
    return view


@pytest.mark.parametrize("k", WIDTHS)
def test_gated_of_views_at_their_storages_end(k):
    gen = torch.Generator().manual_seed(k)
    for m, dtype in ((20, torch.float16), (300, torch.bfloat16)):      # few rows, whole tiles
        a, b = normal(gen, m, k, dtype=dtype), normal(gen, 2 * 70, k, scale=k ** -0.5, dtype=dtype)
        pre = torch.empty((m, 140), dtype=dtype, device="cuda")
        out = gt.mm_tn_gated(at_the_end(a), at_the_end(b, 11), pre=pre)
        h, h_off, p, p_off = ref.gated(a, b, "silu", dtype)
        ref.assert_close(out, h, h_off, "h")
        ref.assert_close(pre, p, p_off, "pre")


@pytest.mark.parametrize("n", WIDTHS)
def test_mm_nt_of_views_at_their_storages_end(n):
    gen = torch.Generator().manual_seed(n)
    for k, m in ((130, 75), (4200, 33)):                               # whole, and cut along K
        a, b = normal(gen, k, m), normal(gen, k, n)
        ref.assert_close(gt.mm_nt(at_the_end(a), at_the_end(b, 11), out_dtype=torch.float32), *ref.mm_nt(a, b, torch.float32))
        ref.assert_close(gt.mm_nt(at_the_end(b), at_the_end(a, 3)), *ref.mm_nt(b, a, torch.bfloat16))


# ---------------------------------------------------------------- what lies around operands and outputs

def amid_nan(x, left, right):
    """x on the GPU inside a larger matrix of NaN, also behind its last row."""
    rows, cols = x.shape
    whole = torch.full((rows + 3, left + cols + right), math.nan).to(x.dtype).cuda()
    whole.view(torch.uint8)[:rows, left * x.element_size():(left + cols) * x.element_size()] = x.cuda().view(torch.uint8)
    return whole[:rows, left:left + cols]


def between(shape, dtype, left, right, onto=None):
    """An output inside a larger matrix of sevens: (output, the larger one). `onto` is what it holds."""
    rows, cols = shape
    whole = torch.full((rows + 2, left + cols + right), 7.0, dtype=dtype, device="cuda")
    out = whole[:rows, left:left + cols]
    if onto is not None:
        out.copy_(onto)
    return out, whole


def assert_sevens_around(out, whole):
    rest = whole.clone()
    left = out.storage_offset()
    rest[:out.shape[0], left:left + out.shape[1]] = 7.0
    assert bool((rest == 7.0).all()), "written outside the output"


TILES = ["pair256", "pair128", "single128"]
#: columns before and behind an output: rows at odd addresses, at even ones, at every 16 bytes
AROUND = [(3, 2), (1, 8), (2, 6), (8, 0)]


@pytest.mark.parametrize("around", AROUND, ids=str)
@pytest.mark.parametrize("which", TILES + ["skinny1", "skinny4"])
@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("out_dtype", ["fp16", "bf16", "fp32", "added"])
def test_e4m3_into_any_rows(out_dtype, rows, which, around):
    m, n, k = 130, 301, 700
    gen = torch.Generator().manual_seed(rows)
    dtype = {"fp16": torch.float16, "bf16": torch.bfloat16}.get(out_dtype, torch.float32)
    a, b = (torch.randn(s, generator=gen).mul(60).clamp(-448, 448).to(torch.float8_e4m3fn) for s in ((m, k), (n, k)))
    sa, sb = (torch.rand(s, generator=gen).add(0.3).mul(0.02) for s in ((m, 6), ((n + rows - 1) // rows, 6)))
    onto = normal(gen, m, n, dtype=torch.float32) if out_dtype == "added" else None
    out, whole = between((m, n), dtype, *around, onto)
    with env_var("GEMM_TN_FF_KERNEL", which):
        gt.mm_tn_e4m3(amid_nan(a, 16, 4), sa.cuda(), amid_nan(b, 0, 4), sb.cuda(), out=out, accumulate=onto is not None)
    ref.assert_close(out, *ref.mm_e4m3(a.float(), sa, b.float(), sb, rows, dtype, onto))
    assert_sevens_around(out, whole)


@pytest.mark.parametrize("around", AROUND, ids=str)
@pytest.mark.parametrize("which", TILES)
@pytest.mark.parametrize("out_dtype", ["bf16", "fp32", "added"])
@pytest.mark.parametrize("k", [130, 4200])
def test_mm_nt_into_any_rows(k, out_dtype, which, around):
    m, n = 130, 301
    gen = torch.Generator().manual_seed(k)
    dtype = torch.bfloat16 if out_dtype == "bf16" else torch.float32
    a, b = normal(gen, k, m), normal(gen, k, n)
    onto = normal(gen, m, n, dtype=torch.float32) if out_dtype == "added" else None
    out, whole = between((m, n), dtype, *around, onto)
    with env_var("GEMM_TN_FF_KERNEL", which):
        gt.mm_nt(amid_nan(a, 8, 6), amid_nan(b, 0, 3), out=out, accumulate=onto is not None)
    ref.assert_close(out, *ref.mm_nt(a, b, dtype, onto))
    assert_sevens_around(out, whole)


@pytest.mark.parametrize("around", AROUND, ids=str)
@pytest.mark.parametrize("which", TILES + ["skinny1", "skinny4"])
def test_gated_into_any_rows(which, around):
    m, n, k = 128, 101, 270
    gen = torch.Generator().manual_seed(k)
    a, b = normal(gen, m, k), normal(gen, 2 * n, k, scale=k ** -0.5)
    (out, whole), (pre, pre_whole) = between((m, n), a.dtype, *around), between((m, 2 * n), a.dtype, *around)
    with env_var("GEMM_TN_FF_KERNEL", which):
        gt.mm_tn_gated(amid_nan(a, 8, 10), amid_nan(b, 0, 2), out=out, pre=pre)
    h, h_off, p, p_off = ref.gated(a, b, "silu", a.dtype)
    ref.assert_close(out, h, h_off, "h")
    ref.assert_close(pre, p, p_off, "pre")
    assert_sevens_around(out, whole)
    assert_sevens_around(pre, pre_whole)


@pytest.mark.parametrize("around", AROUND, ids=str)
@pytest.mark.parametrize("n", [8, 12, 13])
def test_gated_grad_into_any_rows(n, around):
    gen = torch.Generator().manual_seed(n)
    dh, pre = normal(gen, 50, n), normal(gen, 50, 2 * n, scale=3.0)
    for in_place in (False, True):
        out, whole = between((50, 2 * n), dh.dtype, *around, pre if in_place else None)
        gt.gated_grad(amid_nan(dh, 3, 4), out if in_place else amid_nan(pre, 8, 0), out=out)
        ref.assert_close(out, *ref.gated_grad(dh, pre, "silu"))
        assert_sevens_around(out, whole)
