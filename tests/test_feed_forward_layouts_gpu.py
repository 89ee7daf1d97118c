"""Operands and outputs of the feed-forward products in layouts that a user's
views have: rows at odd addresses whose last element is the last of the storage,
of every width around the copies' pieces (``_ff_ref``: the tolerances)."""
from __future__ import annotations

import math

import pytest
import torch

import dense_tiled_gemm_03_gb300 as gt

import _ff_ref as ref
from _parity import require_gpu

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
