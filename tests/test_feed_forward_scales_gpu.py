"""Scales of the e4m3 product near the ends of fp32's range: the product of the
two scales is taken first, in fp32, whatever the kernel, so that a large one meets a
small one before either meets the block's sum (``_ff_ref``: the tolerances)."""
from __future__ import annotations

import math

import pytest
import torch

import dense_tiled_gemm_03_gb300 as gt

import _ff_ref as ref
from _parity import env_var, require_gpu

pytestmark = pytest.mark.gpu

KERNELS = ["pair256", "pair128", "single128", "skinny1", "skinny2", "skinny8", "auto"]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    from dense_tiled_gemm_03_gb300 import build as native_build
    native_build.build()


def operands(m, n, k, rows):
    gen = torch.Generator().manual_seed(m + n + k)
    q = [torch.randn(s, generator=gen).mul(60).clamp(-448, 448).to(torch.float8_e4m3fn) for s in ((m, k), (n, k))]
    s = [torch.rand(s, generator=gen).add(0.5) for s in ((m, k // 128), ((n + rows - 1) // rows, k // 128))]
    return q[0], s[0], q[1], s[1]


def product(which, a, sa, b, sb):
    with env_var("GEMM_TN_FF_KERNEL", None if which == "auto" else which):
        return gt.mm_tn_e4m3(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), out_dtype=torch.float32)


@pytest.mark.parametrize("which", KERNELS)
@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("powers", [(120, -120), (-120, 120), (127, -100), (-126, 100), (60, 40)], ids=str)
def test_large_scales_meet_small_ones(powers, rows, which):
    a, sa, b, sb = operands(24, 200, 1024, rows)
    sa, sb = sa * 2.0 ** powers[0], sb * 2.0 ** powers[1]
    assert bool(sa.isfinite().all()) and bool(sb.isfinite().all())
    ref.assert_close(product(which, a, sa, b, sb), *ref.mm_e4m3(a.float(), sa, b.float(), sb, rows, torch.float32))


@pytest.mark.parametrize("which", KERNELS)
@pytest.mark.parametrize("rows", [1, 128])
def test_scales_whose_product_leaves_fp32(rows, which):
    """It is an infinity or zero then, and times a block's sum of zero NaN or zero: the same from every kernel."""
    a = torch.ones((3, 128)).to(torch.float8_e4m3fn)
    b = torch.ones((5, 128)).to(torch.float8_e4m3fn)
    a.view(torch.uint8)[1] = 0
    big, small = torch.full((3, 1), 2.0 ** 70), torch.full((3, 1), 2.0 ** -80)
    other = lambda s: torch.full((5 if rows == 1 else 1, 1), s)
    got = product(which, a, big, b, other(2.0 ** 70)).cpu()
    assert bool(got[[0, 2]].isposinf().all()) and bool(got[1].isnan().all())
    assert bool((product(which, a, small, b, other(2.0 ** -80)) == 0).all())
