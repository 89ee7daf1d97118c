"""Long rows of calls that copy operands into a workspace first, made as fast as
the host can: each call's workspace is the one that the call before freed, and the
GPU is hundreds of calls behind. The last result has the first one's bits."""
from __future__ import annotations

import pytest
import torch

import dense_tiled_gemm_03_gb300 as gt

from _parity import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    from dense_tiled_gemm_03_gb300 import build as native_build
    native_build.build()


def normal(gen, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=gen, device="cuda").to(dtype)


def row(call, out, count):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    call(status)
    want = out.clone()
    out.zero_()
    torch.cuda.synchronize()
    for _ in range(count):
        call(status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    assert torch.equal(out, want)


@pytest.mark.parametrize("k,m,n,count", [(8192, 16384, 4095, 600), (1000, 5001, 1023, 2000), (5000, 515, 67, 2000), (8192, 512, 512, 2000)])
def test_rows_of_mm_nt(k, m, n, count):
    gen = torch.Generator(device="cuda").manual_seed(k)
    a, b, out = normal(gen, k, m), normal(gen, k, n), torch.empty((m, n), device="cuda")
    row(lambda status: gt.mm_nt(a, b, out=out, status=status), out, count)


@pytest.mark.parametrize("m,n,k,count", [(4096, 4099, 2047, 600), (9, 8001, 4095, 1000)])
def test_rows_of_gated(m, n, k, count):
    gen = torch.Generator(device="cuda").manual_seed(k)
    a, b, out = normal(gen, m, k), normal(gen, 2 * n, k), torch.empty((m, n), dtype=torch.bfloat16, device="cuda")
    row(lambda status: gt.mm_tn_gated(a, b, out=out, status=status), out, count)


def test_rows_of_e4m3_with_scales_copied():
    gen = torch.Generator(device="cuda").manual_seed(3)
    qa, sa = gt.quantize_e4m3(normal(gen, 4096, 4080))
    qb, sb = gt.quantize_e4m3(normal(gen, 4095, 4080))
    sa, sb = sa.contiguous(), sb.contiguous()      # strides that the TMA cannot address
    out = torch.empty((4096, 4095), device="cuda")
    row(lambda status: gt.mm_tn_e4m3(qa, sa, qb, sb, out=out, status=status), out, 600)


@pytest.mark.parametrize("m,n,k,count", [(3001, 5003, 4097, 600), (8192, 8191, 4095, 300)])
def test_rows_of_mm_tn(m, n, k, count):
    gen = torch.Generator(device="cuda").manual_seed(k)
    a, b, out = normal(gen, m, k), normal(gen, n, k), torch.empty((m, n), dtype=torch.bfloat16, device="cuda")
    row(lambda status: gt.mm_tn(a, b, out=out, status=status), out, count)


def test_rows_of_a_blocks_step():
    """Products that use workspaces (a last wave cut along K, copied operands), with kernels of many blocks that may
    start early right behind them: a block's backward pass and its output quantised, again and again."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    m, n, k = 4100, 2303, 2047
    x, w, wd, dy = normal(gen, m, k), normal(gen, 2 * n, k), normal(gen, k, n), normal(gen, m, k)
    h, pre = torch.empty((m, n), dtype=x.dtype, device="cuda"), torch.empty((m, 2 * n), dtype=x.dtype, device="cuda")
    q, s = gt.quantize_e4m3(h.zero_())
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def step():
        gt.mm_tn_gated(x, w, out=h, pre=pre, status=status)
        gt.quantize_e4m3(h, out=q, scale=s)
        d = gt.gated_grad(gt.mm_nn(dy, wd), pre)
        return [gt.mm_nn(d, w), gt.mm_nt(d, x, out_dtype=torch.float32, status=status), q.view(torch.uint8).clone()]

    want = step()
    torch.cuda.synchronize()
    for _ in range(150):
        got = step()
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    assert all(torch.equal(a, b) for a, b in zip(got, want))
