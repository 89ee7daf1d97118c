"""Captured products replayed with new operands: the bits of the same call made
outside a graph, whatever the kernel, a last wave of tiles cut along K included
(its partial rows lie in a workspace that every replay uses again)."""
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


@pytest.mark.parametrize("call", ["mm_tn", "mm_nn", "mm_tn_fused"])
@pytest.mark.parametrize("mnk", [(2304, 4352, 1000), (3000, 5000, 4096), (4096, 4096, 4096), (1024, 1024, 1024), (8, 4096, 4096)],
                         ids=str)
def test_replays_follow_their_operands(mnk, call):
    m, n, k = mnk
    gen = torch.Generator(device="cuda").manual_seed(m)
    new = lambda *s: torch.randn(s, generator=gen, device="cuda").to(torch.bfloat16)
    a, b = new(m, k), new(k, n) if call == "mm_nn" else new(n, k)
    out = torch.empty((m, n), dtype=torch.bfloat16, device="cuda")
    run = lambda: getattr(gt, call)(a, b, out=out)
    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=torch.cuda.Stream()):
        run()
    for _ in range(5):
        a.copy_(new(*a.shape))
        b.copy_(new(*b.shape))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got = out.clone()
        out.zero_()
        run()
        torch.cuda.synchronize()
        assert torch.equal(got, out)
