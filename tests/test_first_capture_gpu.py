"""A process's very first call, captured: what the library sets up at its first
use (kernels' attributes, the workspaces' pool) is no part of the capture and
does not end it."""
from __future__ import annotations

import subprocess
import sys
from pathlib import Path

import pytest

from _parity import require_gpu

pytestmark = pytest.mark.gpu

ROOT = Path(__file__).resolve().parents[1]

CHILD = """
import sys, torch
import dense_tiled_gemm_03_gb300 as gt
new = lambda *s: torch.randn(s, device="cuda").to(torch.bfloat16)
a, b = new(300, 131), new(140, 131)              # rows that are copied to a workspace first
t = new(5000, 136)                               # a sum cut into parts that lie in one
x, w = new(2304, 1000), new(4352, 1000)          # a last wave of tiles whose parts do
q, s = torch.ones((300, 1008), device="cuda").to(torch.float8_e4m3fn)[:, :992], torch.ones((300, 8), device="cuda")
call = {"gated": lambda: gt.mm_tn_gated(a, b), "few rows": lambda: gt.mm_tn_gated(a[:9], b), "nt": lambda: gt.mm_nt(t, t),
        "mm_tn": lambda: gt.mm_tn(a, b), "stream-K": lambda: gt.mm_tn(x, w),
        "e4m3": lambda: gt.mm_tn_e4m3(q, s, q, s), "quantize": lambda: gt.quantize_e4m3(a)[0],
        "gradient": lambda: gt.gated_grad(a[:, :70], a[:, :70].repeat(1, 2))}[sys.argv[1]]
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g, stream=torch.cuda.Stream()):
    out = call()
g.replay()
torch.cuda.synchronize()
got = out.float().clone()
out.zero_()
want = call().float()
torch.cuda.synchronize()
assert torch.equal(got, want) and bool((want != 0).any())
print("the same")
"""


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    from dense_tiled_gemm_03_gb300 import build as native_build
    native_build.build()


@pytest.mark.parametrize("call", ["gated", "few rows", "nt", "mm_tn", "stream-K", "e4m3", "quantize", "gradient"])
def test_the_first_call_may_be_captured(call):
    run = subprocess.run([sys.executable, "-c", CHILD, call], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and "the same" in run.stdout, run.stdout + run.stderr[-2000:]
