"""CPU tests of the feed-forward operators: the C ABI refuses bad arguments
before it touches a device, the binding refuses what is no call, and the 64-bit
references of the GPU tests on closed forms."""
from __future__ import annotations

import math

import pytest
import torch

import dense_tiled_gemm_03_gb300 as gt
from dense_tiled_gemm_03_gb300 import _ff
import _ff_ref as ref


@pytest.fixture(scope="module")
def lib():
    from dense_tiled_gemm_03_gb300 import build as native_build
    native_build.build()
    return gt.library()


# Fake, well-separated addresses: validation never dereferences them.
A, B, C, P, SA, SB = (0x100000000000 + 0x10000000000 * i for i in range(6))
F16, BF16 = gt.GEMM_TN_F16, gt.GEMM_TN_BF16
E16, EBF, E32 = gt.GEMM_TN_ELEM_F16, gt.GEMM_TN_ELEM_BF16, gt.GEMM_TN_ELEM_F32
SILU, RELU = gt.GEMM_TN_ACT_SILU, 1
INVALID, MISALIGNED, DTYPE = gt.GEMM_TN_ERR_INVALID_VALUE, gt.GEMM_TN_ERR_MISALIGNED, gt.GEMM_TN_ERR_UNSUPPORTED_DTYPE
NO_DEVICE = (gt.GEMM_TN_ERR_UNSUPPORTED_DEVICE, gt.GEMM_TN_ERR_CUDA)


def gated(lib, dtype=BF16, m=10, n=20, k=30, a=A, lda=32, b=B, ldb=32, h=C, ldh=20, pre=P, ldp=40, act=SILU):
    return lib.gemm_tn_gated(dtype, m, n, k, a, lda, b, ldb, h, ldh, pre, ldp, act, None, None)


def grad(lib, dtype=F16, m=10, n=20, g=A, ldg=20, pre=P, ldp=40, out=C, ldo=40, act=RELU):
    return lib.gated_grad(dtype, m, n, g, ldg, pre, ldp, out, ldo, act, None)


def nt(lib, dtype=BF16, m=10, n=20, k=30, a=A, lda=10, b=B, ldb=20, c=C, ldc=20, out=0, acc=0):
    return lib.gemm_nt(dtype, m, n, k, a, lda, b, ldb, c, ldc, out, acc, None, None)


def quantize(lib, src=EBF, rows=10, cols=300, x=A, ldx=300, q=C, ldq=304, s=SA, s_line=1, s_blk=12, lines=1, t=0):
    return lib.quantize_e4m3(src, rows, cols, x, ldx, q, ldq, s, s_line, s_blk, lines, t, None)


def e4m3(lib, m=10, n=200, k=300, a=A, lda=304, sa=SA, sar=1, sab=12, b=B, ldb=304, sb=SB, sbr=3, sbb=1, rows=128, c=C, ldc=200,
         out=EBF, acc=0):
    return lib.gemm_tn_e4m3(m, n, k, a, lda, sa, sar, sab, b, ldb, sb, sbr, sbb, rows, c, ldc, out, acc, None, None)


@pytest.mark.parametrize("call", [gated, grad, nt, quantize, e4m3], ids=lambda f: f.__name__)
def test_a_valid_call_gets_as_far_as_the_device(lib, call):
    assert call(lib) in NO_DEVICE


@pytest.mark.parametrize("over,status", [
    (dict(dtype=2), DTYPE), (dict(m=-1), INVALID), (dict(n=1 << 30), INVALID), (dict(k=1 << 30), INVALID), (dict(act=0), INVALID),
    (dict(act=4), INVALID), (dict(h=None), INVALID), (dict(a=None), INVALID), (dict(b=None), INVALID), (dict(lda=29), INVALID),
    (dict(ldb=29), INVALID), (dict(ldh=19), INVALID), (dict(ldp=39), INVALID), (dict(h=C + 1), MISALIGNED),
    (dict(pre=P + 1), MISALIGNED), (dict(a=A + 1), MISALIGNED), (dict(b=B + 1), MISALIGNED), (dict(h=A), INVALID),
    (dict(h=B + 39 * 64), INVALID), (dict(pre=A), INVALID), (dict(h=P), INVALID), (dict(lda=1 << 33), INVALID)])
def test_gated_refusals(lib, over, status):
    assert gated(lib, **over) == status and gt.gemm_tn_last_error_message()


def test_gated_bounds_are_exact(lib):
    assert gated(lib, h=B + 40 * 64) in NO_DEVICE      # right behind B's 40 rows of 32
    assert gated(lib, pre=None, ldp=0) in NO_DEVICE
    assert gated(lib, m=0, h=None) == gt.GEMM_TN_OK and gated(lib, n=0, h=None) == gt.GEMM_TN_OK


@pytest.mark.parametrize("over,status", [
    (dict(dtype=5), DTYPE), (dict(m=-1), INVALID), (dict(n=-1), INVALID), (dict(act=0), INVALID), (dict(g=None), INVALID),
    (dict(pre=None), INVALID), (dict(out=None), INVALID), (dict(ldg=19), INVALID), (dict(ldp=39), INVALID), (dict(ldo=39), INVALID),
    (dict(g=A + 1), MISALIGNED), (dict(out=A), INVALID), (dict(out=P, ldo=41), INVALID), (dict(out=P + 2), INVALID)])
def test_grad_refusals(lib, over, status):
    assert grad(lib, **over) == status


def test_grad_takes_pre_itself(lib):
    assert grad(lib, out=P) in NO_DEVICE and grad(lib, m=0, g=None) == gt.GEMM_TN_OK


@pytest.mark.parametrize("over,status", [
    (dict(dtype=2), DTYPE), (dict(out=2), DTYPE), (dict(acc=1), INVALID), (dict(m=-1), INVALID), (dict(k=1 << 30), INVALID),
    (dict(c=None), INVALID), (dict(a=None), INVALID), (dict(lda=9), INVALID), (dict(ldb=19), INVALID), (dict(ldc=19), INVALID),
    (dict(c=C + 2, out=1), MISALIGNED), (dict(b=B + 1), MISALIGNED), (dict(c=B), INVALID), (dict(c=A + 29 * 20), INVALID)])
def test_nt_refusals(lib, over, status):
    assert nt(lib, **over) == status


@pytest.mark.parametrize("over,status", [
    (dict(src=3), DTYPE), (dict(src=-1), DTYPE), (dict(rows=-1), INVALID), (dict(lines=64), INVALID), (dict(x=None), INVALID),
    (dict(q=None), INVALID), (dict(s=None), INVALID), (dict(ldx=299), INVALID), (dict(ldq=299), INVALID),
    (dict(t=1, ldq=9), INVALID), (dict(x=A + 1), MISALIGNED), (dict(src=E32, x=A + 2), MISALIGNED), (dict(s=SA + 2), MISALIGNED),
    (dict(s_line=0), INVALID), (dict(s_blk=-3), INVALID), (dict(s_line=1, s_blk=9), INVALID), (dict(s_line=2, s_blk=1), INVALID),
    (dict(q=A), INVALID), (dict(s=A), INVALID), (dict(s=C), INVALID)])
def test_quantize_refusals(lib, over, status):
    assert quantize(lib, **over) == status


def test_quantize_strides_that_fit(lib):
    assert quantize(lib, s_line=3, s_blk=1) in NO_DEVICE and quantize(lib, s_line=1, s_blk=10) in NO_DEVICE
    assert quantize(lib, t=1, ldq=16, lines=128, s_line=1, s_blk=1) in NO_DEVICE     # one block along, three lines


@pytest.mark.parametrize("over,status", [
    (dict(out=3), DTYPE), (dict(acc=1), INVALID), (dict(rows=2), INVALID), (dict(n=-1), INVALID), (dict(c=None), INVALID),
    (dict(a=None), INVALID), (dict(sa=None), INVALID), (dict(sb=None), INVALID), (dict(lda=299), INVALID), (dict(ldb=288), INVALID),
    (dict(lda=300), MISALIGNED), (dict(a=A + 8), MISALIGNED), (dict(b=B + 1), MISALIGNED), (dict(sa=SA + 2), MISALIGNED),
    (dict(out=E32, c=C + 2, ldc=200), MISALIGNED), (dict(sar=-1), INVALID), (dict(sbb=1 << 40), INVALID), (dict(ldc=199), INVALID),
    (dict(c=A), INVALID), (dict(c=B + 199 * 304), INVALID), (dict(c=SA), INVALID), (dict(c=SB), INVALID)])
def test_e4m3_refusals(lib, over, status):
    assert e4m3(lib, **over) == status


def test_empty_sums_need_no_operands(lib):
    assert nt(lib, k=0, a=None, b=None) in NO_DEVICE and e4m3(lib, k=0, a=None, b=None, sa=None, sb=None) in NO_DEVICE
    assert nt(lib, m=0, c=None) == gt.GEMM_TN_OK and e4m3(lib, n=0, c=None) == gt.GEMM_TN_OK
    assert quantize(lib, rows=0, x=None) == gt.GEMM_TN_OK and quantize(lib, cols=0, q=None) == gt.GEMM_TN_OK


# ---------------------------------------------------------------- the binding

@pytest.mark.parametrize("call,what", [
    (lambda: gt.mm_tn_gated(), "missing required argument 'a'"), (lambda: gt.mm_tn_gated(1, 2), "a must be a tensor"),
    (lambda: gt.mm_tn_gated(1, 2, 3, b=4), "multiple values"), (lambda: gt.mm_nt(1, 2, trans=1), "unexpected keyword"),
    (lambda: gt.quantize_e4m3(*range(6)), "at most 5"), (lambda: gt.mm_tn_e4m3(1, 2, 3), "missing required argument 'b_scale'")])
def test_the_binding_refuses_what_is_no_call(lib, call, what):
    with pytest.raises(TypeError, match=what):
        call()


def test_the_binding_takes_cuda_tensors_only(lib):
    t = torch.zeros((4, 8), dtype=torch.bfloat16)
    for call in (lambda: gt.mm_tn_gated(t, t), lambda: gt.gated_grad(t, t), lambda: gt.mm_nt(t, t), lambda: gt.quantize_e4m3(t),
                 lambda: gt.mm_tn_e4m3(t, t, t, t)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_the_bindings_names_and_documentation(lib):
    import inspect
    assert set(_ff.BOUND) <= set(dir(gt))
    for name in _ff.BOUND:
        assert getattr(gt, name).__doc__
    assert list(inspect.signature(gt.mm_tn_gated).parameters) == ["a", "b", "out", "pre", "activation", "status"]
    assert inspect.signature(gt.quantize_e4m3).parameters["transpose"].default is False


def test_a_missing_binding_fails_loudly(lib, monkeypatch):
    import sys
    monkeypatch.setitem(sys.modules, "dense_tiled_gemm_03_gb300._feed_forward", None)
    monkeypatch.delattr(gt, "_feed_forward", raising=False)
    with pytest.raises(RuntimeError, match="build it"):
        _ff.binding()


def test_a_binding_built_against_another_torch_is_not_used(lib, monkeypatch):
    from dense_tiled_gemm_03_gb300 import build as b
    here = b.torch_dir()
    assert _ff.binding().built_against == torch.__version__ and not b.ff_binding_is_stale(here)
    monkeypatch.setattr(b, "torch_version", lambda d: "0.0.1+cu1")
    assert b.ff_binding_is_stale(here)
    monkeypatch.setattr(torch, "__version__", "0.0.1+cu1")
    with pytest.raises(RuntimeError, match="build it"):
        _ff.binding()


# ---------------------------------------------------------------- the references

def test_the_slopes_are_the_activations_derivatives():
    g = torch.linspace(-9, 9, 721, dtype=torch.float64)
    for act in ("silu", "gelu"):
        x = g.clone().requires_grad_()
        (x * ref.share(x, act)).sum().backward()
        assert torch.allclose(x.grad, ref.slope(g, act), rtol=1e-12, atol=1e-15)


def test_the_gradient_of_the_reference():
    """gated_grad, and the products behind it, against autograd in 64 bits."""
    gen = torch.Generator().manual_seed(3)
    x, w = torch.randn((7, 12), generator=gen).half(), torch.randn((10, 12), generator=gen).half()
    dh = torch.randn((7, 5), generator=gen).half()
    for act in ("silu", "gelu", "relu"):
        X, W = x.double().requires_grad_(), w.double().requires_grad_()
        g, u = (X @ W.T).chunk(2, 1)
        g.retain_grad(), u.retain_grad()
        (g * ref.share(g, act) * u * dh.double()).sum().backward()
        pre = (x.double() @ w.double().T)
        d, _ = ref.gated_grad(dh.double().to(torch.float16), pre.to(torch.float16), act)
        exact = torch.cat([dh.double() * pre[:, 5:] * ref.slope(pre[:, :5], act), dh.double() * pre[:, :5] * ref.share(pre[:, :5], act)], 1)
        assert torch.allclose(exact, torch.cat([g.grad, u.grad], 1), rtol=1e-12, atol=1e-14)
        assert torch.allclose(d, exact, rtol=2e-2, atol=2e-2)
        assert torch.allclose(exact @ w.double(), X.grad, rtol=1e-12, atol=1e-12)
        assert torch.allclose(exact.T @ x.double(), W.grad, rtol=1e-12, atol=1e-12)


def test_quantized_closed_forms():
    """Values of the format itself come back; the scale is the least power of two that fits; torch rounds the same."""
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    every = every[torch.isfinite(every)]
    x = torch.zeros((1, 256))
    x[0, :every.numel()] = every
    x[0, 127], x[0, 128] = 448.0, 448.0
    q, s = ref.quantized(x, 1, False)
    assert torch.equal(s, torch.ones((1, 2), dtype=torch.float64)) and torch.equal(q, x.double())
    for top, scale in ((448.0, 1.0), (449.0, 2.0), (224.0, 0.5), (225.0, 1.0), (1.0, 2.0 ** -8), (0.0, 1.0), (1e-40, 2.0 ** -126)):
        assert float(ref.quantized(torch.tensor([[top]]), 1, False)[1]) == scale
    gen = torch.Generator().manual_seed(1)
    y = torch.randn((300, 130), generator=gen)
    for rows, transpose in ((1, False), (128, False), (1, True)):
        q, s = ref.quantized(y, rows, transpose)
        z = (y.T if transpose else y) / ref.spread(s, rows, q.shape).float()
        assert torch.equal(q.float(), z.to(torch.float8_e4m3fn).float())
    q, s = ref.quantized(torch.tensor([[math.nan, math.inf, 1.0]]), 1, False)
    assert math.isnan(q[0, 0]) and math.isnan(q[0, 1]) and float(q[0, 2] * s[0, 0]) == 1.0


def test_a_mistake_is_seen():
    """The comparison catches one wrong element, one step of the output's type off, and NaN."""
    a, b = torch.ones((4, 8), dtype=torch.bfloat16), torch.ones((6, 8), dtype=torch.bfloat16)
    h, off, _, _ = ref.gated(a, b, "relu", torch.bfloat16)
    ref.assert_close(h, h, off)
    for wrong in (h[1, 2] * (1 + 2.0 ** -6), torch.tensor(math.nan)):
        bad = h.clone()
        bad[1, 2] = wrong
        with pytest.raises(AssertionError, match="1 of 12"):
            ref.assert_close(bad, h, off)
