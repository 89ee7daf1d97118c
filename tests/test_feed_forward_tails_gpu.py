"""The gate's activations far from zero, against 64 bits, at gates that 16 bits
hold exactly, so that no product's error hides the function's own.

Bounds: _ff_ref.FUNCTION of the function's value (of each of a slope's terms,
which share a factor that vanishes below zero), the one rounding to the output's
type, and where e^-|g| is below fp32's normal numbers its steps of 2^-149. The
projection's gate is an fp32 sum that may be off by half of its last place, |g| 2^-24,
which e^-|g| carries on as a share of itself; its exponent in base 2 is one more such
product, with a constant of 24 bits: 2^-24 + 2^-26 of |g|; together below |g| 2^-22."""
from __future__ import annotations

import math

import pytest
import torch

import dense_tiled_gemm_03_gb300 as gt

import _ff_ref as ref
from _parity import require_gpu

pytestmark = pytest.mark.gpu

STEP = 2.0 ** -149
#: as far as the function is a normal bf16 number below zero, and a little further
REACH = {"silu": 90.0, "gelu": 13.0, "relu": 90.0}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    from dense_tiled_gemm_03_gb300 import build as native_build
    native_build.build()


def gates(act, dtype, count=4000):
    return torch.linspace(-REACH[act], REACH[act], count).to(dtype)


def value(g, act):
    """(act(g), its bound before any rounding)."""
    f = g * ref.share(g, act)
    return f, f.abs() * ref.FUNCTION + g.abs() * STEP


def slope(g, act):
    """(act'(g), its bound before any rounding)."""
    s = ref.share(g, act)
    if act == "silu":
        terms = s * (1 + (g * (1 - s)).abs())
    elif act == "gelu":
        terms = s + g.abs() * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    else:
        terms = s
    return ref.slope(g, act), 4 * ref.FUNCTION * terms + (1 + g.abs()) * STEP


@pytest.mark.parametrize("act", list(REACH))
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("n", [8, 4, 1])      # the widths of the kernel's pieces
def test_gradient_far_from_zero(n, dtype, act):
    g = gates(act, dtype).view(-1, n)
    one = torch.ones_like(g)
    d = gt.gated_grad(one.cuda(), torch.cat([g, one], 1).cuda(), activation=act)
    g = g.double()
    (f, f_off), (s, s_off) = value(g, act), slope(g, act)
    ref.assert_close(d[:, n:], f, f_off + ref.half_step(f, dtype), "dU")
    ref.assert_close(d[:, :n], s, s_off + ref.half_step(s, dtype), "dG")


@pytest.mark.parametrize("act", list(REACH))
@pytest.mark.parametrize("up", [1.0, 2.0 ** 100])
@pytest.mark.parametrize("rows", [20, 400])   # few rows, whole tiles
def test_projection_far_from_zero(rows, up, act):
    """A row's gate is its first element, its other projection the second."""
    bf = torch.bfloat16
    g = gates(act, bf)
    for part in g.split(rows):
        a = torch.zeros((part.numel(), 8), dtype=bf)
        a[:, 0], a[:, 1] = part, up
        b = torch.zeros((2 * 40, 8), dtype=bf)
        b[:40, 0], b[40:, 1] = 1, 1
        h = gt.mm_tn_gated(a.cuda(), b.cuda(), activation=act)
        f, off = value(part.double(), act)
        off = off + f.abs() * part.double().abs() * 2.0 ** -22
        want = (f * up)[:, None].expand(-1, 40)
        ref.assert_close(h, want, (off * up)[:, None] + ref.half_step(want, bf), f"from {float(part[0])}")


@pytest.mark.parametrize("act", list(REACH))
def test_ends_of_the_range(act):
    """Zero and the largest finite gates, infinities and NaN, as torch's own functions have them in 32 bits."""
    bf = torch.bfloat16
    most = torch.finfo(bf).max
    g = torch.tensor([0.0, -0.0, most, -most, math.inf, math.nan, 104.0, -200.0], dtype=bf)[:, None]
    d = gt.gated_grad(torch.ones_like(g).cuda(), torch.cat([g, torch.ones_like(g)], 1).cuda(), activation=act).cpu()
    fn = {"silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu, "relu": torch.relu}[act]
    assert torch.equal(torch.nan_to_num(d[:, 1].float(), nan=7.0), torch.nan_to_num(fn(g[:, 0].float()).to(bf).float(), nan=7.0))
    keep = [0, 1, 2, 3, 6, 7]                 # (the slope of silu and gelu at infinity is infinity times zero)
    want = ref.slope(g[keep, 0].double(), act)
    assert torch.equal(d[keep, 0].double(), want.to(bf).double())
