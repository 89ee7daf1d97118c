"""64-bit references of the feed-forward operators, and how far their kernels
may be off.

Tolerances are bounds, from the arithmetic that include/feed_forward.h states:
  * a sum of K products in fp32: every addition (and the tensor core's
    alignment of a group of products) is off by at most a unit in the last
    place of the sums so far, which S = sum |a b| bounds: K 2^-23 S;
  * an activation: exp and the division or erfc, to 2^-20 of the result;
  * rounding to fewer bits: half a step, eps / 2 of the value (and half the
    smallest subnormal).
"""
from __future__ import annotations

import math

import torch

HALF_STEP = {t: torch.finfo(t).eps / 2 for t in (torch.float16, torch.bfloat16, torch.float32)}
SMALLEST = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -150}
ULP = 2.0 ** -23
FUNCTION = 2.0 ** -20


def half_step(ref, dtype):
    return ref.abs() * HALF_STEP[dtype] + SMALLEST[dtype]


def share(g, act):
    """act(g) / g."""
    if act == "silu":
        return torch.sigmoid(g)
    if act == "gelu":
        return 0.5 * torch.erfc(-g / math.sqrt(2))
    return (g > 0).double()


def slope(g, act):
    s = share(g, act)
    if act == "silu":
        return s * (1 + g * (1 - s))
    if act == "gelu":
        return s + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    return s


def gated(a, b, act, dtype):
    """(h, its bound, pre, its bound) of 16-bit a [m, k] and b [2n, k]."""
    n, k = b.shape[0] // 2, a.shape[1]
    a, b = a.double(), b.double()
    pre, size = a @ b.T, a.abs() @ b.abs().T
    off = k * ULP * size
    g, u, og, ou = pre[:, :n], pre[:, n:], off[:, :n], off[:, n:]
    f = g * share(g, act)
    h = f * u
    of = 1.13 * og + FUNCTION * f.abs()      # |act'| <= 1.13 for silu and gelu, 1 for relu
    return h, of * u.abs() + f.abs() * ou + of * ou + half_step(h, dtype), pre, off + half_step(pre, dtype)


def gated_grad(dh, pre, act):
    """(d, its bound) of 16-bit dh [m, n] and pre [m, 2n]."""
    dtype, n = dh.dtype, dh.shape[1]
    dh, g, u = dh.double(), pre[:, :n].double(), pre[:, n:].double()
    f = g * share(g, act)
    d = torch.cat([dh * u * slope(g, act), dh * f], 1)
    # the slope adds terms of up to 1 + |g|, each to FUNCTION
    off = torch.cat([(dh * u).abs() * (1 + g.abs()) * 2 * FUNCTION, (dh * f).abs() * FUNCTION], 1)
    return d, off + half_step(d, dtype)


def mm_nt(a, b, dtype, onto=None):
    k = a.shape[0]
    a, b = a.double(), b.double()
    c = a.T @ b
    off = k * ULP * (a.abs().T @ b.abs())
    if onto is not None:
        c = c + onto.double()
        off = off + ULP * c.abs()
    return c, off + half_step(c, dtype)


def quantized(x, block_rows, transpose):
    """(q as 64-bit values, scale) by the definition, bit for bit."""
    x = x.double()
    if transpose:
        x = x.T
    m, k = x.shape
    kb, mb = (k + 127) // 128, (m + block_rows - 1) // block_rows
    scale = torch.ones((mb, kb), dtype=torch.float64)
    q = torch.empty((m, k), dtype=torch.float64)
    for i in range(mb):
        for j in range(kb):
            rows, cols = slice(i * block_rows, (i + 1) * block_rows), slice(j * 128, (j + 1) * 128)
            part = x[rows, cols]
            finite = part[torch.isfinite(part)].abs()
            top = float(finite.max()) if finite.numel() else 0.0
            t = 0
            if top > 0:
                t = max(math.frexp(top)[1] - 9 - 2, -126)
                while top > 448.0 * 2.0 ** t:
                    t += 1
            scale[i, j] = 2.0 ** t
            y = part / 2.0 ** t
            step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
            y = torch.round(y / step) * step
            q[rows, cols] = torch.where(torch.isfinite(part), y, math.nan)
    return q, scale


def spread(scale, rows, shape):
    """Each element's scale."""
    return scale.double().repeat_interleave(rows, 0)[:shape[0]].repeat_interleave(128, 1)[:, :shape[1]]


def mm_e4m3(a, sa, b, sb, b_rows, dtype, onto=None):
    k = a.shape[1]
    x, y = a.double() * spread(sa, 1, a.shape), b.double() * spread(sb, b_rows, b.shape)
    c = x @ y.T
    # sums of a block's products, then three roundings a block (its scales' product, the block's, the sum's)
    off = (128 + 3 * ((k + 127) // 128)) * ULP * (x.abs() @ y.abs().T)
    if onto is not None:
        c = c + onto.double()
        off = off + ULP * c.abs()
    return c, off + half_step(c, dtype)


def assert_close(got, ref, bound, what=""):
    got = got.double().cpu()
    ref, bound = ref.cpu(), bound.cpu()
    assert got.shape == ref.shape, what
    bad = ~((got - ref).abs() <= bound)      # NaN is bad
    if bool(bad.any()):
        at = tuple(int(i) for i in bad.nonzero()[0])
        worst = float(((got - ref).abs() / bound).nan_to_num(1e30).max())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {at}: {float(got[at])} for "
                             f"{float(ref[at])} +- {float(bound[at])}; worst {worst:.3g} of the bound")
