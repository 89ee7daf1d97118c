"""The feed-forward operators on the GPU against 64-bit references
(``_ff_ref``: the tolerances and where they come from)."""
from __future__ import annotations

import math

import pytest
import torch

import dense_tiled_gemm_03_gb300 as gt

import _ff_ref as ref
from _parity import env_var, require_gpu

pytestmark = pytest.mark.gpu

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
#: every kernel of whole tiles, and of few rows
TILES = ["pair256", "pair128", "single128"]
SKINNY = ["skinny1", "skinny2", "skinny4", "skinny8"]
ACTS = ["silu", "gelu", "relu"]
#: the output's padding columns and rows, left as they were
FILL = 7.0


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    from dense_tiled_gemm_03_gb300 import build as native_build
    native_build.build()


def kernel(name):
    return env_var("GEMM_TN_FF_KERNEL", None if name == "auto" else name)


def normal(gen, *shape, scale=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=gen) * scale).to(dtype)


def padded(shape, dtype, pitch=None, fill=FILL):
    """A matrix of that shape inside a larger one, all of it `fill`: (matrix, the larger one)."""
    rows, cols = shape
    whole = torch.full((rows + 2, pitch or cols + 24), fill, dtype=torch.float32).to(dtype).cuda()
    return whole[:rows, :cols], whole


def assert_outside(view, whole, fill=FILL):
    w = whole.float().cpu()
    rows, cols = view.shape
    assert bool((w[rows:] == fill).all()) and bool((w[:, cols:] == fill).all()), "written outside the output"


def laid_out(x, layout, to="cuda"):
    """x on the GPU: as it is, or in wider rows from an odd start (which the kernels must copy first)."""
    x = x.to(to)
    if layout == "plain":
        return x
    rows, cols = x.shape
    whole = torch.zeros((rows, cols + 5), dtype=x.dtype, device=to)
    whole[:, 3:3 + cols] = x
    return whole[:, 3:3 + cols]


# ---------------------------------------------------------------- the gated projection

def check_gated(m, n, k, dtype, act, which, train=True, layout="plain", seed=0):
    gen = torch.Generator().manual_seed(seed + m * 7 + n * 3 + k)
    dt = DTYPES[dtype]
    a, b = normal(gen, m, k, dtype=dt), normal(gen, 2 * n, k, scale=k ** -0.5, dtype=dt)
    odd = 1 if layout == "odd" else 0
    out, out_whole = padded((m, n), dt, (n + 7) // 8 * 8 + 8 + odd)
    pre, pre_whole = padded((m, 2 * n), dt, (2 * n + 7) // 8 * 8 + 8 + odd) if train else (None, None)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    with kernel(which):
        got = gt.mm_tn_gated(laid_out(a, layout), laid_out(b, layout), out=out, pre=pre, activation=act, status=status)
    assert got is out and int(status.item()) == 0
    h, h_off, p, p_off = ref.gated(a, b, act, dt)
    ref.assert_close(out, h, h_off, "h")
    assert_outside(out, out_whole)
    if train:
        ref.assert_close(pre, p, p_off, "pre")
        assert_outside(pre, pre_whole)


@pytest.mark.parametrize("which", TILES + SKINNY)
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("mnk", [(1, 1, 1), (7, 64, 520), (16, 128, 512), (33, 65, 530), (100, 200, 640), (128, 333, 1000)],
                         ids=str)
def test_gated_few_rows(mnk, dtype, which):
    check_gated(*mnk, dtype, "silu", which)


@pytest.mark.parametrize("which", ["auto"] + TILES)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("mnk", [(129, 64, 64), (256, 256, 65), (300, 517, 130), (513, 1000, 264)], ids=str)
def test_gated_tiles(mnk, act, which):
    check_gated(*mnk, "bf16", act, which, train=act != "relu")


@pytest.mark.parametrize("which", ["auto", "pair256", "skinny2"])
@pytest.mark.parametrize("mnk", [(40, 100, 129), (1, 72, 257)], ids=str)
def test_gated_odd_layouts(mnk, which):
    check_gated(*mnk, "fp16", "gelu", which, layout="odd")


def test_gated_many_tiles():
    """Several tiles a CTA, the last wave partial; both buffers of tensor memory change hands many times."""
    check_gated(2900, 2600, 192, "bf16", "silu", "pair256", train=False)
    check_gated(2900, 2600, 192, "bf16", "silu", "single128", train=False)


def test_gated_extremes():
    """Large negative and positive gates, NaN and infinities stay in their rows."""
    k, n = 64, 40
    a = torch.zeros((200, k), dtype=torch.bfloat16)
    b = torch.zeros((2 * n, k), dtype=torch.bfloat16)
    a[:, 0] = torch.linspace(-60, 60, 200).to(torch.bfloat16)
    b[:n, 0] = torch.linspace(0.5, 3, n).to(torch.bfloat16)
    a[:, 1] = 1
    b[n:, 1] = 2
    for act in ACTS:
        h, off, _, _ = ref.gated(a, b, act, torch.bfloat16)
        for rows in (200, 20):
            ref.assert_close(gt.mm_tn_gated(a[-rows:].cuda(), b.cuda(), activation=act), h[-rows:], off[-rows:], act)
    a[5, 2], a[9, 2] = math.nan, math.inf
    b[:, 2] = 1
    for rows in (200, 20):
        out = gt.mm_tn_gated(a[:rows].cuda(), b.cuda()).float().cpu()
        assert bool(out[5].isnan().all()) and bool(out[9].isinf().all())
        keep = [i for i in range(rows) if i not in (5, 9)]
        assert bool(out[keep].isfinite().all())


def test_gated_empty():
    a, b = torch.ones((4, 0), dtype=torch.float16, device="cuda"), torch.ones((12, 0), dtype=torch.float16, device="cuda")
    out, pre = torch.full((4, 6), 3.0, dtype=torch.float16, device="cuda"), torch.full((4, 12), 3.0, dtype=torch.float16, device="cuda")
    gt.mm_tn_gated(a, b, out=out, pre=pre)
    assert bool((out == 0).all()) and bool((pre == 0).all())
    assert gt.mm_tn_gated(torch.ones((0, 8), dtype=torch.float16, device="cuda"), torch.ones((4, 8), dtype=torch.float16, device="cuda")).shape == (0, 2)
    assert gt.mm_tn_gated(torch.ones((3, 8), dtype=torch.float16, device="cuda"), torch.ones((0, 8), dtype=torch.float16, device="cuda")).shape == (3, 0)


# ---------------------------------------------------------------- its gradient

@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("mn", [(1, 1), (3, 8), (77, 129), (64, 512), (1, 4096), (1030, 24)], ids=str)
@pytest.mark.parametrize("in_place", [False, True])
def test_gated_grad(mn, dtype, act, in_place):
    gen = torch.Generator().manual_seed(sum(mn))
    m, n = mn
    dh, pre = normal(gen, m, n, dtype=DTYPES[dtype]), normal(gen, m, 2 * n, scale=3.0, dtype=DTYPES[dtype])
    pre[0, 0] = 0.0
    d, off = ref.gated_grad(dh, pre, act)
    p = pre.cuda()
    if in_place:
        out = gt.gated_grad(dh.cuda(), p, out=p, activation=act)
        assert out is p
    else:
        out, whole = padded((m, 2 * n), DTYPES[dtype], (2 * n + 7) // 8 * 8 + 8)
        gt.gated_grad(dh.cuda(), p, out=out, activation=act)
        assert_outside(out, whole)
        assert torch.equal(p.cpu(), pre)
    ref.assert_close(out, d, off, act)


def test_gated_grad_odd_start():
    gen = torch.Generator().manual_seed(5)
    dh, pre = normal(gen, 50, 96, dtype=torch.bfloat16), normal(gen, 50, 192, dtype=torch.bfloat16)
    d, off = ref.gated_grad(dh, pre, "silu")
    ref.assert_close(gt.gated_grad(laid_out(dh, "odd"), laid_out(pre, "odd")), d, off)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gated_grad_differences(act):
    """The gradient against differences of the forward pass (64 bits): h(g + e) - h(g - e) over 2 e."""
    gen = torch.Generator().manual_seed(11)
    dh, pre = normal(gen, 8, 64, dtype=torch.bfloat16), normal(gen, 8, 128, dtype=torch.bfloat16)
    out = gt.gated_grad(dh.cuda(), pre.cuda(), activation=act).double().cpu()
    g, u, e = pre[:, :64].double(), pre[:, 64:].double(), 1e-5
    f = lambda x: x * ref.share(x, act)
    dg, du = dh.double() * u * (f(g + e) - f(g - e)) / (2 * e), dh.double() * f(g)
    d = torch.cat([dg, du], 1)
    # the differences' own error: e^2 / 6 of a third derivative below 2, and 2^-50 / e of rounding
    _, off = ref.gated_grad(dh, pre, act)
    ref.assert_close(out, d, off + 1e-9 * (1 + torch.cat([dh * u, dh * u], 1).double().abs()))


# ---------------------------------------------------------------- A^T B

@pytest.mark.parametrize("which", ["auto"] + TILES)
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("out_dtype", ["input", "fp32", "added"])
@pytest.mark.parametrize("mnk", [(1, 1, 1), (64, 64, 64), (130, 72, 200), (300, 517, 65), (256, 1000, 513)], ids=str)
def test_mm_nt(mnk, dtype, out_dtype, which):
    m, n, k = mnk
    gen = torch.Generator().manual_seed(m + n + k)
    dt = DTYPES[dtype]
    a, b = normal(gen, k, m, dtype=dt), normal(gen, k, n, dtype=dt)
    od = dt if out_dtype == "input" else torch.float32
    out, whole = padded((m, n), od, (n + 7) // 8 * 8 + 8)
    onto = None
    if out_dtype == "added":
        onto = normal(gen, m, n)
        out.copy_(onto)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    with kernel(which):
        gt.mm_nt(a.cuda(), b.cuda(), out=out, accumulate=out_dtype == "added", status=status)
    assert int(status.item()) == 0
    ref.assert_close(out, *ref.mm_nt(a, b, od, onto))
    assert_outside(out, whole)


@pytest.mark.parametrize("od", ["fp16", "fp32"])
def test_mm_nt_odd_layouts(od):
    gen = torch.Generator().manual_seed(3)
    a, b = normal(gen, 150, 77, dtype=torch.float16), normal(gen, 150, 90, dtype=torch.float16)
    out, whole = padded((77, 90), DTYPES[od], 99)
    gt.mm_nt(laid_out(a, "odd"), laid_out(b, "odd"), out=out)
    ref.assert_close(out, *ref.mm_nt(a, b, DTYPES[od]))
    assert_outside(out, whole)


def test_mm_nt_empty():
    a, b = torch.ones((0, 5), dtype=torch.float16, device="cuda"), torch.ones((0, 6), dtype=torch.float16, device="cuda")
    assert bool((gt.mm_nt(a, b) == 0).all())
    onto = torch.full((5, 6), 2.0, device="cuda")
    gt.mm_nt(a, b, out=onto, accumulate=True)
    assert bool((onto == 2).all())


# ---------------------------------------------------------------- quantising

def check_quantized(x, rows, transpose, layout="plain"):
    q, scale = gt.quantize_e4m3(laid_out(x, layout), block_rows=rows, transpose=transpose)
    want_q, want_s = ref.quantized(x, rows, transpose)
    assert q.dtype == torch.float8_e4m3fn and tuple(q.shape) == tuple(want_q.shape)
    assert torch.equal(scale.double().cpu(), want_s)
    got = q.float().double().cpu()
    assert torch.equal(torch.nan_to_num(got, nan=1e9), torch.nan_to_num(want_q, nan=1e9))


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("mk", [(1, 1), (1, 128), (16, 256), (130, 129), (128, 127), (257, 520)], ids=str)
def test_quantize(mk, dtype, rows, transpose):
    gen = torch.Generator().manual_seed(mk[0] * 5 + mk[1])
    x = (torch.randn(mk, generator=gen) * torch.randn(mk[1], generator=gen).mul(2).exp()).to(DTYPES[dtype])
    check_quantized(x, rows, transpose)


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_quantize_odd_layouts(dtype, transpose):
    gen = torch.Generator().manual_seed(2)
    x = torch.randn((150, 200), generator=gen).to(DTYPES[dtype])
    check_quantized(x, 1, transpose, "odd")
    # q in rows of any pitch, scales wherever their strides say
    q = torch.zeros((150, 211), dtype=torch.float8_e4m3fn, device="cuda")[:, 3:203]
    scale = torch.zeros((150, 7), device="cuda")
    if not transpose:
        gt.quantize_e4m3(x.cuda(), out=q, scale=scale[:, :4:2])
        want_q, want_s = ref.quantized(x, 1, False)
        assert torch.equal(q.float().double().cpu(), want_q) and torch.equal(scale[:, :4:2].double().cpu(), want_s)
        assert bool((scale[:, 1::2] == 0).all()) and bool((scale[:, 4:] == 0).all())


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
def test_quantize_edges(dtype, rows, transpose):
    """Zeros, subnormal and largest values, powers of two and 448 times them, ties, NaN and infinities."""
    dt = DTYPES[dtype]
    x = torch.zeros((256, 256), dtype=torch.float32)
    info = torch.finfo(dt)
    for i in range(128):
        x[i, :128] = torch.linspace(-1, 1, 128) * 2.0 ** (i % 20 - 10)
    x[3, :128] = info.smallest_normal / 8
    x[4, :128] = info.max
    x[5, :128] = torch.arange(128) * 0.5          # e4m3's ties among them
    x[6, 0], x[7, 0] = 448.0, 449.0
    x[6, 1:128] = 0.0
    x[128:, 128:] = torch.linspace(-448, 448, 128)
    x[200, 200], x[201, 201], x[202, 202] = math.nan, math.inf, -math.inf
    x[130, 5] = math.inf                          # a block of nothing else
    check_quantized(x.to(dt), rows, transpose)


# ---------------------------------------------------------------- the product in 8 bits

def operands(gen, m, n, k, b_rows):
    """e4m3 matrices with scales that are no powers of two."""
    def one(rows, per):
        q = torch.randn((rows, k), generator=gen).mul(60).clamp(-448, 448).to(torch.float8_e4m3fn)
        s = torch.rand(((rows + per - 1) // per, (k + 127) // 128), generator=gen).add(0.3).mul(0.02)
        return q, s
    return *one(m, 1), *one(n, b_rows)


def on_gpu(q, pitch=None):
    """An e4m3 matrix in rows a multiple of 16 bytes apart, NaN in the padding."""
    rows, cols = q.shape
    whole = torch.full((rows, pitch or (cols + 15) // 16 * 16 + 16), math.nan).to(torch.float8_e4m3fn).cuda()
    whole.view(torch.uint8)[:, :cols] = q.cuda().view(torch.uint8)
    return whole[:, :cols]


def check_e4m3(m, n, k, b_rows, od, which, added=False, side_by_side=True):
    gen = torch.Generator().manual_seed(m * 3 + n * 5 + k)
    a, sa, b, sb = operands(gen, m, n, k, b_rows)
    dt = DTYPES[od]
    out, whole = padded((m, n), dt, (n + 7) // 8 * 8 + 8)
    onto = None
    if added:
        onto = normal(gen, m, n)
        out.copy_(onto)
    gsa, gsb = sa.cuda(), sb.cuda()
    if side_by_side:
        gsa = gsa.t().contiguous().t()
        gsb = gsb.t().contiguous().t()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    with kernel(which):
        gt.mm_tn_e4m3(on_gpu(a), gsa, on_gpu(b), gsb, out=out, accumulate=added, status=status)
    assert int(status.item()) == 0
    ref.assert_close(out, *ref.mm_e4m3(a.float(), sa, b.float(), sb, b_rows, dt, onto))
    assert_outside(out, whole)


@pytest.mark.parametrize("which", TILES + SKINNY)
@pytest.mark.parametrize("b_rows", [1, 128])
@pytest.mark.parametrize("mnk", [(1, 1, 1), (7, 128, 1024), (17, 200, 1040), (33, 129, 1200), (100, 333, 1025), (128, 260, 1100)],
                         ids=str)
def test_e4m3_few_rows(mnk, b_rows, which):
    check_e4m3(*mnk, b_rows, "fp32", which)


@pytest.mark.parametrize("which", ["auto"] + TILES)
@pytest.mark.parametrize("b_rows", [1, 128])
@pytest.mark.parametrize("od", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("mnk", [(129, 64, 128), (256, 256, 100), (300, 517, 257), (513, 1000, 777)], ids=str)
def test_e4m3_tiles(mnk, od, b_rows, which):
    check_e4m3(*mnk, b_rows, od, which, side_by_side=od != "fp16")


@pytest.mark.parametrize("which", TILES + ["skinny1", "skinny2"])
@pytest.mark.parametrize("b_rows", [1, 128])
def test_e4m3_added(b_rows, which):
    check_e4m3(100, 200, 300, b_rows, "fp32", which, added=True)


def test_e4m3_many_tiles():
    for which in ("pair256", "single128"):
        check_e4m3(2900, 5200, 300, 128, "fp32", which)
        check_e4m3(2900, 5200, 300, 1, "bf16", which)


def test_e4m3_empty():
    e = lambda *s: torch.zeros(s, dtype=torch.float8_e4m3fn, device="cuda")
    f = lambda *s: torch.zeros(s, device="cuda")
    assert bool((gt.mm_tn_e4m3(e(5, 0), f(5, 0), e(6, 0), f(6, 0)) == 0).all())
    onto = torch.full((5, 6), 2.0, device="cuda")
    gt.mm_tn_e4m3(e(5, 0), f(5, 0), e(6, 0), f(1, 0), out=onto, accumulate=True)
    assert bool((onto == 2).all())
    assert gt.mm_tn_e4m3(e(0, 16), f(0, 1), e(6, 16), f(6, 1)).shape == (0, 6)
    assert gt.mm_tn_e4m3(e(3, 16), f(3, 1), e(0, 16), f(0, 1)).shape == (3, 0)
