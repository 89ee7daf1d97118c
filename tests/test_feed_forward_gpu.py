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


@pytest.mark.parametrize("which", ["auto"] + TILES)
@pytest.mark.parametrize("out_dtype", ["bf16", "fp32", "added"])
@pytest.mark.parametrize("mnk", [(1, 1, 4096), (70, 90, 4033), (300, 517, 5000), (1100, 513, 8190)], ids=str)
def test_mm_nt_long(mnk, out_dtype, which):
    """Few tiles and many tokens: K is cut into parts, joined in order."""
    m, n, k = mnk
    gen = torch.Generator().manual_seed(m + n + k)
    a, b = normal(gen, k, m, dtype=torch.bfloat16), normal(gen, k, n, dtype=torch.bfloat16)
    od = torch.bfloat16 if out_dtype == "bf16" else torch.float32
    out, whole = padded((m, n), od, n + 9)
    onto = None
    if out_dtype == "added":
        onto = normal(gen, m, n)
        out.copy_(onto)
    before = gt.gemm_tn_launch_count()
    with kernel(which):
        gt.mm_nt(a.cuda(), b.cuda(), out=out, accumulate=out_dtype == "added")
    assert gt.gemm_tn_launch_count() - before >= 2
    ref.assert_close(out, *ref.mm_nt(a, b, od, onto))
    assert_outside(out, whole)


@pytest.mark.parametrize("which", ["auto", "skinny2", "skinny4", "skinny8"])
@pytest.mark.parametrize("mnk", [(129, 70, 2100), (300, 200, 4100), (700, 100, 2048)], ids=str)
def test_several_tiles_of_few_rows(mnk, which):
    """More rows than a skinny tile takes, few columns, a long K."""
    check_gated(*mnk, "bf16", "silu", which)
    for b_rows in (1, 128):
        check_e4m3(mnk[0], mnk[1], 4 * mnk[2], b_rows, "fp32", which)


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


# ---------------------------------------------------------------- together, as they are used

def rounded(x, dtype):
    return x.to(dtype).double()


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("tokens", [5, 200])
def test_a_block_and_its_gradients(tokens, dtype, act):
    """A feed-forward block, forward and backward: y = h Wd^T with h = act(x Wg^T) * (x Wu^T); from dy the gradients of
    x and of all three weights. Every step is checked against 64 bits from the step's own inputs."""
    gen = torch.Generator().manual_seed(tokens)
    dt, k, n = DTYPES[dtype], 192, 328
    x, w = normal(gen, tokens, k, dtype=dt).cuda(), normal(gen, 2 * n, k, scale=k ** -0.5, dtype=dt).cuda()
    wd, dy = normal(gen, k, n, scale=n ** -0.5, dtype=dt).cuda(), normal(gen, tokens, k, dtype=dt).cuda()
    pre = torch.empty((tokens, 2 * n), dtype=dt, device="cuda")
    h = gt.mm_tn_gated(x, w, pre=pre, activation=act)
    y = gt.mm_tn(h, wd)
    dwd = gt.mm_nt(dy, h, out_dtype=torch.float32)          # [k, n], like wd
    dh = gt.mm_nn(dy, wd)
    d = gt.gated_grad(dh, pre, activation=act)
    dx = gt.mm_nn(d, w)
    dw = torch.zeros((2 * n, k), device="cuda")
    for _ in range(2):
        gt.mm_nt(d, x, out=dw, accumulate=True)             # two micro-batches' gradients, here the same
    c = lambda t: t.cpu()
    hr, ho, pr, po = ref.gated(c(x), c(w), act, dt)
    ref.assert_close(h, hr, ho, "h")
    ref.assert_close(pre, pr, po, "pre")
    ref.assert_close(d, *ref.gated_grad(c(dh), c(pre), act), "d")
    ref.assert_close(dwd, *ref.mm_nt(c(dy), c(h), torch.float32), "dwd")
    once, off = ref.mm_nt(c(d), c(x), torch.float32)
    ref.assert_close(dw, 2 * once, 2 * off + 2 * ref.ULP * (2 * once).abs(), "dw")
    # the whole chain against 64 bits without any rounding between: each of the
    # few roundings to 16 bits on the way is half a step of its value, and the
    # products behind it carry it as a sum of signed terms, bounded by their magnitudes
    eps = torch.finfo(dt).eps / 2
    X, W, WD, DY = (c(t).double() for t in (x, w, wd, dy))
    G, U = (X @ W.T).chunk(2, 1)
    a, s = G * ref.share(G, act), ref.slope(G, act)
    DH = DY @ WD
    D = torch.cat([DH * U * s, DH * a], 1)
    # d: dh's rounding, g's and u's (the slope's own slope is below 1.1) and d's own, and fp32 products' far smaller errors
    size_h = DY.abs() @ WD.abs()
    Doff = eps * (4 * D.abs() + torch.cat([1.2 * (DH * U * G).abs(), 1.2 * (DH * G).abs()], 1)) + \
        400 * ref.ULP * torch.cat([size_h * (U * s).abs() + 2 * DH.abs() * (X.abs() @ W.abs().T).chunk(2, 1)[1] * 1.2
                                   + 2 * DH.abs() * U.abs() * (X.abs() @ W.abs().T).chunk(2, 1)[0] * 1.2,
                                   size_h * a.abs() + 2 * DH.abs() * (X.abs() @ W.abs().T).chunk(2, 1)[0] * 1.2], 1) + \
        8 * ref.SMALLEST[dt]
    DX = D @ W
    ref.assert_close(dx, DX, Doff @ W.abs() + 700 * ref.ULP * (D.abs() @ W.abs()) + 2 * eps * DX.abs() + ref.SMALLEST[dt], "dx")
    Y = (a * U) @ WD.T
    Hoff = eps * 3 * (a * U).abs() + 200 * ref.ULP * 1.2 * ((X.abs() @ W.abs().T).chunk(2, 1)[0] * U.abs()
                                                         + a.abs() * (X.abs() @ W.abs().T).chunk(2, 1)[1]) + ref.SMALLEST[dt]
    ref.assert_close(y, Y, Hoff @ WD.abs().T + 400 * ref.ULP * ((a * U).abs() @ WD.abs().T) + 2 * eps * Y.abs() + ref.SMALLEST[dt], "y")


@pytest.mark.parametrize("tokens", [3, 130, 300])
def test_a_linear_layer_in_8_bits(tokens):
    """y = x W^T with both quantised, and from dy the gradients: dx = dy W from the transposed weights, dW = dy^T x
    summed over tokens, both sides quantised along them and added to an fp32 gradient."""
    gen = torch.Generator().manual_seed(tokens)
    k, n = 272, 400
    x, w = normal(gen, tokens, k, dtype=torch.bfloat16).cuda(), normal(gen, n, k, scale=k ** -0.5).cuda()
    dy = normal(gen, tokens, n, scale=1e-3, dtype=torch.bfloat16).cuda()

    def both(t, rows=1, transpose=False):
        q, s = gt.quantize_e4m3(t, block_rows=rows, transpose=transpose)
        want_q, want_s = ref.quantized(t.cpu(), rows, transpose)
        assert torch.equal(q.float().double().cpu(), want_q) and torch.equal(s.double().cpu(), want_s)
        return q, s

    def check(got, a, b, b_rows, dtype, onto=None):
        ref.assert_close(got, *ref.mm_e4m3(a[0].float().cpu(), a[1].cpu(), b[0].float().cpu(), b[1].cpu(), b_rows, dtype, onto))

    xq, wq, wt, dyq = both(x), both(w, 128), both(w, 128, True), both(dy)
    check(gt.mm_tn_e4m3(*xq, *wq), xq, wq, 128, torch.bfloat16)
    check(gt.mm_tn_e4m3(*dyq, *wt, out_dtype=torch.float16), dyq, wt, 128, torch.float16)
    xt, dyt = both(x, 1, True), both(dy, 1, True)
    grad = normal(gen, n, k, scale=1e-2)
    out = grad.cuda()
    assert gt.mm_tn_e4m3(*dyt, *xt, out=out, accumulate=True) is out
    check(out, dyt, xt, 1, torch.float32, grad)
    # how far 8 bits are from none: half a step of either side, as relative 2^-4 and
    # for values below 2^-6 of their scale 2^-10 of it
    Y = x.cpu().double() @ w.cpu().double().T
    y = gt.mm_tn_e4m3(*xq, *wq, out_dtype=torch.float32).cpu().double()

    def step(t, s, rows):
        return t.abs() * 2.0 ** -4 + ref.spread(s.cpu(), rows, t.shape) * 2.0 ** -10

    X, W = x.cpu().double(), w.cpu().double()
    ex, ew = step(X, xq[1], 1), step(W, wq[1], 128)
    off = ex @ W.abs().T + X.abs() @ ew.T + ex @ ew.T + 200 * ref.ULP * (X.abs() @ W.abs().T)
    assert bool(((y - Y).abs() <= off).all())


# ---------------------------------------------------------------- streams, captures, repeats, far offsets

def calls(gen):
    """One call of every operator and kind of kernel, some through workspaces: (name, call, outputs)."""
    bf, out = torch.bfloat16, []
    for m, odd in ((20, False), (300, False), (300, True), (20, True)):
        k = 131 if odd else 136
        a, b = normal(gen, m, k, dtype=bf).cuda(), normal(gen, 2 * 70, k, dtype=bf).cuda()
        h, pre = torch.zeros((m, 70), dtype=bf, device="cuda"), torch.zeros((m, 140), dtype=bf, device="cuda")
        out.append((lambda a=a, b=b, h=h, pre=pre: gt.mm_tn_gated(a, b, out=h, pre=pre), [h, pre]))
        d, dh = torch.zeros((m, 140), dtype=bf, device="cuda"), normal(gen, m, 70, dtype=bf).cuda()
        p = normal(gen, m, 140, dtype=bf).cuda()
        out.append((lambda dh=dh, p=p, d=d: gt.gated_grad(dh, p, out=d), [d]))
        c = torch.zeros((140, k), device="cuda")
        out.append((lambda p=p, a=a, c=c: gt.mm_nt(p, a, out=c), [c]))
        if m == 300:
            long, c2 = normal(gen, 5000, k, dtype=bf).cuda(), torch.zeros((k, k), dtype=bf, device="cuda")
            out.append((lambda t=long, c=c2: gt.mm_nt(t, t, out=c), [c2]))
        x = normal(gen, m, k).cuda()
        for rows, transpose in ((1, False), (128, True)):
            q, s = gt.quantize_e4m3(x, rows, transpose)
            q.zero_()
            s.zero_()
            out.append((lambda x=x, r=rows, t=transpose, q=q, s=s: gt.quantize_e4m3(x, r, t, out=q, scale=s), [q, s]))
        (qa, sa), (qb, sb) = gt.quantize_e4m3(x), gt.quantize_e4m3(normal(gen, 200, k).cuda())
        if odd:
            sa, sb = sa.contiguous(), sb.contiguous()      # strides that whole tiles copy first
        y = torch.zeros((m, 200), dtype=torch.float16, device="cuda")
        out.append((lambda qa=qa, sa=sa, qb=qb, sb=sb, y=y: gt.mm_tn_e4m3(qa, sa, qb, sb, out=y), [y]))
    return out


def bits(tensors):
    return [t.clone().contiguous().view(torch.uint8).clone() for t in tensors]


def test_repeats_streams_and_captures():
    """The same bits again, on other streams at once, and from captures replayed in turn and over one another."""
    work = calls(torch.Generator().manual_seed(17))
    want = []
    for call, outs in work:
        call()
        want.append(bits(outs))
    torch.cuda.synchronize()

    def check(what):
        torch.cuda.synchronize()
        for i, (_, outs) in enumerate(work):
            for got, w in zip(bits(outs), want[i]):
                assert torch.equal(got, w), (what, i)
            for t in outs:
                t.view(torch.uint8).zero_() if t.is_contiguous() else t.zero_()
        torch.cuda.synchronize()

    check("first")
    for call, _ in work:
        call()
        call()
    check("again")
    streams = [torch.cuda.Stream() for _ in range(4)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for i, (call, _) in enumerate(work):
        with torch.cuda.stream(streams[i % 4]):
            for _ in range(3):
                call()
    check("streams")
    graphs = []
    for part in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=streams[part]):
            for call, _ in work[part::2]:
                call()
        graphs.append(g)
    check_zero = [bool((t.float() == 0).all()) for _, outs in work for t in outs]
    assert all(check_zero), "a capture ran"
    for _ in range(2):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    check("replayed")


@pytest.mark.parametrize("tokens", [64, 2304])
def test_a_captured_step_follows_its_inputs(tokens):
    """A block's forward and backward pass captured once and replayed over new tokens, weights and gradients: the bits of
    the same step called. Its products run on every kind of kernel, mm_nn's last tiles cut along K among them."""
    gen = torch.Generator(device="cuda").manual_seed(tokens)
    k, n, bf = 1000, 2176, torch.bfloat16
    new = lambda *s: torch.randn(s, generator=gen, device="cuda").to(bf)
    x, w, wd, dy = new(tokens, k), new(2 * n, k), new(k, n), new(tokens, k)
    pre = torch.empty((tokens, 2 * n), dtype=bf, device="cuda")

    def step():
        h = gt.mm_tn_gated(x, w, pre=pre)
        q, s = gt.quantize_e4m3(h)
        y = gt.mm_tn_e4m3(q, s, *gt.quantize_e4m3(wd, block_rows=128))
        dh = gt.mm_nn(dy, wd)
        d = gt.gated_grad(dh, pre)
        return [h, y, dh, gt.mm_nn(d, w), gt.mm_nt(d, x, out_dtype=torch.float32), gt.mm_nt(dy, h)]

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=torch.cuda.Stream()):
        captured = step()
    for _ in range(4):
        for t in (x, w, wd, dy):
            t.copy_(new(*t.shape))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got = bits(captured)
        want = bits(step())
        assert all(torch.equal(a, b) for a, b in zip(got, want)), [torch.equal(a, b) for a, b in zip(got, want)]


def test_one_scale_for_all():
    """Scales broadcast with strides of zero: a scale for a whole matrix."""
    gen = torch.Generator().manual_seed(31)
    a, _, b, _ = operands(gen, 200, 150, 500, 1)
    sa, sb = torch.full((1, 1), 0.37), torch.full((1, 1), 1.9)
    for rows in (200, 9):
        for lines, per in ((150, 1), (2, 128)):
            got = gt.mm_tn_e4m3(on_gpu(a[:rows]), sa.cuda().expand(rows, 4), on_gpu(b), sb.cuda().expand(lines, 4),
                                out_dtype=torch.float32)
            ref.assert_close(got, *ref.mm_e4m3(a[:rows].float(), sa.expand(rows, 4), b.float(), sb.expand(lines, 4), per, torch.float32))


def test_far_offsets():
    """Rows more than 2^31 elements apart: offsets past 32 bits in outputs and inputs."""
    pitch = (1 << 31) + 64
    gen = torch.Generator().manual_seed(23)
    bf = torch.bfloat16
    whole = torch.empty((2 * pitch + 512,), dtype=bf, device="cuda")
    far = whole.as_strided((3, 256), (pitch, 1))
    a, b = normal(gen, 3, 64, dtype=bf), normal(gen, 512, 64, dtype=bf)
    h, off, _, _ = ref.gated(a, b, "silu", bf)
    for which in ("skinny1", "pair128"):
        far.zero_()
        with kernel(which):
            gt.mm_tn_gated(a.cuda(), b.cuda(), out=far)
        ref.assert_close(far, h, off, which)
    # far rows as an operand: three tokens of a gradient's sum, and of a quantised matrix
    x = normal(gen, 3, 40, dtype=bf)
    ref.assert_close(gt.mm_nt(far, x.cuda(), out_dtype=torch.float32), *ref.mm_nt(far.cpu().contiguous(), x, torch.float32))
    check_quantized_equal(far)
    pre = whole.as_strided((3, 512), (pitch, 1))
    pre.copy_(normal(gen, 3, 512, dtype=bf))
    dh = normal(gen, 3, 256, dtype=bf)
    d, off = ref.gated_grad(dh, pre.cpu(), "silu")
    ref.assert_close(gt.gated_grad(dh.cuda(), pre, out=pre), d, off)
    bytes8 = whole.view(torch.uint8).view(torch.float8_e4m3fn)
    q8 = bytes8.as_strided((3, 256), (pitch, 1))           # (the third row past 2^32 bytes)
    xq = normal(gen, 3, 256)
    _, s = gt.quantize_e4m3(xq.cuda(), out=q8)
    want_q, want_s = ref.quantized(xq, 1, False)
    assert torch.equal(q8.float().double().cpu(), want_q) and torch.equal(s.double().cpu(), want_s)
    bq, bs = gt.quantize_e4m3(normal(gen, 100, 256).cuda())
    ref.assert_close(gt.mm_tn_e4m3(q8, s, bq, bs, out_dtype=torch.float32),
                     *ref.mm_e4m3(q8.float().cpu(), s.cpu(), bq.float().cpu(), bs.cpu(), 1, torch.float32))


def check_quantized_equal(x):
    q, scale = gt.quantize_e4m3(x)
    want_q, want_s = ref.quantized(x.cpu(), 1, False)
    assert torch.equal(q.float().double().cpu(), want_q) and torch.equal(scale.double().cpu(), want_s)


def test_the_watchdog():
    """A load that never comes: the wait runs out, the status says so, and the next call is whole."""
    import time
    gen = torch.Generator().manual_seed(29)
    bf = torch.bfloat16
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    runs = []
    for which in TILES + ["skinny1", "skinny4"]:
        m = 20 if which.startswith("skinny") else 300
        a, b = normal(gen, m, 1024, dtype=bf).cuda(), normal(gen, 400, 1024, dtype=bf).cuda()
        x = normal(gen, m, 1024).cuda()
        q, qs = gt.quantize_e4m3(x)
        w, ws = gt.quantize_e4m3(normal(gen, 300, 1024).cuda())
        w2, ws2 = gt.quantize_e4m3(normal(gen, 300, 1024).cuda(), 128)
        runs += [(which, lambda a=a, b=b: gt.mm_tn_gated(a, b, status=status)),
                 (which, lambda q=q, qs=qs, w=w, ws=ws: gt.mm_tn_e4m3(q, qs, w, ws, status=status)),
                 (which, lambda q=q, qs=qs, w=w2, ws=ws2: gt.mm_tn_e4m3(q, qs, w, ws, status=status))]
        if which in TILES:
            runs.append((which, lambda a=a: gt.mm_nt(a, a, status=status)))
    for which, call in runs:
        with kernel(which):
            before = call().float().clone()
            assert int(status.item()) == 0
            t0 = time.perf_counter()
            with env_var("GEMM_TN_WATCHDOG_MS", "100"), env_var("GEMM_TN_TEST_DROP_LOAD", "0"):
                call()
                torch.cuda.synchronize()
            assert int(status.item()) == gt.GEMM_TN_ERR_TIMEOUT and time.perf_counter() - t0 < 5.0, which
            status.zero_()
            assert torch.equal(call().float(), before) and int(status.item()) == 0, which


# ---------------------------------------------------------------- refusals

def test_refusals():
    bf, f8 = torch.bfloat16, torch.float8_e4m3fn
    z = lambda *s, d=bf: torch.zeros(s, dtype=d, device="cuda")
    a, b, x = z(4, 64), z(16, 64), z(6, 32, d=torch.float32)
    q, s = gt.quantize_e4m3(z(6, 256))
    w, ws = gt.quantize_e4m3(z(10, 256), 128)
    shared = z(4, 80)
    refused = [
        (lambda: gt.mm_tn_gated(a, z(15, 64)), ValueError, "2N"), (lambda: gt.mm_tn_gated(a, z(16, 63)), ValueError, "2N"),
        (lambda: gt.mm_tn_gated(a, z(16, 64, d=torch.float16)), TypeError, "same dtype"),
        (lambda: gt.mm_tn_gated(a.float(), b.float()), TypeError, "unsupported dtype"),
        (lambda: gt.mm_tn_gated(a.cpu(), b), ValueError, "CUDA"), (lambda: gt.mm_tn_gated(a, b.cpu()), ValueError, "CUDA"),
        (lambda: gt.mm_tn_gated(a[0], b), ValueError, "2-D"), (lambda: gt.mm_tn_gated(z(64, 4).t(), b), ValueError, "unit stride"),
        (lambda: gt.mm_tn_gated(a, b, out=z(4, 9)), ValueError, "out must be"),
        (lambda: gt.mm_tn_gated(a, b, out=z(4, 8, d=torch.float32)), TypeError, "out must be"),
        (lambda: gt.mm_tn_gated(a, b, pre=z(4, 8)), ValueError, "pre must be"),
        (lambda: gt.mm_tn_gated(a, b, activation="none"), ValueError, "activation"),
        (lambda: gt.mm_tn_gated(a, b, activation=3), ValueError, "activation"),
        (lambda: gt.mm_tn_gated(a, b, status=z(1)), ValueError, "status"),
        (lambda: gt.mm_tn_gated(shared[:, :64], b, out=shared[:, 56:64]), gt.GemmTnError, "overlaps"),
        (lambda: gt.mm_tn_gated(a, b, out=shared[:, :8], pre=shared[:, 4:20]), gt.GemmTnError, "overlaps"),
        (lambda: gt.mm_tn_gated(a, b, out=z(1, 8).expand(4, 8)), gt.GemmTnError, "ldh"),
        (lambda: gt.gated_grad(z(4, 8), z(4, 15)), ValueError, "pre must be"),
        (lambda: gt.gated_grad(z(4, 8), z(4, 16, d=torch.float16)), TypeError, "pre must be"),
        (lambda: gt.gated_grad(x, z(6, 64, d=torch.float32)), TypeError, "unsupported dtype"),
        (lambda: gt.gated_grad(shared[:, :8], shared[:, 8:24], out=shared[:, 7:23]), gt.GemmTnError, "overlaps"),
        (lambda: gt.gated_grad(z(4, 8), shared[:, 8:24], out=shared[:, 9:25]), gt.GemmTnError, "overlaps"),
        (lambda: gt.mm_nt(a, z(5, 8)), ValueError, "rows"), (lambda: gt.mm_nt(a, a, out_dtype=torch.float16), TypeError, "output dtype"),
        (lambda: gt.mm_nt(a, a, out_dtype="float32"), TypeError, "torch.dtype"),
        (lambda: gt.mm_nt(a, a, accumulate=True), ValueError, "accumulate"),
        (lambda: gt.mm_nt(a, a, out=z(64, 64), accumulate=True), ValueError, "accumulate"),
        (lambda: gt.quantize_e4m3(x, block_rows=64), ValueError, "block_rows"),
        (lambda: gt.quantize_e4m3(x.double()), TypeError, "unsupported dtype"),
        (lambda: gt.quantize_e4m3(x, out=z(6, 31, d=f8)), ValueError, "out must be"),
        (lambda: gt.quantize_e4m3(x, out=z(6, 32)), TypeError, "out must be"),
        (lambda: gt.quantize_e4m3(x, scale=z(6, 2, d=torch.float32)), ValueError, "scale must be"),
        (lambda: gt.quantize_e4m3(z(6, 300, d=torch.float32), scale=z(1, 3, d=torch.float32).expand(6, 3)), gt.GemmTnError, "apart"),
        (lambda: gt.mm_tn_e4m3(z(6, 256), s, w, ws), TypeError, "e4m3"), (lambda: gt.mm_tn_e4m3(q, s.to(bf), w, ws), TypeError, "float32"),
        (lambda: gt.mm_tn_e4m3(q, s[:, :1], w, ws), ValueError, "a_scale"), (lambda: gt.mm_tn_e4m3(q, s, w, s), ValueError, "b_scale"),
        (lambda: gt.mm_tn_e4m3(q, s, w[:, :128], ws[:, :1]), ValueError, "inner"),
        (lambda: gt.mm_tn_e4m3(q, s, w, ws, out_dtype=f8), TypeError, "output dtype"),
        (lambda: gt.mm_tn_e4m3(q, s, w, ws, accumulate=True), ValueError, "accumulate"),
        (lambda: gt.mm_tn_e4m3(q[:, 1:129], s[:, :1], w[:, :128], ws[:, :1]), gt.GemmTnError, "16-byte"),
        (lambda: gt.mm_tn_e4m3(z(6, 250, d=f8), s, z(10, 250, d=f8), ws), gt.GemmTnError, "16-byte"),
    ]
    for i, (call, kind, what) in enumerate(refused):
        with pytest.raises(kind, match=what):
            call()
            raise AssertionError(f"call {i} was taken")
    freed = z(4, 64)
    freed.untyped_storage().resize_(0)
    with pytest.raises(ValueError, match="storage"):
        gt.mm_tn_gated(freed, b)
