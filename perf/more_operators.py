"""The feed-forward operators' cases: the gated projection (both projections,
the activation and their product in one pass), its backward pass, quantising to
8-bit floating point with a scale for each block of 128, and the product of two
matrices quantised so.

Every case names its operator in ``op``. The seed draws the values; the sizes
are the case's alone.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
BLOCK = 128                     # elements that share a scale
LARGEST = 448.0                 # of e4m3
MOST_FLOPS = 1.0e12             # of a drawn case
MOST_BYTES = 1.0e9


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one decoded token: both weight matrices stream past it
        dict(name="gated_token", op="gated", dtype="bf16", act="silu", m=1, n=16384, k=4096, train=False),
        # a few tokens of a small model, odd widths: the call's latency
        dict(name="gated_few", op="gated", dtype="fp16", act="gelu", m=24, n=2049, k=1000, train=False),
        # a prompt of odd length
        dict(name="gated_prompt", op="gated", dtype="fp16", act="silu", m=1111, n=5003, k=2048, train=False),
        # a training step's forward pass keeps what the backward pass needs
        dict(name="gated_train", op="gated", dtype="bf16", act="silu", m=8192, n=16384, k=4096, train=True),
        # backward passes: the gradients of the tokens and of both weight matrices
        dict(name="grad_small", op="grad", dtype="fp16", act="gelu", m=1000, n=2500, k=1024),
        dict(name="grad_train", op="grad", dtype="bf16", act="silu", m=8192, n=8192, k=4096),
        # the tokens of a decode step: the call's latency
        dict(name="quantize_step", op="quantize", dtype="bf16", m=16, k=4096, rows=1, transpose=False),
        # the tokens of prompts: memory bandwidth
        dict(name="quantize_prompts", op="quantize", dtype="bf16", m=16384, k=8192, rows=1, transpose=False),
        # a layer's fp32 weights, transposed for the gradient of its input
        dict(name="quantize_weights", op="quantize", dtype="fp32", m=11001, k=4096, rows=128, transpose=True),
        # a decode step of a small batch: the 8-bit weights stream past it
        dict(name="product_step", op="product", out="bf16", m=8, n=16384, k=8192, rows=128),
        # a weight's gradient: both sides scaled along the tokens, a sum of thousands of them in 32 bits
        dict(name="product_weight_grad", op="product", out="fp32", m=4096, n=5001, k=8191, rows=1),
        # prompts through a layer: tensor-core bound
        dict(name="product_prompts", op="product", out="bf16", m=8192, n=8192, k=8192, rows=128),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi):
    """A size in [lo, hi]: as it falls, or a multiple of 64."""
    x = _log_int(rng, lo, hi)
    return x if rng.random() < 0.5 else max(lo, x // 64 * 64)


def draw(rng):
    op = rng.choice(["gated", "gated", "grad", "quantize", "product", "product"])
    if op == "quantize":
        m, k = _size(rng, 1, 16384), _size(rng, 64, 16384)
        case = dict(op=op, dtype=rng.choice(["fp16", "bf16", "fp32"]), m=m, k=k, rows=rng.choice([1, 1, 128]),
                    transpose=rng.random() < 0.4)
        while work(case)["bytes"] > MOST_BYTES / 2:
            case["m"] = (case["m"] + 1) // 2
        return case
    case = dict(op=op, m=_size(rng, 1, 8192), n=_size(rng, 64, 16384), k=_size(rng, 64, 8192))
    if op == "product":
        case.update(out=rng.choice(["fp16", "bf16", "fp32"]), rows=rng.choice([1, 128, 128]))
    else:
        case.update(dtype=rng.choice(["fp16", "bf16"]), act=rng.choice(["silu", "silu", "gelu", "relu"]))
    if op == "gated":
        case.update(train=rng.random() < 0.5)
    while work(case)["flops"] > MOST_FLOPS or work(case)["bytes"] > MOST_BYTES:
        case["m"], case["n"] = (case["m"] + 1) // 2, max(64, case["n"] * 3 // 4)
    return case


# ---------------------------------------------------------------- inputs

def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def _quantized(x, rows):
    """x [m, k] (32 bits) as e4m3 with a power of two for each `rows` x 128 block: the values, and the scales
    [ceil(m / rows), ceil(k / 128)]."""
    m, k = x.shape
    mb, kb = (m + rows - 1) // rows, _blocks(k)
    mag = x.abs()
    mag = torch.where(torch.isfinite(mag), mag, 0.0)
    mag = torch.nn.functional.pad(mag, (0, kb * BLOCK - k, 0, mb * rows - m))
    top = mag.view(mb, rows, kb, BLOCK).amax((1, 3))
    # the least power of two that brings the block's largest value to 448 = 0.875 * 2^9 at most
    frac, expo = torch.frexp(top)
    expo = torch.where(top > 0, expo - 9 + (frac > 0.875).to(expo.dtype), torch.zeros_like(expo)).clamp(min=-126)
    scale = torch.ldexp(torch.ones_like(top), expo)
    each = scale.repeat_interleave(rows, 0)[:m].repeat_interleave(BLOCK, 1)[:, :k]
    y = x / each
    return torch.where(torch.isfinite(x), y, math.nan).to(torch.float8_e4m3fn), scale


def _with_pitch(q):
    """q in rows a multiple of 16 bytes apart."""
    m, k = q.shape
    wide = torch.zeros((m, (k + 15) // 16 * 16), dtype=torch.uint8, device=q.device).view(q.dtype)
    wide.view(torch.uint8)[:, :k] = q.view(torch.uint8)
    return wide[:, :k]


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, scale=1.0, dtype=torch.float32):
        return (torch.randn(shape, generator=gen, device=dev) * scale).to(dtype)

    op, m, k, s = case["op"], case["m"], case["k"], dict(case=case)
    if op == "quantize":
        # a few channels far larger than the others
        s["x"] = (normal(m, k) * (normal(k) * 1.5).exp()).to(DTYPES[case["dtype"]])
    elif op == "product":
        n = case["n"]
        a, b = normal(m, k), normal(n, k, scale=k ** -0.5)
        qa, sa = _quantized(a * (normal(k) * 0.5).exp(), 1)
        qb, sb = _quantized(b, case["rows"])
        s.update(a=_with_pitch(qa), b=_with_pitch(qb))
        # scales of single rows lie side by side for the rows, as the quantiser writes them
        s.update(a_scale=sa.t().contiguous().t(), b_scale=sb.t().contiguous().t() if case["rows"] == 1 else sb)
        s["out"] = torch.zeros((m, n), dtype=DTYPES[case["out"]], device=dev)
    else:
        n, dt = case["n"], DTYPES[case["dtype"]]
        s["x"] = normal(m, k, dtype=dt)
        s["w"] = normal(2 * n, k, scale=k ** -0.5, dtype=dt)     # the gate's rows, then the other projection's
        if op == "gated":
            s["out"] = torch.zeros((m, n), dtype=dt, device=dev)
            s["pre"] = torch.zeros((m, 2 * n), dtype=dt, device=dev) if case["train"] else None
        else:
            s["pre"] = normal(m, 2 * n, dtype=dt)
            s["grad"] = normal(m, n, scale=0.1, dtype=dt)
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    case, op = s["case"], s["case"]["op"]
    if own:
        import dense_tiled_gemm_03_gb300 as gt
        if op == "gated":
            gt.mm_tn_gated(s["x"], s["w"], out=s["out"], pre=s["pre"], activation=case["act"])
            return [s["out"]] if s["pre"] is None else [s["out"], s["pre"]]
        if op == "grad":
            d = gt.gated_grad(s["grad"], s["pre"], activation=case["act"])
            return [gt.mm_nn(d, s["w"]), gt.mm_nt(d, s["x"])]
        if op == "quantize":
            return list(gt.quantize_e4m3(s["x"], block_rows=case["rows"], transpose=case["transpose"]))
        return [gt.mm_tn_e4m3(s["a"], s["a_scale"], s["b"], s["b_scale"], out=s["out"])]
    if op == "gated":
        both = torch.matmul(s["x"].float(), s["w"].float().t())
        gate, up = both.chunk(2, dim=1)
        s["out"].copy_(_act(gate, case["act"]) * up)
        if s["pre"] is None:
            return [s["out"]]
        s["pre"].copy_(both)
        return [s["out"], s["pre"]]
    if op == "grad":
        gate, up = s["pre"].float().chunk(2, dim=1)
        dh = s["grad"].float()
        d = torch.cat([dh * up * _act_slope(gate, case["act"]), dh * _act(gate, case["act"])], 1)
        dt = s["x"].dtype
        return [torch.matmul(d, s["w"].float()).to(dt), torch.matmul(d.t(), s["x"].float()).to(dt)]
    if op == "quantize":
        x = s["x"].float()
        q, scale = _quantized(x.t().contiguous() if case["transpose"] else x, case["rows"])
        return [q, scale]
    s["out"].copy_(torch.matmul(_values(s["a"], s["a_scale"], 1), _values(s["b"], s["b_scale"], case["rows"]).t()))
    return [s["out"]]


def _values(q, scale, rows):
    m, k = q.shape
    return q.float() * scale.repeat_interleave(rows, 0)[:m].repeat_interleave(BLOCK, 1)[:, :k]


def _act(x, act):
    if act == "silu":
        return x / (1.0 + torch.exp(-x))
    if act == "gelu":
        return 0.5 * x * torch.erfc(x * -math.sqrt(0.5))
    return torch.where(x > 0, x, 0.0)


def _act_slope(x, act):
    if act == "silu":
        z = 1.0 / (1.0 + torch.exp(-x))
        return z * (1.0 + x * (1.0 - z))
    if act == "gelu":
        return 0.5 * torch.erfc(x * -math.sqrt(0.5)) + x * torch.exp(-0.5 * x * x) * (1.0 / math.sqrt(2.0 * math.pi))
    return (x > 0).to(x.dtype)


# ---------------------------------------------------------------- what a pass needs

def work(case):
    op, m, k = case["op"], case["m"], case["k"]
    e = {"fp16": 2, "bf16": 2, "fp32": 4}
    if op == "quantize":
        size = e[case["dtype"]]
        lines, along = (k, m) if case["transpose"] else (m, k)
        scales = (lines + case["rows"] - 1) // case["rows"] * _blocks(along)
        return {"bytes": m * k * (size + 1) + 4 * scales, "flops": 0}
    n = case["n"]
    if op == "product":
        scales = m * _blocks(k) + (n + case["rows"] - 1) // case["rows"] * _blocks(k)
        return {"bytes": m * k + n * k + 4 * scales + m * n * e[case["out"]], "flops": 2 * m * n * k}
    if op == "gated":
        return {"bytes": 2 * (m * k + 2 * n * k + m * n * (3 if case["train"] else 1)), "flops": 4 * m * n * k}
    # the gradients of the tokens and of the weights are a product of this size each
    return {"bytes": 2 * (m * n * 3 + 2 * (m * k + 2 * n * k)), "flops": 8 * m * n * k}


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        return _exact_quantized(s["x"].double(), case)
    if op == "product":
        a, b = s["a"].double(), s["b"].double()
        total = torch.zeros(s["out"].shape, dtype=torch.float64, device=a.device)
        for i in range(_blocks(case["k"])):
            part = slice(i * BLOCK, (i + 1) * BLOCK)
            sb = s["b_scale"][:, i].double()
            if case["rows"] > 1:
                sb = sb[torch.arange(case["n"], device=sb.device) // case["rows"]]
            total += torch.outer(s["a_scale"][:, i].double(), sb) * (a[:, part] @ b[:, part].T)
        return [total]
    n, act = case["n"], case["act"]
    x, wg, wu = s["x"].double(), s["w"][:n].double(), s["w"][n:].double()
    if op == "gated":
        g, u = x @ wg.T, x @ wu.T
        h = g * u * _share(g, act)
        return [h, torch.cat([g, u], 1)] if case["train"] else [h]
    g, u, dh = s["pre"][:, :n].double(), s["pre"][:, n:].double(), s["grad"].double()
    share = _share(g, act)
    if act == "silu":
        slope = share + g * share * (1 - share)
    elif act == "gelu":
        slope = share + g * torch.exp(-g.square() / 2) / math.sqrt(2 * math.pi)
    else:
        slope = share
    dg, du = dh * u * slope, dh * g * share
    return [dg @ wg + du @ wu, torch.cat([dg.T @ x, du.T @ x])]


def _share(g, act):
    """act(g) / g in 64 bits."""
    if act == "silu":
        return torch.sigmoid(g)
    if act == "gelu":
        return torch.special.ndtr(g)
    return (g > 0).double()


def _exact_quantized(x, case):
    if case["transpose"]:
        x = x.T
    m, k = x.shape
    rows = case["rows"]
    scale = torch.empty(((m + rows - 1) // rows, _blocks(k)), dtype=torch.float64, device=x.device)
    q = torch.empty((m, k), dtype=torch.float64, device=x.device)
    for j in range(scale.shape[1]):
        part = x[:, j * BLOCK:(j + 1) * BLOCK]
        top = part.abs().amax(1)
        if rows > 1:
            top = torch.stack([t.max() for t in top.split(rows)])
        # candidates around the logarithm, the least that fits
        guess = torch.floor(torch.log2(torch.where(top > 0, top, 448.0) / 448.0))
        fits = [top <= 448.0 * torch.exp2(guess + c) for c in (-1, 0, 1, 2)]
        first = torch.where(fits[0], -1, torch.where(fits[1], 0, torch.where(fits[2], 1, 2)))
        t = torch.where(top > 0, torch.exp2((guess + first).clamp(min=-126)), 1.0)
        scale[:, j] = t
        y = part / (t[:, None] if rows == 1 else t[torch.arange(m, device=x.device) // rows][:, None])
        # e4m3 has steps of 2^(e - 3) in [2^e, 2^(e + 1)), and of 2^-9 below 2^-6; torch.round takes ties to even
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
        q[:, j * BLOCK:(j + 1) * BLOCK] = torch.round(y / step) * step
    return [q, scale]
