"""A plain 64-bit implementation of the paged cache's operators, and the inputs
and tolerances of their tests. Loops over sequences and heads; shares nothing
with the kernels."""
from __future__ import annotations

import math
from dataclasses import dataclass, field

import torch

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


@dataclass
class Setup:
    """A cache and new tokens on the CPU; every element that no result may
    depend on is NaN (or a wild number, for whole numbers)."""
    dtype: torch.dtype
    k: torch.Tensor            # [pages, page, kv_heads, dim]
    v: torch.Tensor
    table: torch.Tensor        # [batch, max_pages]
    lens: torch.Tensor
    q: torch.Tensor            # [batch, tokens, heads, dim]
    k_new: torch.Tensor
    v_new: torch.Tensor
    token_lens: torch.Tensor
    weight: torch.Tensor
    pos: torch.Tensor
    seen: torch.Tensor
    extra: dict = field(default_factory=dict)

    @property
    def batch(self):
        return self.table.shape[0]

    @property
    def page(self):
        return self.k.shape[1]

    @property
    def kv_heads(self):
        return self.k.shape[2]

    @property
    def group(self):
        return self.q.shape[2] // self.kv_heads

    def rows_of(self, pool, b, h, n):
        """[n, dim] of slots 0 .. n-1 of sequence b, head h, in 64 bits."""
        s = torch.arange(n)
        return pool[self.table[b].long()[s // self.page], s % self.page, h].double()


def make(dtype, dim, lens, tokens, kv_heads, group, page, token_lens=None, seed=0, max_pages=None, q_scale=1.5):
    dt = DTYPES[dtype]
    g = torch.Generator().manual_seed(seed)
    batch = len(lens)
    need = max(1, -(-max(lens) // page))
    max_pages = need if max_pages is None else max_pages
    pages = batch * max_pages + 2
    token_lens = [tokens] * batch if token_lens is None else list(token_lens)

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=g) * scale).to(dt)

    k, v = normal(pages, page, kv_heads, dim), normal(pages, page, kv_heads, dim)
    table = torch.randperm(pages, generator=g)[:batch * max_pages].view(batch, max_pages).to(torch.int32)
    used = torch.zeros((pages, page), dtype=torch.bool)
    for b, n in enumerate(lens):
        s = torch.arange(n)
        used[table[b].long()[s // page], s % page] = True
        table[b, -(-n // page):] = 2 ** 31 - 1 if b % 2 else -7      # entries that nothing uses
    k[~used] = float("nan")
    v[~used] = float("nan")
    heads = kv_heads * group
    q, kn, vn = normal(batch, tokens, heads, dim, scale=q_scale), normal(batch, tokens, kv_heads, dim), \
        normal(batch, tokens, kv_heads, dim)
    for b, n in enumerate(token_lens):
        q[b, n:] = float("nan")
        kn[b, n:] = float("nan")
        vn[b, n:] = float("nan")
    cap = max_pages * page
    weight = torch.rand((batch, kv_heads, cap), generator=g)
    pos = torch.stack([torch.stack([torch.randperm(cap, generator=g) for _ in range(kv_heads)]) for _ in range(batch)])
    return Setup(dt, k, v, table, torch.tensor(lens, dtype=torch.int32), q, kn, vn,
                 torch.tensor(token_lens, dtype=torch.int32), weight, pos.to(torch.int32),
                 torch.full((batch,), cap, dtype=torch.int32))


def visible(tokens, mask_words=None):
    """[batch or 1, tokens, tokens] truth values of the chain or of mask words."""
    j = torch.arange(tokens)
    if mask_words is None:
        return (j[None, :] <= j[:, None])[None]
    return ((mask_words[:, :, j // 64] >> (j % 64)) & 1) != 0


def attention(s: Setup, mask_words=None, use_new=True, scale=None):
    """o, lse, sum_k p_k |v_k|, sum over seen keys of |v|, and the largest
    scale * sum |q||k| of each row, all [batch, tokens, heads, ...] in 64 bits;
    rows that do not exist hold NaN."""
    batch, tokens, heads, dim = s.q.shape
    scale = 1.0 / math.sqrt(dim) if scale is None else scale
    nan = float("nan")
    o = torch.full((batch, tokens, heads, dim), nan, dtype=torch.float64)
    pv, av = o.clone(), o.clone()
    lse = torch.full((batch, tokens, heads), nan, dtype=torch.float64)
    amp = lse.clone()
    sees = visible(tokens, mask_words).expand(batch, tokens, tokens)
    for b in range(batch):
        n, ln = int(s.token_lens[b]), int(s.lens[b])
        if n == 0:
            continue
        see = torch.ones((n, ln), dtype=torch.bool)
        if use_new:
            see = torch.cat([see, sees[b, :n, :n]], 1)
        for x in range(heads):
            h = x // s.group
            k, v = s.rows_of(s.k, b, h, ln), s.rows_of(s.v, b, h, ln)
            if use_new:
                k, v = torch.cat([k, s.k_new[b, :n, h].double()]), torch.cat([v, s.v_new[b, :n, h].double()])
            q = s.q[b, :n, x].double()
            sc = (q @ k.T * scale).masked_fill(~see, -math.inf)
            z = torch.logsumexp(sc, 1) if sc.shape[1] else torch.full((n,), -math.inf, dtype=torch.float64)
            p = torch.where(see, torch.exp(sc - torch.where(z == -math.inf, 0.0, z)[:, None]), 0.0)
            o[b, :n, x], pv[b, :n, x], av[b, :n, x] = p @ v, p @ v.abs(), see.double() @ v.abs()
            lse[b, :n, x] = z
            a = (q.abs() @ k.abs().T * scale).masked_fill(~see, 0.0)
            amp[b, :n, x] = a.amax(1) if a.shape[1] else 0.0
    return o, lse, pv, av, amp


def score_error(amp):
    """Bound of a score's error in natural-log units: dim <= 128 products
    accumulated in fp32, each addition off by at most one unit in the last place
    (2^-23) of a partial sum that sum |q||k| bounds, and the rounding of the
    scaled score and of its reference (2^-23 of their size, which amp bounds)."""
    return 130 * 2.0 ** -23 * amp


def check_attention(out, lse, ref, s: Setup, untouched):
    """Every existing row within its bound, every other one as it was.

    A probability is off by its rounding to the input type (eps / 2), and by
    the error d of its score and of its row's sum (a factor e^2d each way,
    2 e^... below 1 + 4 d for d < 0.1) plus a few fp32 units (2^-20); the output
    is rounded once more. fp16 probabilities below 2^-14 of the row's
    reference (which is at most 2^8 under its maximum, so the sum is at least
    2^-0) are off by 2^-25 at most each, and fp16 outputs by 2^-25.
    """
    o, z, pv, av, amp = ref
    eps = torch.finfo(s.dtype).eps / 2
    live = ~torch.isnan(z)
    d = score_error(amp)
    tiny = 2.0 ** -25 if s.dtype == torch.float16 else 0.0
    tol = pv * (eps + 4 * d[..., None] + 2.0 ** -20) * (1 + 2 * eps) + eps * o.abs() + tiny * (av + 1)
    got = out.double()
    err = (got - o).abs()
    bad = ~(err <= tol) & live[..., None]
    assert not bad.any(), (f"{int(bad.sum())} outputs off, worst {float((err - tol)[bad].max()):.3g} past the bound "
                           f"(first at {bad.nonzero()[0].tolist()})")
    assert torch.equal(out[~live], torch.full_like(out[~live], untouched)), "rows that do not exist were written"
    if lse is not None:
        none = live & (z == -math.inf)
        assert (lse[none] == -math.inf).all() and (out[none] == 0).all()
        some = live & (z != -math.inf)
        # the row's sum: each term off by a factor e^d, fp32 sums and the logarithm by 2^-20
        lim = d + 2.0 ** -20 * (1 + z.abs())
        off = (lse.double() - z).abs()
        assert bool((off[some] <= lim[some]).all()), f"lse off by {float((off - lim)[some].max()):.3g} past the bound"
        assert torch.equal(lse[~live], torch.full_like(lse[~live], untouched))


def weigh(s: Setup, lse, rows, counts, causal=True, scale=None):
    """weight + sums in 64 bits (slots in use only; the others stay), and the bound of the error."""
    batch, tokens, heads, dim = s.q.shape
    scale = 1.0 / math.sqrt(dim) if scale is None else scale
    out = s.weight.double()
    tol = torch.zeros_like(out)
    for b in range(batch):
        ln, n = int(s.lens[b]), int(counts[b])
        if ln == 0:
            continue
        pick = (rows[b, :n] if rows is not None else torch.arange(n)).long()
        i = torch.arange(n)
        see = torch.arange(ln)[None, :] < (ln - n + i + 1)[:, None] if causal else torch.ones((n, ln), dtype=torch.bool)
        for x in range(heads):
            h = x // s.group
            k = s.rows_of(s.k, b, h, ln)
            q = s.q[b, pick, x].double()
            z = lse[b, pick, x].double()[:, None]
            p = torch.where(see, torch.exp(q @ k.T * scale - z), 0.0)
            amp = q.abs() @ k.abs().T * scale
            out[b, h, :ln] += p.sum(0)
            # the score's error, lse in units of 1/log2e and the exponential: 2^-21 of their sizes
            tol[b, h, :ln] += (p * (score_error(amp) + 2.0 ** -21 * (1 + amp + z.abs()))).sum(0)
        # fp32 sums of up to n * group terms and the weight
        tol[b, :, :ln] += out[b, :, :ln] * 2.0 ** -23 * (2 + n * s.group)
    return out, tol


def evict(s: Setup, keep, recent):
    """New k, v, weight, pos, lens: the definition, slot by slot."""
    k, v, weight, pos, lens = (t.clone() for t in (s.k, s.v, s.weight, s.pos, s.lens))
    for b in range(s.batch):
        ln = int(s.lens[b])
        if ln <= keep:
            continue
        lens[b] = keep
        for h in range(s.kv_heads):
            def rank(x):
                w = float(s.weight[b, h, x])
                new = recent > 0 and int(s.pos[b, h, x]) >= int(s.seen[b]) - recent
                return (0 if new else 1, 0 if math.isnan(w) else 1, 0.0 if new or math.isnan(w) else -w, x)
            kept = set(sorted(range(ln), key=rank)[:keep])
            holes = [x for x in range(keep) if x not in kept]
            movers = [x for x in range(keep, ln) if x in kept]
            assert len(holes) == len(movers)
            for a, c in zip(movers, holes):
                weight[b, h, c], pos[b, h, c] = s.weight[b, h, a], s.pos[b, h, a]
                pa, pc = int(s.table[b, a // s.page]), int(s.table[b, c // s.page])
                k[pc, c % s.page, h], v[pc, c % s.page, h] = s.k[pa, a % s.page, h], s.v[pa, a % s.page, h]
    return k, v, weight, pos, lens


def same(a, b):
    """Equal to the bit, NaN included."""
    if a.dtype.is_floating_point:
        kind = {2: torch.int16, 4: torch.int32}[a.element_size()]
        return torch.equal(a.view(kind), b.view(kind))
    return torch.equal(a, b)
