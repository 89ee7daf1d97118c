"""The cache operators' cases: attention of new (drafted) tokens over a paged
key/value cache, appending accepted tokens, accumulating the attention weight
of cached keys, and evicting the lightest ones.

Every case names its operator in ``op``. Sequence lengths, page tables and
trees follow from the case alone; the seed draws the values.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
LARGEST_PAIR_FLOPS = 4.0e11     # 4 * dim * heads * (token, key) pairs of the largest attention case
LARGEST_BYTES = 1.3e9           # K and V of the largest cache


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one user, one token, a short context: the call's latency
        dict(name="decode_one_user", op="attn", dtype="fp16", batch=1, tokens=1, heads=8, kv_heads=8, dim=64,
             min_len=517, max_len=517, page=16, branch=0),
        # a decode batch with ragged contexts: HBM bandwidth
        dict(name="decode_batch", op="attn", dtype="bf16", batch=64, tokens=1, heads=32, kv_heads=8, dim=128,
             min_len=900, max_len=8192, page=64, branch=0),
        # drafted trees of 26 tokens for a few users
        dict(name="tree_mid", op="attn", dtype="bf16", batch=8, tokens=26, heads=32, kv_heads=8, dim=128,
             min_len=1000, max_len=4096, page=32, branch=3),
        # wide trees over long contexts, 8 query heads a KV head
        dict(name="tree_long", op="attn", dtype="fp16", batch=4, tokens=63, heads=16, kv_heads=2, dim=128,
             min_len=20011, max_len=32768, page=128, branch=2),
        # a prompt's next 1024 tokens over the 8192 before them: tensor-core bound
        dict(name="chunked_prefill", op="attn", dtype="bf16", batch=2, tokens=1024, heads=32, kv_heads=8, dim=128,
             min_len=7777, max_len=8192, page=64, branch=0),
        # the accepted tokens of a batch's trees go into the cache
        dict(name="append_accepted", op="append", dtype="bf16", batch=64, tokens=26, heads=32, kv_heads=8, dim=128,
             min_len=100, max_len=1024, page=32, most=5),
        # two prompts of 8192 tokens go into the cache
        dict(name="append_prompts", op="append", dtype="fp16", batch=2, tokens=8192, heads=32, kv_heads=8, dim=128,
             min_len=0, max_len=64, page=64, most=8192),
        # one decoded token's weights for a small batch
        dict(name="weigh_decode", op="weigh", dtype="fp16", batch=4, tokens=1, heads=16, kv_heads=16, dim=64,
             min_len=300, max_len=1024, page=16, most=1),
        # the last 32 queries of long prompts choose what stays
        dict(name="weigh_window", op="weigh", dtype="bf16", batch=8, tokens=32, heads=32, kv_heads=8, dim=128,
             min_len=9001, max_len=16384, page=64, most=32),
        # a budget of 512 slots, overrun by a few tokens
        dict(name="evict_step", op="evict", dtype="bf16", batch=16, heads=32, kv_heads=8, dim=128,
             min_len=513, max_len=544, page=32, keep=512, recent=64),
        # long prompts cut to half
        dict(name="evict_prompts", op="evict", dtype="fp16", batch=8, heads=32, kv_heads=8, dim=128,
             min_len=12001, max_len=16384, page=64, keep=8192, recent=256),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "append", "weigh", "evict"])
    dtype = rng.choice(["fp16", "bf16"])
    dim = rng.choice([64, 128])
    kv_heads = rng.choice([1, 2, 4, 5, 8, 16])
    group = rng.choice([1, 2, 3, 4, 7, 8])
    page = rng.choice([8, 16, 32, 64, 128, 256])
    heads = kv_heads * group
    max_len = _log_int(rng, 40, 32768)
    min_len = rng.randint(max_len // 3, max_len)
    batch = _log_int(rng, 1, 64)
    row = 4 * kv_heads * dim       # bytes of one slot's K and V
    while batch > 1 and batch * max_len * row > LARGEST_BYTES / 2:
        batch = (batch + 1) // 2
    case = dict(op=op, dtype=dtype, batch=batch, heads=heads, kv_heads=kv_heads, dim=dim, min_len=min_len,
                max_len=max_len, page=page)
    if op == "attn":
        branch = rng.choice([0, 1, 2, 3, 4])
        tokens = _log_int(rng, 1, 160) if branch else rng.choice([1, _log_int(rng, 1, 1000)])
        while tokens > 1 and 4.0 * dim * heads * batch * tokens * (max_len + tokens) > LARGEST_PAIR_FLOPS / 4:
            tokens = (tokens + 1) // 2
        case.update(tokens=tokens, branch=branch)
    elif op == "append":
        tokens = _log_int(rng, 1, 4096)
        while tokens > 1 and batch * tokens * row > LARGEST_BYTES / 4:
            tokens = (tokens + 1) // 2
        case.update(tokens=tokens, most=rng.randint(1, tokens))
    elif op == "weigh":
        tokens = min(_log_int(rng, 1, 128), max_len // 3 + 1)
        while tokens > 1 and 2.0 * dim * heads * batch * tokens * max_len > LARGEST_PAIR_FLOPS / 8:
            tokens = (tokens + 1) // 2
        case.update(tokens=tokens, most=rng.randint(1, tokens))
    else:
        keep = rng.randint(max(1, min_len // 4), min_len)
        case.update(keep=keep, recent=rng.randint(0, keep // 2))
    return case


def _spread(case, lo, hi, salt):
    """One whole number in [lo, hi] for each sequence, spread evenly, from the case alone."""
    return [lo + int((hi - lo + 0.999) * ((b * 0.6180339887 + salt) % 1.0)) for b in range(case["batch"])]


def _lens(case):
    """Slots of each sequence in use before the call (the longest is max_len)."""
    lens = _spread(case, case["min_len"], case["max_len"], 0.37)
    lens[0] = case["max_len"]
    return lens


def _counts(case):
    """New tokens of each sequence: all for a chunk, ragged for trees, the accepted ones for append and weigh."""
    if case["op"] == "attn":
        return _spread(case, max(1, case["tokens"] * 2 // 3), case["tokens"], 0.11) if case["branch"] else \
            [case["tokens"]] * case["batch"]
    most = case["most"]
    return [most] * case["batch"] if most == case["tokens"] else _spread(case, 1, most, 0.11)


def _parents(case):
    """The drafted tree: token 0 is the root, token i hangs below token (i - 1) // branch."""
    return [-1] + [(i - 1) // case["branch"] for i in range(1, case["tokens"])]


def _pairs(case):
    """(query token, key) pairs that the case's mask shows."""
    lens, counts = _lens(case), _counts(case)
    if case["op"] == "weigh":
        return sum(n * (l - n) + n * (n + 1) // 2 for l, n in zip(lens, counts))
    depth = list(range(1, case["tokens"] + 1))
    if case["branch"]:
        depth, par = [], _parents(case)
        for p in par:
            depth.append(1 if p < 0 else depth[p] + 1)
    return sum(n * l + sum(depth[:n]) for l, n in zip(lens, counts))


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev).manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    b, hq, hkv, d, ps = case["batch"], case["heads"], case["kv_heads"], case["dim"], case["page"]

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=gen, device=dev) * scale).to(dt)

    lens, grow = _lens(case), 0
    if case["op"] == "append":
        grow = case["most"]
    per_seq = (max(lens) + grow + ps - 1) // ps
    pages = b * per_seq + 3       # a few pages are someone else's
    cap = per_seq * ps
    s = dict(case=case, scale=d ** -0.5,
             k=normal(pages, ps, hkv, d), v=normal(pages, ps, hkv, d),
             table=torch.randperm(pages, generator=gen, device=dev)[:b * per_seq].view(b, per_seq).to(torch.int32),
             lens=torch.tensor(lens, dtype=torch.int32, device=dev))
    if case["op"] != "attn":
        s["weight"] = torch.randn((b, hkv, cap), generator=gen, device=dev).exp_()
        s["pos"] = torch.arange(cap, device=dev, dtype=torch.int32).expand(b, hkv, cap).contiguous()
        s["seen"] = s["lens"].clone()
    if case["op"] == "evict":
        s["weight_out"] = torch.zeros_like(s["weight"])
        s["pos_out"] = torch.zeros_like(s["pos"])
        s["lens_out"] = torch.zeros_like(s["lens"])
    else:
        t = case["tokens"]
        s["counts"] = torch.tensor(_counts(case), dtype=torch.int32, device=dev)
        # the projections' output: q, k and v of a token side by side
        qkv = normal(b, t, hq + 2 * hkv, d)
        qkv[:, :, :hq] *= 1.5
        s["q"], s["k_new"], s["v_new"] = qkv[:, :, :hq], qkv[:, :, hq:hq + hkv], qkv[:, :, hq + hkv:]
    if case["op"] == "attn":
        s["mask"] = None
        if case["branch"]:
            words = (t + 63) // 64
            seen = [[0] * words for _ in range(t)]
            for i, p in enumerate(_parents(case)):
                if p >= 0:
                    seen[i] = list(seen[p])
                seen[i][i // 64] |= 1 << (i % 64)
            signed = [[w - (1 << 64) if w >> 63 else w for w in r] for r in seen]
            s["mask"] = torch.tensor(signed, dtype=torch.int64, device=dev).expand(b, t, words).contiguous()
        s["out"] = torch.zeros((b, t, hq, d), dtype=dt, device=dev)
        s["lse"] = torch.zeros((b, t, hq), dtype=torch.float32, device=dev)
    if case["op"] in ("append", "weigh"):
        # the accepted path: ascending tokens of the tree (all of them where every token counts)
        a = case["most"]
        pick = torch.rand((b, t), generator=gen, device=dev).argsort(dim=1)[:, :a].sort(dim=1).values
        s["rows"] = pick.to(torch.int32)
    if case["op"] == "append":
        s["lens_out"] = torch.zeros_like(s["lens"])
        s["seen_out"] = torch.zeros_like(s["seen"])
    if case["op"] == "weigh":
        # what the attention gave these queries: the log of their scores' sum of exponentials
        q = _rows_of(s["q"], s["rows"])
        s["lse"] = torch.zeros((b, t, hq), dtype=torch.float32, device=dev)
        sc, see = _weigh_scores(s, q)
        l = torch.logsumexp(sc.masked_fill(~see, -math.inf), dim=-1)           # [b, hkv, group, a]
        l = l.permute(0, 3, 1, 2).reshape(b, a, hq)
        s["lse"].scatter_(1, s["rows"].long()[:, :, None].expand(b, a, hq), l)
        s["weight_out"] = torch.zeros_like(s["weight"])
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    op = s["case"]["op"]
    if own:
        import dense_tiled_gemm_03_gb300 as gt
        cache = gt.KVCache(s["k"], s["v"], s["table"], s["lens"], weight=s.get("weight"), pos=s.get("pos"),
                           seen=s.get("seen"))
        if op == "attn":
            gt.tree_attn(s["q"], cache, s["k_new"], s["v_new"], mask=s["mask"], token_lens=s["counts"],
                         out=s["out"], lse=s["lse"])
        elif op == "append":
            gt.cache_append(cache, s["k_new"], s["v_new"], counts=s["counts"], rows=s["rows"],
                            lens_out=s["lens_out"], seen_out=s["seen_out"])
        elif op == "weigh":
            gt.cache_weigh(cache, s["q"], s["lse"], counts=s["counts"], rows=s["rows"], out=s["weight_out"])
        else:
            gt.cache_evict(cache, s["case"]["keep"], s["case"]["recent"], weight_out=s["weight_out"],
                           pos_out=s["pos_out"], lens_out=s["lens_out"])
    elif op == "attn":
        _plain_attn(s)
    elif op == "append":
        _plain_append(s)
    elif op == "weigh":
        _plain_weigh(s)
    else:
        _plain_evict(s)
    if op == "attn":
        return [s["out"], s["lse"]]
    if op == "append":
        return [s["k"], s["v"], s["weight"], s["pos"], s["lens_out"], s["seen_out"]]
    if op == "weigh":
        return [s["weight_out"]]
    return [s["k"], s["v"], s["weight_out"], s["pos_out"], s["lens_out"]]


def _slots(pool, table):
    """[batch, slots, kv heads, dim] of the pages in order, in 32 bits."""
    x = pool[table.long()]
    return x.reshape(x.shape[0], -1, *x.shape[3:]).float()


def _rows_of(x, rows):
    idx = rows.long()[:, :, None, None].expand(rows.shape[0], rows.shape[1], x.shape[2], x.shape[3])
    return torch.gather(x, 1, idx)


def _plain_attn(s):
    case = s["case"]
    b, t, hq, hkv, d = case["batch"], case["tokens"], case["heads"], case["kv_heads"], case["dim"]
    g, dev = hq // hkv, s["q"].device
    k = torch.cat([_slots(s["k"], s["table"]), s["k_new"].float()], 1).permute(0, 2, 1, 3)
    v = torch.cat([_slots(s["v"], s["table"]), s["v_new"].float()], 1).permute(0, 2, 1, 3)
    cap = k.shape[2] - t
    q = s["q"].float().reshape(b, t, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, g * t, d)
    j = torch.arange(t, device=dev)
    live = j[None, :] < s["counts"][:, None]
    if s["mask"] is None:
        tree = (j[None, :] <= j[:, None]).expand(b, t, t)
    else:
        tree = ((s["mask"][:, :, j // 64] >> (j % 64)) & 1) != 0
    old = torch.arange(cap, device=dev)[None, :] < s["lens"][:, None]
    see = torch.cat([old[:, None, :].expand(b, t, cap), tree & live[:, None, :]], 2)
    sc = torch.matmul(q, k.transpose(2, 3)).mul_(s["scale"]).view(b, hkv, g, t, cap + t)
    sc.masked_fill_(~see[:, None, None], -math.inf)
    m = sc.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = sc.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    v = v * torch.cat([old, live], 1)[:, None, :, None]
    o = torch.matmul(p.view(b, hkv, g * t, cap + t), v).view(b, hkv, g, t, d) / torch.where(l == 0, 1.0, l)
    o = o.permute(0, 3, 1, 2, 4).reshape(b, t, hq, d)
    lse = (m + l.log())[..., 0].permute(0, 3, 1, 2).reshape(b, t, hq)
    s["out"].copy_(torch.where(live[:, :, None, None], o, s["out"].float()))
    s["lse"].copy_(torch.where(live[:, :, None], lse, s["lse"]))


def _plain_append(s):
    ps, rows = s["case"]["page"], s["rows"]
    i = torch.arange(rows.shape[1], device=rows.device)
    bi, ii = torch.nonzero(i[None, :] < s["counts"][:, None], as_tuple=True)
    slot = s["lens"].long()[bi] + ii
    page = s["table"].long()[bi, slot // ps]
    src = rows.long()[bi, ii]
    s["k"][page, slot % ps] = s["k_new"][bi, src]
    s["v"][page, slot % ps] = s["v_new"][bi, src]
    s["weight"][bi, :, slot] = 0.0
    s["pos"][bi, :, slot] = (s["seen"][bi] + ii.to(torch.int32))[:, None].expand(-1, s["pos"].shape[1])
    s["lens_out"].copy_(s["lens"] + s["counts"])
    s["seen_out"].copy_(s["seen"] + s["counts"])


def _weigh_scores(s, q):
    """Scores [b, hkv, group, a, slots] of the chosen queries and which of them the mask shows."""
    case = s["case"]
    b, hkv, d = case["batch"], case["kv_heads"], case["dim"]
    g, a = case["heads"] // hkv, q.shape[1]
    k = _slots(s["k"], s["table"]).permute(0, 2, 1, 3)
    cap = k.shape[2]
    q = q.float().reshape(b, a, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, g * a, d)
    sc = torch.matmul(q, k.transpose(2, 3)).mul_(s["scale"]).view(b, hkv, g, a, cap)
    i = torch.arange(a, device=q.device)
    # query i of the newest `counts` slots sees the slots up to its own
    end = torch.where(i[None, :] < s["counts"][:, None], (s["lens"] - s["counts"])[:, None] + i[None, :] + 1, 0)
    see = torch.arange(cap, device=q.device)[None, None, :] < end[:, :, None]
    return sc, see[:, None, None]


def _plain_weigh(s):
    case = s["case"]
    b, hq, hkv = case["batch"], case["heads"], case["kv_heads"]
    a = s["rows"].shape[1]
    sc, see = _weigh_scores(s, _rows_of(s["q"], s["rows"]))
    lse = torch.gather(s["lse"], 1, s["rows"].long()[:, :, None].expand(b, a, hq))
    lse = lse.reshape(b, a, hkv, hq // hkv).permute(0, 2, 3, 1)[..., None]
    p = torch.where(see, sc.sub_(lse).exp_(), 0.0).sum((2, 3))
    live = torch.arange(p.shape[2], device=p.device)[None, None, :] < s["lens"][:, None, None]
    s["weight_out"].copy_(torch.where(live, s["weight"] + p, s["weight_out"]))


def _plain_evict(s):
    case = s["case"]
    ps, keep = case["page"], case["keep"]
    w, pos, lens = s["weight"], s["pos"], s["lens"]
    b, hkv, cap = w.shape
    slot = torch.arange(cap, device=w.device)
    live = slot < lens[:, None, None]
    key = torch.where(pos >= (s["seen"] - case["recent"])[:, None, None], math.inf, w)
    key = torch.where(live, key, -1.0)             # weights are sums of probabilities: never negative
    order = torch.sort(key, dim=2, descending=True, stable=True).indices
    kept = torch.zeros_like(live.expand(b, hkv, cap)).scatter(2, order[:, :, :keep], True) & live
    small = (lens <= keep)[:, None, None]
    mover = kept & (slot >= keep) & ~small
    hole = ~kept & (slot < keep) & ~small
    mb, mh, ms = torch.nonzero(mover, as_tuple=True)      # in ascending order for each head, as many as holes
    hb, hh, hs = torch.nonzero(hole, as_tuple=True)
    stay = live & (slot < keep)
    s["weight_out"].copy_(torch.where(stay, w, s["weight_out"]))
    s["pos_out"].copy_(torch.where(stay, pos, s["pos_out"]))
    s["weight_out"][hb, hh, hs] = w[mb, mh, ms]
    s["pos_out"][hb, hh, hs] = pos[mb, mh, ms]
    src, dst = s["table"].long()[mb, ms // ps], s["table"].long()[hb, hs // ps]
    for pool in (s["k"], s["v"]):
        pool[dst, hs % ps, hh] = pool[src, ms % ps, mh]
    s["lens_out"].copy_(torch.minimum(lens, torch.full_like(lens, keep)))


# ---------------------------------------------------------------- what a pass needs

def work(case):
    lens, e = _lens(case), 2
    hq, hkv, d = case["heads"], case["kv_heads"], case["dim"]
    row = 2 * hkv * d * e                       # one slot's K and V
    if case["op"] == "attn":
        n = sum(_counts(case))
        return {"bytes": sum(lens) * row + n * (row + 2 * hq * d * e + 4 * hq), "flops": 4 * d * hq * _pairs(case)}
    if case["op"] == "append":
        n = sum(_counts(case))
        return {"bytes": n * (2 * row + 8 * hkv + 4), "flops": 0}
    if case["op"] == "weigh":
        n = sum(_counts(case))
        return {"bytes": sum(lens) * (row // 2 + 8 * hkv) + n * hq * (d * e + 4), "flops": 2 * d * hq * _pairs(case)}
    over = [l for l in lens if l > case["keep"]]
    keep = case["keep"]
    # weights and positions read once, the kept ones written; of the kept slots the share behind `keep` moves,
    # the newest among them whatever their weight
    moved = sum(min(l - keep, case["recent"]) + max(0, l - keep - case["recent"]) * (keep - case["recent"])
                // max(1, l - case["recent"]) for l in over)
    return {"bytes": hkv * (8 * sum(lens) + 8 * sum(min(l, keep) for l in lens)) + moved * 2 * row, "flops": 0}


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op, dev = case["op"], s["k"].device
    b_all, hkv, d, ps = case["batch"], case["kv_heads"], case["dim"], case["page"]
    lens = _lens(case)

    def cached(pool, b, h, n):
        at = torch.arange(n, device=dev)
        return pool[s["table"][b].long()[at // ps], at % ps, h].double()

    if op == "attn":
        counts, g = _counts(case), case["heads"] // hkv
        out, lse = s["out"].double(), s["lse"].double()
        par = _parents(case) if case["branch"] else list(range(-1, case["tokens"] - 1))
        line = torch.zeros((case["tokens"], case["tokens"]), dtype=torch.bool)
        for i, p in enumerate(par):
            if p >= 0:
                line[i] = line[p]
            line[i, i] = True
        line = line.to(dev)
        for b in range(b_all):
            n, ln = counts[b], lens[b]
            for h in range(hkv):
                keys = torch.cat([cached(s["k"], b, h, ln), s["k_new"][b, :n, h].double()])
                vals = torch.cat([cached(s["v"], b, h, ln), s["v_new"][b, :n, h].double()])
                see = torch.cat([torch.ones((n, ln), dtype=torch.bool, device=dev), line[:n, :n]], 1)
                for x in range(h * g, (h + 1) * g):
                    sc = (s["q"][b, :n, x].double() @ keys.T) / math.sqrt(d)
                    sc = sc.masked_fill(~see, -math.inf)
                    z = torch.logsumexp(sc, 1)
                    lse[b, :n, x] = z
                    out[b, :n, x] = torch.exp(sc - z[:, None]) @ vals
        return [out, lse]
    if op == "weigh":
        counts, g = _counts(case), case["heads"] // hkv
        w = s["weight_out"].double()
        for b in range(b_all):
            n, ln = counts[b], lens[b]
            rows = s["rows"][b, :n].long()
            see = torch.arange(ln, device=dev)[None] <= (ln - n + torch.arange(n, device=dev))[:, None]
            for h in range(hkv):
                keys = cached(s["k"], b, h, ln)
                total = s["weight"][b, h, :ln].double()
                for x in range(h * g, (h + 1) * g):
                    sc = (s["q"][b, rows, x].double() @ keys.T) / math.sqrt(d)
                    p = torch.exp(sc - s["lse"][b, rows, x].double()[:, None])
                    total = total + torch.where(see, p, 0.0).sum(0)
                w[b, h, :ln] = total
        return [w]
    return None     # append and evict move values, and compute none
