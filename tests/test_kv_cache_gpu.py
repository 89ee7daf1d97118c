"""GPU tests of the paged cache's operators (include/kv_cache.h) against a plain
64-bit implementation: attention of new tokens over the cache, append,
accumulated weights, eviction, and a run of them as a serving loop uses them.

Whatever no result may depend on holds NaN: rows behind the last slot, unused
pages, tokens behind the end of a sequence's own.
"""
from __future__ import annotations

import gc
import math
import sys
import time

import pytest
import torch

import dense_tiled_gemm_03_gb300 as gt
import _cache_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    from _parity import require_gpu
    require_gpu()


DEV = "cuda:0"


def on_gpu(s: ref.Setup, **over):
    """The cache on the GPU (own copies of everything), and the status word."""
    t = dict(k=s.k, v=s.v, page_table=s.table, lens=s.lens, weight=s.weight, pos=s.pos, seen=s.seen)
    t.update(over)
    t = {n: None if x is None else x.to(DEV).clone() for n, x in t.items()}
    return gt.KVCache(**t), torch.zeros(1, dtype=torch.int32, device=DEV)


def run_attn(s: ref.Setup, mask=None, use_new=True, scale=None, fill=7.0, cache=None):
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    if cache is None:
        cache, status = on_gpu(s)
    out = torch.full(s.q.shape, fill, dtype=s.dtype, device=DEV)
    lse = torch.full(s.q.shape[:3], fill, device=DEV)
    kn, vn = (s.k_new.to(DEV), s.v_new.to(DEV)) if use_new else (None, None)
    gt.tree_attn(s.q.to(DEV), cache, kn, vn, mask=None if mask is None else mask.to(DEV),
                 token_lens=s.token_lens.to(DEV), scale=scale, out=out, lse=lse, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    return out.cpu(), lse.cpu()


def random_mask(batch, tokens, seed, empty_row=False):
    """Any mask: not a tree, some rows see nothing, bits behind the end set."""
    g = torch.Generator().manual_seed(seed)
    words = (tokens + 63) // 64
    m = torch.randint(-2 ** 63, 2 ** 63 - 1, (batch, tokens, words), generator=g, dtype=torch.int64)
    if empty_row:
        m[:, tokens // 2] = 0
    return m


def random_tree(batch, tokens, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.stack([torch.stack([torch.tensor(-1) if i == 0 else torch.randint(-1, i, (), generator=g)
                                     for i in range(tokens)]) for _ in range(batch)])


# lens, tokens, kv_heads, group, page, token_lens
SHAPES = [
    ([1], 1, 1, 1, 8, None),
    ([0, 5], 1, 2, 1, 8, None),
    ([127, 128, 129], 1, 2, 4, 16, None),
    ([300, 0, 1, 640], 2, 1, 8, 64, [2, 1, 0, 2]),
    ([255, 257], 7, 3, 3, 32, [7, 4]),
    ([1000], 16, 2, 7, 128, None),
    ([513, 90], 33, 1, 4, 256, [33, 17]),          # two row tiles: pair mode
    ([40, 200], 65, 2, 2, 16, [64, 65]),           # 130 rows
    ([70], 130, 1, 1, 8, None),
    ([0, 0], 200, 2, 3, 32, [200, 129]),           # the new tokens alone
    ([2500, 31], 3, 2, 128, 64, [3, 2]),           # one token per row tile
]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("kind", ["chain", "mask", "cache_only"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "len{}_t{}_h{}x{}_p{}".format("-".join(map(str, s[0])), *s[1:5]))
def test_attention(shape, kind, dim, dtype):
    lens, tokens, kv_heads, group, page, token_lens = shape
    s = ref.make(dtype, dim, lens, tokens, kv_heads, group, page, token_lens, seed=tokens + dim)
    mask = random_mask(len(lens), tokens, seed=tokens, empty_row=True) if kind == "mask" else None
    out, lse = run_attn(s, mask, use_new=kind != "cache_only")
    ref.check_attention(out, lse, ref.attention(s, mask, use_new=kind != "cache_only"), s, 7.0)


@pytest.mark.parametrize("tokens", [1, 26, 64, 97])
def test_attention_of_drafted_trees(tokens):
    s = ref.make("bf16", 128, [333, 1200, 64], tokens, 2, 4, 32, seed=tokens)
    mask = gt.tree_mask(random_tree(3, tokens, seed=tokens))
    out, lse = run_attn(s, mask)
    ref.check_attention(out, lse, ref.attention(s, mask), s, 7.0)


def test_many_short_sequences_and_one_long():
    """Ragged lengths: chunks that hold many items, and an item cut many times."""
    lens = [1 + 37 * i % 211 for i in range(70)] + [20000]
    s = ref.make("bf16", 64, lens, 2, 1, 2, 16, [1 + i % 2 for i in range(71)], seed=3, max_pages=1250)
    out, lse = run_attn(s)
    ref.check_attention(out, lse, ref.attention(s), s, 7.0)


@pytest.mark.parametrize("tokens,group", [(1, 2), (3, 16)])
def test_more_sequences_than_threads(tokens, group):
    """The search for a CTA's first tile goes round more than once; some sequences have no work."""
    lens = [(17 * i) % 150 if i % 5 else 0 for i in range(700)]
    s = ref.make("bf16", 64, lens, tokens, 1, group, 16, [i % (tokens + 1) for i in range(700)], seed=7)
    out, lse = run_attn(s)
    ref.check_attention(out, lse, ref.attention(s), s, 7.0)
    lse = torch.nan_to_num(lse, nan=5.0) + 1.0
    counts = [min(n, int(m)) for n, m in zip(lens, s.token_lens)]
    want, tol = ref.weigh(s, lse, None, counts)
    cache, status = on_gpu(s)
    gt.cache_weigh(cache, s.q.to(DEV), lse.to(DEV), counts=torch.tensor(counts, dtype=torch.int32, device=DEV), status=status)
    assert int(status.item()) == 0
    live = (torch.arange(want.shape[2])[None, None, :] < s.lens[:, None, None]).expand(want.shape)
    assert bool(((cache.weight.cpu().double() - want).abs()[live] <= tol[live]).all())


@pytest.mark.parametrize("tokens", [1, 30, 70, 200])
@pytest.mark.parametrize("batch,max_pages", [(19, 6), (19, 70), (5, 6), (5, 70), (45, 3)])
def test_ragged_items_over_the_ctas(batch, max_pages, tokens):
    """Items whole or cut (70 pages are more tiles than stay whole), with sequences and new tokens missing among them."""
    lens = [(97 * b * b + 41 * b) % (64 * min(max_pages, 6) + 1) if b % 4 else 0 for b in range(batch)]
    counts = [0 if b % 5 == 2 else 1 + (7 * b + tokens - 1) % tokens for b in range(batch)]
    s = ref.make("bf16", 64, lens, tokens, 8, 4, 64, token_lens=counts, seed=tokens + batch, max_pages=max_pages)
    mask = random_mask(batch, tokens, 8, empty_row=True) if batch % 2 and tokens < 100 else None
    out, lse = run_attn(s, mask)
    ref.check_attention(out, lse, ref.attention(s, mask), s, 7.0)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("tokens", [1, 4, 30])
@pytest.mark.parametrize("batch,kv_heads,longest", [(1, 1, 640), (3, 5, 700), (1, 2, 4000), (8, 4, 1500), (13, 5, 900)])
def test_items_shared_by_a_cluster(batch, kv_heads, longest, tokens, dim):
    """Clusters of 8, 4 and 2; lengths far below the capacity leave CTAs of a cluster without tiles, or all of them."""
    lens = [longest] + [(211 * b * b + 3) % longest if b % 3 else 0 for b in range(1, batch)]
    counts = [tokens] + [(5 * b) % (tokens + 1) for b in range(1, batch)]
    s = ref.make("fp16" if dim == 64 else "bf16", dim, lens, tokens, kv_heads, 4, 32, token_lens=counts, seed=batch + tokens)
    out, lse = run_attn(s)
    ref.check_attention(out, lse, ref.attention(s), s, 7.0)
    out, lse = run_attn(s, use_new=False)      # rows that see no key at all
    ref.check_attention(out, lse, ref.attention(s, use_new=False), s, 7.0)


@pytest.mark.parametrize("page", [8, 128, 384, 1024])
def test_page_sizes(page):
    """Pages longer than a tile, and lengths that end everywhere in them."""
    s = ref.make("fp16", 128, [page - 1, page + 1, 3 * page - 130 if page > 128 else 77, 900], 6, 1, 3, page, seed=page)
    for use_new in (True, False):
        out, lse = run_attn(s, use_new=use_new)
        ref.check_attention(out, lse, ref.attention(s, use_new=use_new), s, 7.0)
    check_evict(s, 64, 7, False)


def test_a_bad_query_spoils_its_own_row_alone():
    """NaN and infinite queries of one token beside finite ones, in each kernel's row layout."""
    for tokens, group in ((4, 2), (9, 8), (70, 4)):
        s = ref.make("bf16", 64, [300, 40], tokens, 1, group, 16, seed=tokens)
        want = ref.attention(s)
        s.q[0, 1, 0] = float("nan")
        s.q[0, 2, 1] = float("inf")
        out, lse = run_attn(s)
        assert torch.isnan(out[0, 1, 0].float()).all() and torch.isnan(lse[0, 1, 0])
        out[0, 1, 0], lse[0, 1, 0] = 7.0, 7.0
        out[0, 2, 1], lse[0, 2, 1] = 7.0, 7.0
        for t in want:
            t[0, 1, 0] = float("nan")
            t[0, 2, 1] = float("nan")
        ref.check_attention(out, lse, want, s, 7.0)


def test_long_chunk_over_a_cache():
    """The next tokens of a prompt: several row tiles and key tiles, the causal chain across them."""
    s = ref.make("fp16", 64, [500, 77], 700, 1, 2, 64, [700, 389], seed=5)
    out, lse = run_attn(s)
    ref.check_attention(out, lse, ref.attention(s), s, 7.0)


def test_scale_and_wide_scores():
    """A given scale; scores that rise along the keys, so that references move many times."""
    s = ref.make("fp16", 64, [900], 4, 2, 2, 64, seed=6, q_scale=4.0)
    page = s.table[0].long()
    ramp = torch.linspace(0.1, 3.0, 15 * 64).view(15, 64, 1, 1)
    s.k[page] = (s.k[page].float() * ramp).to(s.dtype)
    for scale in (None, 0.05, 0.4):
        out, lse = run_attn(s, scale=scale)
        ref.check_attention(out, lse, ref.attention(s, scale=scale), s, 7.0)


def test_scores_far_below_the_first_tiles():
    """Keys whose scores drop by hundreds behind the first tile, and the other way round."""
    s = ref.make("bf16", 64, [400], 3, 1, 4, 16, seed=8, q_scale=0.25)
    q = s.q.float()
    q[..., 0] = 40.0
    s.q = q.to(s.dtype)
    for first, rest in ((8.0, -8.0), (-8.0, 8.0)):
        k = s.k.float()
        page = s.table[0].long()
        k[page, :, :, 0] = rest
        k[page[:8], :, :, 0] = first
        s.k = k.to(s.dtype)
        out, lse = run_attn(s)
        ref.check_attention(out, lse, ref.attention(s), s, 7.0)


def replayed_us(calls, times=24, rounds=5, replays=5):
    """Shortest time of each call in a replayed graph of several, the calls' graphs in turn."""
    stream = torch.cuda.Stream()
    graphs, best = [], [float("inf")] * len(calls)
    with torch.cuda.stream(stream):
        for call in calls:
            call()
            stream.synchronize()
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1], stream=stream):
                for _ in range(times):
                    call()
        for _ in range(rounds):
            for i, graph in enumerate(graphs):
                for _ in range(replays):
                    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
                    start.record()
                    graph.replay()
                    end.record()
                    stream.synchronize()
                    best[i] = min(best[i], start.elapsed_time(end) * 1e3 / times)
    return best


def risen(tokens, lens, heads, group, dim, rise, dtype=torch.bfloat16):
    """Queries and keys whose scores lie `rise` powers of two above the first 128 keys' from there on."""
    s = ref.make("bf16", dim, lens, tokens, heads, group, 64, seed=13, q_scale=0.05)
    q, k = s.q.float(), s.k.float() * 0.05
    q[..., 0], k[..., 0] = 10.0, 1.0 + rise * math.log(2) * math.sqrt(dim) / 10.0
    for b in range(len(lens)):
        k[s.table[b, :2].long(), :, :, 0] = 1.0
    s.q, s.k = q.to(s.dtype), k.to(s.dtype)
    return s


@pytest.mark.parametrize("tokens,group", [(1, 4), (20, 4), (70, 4)])
@pytest.mark.parametrize("rise", [1.5, 3.0, 7.0, 9.0])
def test_scores_a_little_above_the_first_tiles(rise, tokens, group):
    s = risen(tokens, [900, 333], 2, group, 64, rise)
    out, lse = run_attn(s, use_new=False)
    ref.check_attention(out, lse, ref.attention(s, use_new=False), s, 7.0)


def test_scores_a_little_above_the_first_tiles_take_no_longer():
    """Their exponentials once a tile, as where no reference moves. (Twice, they are over half of a tile's time: 1.28 of it.)"""
    calls = []
    for rise in (0.0, 3.0):
        s = risen(256, [8192, 8192], 8, 4, 128, rise)
        cache, q = on_gpu(s)[0], s.q.to(DEV)
        calls.append(lambda q=q, cache=cache, out=torch.zeros_like(q): gt.tree_attn(q, cache, out=out))
    times = replayed_us(calls)
    assert times[1] <= 1.1 * times[0], times


@pytest.mark.parametrize("fill", [0.0, 100.0, -60000.0, float("inf"), float("nan")])
def test_what_lies_in_rows_that_do_not_exist(fill):
    """Queries, keys and values from token_lens on hold anything; the rows that exist come out the same to the bit."""
    for tokens, group, counts in ((4, 4, [1, 3]), (8, 4, [1, 0]), (32, 1, [5, 17]), (50, 4, [20, 33])):
        s = ref.make("fp16", 64, [700, 300], tokens, 2, group, 16, counts, seed=14)
        want = run_attn(s)
        ref.check_attention(*want, ref.attention(s), s, 7.0)
        for b, n in enumerate(counts):
            for t in (s.q, s.k_new, s.v_new):
                t[b, n:] = fill
        got = run_attn(s)
        assert ref.same(got[0], want[0]) and ref.same(got[1], want[1])


def test_rows_that_do_not_exist_take_no_time():
    """Padding tokens with large scores beside ones of zeros: the same work. (They called for new references, 1.14 times
    the time; shortest times of graphs in turn lie within 1% of one another.)"""
    g = torch.Generator(device=DEV).manual_seed(15)
    pool = torch.randn((2, 256, 64, 8, 64), generator=g, device=DEV).bfloat16()
    cache = gt.KVCache(pool[0], pool[1], torch.arange(256, dtype=torch.int32, device=DEV).view(4, 64),
                       torch.full((4,), 4096, dtype=torch.int32, device=DEV))
    q = torch.randn((2, 4, 4, 64, 64), generator=g, device=DEV).bfloat16()
    q[0, :, 1:], q[1, :, 1:] = 0.0, 100.0
    lens, out = torch.ones(4, dtype=torch.int32, device=DEV), torch.zeros_like(q[0])
    times = replayed_us([lambda x=x: gt.tree_attn(x, cache, token_lens=lens, out=out) for x in q])
    assert times[1] <= 1.05 * times[0], times


def test_pool_and_input_layouts():
    """[page][head][row] pools, K and V in one tensor, q, k, v side by side in one projection."""
    s = ref.make("bf16", 128, [200, 131], 5, 4, 2, 16, [5, 3], seed=9)
    want = ref.attention(s)
    pools = torch.empty((s.k.shape[0], 2, 4, 16, 128), dtype=s.dtype, device=DEV)
    pools[:, 0] = s.k.permute(0, 2, 1, 3).to(DEV)
    pools[:, 1] = s.v.permute(0, 2, 1, 3).to(DEV)
    cache = gt.KVCache(pools[:, 0].permute(0, 2, 1, 3), pools[:, 1].permute(0, 2, 1, 3), s.table.to(DEV), s.lens.to(DEV))
    qkv = torch.cat([s.q, s.k_new, s.v_new], 2).to(DEV)
    out = torch.full(s.q.shape, 7.0, dtype=s.dtype, device=DEV)
    gt.tree_attn(qkv[:, :, :8], cache, qkv[:, :, 8:12], qkv[:, :, 12:], token_lens=s.token_lens.to(DEV), out=out)
    ref.check_attention(out.cpu(), None, want, s, 7.0)


def test_page_offsets_past_32_bits():
    """A pool whose used pages lie more than 2^32 elements apart."""
    s = ref.make("bf16", 128, [1000], 4, 8, 2, 128, seed=10)
    far = 4300
    pages = 33000
    pool = torch.empty((2, pages, 128, 8, 128), dtype=s.dtype, device=DEV)   # 2 x 8.65 GB: 4.3e9 elements each
    where = torch.tensor([0, far, 2 * far, 7 * far, 32999, 5, 32998, 32771])[:s.table.shape[1]]
    for dst, src in ((pool[0], s.k), (pool[1], s.v)):
        dst[where.to(DEV)] = src[s.table[0].long()].to(DEV)
    cache = gt.KVCache(pool[0], pool[1], where[None].to(torch.int32).to(DEV), s.lens.to(DEV))
    out, lse = run_attn(s, cache=cache)
    ref.check_attention(out, lse, ref.attention(s), s, 7.0)
    gt.cache_append(cache, s.k_new.to(DEV)[:, :1], s.v_new.to(DEV)[:, :1])
    assert ref.same(pool[0, 32771, 1000 % 128].cpu(), s.k_new[0, 0])


def test_repeated_calls_are_bit_identical():
    s = ref.make("bf16", 128, [3000, 170, 901], 9, 2, 4, 32, seed=11)
    a, b = run_attn(s), run_attn(s)
    assert ref.same(a[0], b[0]) and ref.same(a[1], b[1])


def test_lengths_on_the_device_are_clamped():
    """Lengths and counts past what the arrays hold, and negative ones."""
    s = ref.make("bf16", 64, [64, 32], 4, 1, 2, 16, [4, 3], seed=12, max_pages=4)
    want = ref.attention(s)
    cache, _ = on_gpu(s, lens=torch.tensor([1000, 32], dtype=torch.int32))
    s.token_lens = torch.tensor([2 ** 31 - 1, 3], dtype=torch.int32)
    out, _ = run_attn(s, cache=cache)
    s.token_lens = torch.tensor([4, 3], dtype=torch.int32)
    ref.check_attention(out, None, want, s, 7.0)
    cache, _ = on_gpu(s, lens=torch.tensor([-5, -2 ** 31], dtype=torch.int32))
    s.token_lens = torch.tensor([4, -1], dtype=torch.int32)
    out, lse = run_attn(s, cache=cache)
    s.lens, s.token_lens = torch.tensor([0, 0]), torch.tensor([4, 0])
    ref.check_attention(out, lse, ref.attention(s), s, 7.0)


def test_page_numbers_out_of_range_are_reported_and_not_followed():
    s = ref.make("bf16", 64, [100, 100], 1, 1, 1, 16, seed=13)
    for bad in (-1, s.k.shape[0], 2 ** 31 - 1):
        s2 = ref.make("bf16", 64, [100, 100], 1, 1, 1, 16, seed=13)
        s2.table[0, 3] = bad
        cache, status = on_gpu(s2)
        out = torch.zeros(s2.q.shape, dtype=s2.dtype, device=DEV)
        lse = torch.zeros(s2.q.shape[:3], device=DEV)
        gt.tree_attn(s2.q.to(DEV), cache, out=out, lse=lse, status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == gt.GEMM_TN_ERR_INVALID_VALUE
        want = ref.attention(s, use_new=False)
        s_other = ref.Setup(**{**s.__dict__})
        ref.check_attention(out.cpu()[1:], lse.cpu()[1:], tuple(t[1:] for t in want), s_other, 0.0)
        for call in (lambda: gt.cache_weigh(cache, s2.q.to(DEV), lse, status=status),
                     lambda: gt.cache_evict(cache, 40, status=status)):
            status.zero_()
            call()
            torch.cuda.synchronize()
            assert int(status.item()) == gt.GEMM_TN_ERR_INVALID_VALUE


# ---------------------------------------------------------------- append

@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("dim,kv_heads,page", [(64, 1, 8), (128, 3, 16), (64, 8, 128)])
def test_append(dim, kv_heads, page, in_place):
    tokens, lens, counts = 9, [0, 7, 16, 100, 33], [9, 0, 1, 5, 4]
    s = ref.make("bf16", dim, lens, tokens, kv_heads, 2, page, seed=20, max_pages=-(-140 // page))
    g = torch.Generator().manual_seed(1)
    s.table = torch.randperm(s.k.shape[0], generator=g)[:s.table.numel()].view(s.table.shape).to(torch.int32)
    rows = torch.stack([torch.randperm(tokens, generator=g) for _ in lens]).to(torch.int32)
    rows[3, 1] = rows[3, 0]                      # the same token twice
    s.seen = torch.tensor([50, 7, 99, 1000, 0], dtype=torch.int32)
    k, v, weight, pos = s.k.clone(), s.v.clone(), s.weight.clone(), s.pos.clone()
    for b, n in enumerate(counts):
        for i in range(n):
            slot = lens[b] + i
            page_no = int(s.table[b, slot // page])
            k[page_no, slot % page] = s.k_new[b, int(rows[b, i])]
            v[page_no, slot % page] = s.v_new[b, int(rows[b, i])]
            weight[b, :, slot] = 0
            pos[b, :, slot] = s.seen[b] + i
    cache, status = on_gpu(s)
    new = torch.tensor(counts, dtype=torch.int32)
    lens_out, seen_out = (None, None) if in_place else (torch.zeros(5, dtype=torch.int32, device=DEV) for _ in range(2))
    gt.cache_append(cache, s.k_new.to(DEV), s.v_new.to(DEV), counts=new.to(DEV), rows=rows.to(DEV), lens_out=lens_out,
                    seen_out=seen_out, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    for got, want in ((cache.k, k), (cache.v, v), (cache.weight, weight), (cache.pos, pos),
                      (cache.lens if in_place else lens_out, s.lens + new),
                      (cache.seen if in_place else seen_out, s.seen + new)):
        assert ref.same(got.cpu(), want)
    if not in_place:
        assert torch.equal(cache.lens.cpu(), s.lens) and torch.equal(cache.seen.cpu(), s.seen)


def test_append_without_rows_and_statistics():
    s = ref.make("fp16", 64, [3, 0], 40, 2, 1, 8, seed=21, max_pages=6)
    s.table = torch.arange(12, dtype=torch.int32).view(2, 6)
    cache, status = on_gpu(s, weight=None, pos=None, seen=None)
    gt.cache_append(cache, s.k_new.to(DEV), s.v_new.to(DEV), status=status)
    assert cache.lens.tolist() == [43, 40] and int(status.item()) == 0
    s.lens = torch.tensor([43, 40])
    for b, at in ((0, 3), (1, 0)):
        for h in range(2):
            assert torch.equal(s.rows_of(cache.k.cpu(), b, h, at + 40)[at:], s.k_new[b, :, h].double())
            assert torch.equal(s.rows_of(cache.v.cpu(), b, h, at + 40)[at:], s.v_new[b, :, h].double())


def test_append_past_the_capacity_and_from_rows_out_of_range():
    s = ref.make("fp16", 64, [14, 2], 4, 1, 1, 8, seed=22, max_pages=2)
    s.table = torch.tensor([[2, 1], [0, 4]], dtype=torch.int32)
    cache, status = on_gpu(s)
    before = cache.k.clone()
    gt.cache_append(cache, s.k_new.to(DEV), s.v_new.to(DEV), status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == gt.GEMM_TN_ERR_INVALID_VALUE and cache.lens.tolist() == [16, 6]
    assert ref.same(cache.k[1, 6:8].cpu(), s.k_new[0, :2])          # the two that fit
    assert ref.same(cache.k[0, 2:6].cpu(), s.k_new[1])
    assert ref.same(cache.k[[3, 5]], before[[3, 5]])
    status.zero_()
    rows = torch.tensor([[0], [4]], dtype=torch.int32, device=DEV)
    out = torch.zeros(2, dtype=torch.int32, device=DEV)
    at = cache.k[0, 6].clone()
    gt.cache_append(cache, s.k_new.to(DEV), s.v_new.to(DEV), rows=rows, lens_out=out,
                    counts=torch.tensor([0, 1], dtype=torch.int32, device=DEV), status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == gt.GEMM_TN_ERR_INVALID_VALUE and ref.same(cache.k[0, 6], at)


@pytest.mark.parametrize("in_place", [False, True])
def test_append_more_rows_than_any_cache_has_slots(in_place):
    """max_rows at its limit, the one token over and over: len + max_rows is past 32 bits, and the slots end at the capacity."""
    if torch.cuda.mem_get_info()[0] < 12 * 2 ** 30:
        pytest.skip("the list of rows takes 8.6 GB")
    s = ref.make("bf16", 64, [13], 1, 1, 1, 8, seed=24, max_pages=4)
    s.table = torch.tensor([[4, 1, 5, 2]], dtype=torch.int32)
    k, v, weight, pos = s.k.clone(), s.v.clone(), s.weight.clone(), s.pos.clone()
    for slot in range(13, 32):
        k[s.table[0, slot // 8], slot % 8], v[s.table[0, slot // 8], slot % 8] = s.k_new[0, 0], s.v_new[0, 0]
        weight[0, 0, slot], pos[0, 0, slot] = 0.0, int(s.seen[0]) + slot - 13
    cache, status = on_gpu(s)
    out = cache.lens if in_place else torch.zeros(1, dtype=torch.int32, device=DEV)
    rows = torch.zeros((1, 2 ** 31 - 1), dtype=torch.int32, device=DEV)
    gt.cache_append(cache, s.k_new.to(DEV), s.v_new.to(DEV), rows=rows, lens_out=out,
                    seen_out=torch.zeros(1, dtype=torch.int32, device=DEV), status=status)
    torch.cuda.synchronize()
    del rows
    torch.cuda.empty_cache()
    assert out.tolist() == [32] and int(status.item()) == gt.GEMM_TN_ERR_INVALID_VALUE
    for got, want in ((cache.k, k), (cache.v, v), (cache.weight, weight), (cache.pos, pos)):
        assert ref.same(got.cpu(), want)


# ---------------------------------------------------------------- accumulated weights

# lens, tokens, kv_heads, group, page, counts
WEIGH = [
    ([1], 1, 1, 1, 8, None),
    ([5, 0, 128], 1, 2, 4, 16, None),
    ([300, 129], 9, 1, 8, 64, [9, 4]),
    ([700, 64], 32, 2, 8, 32, [32, 7]),          # 256 rows: one full block
    ([513, 900], 70, 1, 7, 128, [70, 33]),       # several blocks of rows
    ([260], 3, 1, 128, 256, None),               # two tokens per block
    ([90, 40], 5, 3, 3, 8, [0, 5]),              # no row counts: the weights come back
    ([3, 200], 9, 1, 40, 16, [9, 8]),            # more rows than slots; 360 columns in blocks of 240
]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("shape", WEIGH, ids=lambda s: "len{}_t{}_h{}x{}_p{}".format("-".join(map(str, s[0])), *s[1:5]))
def test_weigh(shape, causal, dim, dtype):
    lens, tokens, kv_heads, group, page, counts = shape
    counts = [min(tokens, n) for n in lens] if counts is None else counts
    s = ref.make(dtype, dim, lens, tokens, kv_heads, group, page, seed=tokens + dim)
    g = torch.Generator().manual_seed(2)
    rows = torch.stack([torch.randperm(tokens, generator=g) for _ in lens]).to(torch.int32)
    lse = torch.rand(s.q.shape[:3], generator=g) * 3 + math.log(max(max(lens), 2)) + 1.0
    for b, n in enumerate(counts):               # tokens that do not count
        for i in rows[b, n:].tolist():
            s.q[b, i] = float("nan")
            lse[b, i] = float("nan")
    want, tol = ref.weigh(s, lse, rows, counts, causal)
    cache, status = on_gpu(s)
    out = torch.full_like(cache.weight, 5.0)
    got = gt.cache_weigh(cache, s.q.to(DEV), lse.to(DEV), counts=torch.tensor(counts, dtype=torch.int32, device=DEV),
                         rows=rows.to(DEV), causal=causal, out=out, status=status)
    torch.cuda.synchronize()
    assert got is out and int(status.item()) == 0
    assert ref.same(cache.weight.cpu(), s.weight)
    live = torch.arange(out.shape[2])[None, None, :] < s.lens[:, None, None]
    live = live.expand(out.shape)
    off = (out.cpu().double() - want).abs()
    assert bool((off[live] <= tol[live]).all()), float((off - tol)[live].max())
    assert (out.cpu()[~live] == 5.0).all()
    gt.cache_weigh(cache, s.q.to(DEV), lse.to(DEV), counts=torch.tensor(counts, dtype=torch.int32, device=DEV),
                   rows=rows.to(DEV), causal=causal, status=status)
    assert ref.same(cache.weight.cpu()[live], out.cpu()[live]), "in place: the same sums"
    assert ref.same(cache.weight.cpu()[~live], s.weight[~live])


@pytest.mark.parametrize("tokens", [1, 20, 40, 130])
@pytest.mark.parametrize("batch,longest", [(3, 4500), (19, 700), (45, 130)])
def test_weights_of_ragged_items_over_the_ctas(batch, longest, tokens):
    """Few long and many short items, empty sequences and sequences without counted tokens among them."""
    lens = [(97 * b * b + longest) % (longest + 1) if b % 4 != 1 else 0 for b in range(batch)]
    counts = [0 if b % 5 == 2 else min(n, 1 + (7 * b + tokens - 1) % tokens) for b, n in enumerate(lens)]
    s = ref.make("fp16", 64, lens, tokens, 4, 4, 32, seed=tokens + batch)
    rows = torch.arange(tokens, dtype=torch.int32).repeat(batch, 1)
    lse = torch.full(s.q.shape[:3], math.log(longest) + 2.0)
    want, tol = ref.weigh(s, lse, rows, counts, True)
    cache, status = on_gpu(s)
    gt.cache_weigh(cache, s.q.to(DEV), lse.to(DEV), counts=torch.tensor(counts, dtype=torch.int32, device=DEV),
                   status=status)
    out = cache.weight.cpu()
    live = (torch.arange(out.shape[2])[None, None, :] < s.lens[:, None, None]).expand(out.shape)
    off = (out.double() - want).abs()
    assert bool((off[live] <= tol[live]).all()), float((off - tol)[live].max())
    assert ref.same(out[~live], s.weight[~live]) and int(status.item()) == 0


@pytest.mark.parametrize("none", [False, True])
@pytest.mark.parametrize("tokens,group", [(1, 4), (20, 4), (32, 4), (40, 4), (70, 7)])
@pytest.mark.parametrize("batch,longest", [(19, 700), (45, 130)])
def test_weights_of_chosen_rows_over_the_ctas(batch, longest, tokens, group, none):
    """Listed rows where a CTA has several items, so that each way of gathering queries looks them up (up to 128 rows ahead of
    the item, more between items); uncounted tokens hold NaN; rows that are no token are reported and weigh nothing."""
    lens = [(97 * b * b + longest) % (longest + 1) if b % 4 != 1 else 0 for b in range(batch)]
    counts = [0 if b % 5 == 2 else min(n, 1 + (7 * b + tokens - 1) % tokens) for b, n in enumerate(lens)]
    s = ref.make("fp16", 64, lens, tokens, 8, group, 32, seed=tokens + batch)
    g = torch.Generator().manual_seed(33)
    rows = torch.stack([torch.randperm(tokens, generator=g) for _ in lens]).to(torch.int32)
    lse = math.log(longest) + 2.0 + torch.rand(s.q.shape[:3], generator=g)
    for b, n in enumerate(counts):
        s.q[b, rows[b, n:].long()] = float("nan")
        lse[b, rows[b, n:].long()] = float("nan")
    clean_lse = lse.clone()
    if none:
        hit = [b for b, n in enumerate(counts) if n > 0 and b % 3 == 0]
        assert hit
        for b in hit:                    # for the reference: a token whose lse leaves it no weight
            clean_lse[b, int(rows[b, counts[b] // 2])] = 1e30
    want, tol = ref.weigh(s, clean_lse, rows, counts, True)
    if none:
        for x, b in enumerate(hit):
            rows[b, counts[b] // 2] = (-1, tokens, 2 ** 31 - 1, -2 ** 31)[x % 4]
    cache, status = on_gpu(s)
    gt.cache_weigh(cache, s.q.to(DEV), lse.to(DEV), counts=torch.tensor(counts, dtype=torch.int32, device=DEV),
                   rows=rows.to(DEV), status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == (gt.GEMM_TN_ERR_INVALID_VALUE if none else 0)
    out = cache.weight.cpu()
    live = (torch.arange(out.shape[2])[None, None, :] < s.lens[:, None, None]).expand(out.shape)
    off = (out.double() - want).abs()
    assert bool((off[live] <= tol[live]).all()), float((off - tol)[live].max())
    assert ref.same(out[~live], s.weight[~live])


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("batch,tokens,kv_heads,group", [(1, 3, 1, 2), (3, 9, 2, 8), (2, 70, 1, 7), (3, 32, 1, 8), (40, 1, 8, 4), (40, 5, 8, 3)])
def test_keys_that_weigh_nothing_keep_their_weight_whatever_they_hold(batch, tokens, kv_heads, group, causal):
    """Infinities and NaN in keys that no query counts for, and infinite keys whose scores are all -inf: no row that the
    kernel pads with, and no row that is none, may bring them in."""
    lens = [200 + 37 * b % 190 for b in range(batch)]
    counts = [0 if b % 3 == 2 else 1 + (5 * b + tokens - 1) % tokens for b in range(batch)]
    s = ref.make("bf16", 64, lens, tokens, kv_heads, group, 16, seed=31 + tokens)
    s.q[..., 5] = -s.q[..., 5].abs() - 0.5
    g = torch.Generator().manual_seed(32)
    rows = torch.stack([torch.randperm(tokens, generator=g) for _ in lens]).to(torch.int32)
    lse = torch.full(s.q.shape[:3], 7.0)
    want, tol = ref.weigh(s, lse, rows, counts, causal)
    bad = torch.zeros(want.shape, dtype=torch.bool)
    for b, n in enumerate(lens):
        at = torch.arange(b % 7, n, 7)
        bad[b, :, at] = True
        s.k[s.table[b].long()[at // 16], at % 16, :, 5] = float("nan") if counts[b] == 0 and b % 2 else float("inf")
    live = (torch.arange(want.shape[2])[None, None, :] < s.lens[:, None, None]).expand(want.shape)
    for none in (None, -1, tokens):              # a counted row of sequence 0 that is no token weighs nothing
        if none is not None:
            if counts[0] > 1:
                continue
            rows[0, 0] = none
            want[0] = s.weight[0].double()
        cache, status = on_gpu(s)
        gt.cache_weigh(cache, s.q.to(DEV), lse.to(DEV), counts=torch.tensor(counts, dtype=torch.int32, device=DEV),
                       rows=rows.to(DEV), causal=causal, status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == (0 if none is None else gt.GEMM_TN_ERR_INVALID_VALUE)
        out = cache.weight.cpu()
        assert ref.same(out[bad | ~live], s.weight[bad | ~live])
        off = (out.double() - want).abs()
        assert bool((off[live & ~bad] <= tol[live & ~bad]).all()), float((off - tol)[live & ~bad].max())


def test_weights_of_one_pass_sum_to_the_rows():
    """With the attention's own lse every counted row's weights over the slots sum to one."""
    s = ref.make("bf16", 128, [2000, 333], 6, 2, 4, 64, seed=30)
    cache, status = on_gpu(s, weight=torch.zeros_like(s.weight))
    q = s.q.to(DEV)
    lse = torch.zeros(s.q.shape[:3], device=DEV)
    gt.tree_attn(q, cache, lse=lse, status=status)
    gt.cache_weigh(cache, q, lse, causal=False, status=status)
    total = cache.weight.double().cpu()
    for b in range(2):
        got = total[b, :, :int(s.lens[b])].sum(1)
        # 24 rows; each sum of probabilities is off by the scores' errors (amp < 40: 130 * 2^-23 * 40 < 1e-3)
        assert (got - 24.0).abs().max().item() < 24 * 1e-3
    assert int(status.item()) == 0


# ---------------------------------------------------------------- evict

@pytest.mark.parametrize("recent", [0, 5])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("lens,keep,page,dim,kv_heads", [
    ([1, 9], 8, 8, 64, 1), ([40, 41, 200, 0], 40, 16, 128, 3), ([300, 130], 129, 64, 64, 2),
    ([2049, 1500], 1024, 128, 64, 1), ([33], 5, 8, 128, 2), ([1200], 1199, 32, 64, 1)])
def test_evict(lens, keep, page, dim, kv_heads, in_place, recent):
    s = ref.make("bf16", dim, lens, 1, kv_heads, 1, page, seed=keep)
    check_evict(s, keep, recent, in_place)


def check_evict(s, keep, recent, in_place):
    k, v, weight, pos, lens = ref.evict(s, keep, recent)
    cache, status = on_gpu(s)
    outs = [None] * 3 if in_place else [torch.full_like(t, 3) for t in (cache.weight, cache.pos, cache.lens)]
    gt.cache_evict(cache, keep, recent, *outs, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    assert ref.same(cache.k.cpu(), k) and ref.same(cache.v.cpu(), v)
    got = [cache.weight, cache.pos, cache.lens] if in_place else outs
    assert torch.equal(got[2].cpu(), lens)
    written = (torch.arange(weight.shape[2])[None, None, :] < lens[:, None, None]).expand(weight.shape)
    for x, want, old in ((got[0].cpu(), weight, s.weight), (got[1].cpu(), pos, s.pos)):
        assert ref.same(x[written], want[written])
        assert ref.same(x[~written], old[~written] if in_place else torch.full_like(old, 3)[~written])
    if not in_place:
        assert ref.same(cache.weight.cpu(), s.weight) and ref.same(cache.pos.cpu(), s.pos)


def test_evict_in_place_but_for_the_lengths():
    """Weights and positions in place with lengths elsewhere (the form that moves its rows in one kernel), and the other way."""
    s = ref.make("bf16", 64, [300, 90, 130], 1, 2, 1, 16, seed=44)
    k, v, weight, pos, lens = ref.evict(s, 100, 9)
    for lens_apart in (True, False):
        cache, status = on_gpu(s)
        outs = dict(lens_out=torch.zeros_like(cache.lens)) if lens_apart else \
            dict(weight_out=torch.zeros_like(cache.weight), pos_out=torch.zeros_like(cache.pos))
        gt.cache_evict(cache, 100, 9, **outs, status=status)
        got = dict(weight_out=cache.weight, pos_out=cache.pos, lens_out=cache.lens) | outs
        assert int(status.item()) == 0 and ref.same(cache.k.cpu(), k) and ref.same(cache.v.cpu(), v)
        assert torch.equal(got["lens_out"].cpu(), lens)
        live = (torch.arange(weight.shape[2])[None, None, :] < lens[:, None, None]).expand(weight.shape)
        assert ref.same(got["weight_out"].cpu()[live], weight[live]) and ref.same(got["pos_out"].cpu()[live], pos[live])


def test_evict_more_slots_than_the_newest_leave_room_for():
    """Positions as an eviction leaves them twice over: more slots count as newest than are kept; the lowest stay."""
    s = ref.make("bf16", 64, [200], 1, 1, 1, 8, seed=45)
    s.pos = (s.pos % 40).contiguous()
    s.seen[:] = 40
    check_evict(s, 60, 30, False)
    check_evict(s, 100, 30, True)


@pytest.mark.parametrize("keep", [0, 1, 63, 64])
def test_evict_ties_and_odd_weights(keep):
    """Equal weights keep the lowest slots; zeros of both signs are equal; infinities, NaN, negative and denormal values."""
    s = ref.make("fp16", 64, [100, 97], 1, 1, 1, 16, seed=40)
    odd = torch.tensor([0.0, -0.0, float("inf"), -float("inf"), float("nan"), 1.0, 1.0, -2.5, 1e-42, -1e-42, 3e38])
    g = torch.Generator().manual_seed(3)
    s.weight = odd[torch.randint(0, len(odd), s.weight.shape, generator=g)]
    check_evict(s, keep, 0, False)
    check_evict(s, keep, min(keep, 10), True)


def test_evict_a_sequence_longer_than_shared_memory_holds():
    s = ref.make("fp16", 64, [50000], 1, 1, 1, 128, seed=41)
    check_evict(s, 20001, 100, False)


@pytest.mark.parametrize("lens,kv_heads,keep,recent,odd", [
    ([17000, 30, 9000], 2, 5000, 64, True), ([17000, 16300], 1, 8191, 0, True), ([16500, 40, 5001], 1, 5000, 100, False),
    ([17000] + [90, 0, 200] * 8, 3, 77, 5, True), ([70001], 1, 40000, 33, False), ([170000], 1, 90001, 64, True)])
def test_evict_lists_shared_by_a_cluster(lens, kv_heads, keep, recent, odd):
    """Ties and the newest slots spread over several blocks, blocks without slots, and more slots a block than its shared memory holds."""
    s = ref.make("bf16", 64, lens, 1, kv_heads, 1, 128, seed=keep)
    if odd:
        few = torch.tensor([0.0, -0.0, 0.5, 0.25, 2.0, float("nan"), -1.0, float("inf")])
        s.weight = few[torch.randint(0, len(few), s.weight.shape, generator=torch.Generator().manual_seed(4))]
    check_evict(s, keep, recent, keep % 2 == 0)


def test_evict_without_positions():
    s = ref.make("fp16", 64, [60], 1, 2, 1, 16, seed=42)
    k, v, weight, _, lens = ref.evict(s, 30, 0)
    cache, status = on_gpu(s, pos=None, seen=None)
    gt.cache_evict(cache, 30, status=status)
    assert ref.same(cache.k.cpu(), k) and ref.same(cache.v.cpu(), v) and cache.lens.tolist() == [30]
    assert ref.same(cache.weight.cpu()[:, :, :30], weight[:, :, :30]) and int(status.item()) == 0


# ---------------------------------------------------------------- together

def serve(s: ref.Setup, steps, seed, capture=False):
    """A serving loop: drafted trees attended, the accepted path appended, its
    weights added, the cache cut to its budget; everything on the device."""
    cache, status = on_gpu(s, weight=torch.zeros_like(s.weight))
    g = torch.Generator().manual_seed(seed)
    batch, tokens, heads, dim = s.q.shape
    q, kn, vn = torch.empty_like(s.q, device=DEV), torch.empty_like(s.k_new, device=DEV), torch.empty_like(s.v_new, device=DEV)
    mask = torch.zeros((batch, tokens, 1), dtype=torch.int64, device=DEV)
    rows = torch.zeros((batch, tokens), dtype=torch.int32, device=DEV)
    counts = torch.zeros(batch, dtype=torch.int32, device=DEV)
    out, lse = torch.zeros_like(q), torch.zeros((batch, tokens, heads), device=DEV)

    def step():
        gt.tree_attn(q, cache, kn, vn, mask=mask, out=out, lse=lse, status=status)
        gt.cache_append(cache, kn, vn, counts=counts, rows=rows, status=status)
        gt.cache_weigh(cache, q, lse, counts=counts, rows=rows, status=status)
        gt.cache_evict(cache, 150, 20, status=status)

    graph = None
    seen = []
    for n in range(steps):
        parents = random_tree(batch, tokens, seed=seed + n)
        path = torch.zeros((batch, tokens), dtype=torch.int32)
        length = torch.zeros(batch, dtype=torch.int32)
        for b in range(batch):
            at, line = int(torch.randint(0, tokens, (), generator=g)), []
            while at >= 0:
                line.append(at)
                at = int(parents[b, at])
            path[b, :len(line)] = torch.tensor(line[::-1], dtype=torch.int32)
            length[b] = len(line)
        inputs = [(q, torch.randn(q.shape, generator=g).to(s.dtype)), (kn, torch.randn(kn.shape, generator=g).to(s.dtype)),
                  (vn, torch.randn(vn.shape, generator=g).to(s.dtype)), (mask, gt.tree_mask(parents)), (rows, path),
                  (counts, length)]
        for dst, src in inputs:
            dst.copy_(src)
        if capture and n == 1:
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
        if graph is not None:
            graph.replay()
        else:
            step()
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        seen.append([t.cpu().clone() for t in (out, lse, cache.k, cache.v, cache.weight, cache.pos, cache.lens, cache.seen)] +
                    [x[1] for x in inputs])
    return seen


def serving_setup():
    s = ref.make("bf16", 64, [140, 3, 90], 12, 2, 2, 16, seed=50, max_pages=14)
    # every sequence gets all the pages it can grow into; what the slots in use held moves along
    rows = [[s.rows_of(pool, b, h, int(s.lens[b])).to(s.dtype) for pool in (s.k, s.v)] for b in range(3) for h in range(2)]
    s.table = torch.randperm(s.k.shape[0], generator=torch.Generator().manual_seed(51))[:42].view(3, 14).to(torch.int32)
    s.k.fill_(float("nan"))
    s.v.fill_(float("nan"))
    for b in range(3):
        for h in range(2):
            at = torch.arange(int(s.lens[b]))
            for pool, x in zip((s.k, s.v), rows[2 * b + h]):
                pool[s.table[b].long()[at // 16], at % 16, h] = x
    s.pos = torch.arange(s.pos.shape[2], dtype=torch.int32).expand(s.pos.shape).contiguous()
    s.seen = s.lens.clone()
    return s


def test_a_serving_loop():
    """Each step of the loop against the 64-bit operators run on the state that the step before left."""
    s = serving_setup()
    state = ref.Setup(**{**s.__dict__})
    state.weight = torch.zeros_like(s.weight)
    for out, lse, k, v, weight, pos, lens, seen, q, kn, vn, mask, rows, counts in serve(s, 6, seed=52):
        state.q, state.k_new, state.v_new = q, kn, vn
        state.token_lens = torch.full((3,), 12, dtype=torch.int32)
        ref.check_attention(out, lse, ref.attention(state, mask), state, 0.0)
        for b in range(3):
            for i in range(int(counts[b])):
                slot = int(state.lens[b]) + i
                page = int(state.table[b, slot // 16])
                state.k[page, slot % 16], state.v[page, slot % 16] = kn[b, rows[b, i]], vn[b, rows[b, i]]
                state.weight[b, :, slot], state.pos[b, :, slot] = 0.0, state.seen[b] + i
        state.lens, state.seen = state.lens + counts, state.seen + counts
        want, tol = ref.weigh(state, lse, rows, counts)
        # the sums differ by rounding, so which slots go is taken from the kernel's own weights
        long = state.lens > 150
        assert torch.equal(lens, torch.where(long, 150, state.lens).to(torch.int32)) and torch.equal(seen, state.seen)
        for b in range(3):
            for h in range(2):
                n = int(lens[b])
                where = {int(p): i for i, p in enumerate(state.pos[b, h, :int(state.lens[b])])}
                at = torch.tensor([where[int(p)] for p in pos[b, h, :n]])
                assert len(set(at.tolist())) == n
                assert bool(((weight[b, h, :n].double() - want[b, h, at]).abs() <= tol[b, h, at]).all())
                if bool(long[b]):
                    gone = sorted(set(range(int(state.lens[b]))) - set(at.tolist()))
                    newest = state.pos[b, h, gone] >= state.seen[b] - 20
                    assert not newest.any()
                    old = [i for i in at.tolist() if int(state.pos[b, h, i]) < int(state.seen[b]) - 20]
                    assert float((want - tol)[b, h, gone].max()) <= float((want + tol)[b, h, old].min())
                for pool, got in ((state.k, k), (state.v, v)):
                    assert torch.equal(state.rows_of(got, b, h, n), state.rows_of(pool, b, h, int(state.lens[b]))[at])
        state.k, state.v, state.weight, state.pos, state.lens, state.seen = k, v, weight, pos, lens, seen


def test_a_serving_loop_in_a_graph():
    """The same loop with the steps from the second on replayed from one capture, to the bit."""
    a, b = serve(serving_setup(), 5, seed=53), serve(serving_setup(), 5, seed=53, capture=True)
    for x, y in zip(a, b):
        for p, q in zip(x, y):
            assert ref.same(p, q)


def test_two_streams_at_once_and_two_graphs_in_turn():
    """Workspaces are each call's own: calls in flight on two streams, and two captures replayed over one another."""
    s1 = ref.make("bf16", 128, [4000, 1500], 4, 2, 4, 64, seed=60)
    s2 = ref.make("fp16", 64, [2500, 3, 700], 20, 1, 8, 16, seed=61)
    want = [run_attn(s) for s in (s1, s2)]
    args = []
    for s in (s1, s2):
        cache, status = on_gpu(s)
        out, lse = torch.full(s.q.shape, 7.0, dtype=s.dtype, device=DEV), torch.full(s.q.shape[:3], 7.0, device=DEV)
        args.append((s.q.to(DEV), cache, s.k_new.to(DEV), s.v_new.to(DEV), out, lse, status))

    def call(a):
        q, cache, kn, vn, out, lse, status = a
        gt.tree_attn(q, cache, kn, vn, out=out, lse=lse, status=status)

    def check():
        torch.cuda.synchronize()
        for a, w in zip(args, want):
            assert ref.same(a[4].cpu(), w[0]) and ref.same(a[5].cpu(), w[1]) and int(a[6].item()) == 0
            a[4].fill_(float("nan"))
            a[5].fill_(float("nan"))
        torch.cuda.synchronize()

    streams = [torch.cuda.Stream() for _ in args]
    torch.cuda.synchronize()
    for _ in range(10):
        for a, st in zip(args, streams):
            with torch.cuda.stream(st):
                call(a)
    check()
    graphs = []
    for a in args:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(a)
        graphs.append(graph)
    for _ in range(3):
        for graph in graphs:
            graph.replay()
    check()
    for graph, st in zip(graphs, streams):
        with torch.cuda.stream(st):
            graph.replay()
    check()


def test_watchdog_reports_a_timeout_and_the_context_survives():
    """The first CTA's producer skips one copy (test hook), so a bounded wait expires."""
    from _parity import env_var
    s = ref.make("bf16", 128, [3000], 2, 2, 4, 64, seed=62)
    cache, status = on_gpu(s)
    q, lse = s.q.to(DEV), torch.zeros(s.q.shape[:3], device=DEV)
    for call in (lambda: gt.tree_attn(q, cache, s.k_new.to(DEV), s.v_new.to(DEV), status=status),
                 lambda: gt.cache_weigh(cache, q, lse, out=torch.zeros_like(cache.weight), status=status)):
        status.zero_()
        t0 = time.perf_counter()
        with env_var("GEMM_TN_WATCHDOG_MS", "200"), env_var("GEMM_TN_TEST_DROP_LOAD", "0"):
            call()
            torch.cuda.synchronize()
        assert int(status.item()) == gt.GEMM_TN_ERR_TIMEOUT and time.perf_counter() - t0 < 5.0
    out, lse = run_attn(s)
    ref.check_attention(out, lse, ref.attention(s), s, 7.0)


def test_the_binding_refuses_tensors_that_do_not_fit():
    s = ref.make("bf16", 64, [30, 40], 3, 2, 2, 16, seed=66)
    cache, _ = on_gpu(s)
    q, kn, vn = s.q.to(DEV), s.k_new.to(DEV), s.v_new.to(DEV)
    lse = torch.zeros(s.q.shape[:3], device=DEV)
    whole = dict(k=cache.k, v=cache.v, page_table=cache.page_table, lens=cache.lens, weight=cache.weight, pos=cache.pos,
                 seen=cache.seen)
    i32 = torch.int32

    def other(**over):
        return lambda: gt.KVCache(**{**whole, **over})

    refused = [
        (other(v=cache.v.cpu()), ValueError), (other(lens=cache.lens.cpu()), ValueError), (other(v=cache.v.half()), TypeError),
        (other(k=cache.k.float(), v=cache.v.float()), TypeError), (other(k=cache.k[0], v=cache.v[0]), ValueError),
        (other(v=cache.v[:-1]), ValueError), (other(v=cache.v.transpose(1, 2).contiguous().transpose(1, 2)), ValueError),
        (other(k=cache.k.transpose(0, 3), v=cache.v.transpose(0, 3)), ValueError), (other(lens=cache.lens.long()), TypeError),
        (other(page_table=cache.page_table[0]), ValueError), (other(page_table=cache.page_table.t().contiguous().t()), ValueError),
        (other(lens=cache.lens[:1]), ValueError), (other(lens=torch.zeros(4, dtype=i32, device=DEV)[::2]), ValueError),
        (other(weight=cache.weight[:, :1]), ValueError), (other(weight=cache.weight.double()), ValueError),
        (other(pos=cache.pos.long()), ValueError), (other(seen=cache.seen[:1]), ValueError),
        (lambda: gt.tree_attn(q[0], cache), ValueError), (lambda: gt.tree_attn(q[:1], cache), ValueError),
        (lambda: gt.tree_attn(q.half(), cache), TypeError), (lambda: gt.tree_attn(s.q, cache), ValueError),
        (lambda: gt.tree_attn(q.transpose(1, 3), cache), ValueError), (lambda: gt.tree_attn(q, cache, kn), ValueError),
        (lambda: gt.tree_attn(q, cache, None, vn), ValueError), (lambda: gt.tree_attn(q, cache, kn[:, :2], vn), ValueError),
        (lambda: gt.tree_attn(q, cache, kn, vn, mask=torch.zeros((2, 3, 1), dtype=i32, device=DEV)), ValueError),
        (lambda: gt.tree_attn(q, cache, kn, vn, mask=torch.zeros((2, 3, 2), dtype=torch.int64, device=DEV)), ValueError),
        (lambda: gt.tree_attn(q, cache, token_lens=torch.zeros(3, dtype=i32, device=DEV)), ValueError),
        (lambda: gt.tree_attn(q, cache, out=q.transpose(1, 2)), ValueError), (lambda: gt.tree_attn(q, cache, out=q.half()), ValueError),
        (lambda: gt.tree_attn(q, cache, lse=lse[:1]), ValueError), (lambda: gt.tree_attn(q, cache, scale=0.0), ValueError),
        (lambda: gt.tree_attn(q, cache, scale="x"), TypeError), (lambda: gt.tree_attn(q, cache, status=lse), ValueError),
        (lambda: gt.tree_attn(q, cache, out=q), gt.GemmTnError), (lambda: gt.tree_attn(q, cache, scale=-1.0), gt.GemmTnError),
        (lambda: gt.cache_append(cache, kn[:, :, :1], vn), ValueError), (lambda: gt.cache_append(cache, kn, vn[:, :2]), ValueError),
        (lambda: gt.cache_append(cache, kn, vn, rows=torch.zeros(2, dtype=i32, device=DEV)), ValueError),
        (lambda: gt.cache_append(other(seen=None)(), kn, vn, seen_out=cache.seen), ValueError),
        (lambda: gt.cache_append(cache, kn, vn, lens_out=cache.seen), gt.GemmTnError),
        (lambda: gt.cache_weigh(other(weight=None)(), q, lse), ValueError), (lambda: gt.cache_weigh(cache, q, lse[0]), ValueError),
        (lambda: gt.cache_weigh(cache, q, lse, out=cache.weight[:1]), ValueError), (lambda: gt.cache_weigh(cache, q, None), TypeError),
        (lambda: gt.cache_evict(other(weight=None)(), 8), ValueError), (lambda: gt.cache_evict(cache, 8.5), TypeError),
        (lambda: gt.cache_evict(other(pos=None)(), 8, pos_out=cache.pos), ValueError), (lambda: gt.cache_evict(cache, -1), gt.GemmTnError),
        (lambda: gt.cache_evict(cache, 8, 9), gt.GemmTnError)]
    before = {n: sys.getrefcount(t) for n, t in [*whole.items(), ("q", q), ("lse", lse)]}
    for i, (call, error) in enumerate(refused):
        with pytest.raises(error) as caught:
            call()
        assert str(caught.value), i
        del caught
    gc.collect()
    assert before == {n: sys.getrefcount(t) for n, t in [*whole.items(), ("q", q), ("lse", lse)]}


def test_a_cache_keeps_its_tensors_and_shows_them():
    s = ref.make("fp16", 128, [9], 1, 2, 1, 8, seed=67)
    cache, _ = on_gpu(s)
    lens = torch.tensor([5], dtype=torch.int32, device=DEV)
    count = sys.getrefcount(lens)
    other = gt.KVCache(cache.k, cache.v, cache.page_table, lens)
    assert sys.getrefcount(lens) == count + 1 and other.lens is lens and other.weight is None and other.seen is None
    assert (other.batch, other.capacity, other.index, other.kv_heads, other.head_dim) == (1, 16, 0, 2, 128)
    assert other.dtype is torch.float16
    with pytest.raises(AttributeError):
        other.lens = cache.lens      # the description was made of the tensor
    del other
    assert sys.getrefcount(lens) == count
    out = gt.tree_attn(s.q.to(DEV), cache)
    assert sys.getrefcount(out) == 2 and gt.tree_attn(s.q.to(DEV), cache, out=out) is out


def test_a_cache_follows_its_tensors_to_other_storage():
    """Tensors given other storage after the cache was made: .data, set_ and resize_ to the same sizes; every call goes there."""
    s = ref.make("bf16", 64, [30, 41], 3, 2, 2, 16, seed=68)
    want = ref.attention(s)
    for move in ("data", "set_", "resize_"):
        wrong = ref.make("bf16", 64, [9, 5], 3, 2, 2, 16, seed=69, max_pages=s.table.shape[1])
        cache, status = on_gpu(wrong)
        for name in ("k", "v", "page_table", "lens", "weight", "pos", "seen"):
            held, now = getattr(cache, name), {"page_table": s.table}.get(name, getattr(s, name, None)).to(DEV)
            if move == "data":
                held.data = now
            elif move == "set_":
                held.set_(now)
            else:
                shape = held.shape
                held.resize_(4 * held.numel()).resize_(shape)      # the storage moves as it grows
                held.copy_(now)
        out, lse = run_attn(s, cache=cache)
        ref.check_attention(out, lse, want, s, 7.0)
        pool = cache.k
        gt.cache_append(cache, s.k_new[:, :1].to(DEV), s.v_new[:, :1].to(DEV), status=status)
        assert cache.lens.tolist() == [31, 42] and int(status.item()) == 0
        assert ref.same(pool[int(s.table[1, 2]), 41 % 16].cpu(), s.k_new[1, 0])
        kept = cache.weight.clone()
        gt.cache_weigh(cache, s.q.to(DEV), lse.to(DEV), counts=torch.zeros(2, dtype=torch.int32, device=DEV))
        assert ref.same(cache.weight, kept)
        gt.cache_evict(cache, 20)
        assert cache.lens.tolist() == [20, 20]


def test_a_cache_refuses_tensors_that_no_longer_fit():
    """Other sizes, types or a freed storage behind a cache's tensors: every call refuses, and touches nothing."""
    s = ref.make("bf16", 64, [30, 40], 3, 2, 2, 16, seed=70)
    q, kn, vn, lse = s.q.to(DEV), s.k_new.to(DEV), s.v_new.to(DEV), torch.zeros(s.q.shape[:3], device=DEV)

    def freed(c):
        c.v.untyped_storage().resize_(0)

    def shorter(c):
        c.weight.untyped_storage().resize_(c.weight.numel() * 4 - 4)

    for spoil, what in [(lambda c: c.k.resize_(c.k.shape[0] - 1, *c.k.shape[1:]), "same strides"), (freed, "smaller than"),
                        (shorter, "smaller than"), (lambda c: c.lens.resize_(1), "contiguous \\[batch\\]"),
                        (lambda c: c.pos.resize_(3), "pos must be"),
                        (lambda c: [c.k.resize_(1, *c.k.shape[1:]), c.v.resize_(1, *c.v.shape[1:])], "have changed"),
                        (lambda c: [t.resize_(1, *t.shape[1:]) for t in (c.page_table, c.weight, c.pos)] +
                         [t.resize_(1) for t in (c.lens, c.seen)], "have changed")]:
        cache, _ = on_gpu(s)
        spoil(cache)
        for call in (lambda: gt.tree_attn(q, cache, kn, vn), lambda: gt.cache_append(cache, kn, vn),
                     lambda: gt.cache_weigh(cache, q, lse), lambda: gt.cache_evict(cache, 8)):
            with pytest.raises(ValueError, match=what):
                call()
    torch.cuda.synchronize()


def test_empty_calls():
    s = ref.make("bf16", 64, [5], 2, 1, 1, 8, seed=63)
    cache, status = on_gpu(s)
    q = torch.zeros((1, 0, 1, 64), dtype=s.dtype, device=DEV)
    assert gt.tree_attn(q, cache).shape == q.shape
    gt.cache_append(cache, q, q, status=status)
    assert cache.lens.tolist() == [5]
    before = cache.weight.clone()
    gt.cache_weigh(cache, q, torch.zeros((1, 0, 1), device=DEV), status=status)
    gt.cache_evict(cache, 5, status=status)
    assert ref.same(cache.weight, before) and cache.lens.tolist() == [5] and int(status.item()) == 0


def test_the_cache_continues_a_prompts_attention():
    """flash_attn over a prompt gives what tree_attn gives for its last tokens over a cache of the others."""
    from dense_tiled_gemm_03_gb300.workloads import make_qkv
    q, k, v = (t.to(DEV) for t in make_qkv(2, 300, 2, 64, "bf16", seed=64))
    full = gt.flash_attn(q, k, v, causal=True)
    pool_k = torch.zeros((2 * 16, 16, 2, 64), dtype=k.dtype, device=DEV)
    cache = gt.KVCache(pool_k, torch.zeros_like(pool_k), torch.arange(32, dtype=torch.int32, device=DEV).view(2, 16),
                       torch.zeros(2, dtype=torch.int32, device=DEV))
    gt.cache_append(cache, k[:, :250].contiguous(), v[:, :250].contiguous())
    part = gt.tree_attn(q[:, 250:], cache, k[:, 250:], v[:, 250:])
    # both round their probabilities (2^-9 of the mean |v| <= 4) and their outputs
    assert (part.float() - full[:, 250:].float()).abs().max().item() <= 2 * (2.0 ** -9 * 4 + 2.0 ** -9 * 4)
