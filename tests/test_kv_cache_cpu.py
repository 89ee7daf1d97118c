"""CPU tests of the paged cache's operators: the C ABI refuses bad arguments
before it touches a device, the binding refuses tensors it cannot hand over, the
tree masks, and the 64-bit reference of the GPU tests on closed forms."""
from __future__ import annotations

import ctypes
import math

import pytest
import torch

import dense_tiled_gemm_03_gb300 as gt
from dense_tiled_gemm_03_gb300 import _cache
import _cache_ref as ref


@pytest.fixture(scope="module")
def lib():
    from dense_tiled_gemm_03_gb300 import build as native_build
    native_build.build()
    return gt.library()


# Fake, well-separated addresses: validation never dereferences them.
K, V, TABLE, LENS, Q, KN, VN, O, LSE, W, POS, SEEN, OUT = (0x100000000000 + 0x10000000000 * i for i in range(13))
F16, BF16 = gt.GEMM_TN_F16, gt.GEMM_TN_BF16
INVALID, MISALIGNED = gt.GEMM_TN_ERR_INVALID_VALUE, gt.GEMM_TN_ERR_MISALIGNED
NO_DEVICE = (gt.GEMM_TN_ERR_UNSUPPORTED_DEVICE, gt.GEMM_TN_ERR_CUDA)


def cache(**over):
    """A valid cache: 100 pages of 16 rows of 2 heads of 64."""
    f = dict(k=K, v=V, num_pages=100, page_size=16, kv_heads=2, head_dim=64, page_stride=2048, slot_stride=128,
             head_stride=64, page_table=TABLE, table_stride=10, max_pages=10, lens=LENS, weight=W, pos=POS, seen=SEEN)
    f.update(over)
    return _cache.KvCacheStruct(**f)


def rows(data=Q, b=4 * 8 * 64, t=8 * 64, h=64):
    return _cache.KvRows(data, b, t, h)


def ref_or_null(x):
    return None if x is None else ctypes.byref(x)


def attn(lib, dtype=BF16, batch=3, tokens=4, heads=8, c=cache(), q=rows(), kn=rows(KN, 512, 128), vn=rows(VN, 512, 128),
         mask=None, token_lens=None, o=O, lse=LSE, scale=0.0):
    return lib.tree_attn_fwd(dtype, batch, tokens, heads, ref_or_null(c), ref_or_null(q), ref_or_null(kn), ref_or_null(vn), mask,
                             token_lens, o, lse, scale, None, None)


def append(lib, dtype=BF16, batch=3, tokens=4, c=cache(), kn=rows(KN, 512, 128), vn=rows(VN, 512, 128), r=None, counts=None,
           max_rows=4, lens_out=OUT, seen_out=None):
    return lib.kv_cache_append(dtype, batch, tokens, ref_or_null(c), ref_or_null(kn), ref_or_null(vn), r, counts, max_rows,
                               lens_out, seen_out, None, None)


def weigh(lib, dtype=BF16, batch=3, tokens=4, heads=8, c=cache(), q=rows(), lse=LSE, r=None, counts=None, max_rows=4, causal=1,
          scale=0.0, out=OUT):
    return lib.kv_cache_weigh(dtype, batch, tokens, heads, ref_or_null(c), ref_or_null(q), lse, r, counts, max_rows, causal,
                              scale, out, None, None)


def evict(lib, dtype=BF16, batch=3, c=cache(), keep=50, recent=5, w=OUT, p=POS, lens_out=LENS):
    return lib.kv_cache_evict(dtype, batch, ref_or_null(c), keep, recent, w, p, lens_out, None, None)


def test_valid_calls_get_as_far_as_the_device(lib):
    if torch.cuda.is_available():
        pytest.skip("the addresses are not real")
    for call in (attn, append, weigh, evict):
        assert call(lib) in NO_DEVICE, call.__name__
    assert attn(lib, kn=None, vn=None) in NO_DEVICE
    assert attn(lib, lse=None, mask=0x1000, token_lens=0x2000) in NO_DEVICE
    # a pool of [page][head][row] order, and one page, one head with strides nobody reads
    assert attn(lib, c=cache(slot_stride=64, head_stride=1024)) in NO_DEVICE
    assert attn(lib, c=cache(num_pages=1, page_stride=0, kv_heads=1, head_stride=0)) in NO_DEVICE
    assert evict(lib, recent=0, p=None, c=cache(pos=None, seen=None)) in NO_DEVICE


CACHE_FAULTS = [
    (None, INVALID), (cache(k=None), INVALID), (cache(v=None), INVALID), (cache(page_table=None), INVALID),
    (cache(lens=None), INVALID), (cache(head_dim=96), INVALID), (cache(kv_heads=0), INVALID), (cache(page_size=12), INVALID),
    (cache(page_size=0), INVALID), (cache(page_size=200), INVALID), (cache(page_size=1 << 21), INVALID),
    (cache(num_pages=0), INVALID), (cache(num_pages=2 ** 31), INVALID), (cache(max_pages=0), INVALID),
    (cache(max_pages=2 ** 27), INVALID), (cache(table_stride=9), INVALID), (cache(page_stride=2047), INVALID),
    (cache(slot_stride=-128), INVALID), (cache(slot_stride=0), INVALID), (cache(head_stride=0), INVALID),
    (cache(head_stride=2 ** 39), INVALID), (cache(k=K + 2), MISALIGNED), (cache(v=V + 8), MISALIGNED),
    (cache(lens=LENS + 2), MISALIGNED), (cache(page_table=TABLE + 1), MISALIGNED),
]


@pytest.mark.parametrize("fault,status", CACHE_FAULTS)
@pytest.mark.parametrize("call", [attn, append, weigh, evict])
def test_a_bad_cache_is_refused(lib, call, fault, status):
    assert call(lib, c=fault) == status
    assert gt.gemm_tn_last_error_message() != ""


@pytest.mark.parametrize("call", [attn, append, weigh, evict])
def test_types_and_sizes(lib, call):
    assert call(lib, dtype=2) == gt.GEMM_TN_ERR_UNSUPPORTED_DTYPE
    assert call(lib, batch=-1) == INVALID and call(lib, batch=2 ** 31) == INVALID
    assert call(lib, batch=2 ** 31 - 1) == INVALID      # times kv_heads
    assert call(lib, batch=0) == gt.GEMM_TN_OK


@pytest.mark.parametrize("over,status", [
    (dict(heads=7), INVALID), (dict(heads=2 * 129), INVALID), (dict(tokens=-1), INVALID), (dict(tokens=2 ** 31), INVALID),
    (dict(scale=-1.0), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(q=None), INVALID), (dict(q=rows(None)), INVALID), (dict(q=rows(Q + 8)), MISALIGNED), (dict(q=rows(t=513)), INVALID),
    (dict(q=rows(h=0)), INVALID), (dict(q=rows(b=-512)), INVALID), (dict(kn=None), INVALID), (dict(vn=None), INVALID),
    (dict(kn=rows(KN, 512, 120)), gt.GEMM_TN_OK), (dict(vn=rows(VN, 512, 4)), INVALID), (dict(o=None), INVALID),
    (dict(o=O + 8), MISALIGNED), (dict(lse=LSE + 2), MISALIGNED), (dict(mask=0x1004), MISALIGNED),
    (dict(token_lens=0x1001), MISALIGNED), (dict(o=Q + 64), INVALID), (dict(o=K + 4096), INVALID), (dict(o=VN), INVALID),
    (dict(kn=None, vn=None, mask=0x1000), INVALID)])
def test_attention_refusals(lib, over, status):
    rc = attn(lib, **over)
    assert rc == status or (status == gt.GEMM_TN_OK and rc in NO_DEVICE)


@pytest.mark.parametrize("over,status", [
    (dict(tokens=-1), INVALID), (dict(max_rows=5), INVALID), (dict(max_rows=-1), INVALID), (dict(tokens=0, r=0x1000), INVALID),
    (dict(lens_out=None), INVALID), (dict(c=cache(seen=None), seen_out=OUT), INVALID), (dict(r=0x1002), MISALIGNED),
    (dict(counts=0x1001), MISALIGNED), (dict(kn=rows(K + 4096, 512, 128)), INVALID), (dict(vn=None), INVALID),
    (dict(batch=2 ** 29, tokens=128, max_rows=128), INVALID)])
def test_append_refusals(lib, over, status):
    assert append(lib, **over) == status


@pytest.mark.parametrize("over,status", [
    (dict(heads=0), INVALID), (dict(heads=3), INVALID), (dict(max_rows=5), INVALID), (dict(tokens=0, r=0x1000), INVALID),
    (dict(lse=None), INVALID), (dict(out=None), INVALID), (dict(c=cache(weight=None)), INVALID), (dict(out=OUT + 2), MISALIGNED),
    (dict(r=0x1001), MISALIGNED), (dict(scale=-0.5), INVALID), (dict(max_rows=2 ** 23, r=0x1000), INVALID)])
def test_weigh_refusals(lib, over, status):
    assert weigh(lib, **over) == status


@pytest.mark.parametrize("over,status", [
    (dict(keep=-1), INVALID), (dict(keep=2 ** 31), INVALID), (dict(recent=-1), INVALID), (dict(recent=51), INVALID),
    (dict(c=cache(pos=None), p=None), INVALID), (dict(c=cache(seen=None)), INVALID), (dict(p=None), INVALID),
    (dict(c=cache(pos=None), recent=0), INVALID), (dict(c=cache(weight=None)), INVALID), (dict(w=None), INVALID),
    (dict(lens_out=None), INVALID), (dict(lens_out=LENS + 1), MISALIGNED)])
def test_evict_refusals(lib, over, status):
    assert evict(lib, **over) == status


@pytest.mark.parametrize("call,over", [
    (attn, dict(lse=O)), (attn, dict(lse=O + 3 * 4 * 8 * 64 * 2 - 4)), (attn, dict(lse=Q + 64)), (attn, dict(lse=LENS)),
    (attn, dict(lse=TABLE + 96)), (attn, dict(o=TABLE)), (attn, dict(o=0x1000, token_lens=0x1000)), (attn, dict(o=0x1000, mask=0x1010)),
    (append, dict(lens_out=LENS + 4)), (append, dict(lens_out=SEEN)), (append, dict(lens_out=OUT, seen_out=OUT + 8)),
    (append, dict(lens_out=OUT, counts=OUT)), (append, dict(lens_out=OUT, r=OUT - 40)), (append, dict(seen_out=LENS)),
    (append, dict(seen_out=SEEN + 4)), (append, dict(lens_out=TABLE + 116)), (weigh, dict(out=W + 4)), (weigh, dict(out=LSE)),
    (weigh, dict(out=LENS - 8)), (weigh, dict(out=K)), (weigh, dict(out=0x1000, counts=0x1100)), (evict, dict(w=W + 64)),
    (evict, dict(w=POS)), (evict, dict(p=W)), (evict, dict(p=POS - 4)), (evict, dict(w=OUT, p=OUT + 3 * 2 * 160 * 4 - 4)),
    (evict, dict(lens_out=LENS - 4)), (evict, dict(lens_out=SEEN)), (evict, dict(lens_out=TABLE)), (evict, dict(lens_out=W))])
def test_outputs_that_lie_in_other_arrays_are_refused(lib, call, over):
    assert call(lib, **over) == INVALID
    assert "overlap" in gt.gemm_tn_last_error_message()


def with_status(lib, name, at):
    """A call of the C function with a status word at that address."""
    c, q, kn, vn = cache(), rows(), rows(KN, 512, 128), rows(VN, 512, 128)
    r = ctypes.byref
    return {"attn": lambda: lib.tree_attn_fwd(BF16, 3, 4, 8, r(c), r(q), r(kn), r(vn), None, None, O, LSE, 0.0, at, None),
            "append": lambda: lib.kv_cache_append(BF16, 3, 4, r(c), r(kn), r(vn), None, None, 4, OUT, None, at, None),
            "weigh": lambda: lib.kv_cache_weigh(BF16, 3, 4, 8, r(c), r(q), LSE, None, None, 4, 1, 0.0, OUT, at, None),
            "evict": lambda: lib.kv_cache_evict(BF16, 3, r(c), 50, 5, W, POS, LENS, at, None)}[name]()


@pytest.mark.parametrize("call,over", [
    (append, dict(lens_out=KN)), (append, dict(lens_out=VN + 64)), (append, dict(lens_out=K + 4096)), (append, dict(lens_out=V)),
    (append, dict(lens_out=W + 8)), (append, dict(lens_out=POS)), (append, dict(seen_out=K)), (append, dict(seen_out=W)),
    (append, dict(c=cache(weight=KN))), (append, dict(c=cache(pos=LENS))), (append, dict(c=cache(pos=SEEN))),
    (append, dict(c=cache(pos=W))), (append, dict(c=cache(pos=W + 3 * 2 * 160 * 4 - 4))), (append, dict(c=cache(weight=K))),
    (append, dict(c=cache(lens=K))), (append, dict(c=cache(page_table=V))), (append, dict(c=cache(v=K))),
    (append, dict(c=cache(v=K + 128))), (append, dict(counts=K)), (append, dict(r=W)),
    (evict, dict(w=K)), (evict, dict(p=V)), (evict, dict(lens_out=K)), (evict, dict(lens_out=V + 8)), (evict, dict(c=cache(v=K))),
    (evict, dict(c=cache(seen=K))), (evict, dict(c=cache(page_table=K))), (evict, dict(c=cache(weight=K))),
    (evict, dict(c=cache(weight=POS), w=POS, p=OUT)), (weigh, dict(out=V)), (weigh, dict(out=POS)), (weigh, dict(out=SEEN)),
    (attn, dict(o=W)), (attn, dict(lse=POS)), (attn, dict(o=SEEN))])
def test_what_a_call_writes_lies_apart_from_all_its_arrays(lib, call, over):
    assert call(lib, **over) == INVALID
    assert "overlap" in gt.gemm_tn_last_error_message()


@pytest.mark.parametrize("name,places", [
    ("attn", [O, LSE, Q, KN, VN, K, V, LENS, TABLE, W]), ("append", [OUT, K, V, W, POS, LENS, SEEN, TABLE, KN]),
    ("weigh", [OUT, W, Q, LSE, K, LENS, TABLE]), ("evict", [W, POS, LENS, SEEN, TABLE, K, V])])
def test_the_status_word_lies_apart_too(lib, name, places):
    for at in places:
        assert with_status(lib, name, at) == INVALID and "overlap" in gt.gemm_tn_last_error_message()
    if not torch.cuda.is_available():
        assert with_status(lib, name, 0x1000) in NO_DEVICE


def test_pools_may_lie_between_one_another(lib):
    """K and V of a page, of a slot, of a head or of all heads side by side; reading may share them outright."""
    if torch.cuda.is_available():
        pytest.skip("the addresses are not real")
    for over in (dict(page_stride=4096, v=K + 2048 * 2), dict(page_stride=4096, slot_stride=256, v=K + 128 * 2),
                 dict(page_stride=4096, slot_stride=256, head_stride=128, v=K + 64 * 2), dict(v=K + 100 * 2048 * 2),
                 dict(k=K + 2048 * 2, v=K, page_stride=4096), dict(num_pages=1, page_stride=0, v=K + 2048 * 2)):
        for call in (append, evict):
            assert call(lib, c=cache(**over)) in NO_DEVICE, over
    for call in (attn, weigh):
        assert call(lib, c=cache(v=K)) in NO_DEVICE
    assert append(lib, max_rows=0, kn=None, vn=None) in NO_DEVICE


def test_whether_pools_share_rows_is_found_for_any_strides(lib):
    """Random strides and distances against the rows listed one by one; 8-element steps are what 16-byte rows allow."""
    if torch.cuda.is_available():
        pytest.skip("the addresses are not real")
    import random
    rng = random.Random(7)
    shared = apart = 0
    for _ in range(1500):
        heads, pages = rng.randint(1, 3), rng.randint(1, 4)
        inner, n_inner, outer, n_outer = rng.choice([("head", heads, "slot", 8), ("slot", 8, "head", heads)])
        s = {inner: 64 + 8 * rng.choice([0, 0, 1, 8, 9])}
        s[outer] = s[inner] * (n_inner - 1) + 64 + 8 * rng.choice([0, 0, 3, 8, 16])
        s["page"] = s[outer] * (n_outer - 1) + s[inner] * (n_inner - 1) + 64 + 8 * rng.choice([0, 0, 8, 40, 80])
        reach = s["page"] * pages
        d = 8 * rng.randint(-reach // 8 - 4, reach // 8 + 4) if rng.random() < 0.5 else \
            64 * rng.randint(-3, 3) + rng.choice([0, s["slot"], s["head"], s["page"]]) * rng.randint(-9, 9)
        at = {p * s["page"] + r * s["slot"] + h * s["head"] for p in range(pages) for r in range(8) for h in range(heads)}
        spans = {x // 8 + e for x in at for e in range(8)}                     # in steps of 8 elements
        want = any((x + d) // 8 + e in spans for x in at for e in range(8))
        c = cache(kv_heads=heads, num_pages=pages, page_size=8, page_stride=s["page"], slot_stride=s["slot"],
                  head_stride=s["head"], v=K + 2 * d)
        rc = evict(lib, c=c)
        assert (rc == INVALID) == want and (want or rc in NO_DEVICE), (s, d, heads, pages)
        shared, apart = shared + want, apart + (not want)
    assert shared > 200 and apart > 200


def test_outputs_that_replace_the_caches_own_arrays_are_not(lib):
    if torch.cuda.is_available():
        pytest.skip("the addresses are not real")
    for rc in (append(lib, lens_out=LENS, seen_out=SEEN), append(lib, lens_out=LENS), append(lib, lens_out=OUT, seen_out=OUT + 12),
               weigh(lib, out=W), evict(lib, w=W, p=POS, lens_out=LENS), evict(lib, w=OUT, p=OUT + 3 * 2 * 160 * 4),
               attn(lib, lse=O + 3 * 4 * 8 * 64 * 2)):
        assert rc in NO_DEVICE


def test_evict_refuses_sizes_that_its_32_bit_walks_cannot_hold(lib):
    """The walk over slots steps up to 2^16 past the last one, the walk over lists by up to 65535."""
    wide = cache(page_size=128, max_pages=(2 ** 31 - 257) // 128, table_stride=2 ** 24)
    assert evict(lib, c=wide) == INVALID and "2^31 - 2^16" in gt.gemm_tn_last_error_message()
    many = cache(kv_heads=1, table_stride=10)
    for batch in (2 ** 31 - 1, 2 ** 30 + 1):
        assert evict(lib, batch=batch, c=many) == INVALID and "2^30" in gt.gemm_tn_last_error_message()


def test_as_many_key_tiles_as_32_bits_hold_leave_room_for_whole_chunks(lib):
    """192 lists of 11184810 tiles and places between them: 2^31 - 128, which rounding up to chunks would carry past 2^31."""
    c = cache(page_size=128, max_pages=11184810 - 9, table_stride=2 ** 24)
    assert 192 * 11184810 == 2 ** 31 - 128
    assert weigh(lib, batch=96, c=c) == INVALID and "key tiles" in gt.gemm_tn_last_error_message()


def test_empty_calls_need_no_device(lib):
    assert attn(lib, tokens=0) == gt.GEMM_TN_OK and attn(lib, heads=0) == gt.GEMM_TN_OK


def test_the_binding_takes_cuda_tensors_only(lib):
    k = torch.zeros((2, 8, 1, 64), dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA"):
        gt.KVCache(k, k, torch.zeros((1, 2), dtype=torch.int32), torch.zeros(1, dtype=torch.int32))


@pytest.mark.parametrize("call,what", [
    (lambda: gt.KVCache(), "missing required argument 'k'"), (lambda: gt.KVCache(1, 2, 3, 4), "k must be a tensor"),
    (lambda: gt.KVCache(None, None, None, None), "k must be a tensor"),
    (lambda: gt.KVCache(1, 2, 3, 4, k=1), "multiple values for argument 'k'"),
    (lambda: gt.KVCache(1, 2, 3, 4, table=1), "unexpected keyword argument 'table'"),
    (lambda: gt.KVCache(*range(8)), "at most 7 arguments"), (lambda: gt.tree_attn(torch.zeros(1), None), "must be a KVCache"),
    (lambda: gt.tree_attn(torch.zeros(1), torch.zeros(1)), "must be a KVCache"),
    (lambda: gt.cache_append(3, 4), "missing required argument 'v_new'"), (lambda: gt.cache_weigh(3, 4, 5), "must be a KVCache"),
    (lambda: gt.cache_evict(cache=3, keep=4), "must be a KVCache"), (lambda: gt.cache_evict(), "missing required argument 'cache'")])
def test_the_binding_refuses_what_is_no_call(lib, call, what):
    with pytest.raises(TypeError, match=what):
        call()


def test_the_bindings_names_and_documentation(lib):
    import inspect
    assert set(_cache.BOUND) <= set(dir(gt)) and not hasattr(gt, "no_such_name")
    for name in _cache.BOUND:
        assert getattr(gt, name).__doc__
    names = list(inspect.signature(gt.tree_attn).parameters)
    assert names == ["q", "cache", "k_new", "v_new", "mask", "token_lens", "scale", "out", "lse", "status"]
    assert inspect.signature(gt.cache_weigh).parameters["causal"].default is True


def test_a_missing_binding_fails_loudly(lib, monkeypatch):
    import sys
    monkeypatch.setitem(sys.modules, "dense_tiled_gemm_03_gb300._kv_cache", None)
    monkeypatch.delattr(gt, "_kv_cache", raising=False)
    with pytest.raises(RuntimeError, match="build it"):
        _cache.binding()


# ---------------------------------------------------------------- the build

@pytest.fixture
def small_build(monkeypatch, tmp_path):
    """The build step with one source, and everything that it makes elsewhere."""
    from dense_tiled_gemm_03_gb300 import build as b
    for name, value in (("SOURCES", ["repack.cu"]), ("BUILD_DIR", tmp_path / "objects"), ("LIBRARY", tmp_path / "lib.so"),
                        ("BINDING", tmp_path / "binding.so")):
        monkeypatch.setattr(b, name, value)
    return b


@pytest.mark.parametrize("torch_is", ["missing", "without CUDA"])
def test_the_library_builds_without_torch(small_build, monkeypatch, tmp_path, torch_is, capsys):
    import importlib.util
    from types import SimpleNamespace
    find = importlib.util.find_spec
    spec = None if torch_is == "missing" else SimpleNamespace(submodule_search_locations=[str(tmp_path)])
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: spec if name == "torch" else find(name, *a))
    assert small_build.build() == small_build.LIBRARY and small_build.LIBRARY.exists()
    assert not small_build.BINDING.exists() and "no torch" in capsys.readouterr().err


def test_a_binding_that_does_not_compile_leaves_the_library(small_build, monkeypatch, tmp_path):
    broken = tmp_path / "broken.cpp"
    broken.write_text("#error no binding\n")
    monkeypatch.setattr(small_build, "BINDING_SOURCE", broken)
    with pytest.raises(RuntimeError, match="no binding"):
        small_build.build()
    assert small_build.LIBRARY.exists() and not small_build.BINDING.exists()


def test_a_binding_built_against_another_torch_is_stale(lib, monkeypatch, tmp_path):
    from dense_tiled_gemm_03_gb300 import build as b
    here = b.torch_dir()
    assert b.torch_version(here) == torch.__version__ and not b.binding_is_stale(here)
    other = tmp_path / "torch"
    other.mkdir()
    (other / "version.py").write_text((here / "version.py").read_text())
    assert b.binding_is_stale(other)                       # elsewhere
    monkeypatch.setattr(b, "torch_version", lambda d: "0.0.1+cu1")
    assert b.binding_is_stale(here)                        # there, another version


def test_a_binding_built_against_another_torch_is_not_used(lib, monkeypatch):
    assert _cache.binding().built_against == torch.__version__
    monkeypatch.setattr(torch, "__version__", "0.0.1+cu1")
    with pytest.raises(RuntimeError, match="build it"):
        _cache.binding()


def test_the_package_loads_its_library_without_torch(lib):
    import subprocess
    import sys
    from pathlib import Path
    code = ("import sys; sys.modules['torch'] = None\n"
            "import dense_tiled_gemm_03_gb300 as gt\n"
            "assert gt.gemm_tn_version() > 0 and gt.gemm_tn_select_config(0, 256, 256, 256) >= 0\n")
    subprocess.run([sys.executable, "-c", code], check=True, cwd=Path(__file__).resolve().parents[1])


# ---------------------------------------------------------------- tree masks

def test_tree_mask():
    parents = torch.tensor([[-1, 0, 0, 1, 2, -1], [-1, 0, 1, 2, 3, 4]])
    m = gt.tree_mask(parents)
    assert m.shape == (2, 6, 1) and m.dtype == torch.int64
    assert m[0, :, 0].tolist() == [0b1, 0b11, 0b101, 0b1011, 0b10101, 0b100000]
    assert m[1, :, 0].tolist() == [2 ** (i + 1) - 1 for i in range(6)]
    chain = torch.arange(-1, 129)[None]
    see = ref.visible(130, gt.tree_mask(chain))
    assert torch.equal(see, ref.visible(130)) and gt.tree_mask(chain).shape == (1, 130, 3)
    assert gt.tree_mask(torch.zeros((2, 0), dtype=torch.int32)).shape == (2, 0, 0)


@pytest.mark.parametrize("parents", [[[0]], [[-1, 1]], [[-2]], [[-1, 5]]])
def test_tree_mask_refuses_parents_that_do_not_come_first(parents):
    with pytest.raises(ValueError):
        gt.tree_mask(torch.tensor(parents))


def test_tree_mask_refuses_other_types():
    for bad in (torch.zeros((1, 2)), torch.zeros(3, dtype=torch.int64), torch.zeros((1, 1), dtype=torch.bool)):
        with pytest.raises(ValueError):
            gt.tree_mask(bad)


# ---------------------------------------------------------------- the reference

def test_the_reference_on_closed_forms():
    s = ref.make("bf16", 64, [20, 0], 3, 2, 2, 8, [3, 2], seed=1)
    s.q.nan_to_num_(0.0)
    s.q[:] = 0.0
    o, lse, *_ = ref.attention(s)
    assert abs(float(lse[0, 1, 0]) - math.log(22)) < 1e-12 and abs(float(lse[1, 0, 3])) < 1e-12
    mean = torch.cat([s.rows_of(s.v, 0, 1, 20), s.v_new[0, :2, 1].double()]).mean(0)
    assert torch.allclose(o[0, 1, 2], mean)
    assert torch.isnan(lse[1, 2]).all() and not torch.isnan(o[0]).any()
    w, _ = ref.weigh(s, torch.full((2, 3, 4), math.log(20.0)), None, [3, 0])
    # three queries of two heads; the newest slot is seen by the last query alone
    gain = (w - s.weight.double())[0, 0, :20]
    assert torch.allclose(gain, torch.tensor([6.0] * 18 + [4.0, 2.0], dtype=torch.float64) / 20)


def test_the_reference_evicts_the_lightest():
    s = ref.make("bf16", 64, [6], 1, 1, 1, 8, seed=2)
    s.weight[0, 0, :6] = torch.tensor([5.0, 1.0, 4.0, 1.0, 3.0, 0.0])
    s.pos[0, 0] = torch.arange(8)
    s.seen[0] = 6
    k, v, weight, pos, lens = ref.evict(s, 4, 1)      # slot 5 is the newest; 0, 2, 4 the heaviest; 5, 4 fill 1, 3
    assert lens.tolist() == [4] and pos[0, 0, :4].tolist() == [0, 4, 2, 5] and weight[0, 0, :4].tolist() == [5.0, 3.0, 4.0, 0.0]
    page = int(s.table[0, 0])
    assert torch.equal(k[page, 1], s.k[page, 4]) and torch.equal(v[page, 3], s.v[page, 5])
