"""Outputs of the paged-cache calls that lie over their inputs are refused by
address range, whatever the tensors' first addresses. Made-up addresses: every
call here is refused before any device work."""
import ctypes as C
import os

import pytest

from ranking_prefill_gb300 import lib

MB = 1 << 20


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(lib.LIB_PATH):
        from ranking_prefill_gb300 import build
        build.build()
    return lib.load()


# 10 pages of 16 rows, 2 heads of 64: 40960 bytes each
CACHE = dict(k=64 * MB, v=65 * MB, n_pages=10, page_size=16, Hkv=2, D=64, page_stride=16 * 128, row_stride=128,
             head_stride=64)
BYTES = 40960
LAYOUTS = {"rows": {}, "heads": dict(head_stride=16 * 64, row_stride=64),
           "apart": dict(page_stride=3 * 16 * 128), "pages inside": dict(page_stride=128, row_stride=1280)}


def cache(**kw):
    d = dict(CACHE)
    d.update(kw)
    return lib.mis_paged_cache(*[d[f] for f, _ in lib.mis_paged_cache._fields_])


EXTEND = dict(B=3, T=8, page_size=16, n_pages=100, new_len=MB, cache_len=2 * MB, cache_len_out=3 * MB,
              block_table=4 * MB, max_pages=4, stride=6, free_pages=5 * MB, n_free=50, free_head=6 * MB,
              free_head_out=7 * MB, cu_new=8 * MB, slot_map=9 * MB, position_ids=10 * MB, ws=11 * MB,
              ws_bytes=1 << 20, stream=None)
# table rows: 4 columns of 6, so an int at 4 MB + 16 or + 20 lies beside them


@pytest.mark.parametrize("kw", [
    dict(cache_len_out=MB), dict(cache_len_out=2 * MB + 4), dict(cache_len_out=5 * MB + 196), dict(free_head_out=6 * MB, free_head=6 * MB, new_len=6 * MB),
    dict(free_head_out=5 * MB + 8), dict(cu_new=2 * MB - 12), dict(cu_new=3 * MB + 8), dict(slot_map=9 * MB, position_ids=9 * MB + 28),
    dict(slot_map=5 * MB - 4), dict(position_ids=2 * MB + 8), dict(block_table=5 * MB + 100), dict(free_head=4 * MB + 12),
    dict(free_head_out=4 * MB + 24), dict(ws=4 * MB), dict(ws=9 * MB), dict(new_len=11 * MB + 256)])
def test_extend(L, kw):
    a = dict(EXTEND)
    a.update(kw)
    assert L.mis_paged_extend(*a.values()) == lib.MIS_ERR_INVALID_ARG


WRITE = dict(k=MB, v=2 * MB, ks=128, vs=160, T=4, src=3 * MB, slot=4 * MB, n=4, pos=5 * MB, base=1e6, ws=6 * MB,
             ws_bytes=256, stream=None)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("name", ["k", "v", "src", "slot", "pos"])
@pytest.mark.parametrize("buffer", ["k", "v"])
@pytest.mark.parametrize("at", [0, 64 * 256, BYTES - 16])
def test_write(L, layout, name, buffer, at):
    a = dict(WRITE)
    a[name] = CACHE[buffer] + at
    if layout == "apart":                                    # the same row and page: pages of 4096 bytes, 12288 apart
        a[name] += at // 4096 * 8192
    c = cache(**LAYOUTS[layout])
    assert L.mis_paged_write_kv(C.byref(c), *a.values()) == lib.MIS_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(ws=MB), dict(ws=4 * MB), dict(slot=6 * MB + 252)])
def test_write_workspace(L, kw):
    a = dict(WRITE)
    a.update(kw)
    c = cache()
    assert L.mis_paged_write_kv(C.byref(c), *a.values()) == lib.MIS_ERR_INVALID_ARG


TREE = dict(q=MB, k=2 * MB, v=3 * MB, o=4 * MB, lse=5 * MB, qs=256, ks=128, vs=128, os=256, table=6 * MB, max_pages=4,
            stride=4, cache_len=7 * MB, cu=8 * MB, parents=9 * MB, ws=128 * MB, ws_bytes=1 << 40, stream=None)
# 8 rows: q and o 4096 bytes, k and v 2048; lse 128, parents 32, cu 12, table 32


@pytest.mark.parametrize("kw", [
    dict(o=MB), dict(o=MB + 512), dict(o=MB - 3584 - 128), dict(o=2 * MB + 1920), dict(o=3 * MB - 4080), dict(o=CACHE["k"] + 512),
    dict(o=CACHE["v"] + BYTES - 16), dict(o=6 * MB - 4080), dict(o=7 * MB), dict(o=8 * MB), dict(o=9 * MB - 4064),
    dict(lse=MB + 4092), dict(lse=2 * MB - 124), dict(lse=4 * MB + 100), dict(lse=CACHE["v"] + 20000), dict(lse=7 * MB + 4),
    dict(lse=9 * MB), dict(o=5 * MB - 64), dict(q=128 * MB + 4096), dict(ws=4 * MB), dict(ws=64 * MB),
    # columns of one buffer that meet, at one row stride and at two
    dict(q=MB, o=MB + 2 * 192, qs=640, os=640), dict(q=MB, o=MB + 2 * 512, qs=640, os=640), dict(q=MB, o=MB + 512, qs=1024, os=2048)])
def test_tree_attention(L, kw):
    a = dict(TREE)
    a.update(kw)
    d, c = lib.mis_tree_desc(2, 8, 4, 4, 0.0), cache()
    assert L.mis_tree_attention_fwd(C.byref(d), C.byref(c), *a.values()) == lib.MIS_ERR_INVALID_ARG


@pytest.mark.parametrize("layout", LAYOUTS)
def test_tree_attention_over_any_cache(L, layout):
    d, c = lib.mis_tree_desc(2, 8, 4, 4, 0.0), cache(**LAYOUTS[layout])
    for o in (CACHE["k"] + 1024, CACHE["v"] + 2048):
        a = dict(TREE, o=o)
        assert L.mis_tree_attention_fwd(C.byref(d), C.byref(c), *a.values()) == lib.MIS_ERR_INVALID_ARG
