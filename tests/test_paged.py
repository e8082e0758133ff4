"""Paged-cache operators on the CPU: the oracle's own pins, and the refusals of
the C calls (every argument error is found before any device work, so the
calls below only ever see made-up addresses)."""
import ctypes as C
import os

import numpy as np
import pytest

from oracle import paged_oracle as P
from ranking_prefill_gb300 import lib


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(lib.LIB_PATH):
        from ranking_prefill_gb300 import build
        build.build()
    return lib.load()


# ------------------------------------------------------------------- oracle

def test_oracle_extend_by_hand():
    # 2 pages of 4 held by request 0 (5 rows), none by request 1; free list 7, 3, 9
    table = np.array([[1, 4, -1], [-1, -1, -1]])
    r = P.extend([4, 2], [5, 0], table, [8, 7, 3, 9], 1, 4, 10, 8)
    assert r["table"].tolist() == [[1, 4, 7], [3, -1, -1]]
    assert r["cu_new"].tolist() == [0, 4, 6] and r["cache_len"].tolist() == [9, 2]
    assert r["slot_map"].tolist() == [17, 18, 19, 28, 12, 13, -1, -1]
    assert r["position_ids"].tolist() == [5, 6, 7, 8, 0, 1, 0, 0]
    assert r["free_head"] == 3 and not r["bad_index"] and not r["out_of_pages"]


def test_oracle_tree_equals_separate_chains():
    # a node's output is that of plain causal attention on its root-to-node path
    rng = np.random.default_rng(0)
    n, Hq, H, D, ps = 7, 4, 2, 8, 4
    par = np.array([-1, 0, 0, 1, 2, -1, 5])
    q, k, v = rng.normal(size=(n, Hq, D)), rng.normal(size=(n, H, D)), rng.normal(size=(n, H, D))
    kc, vc = rng.normal(size=(5, ps, H, D)), rng.normal(size=(5, ps, H, D))
    table, Lc = np.array([[3, 0, 2]]), 10
    o, lse, _, _ = P.tree_attention(q, k, v, kc, vc, table, [Lc], [0, n], par)
    for i in range(n):
        path = [i]
        while par[path[0]] >= 0:
            path.insert(0, int(par[path[0]]))
        oc, lc, _, _ = P.tree_attention(q[path], k[path], v[path], kc, vc, table, [Lc],
                                        [0, len(path)], None)
        assert np.allclose(o[i], oc[-1]) and np.allclose(lse[:, i], lc[:, -1])


def test_oracle_rotation_is_a_rotation():
    rng = np.random.default_rng(1)
    x = rng.normal(size=(3, 2, 16))
    y = P.rotate(x, [0, 5, 9], 1e4)
    assert np.allclose(y[0], x[0])
    assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1))
    # scores depend on the distance only
    a = P.rotate(x[:1], [3], 1e4)[0] @ P.rotate(x[1:2], [8], 1e4)[0].T
    b = P.rotate(x[:1], [103], 1e4)[0] @ P.rotate(x[1:2], [108], 1e4)[0].T
    assert np.allclose(a, b)


# ----------------------------------------------------------------- refusals

A = 1 << 20      # an aligned made-up address


def _cache(**kw):
    d = dict(k=A, v=A, n_pages=10, page_size=16, Hkv=2, D=64, page_stride=16 * 128, row_stride=128,
             head_stride=64)
    d.update(kw)
    return lib.mis_paged_cache(*[d[f] for f, _ in lib.mis_paged_cache._fields_])


CACHE_ERRORS = [
    (dict(k=None), "MIS_ERR_INVALID_ARG"), (dict(v=A + 8), "MIS_ERR_INVALID_ARG"),
    (dict(n_pages=0), "MIS_ERR_INVALID_ARG"), (dict(Hkv=0), "MIS_ERR_INVALID_ARG"),
    (dict(page_size=24), "MIS_ERR_UNSUPPORTED"), (dict(page_size=8), "MIS_ERR_UNSUPPORTED"),
    (dict(page_size=512), "MIS_ERR_UNSUPPORTED"), (dict(D=96), "MIS_ERR_UNSUPPORTED"),
    (dict(n_pages=1 << 27), "MIS_ERR_SHAPE"), (dict(row_stride=132), "MIS_ERR_SHAPE"),
    (dict(row_stride=120), "MIS_ERR_SHAPE"),               # heads of neighbouring rows overlap
    (dict(page_stride=15 * 128), "MIS_ERR_SHAPE"), (dict(head_stride=-64), "MIS_ERR_SHAPE"),
]


@pytest.mark.parametrize("kw,want", CACHE_ERRORS)
def test_cache_refusals(L, kw, want):
    c = _cache(**kw)
    d = lib.mis_tree_desc(1, 1, 2, 1, 0.0)
    assert L.mis_tree_attention_workspace_size(C.byref(d), C.byref(c)) == 0
    st = L.mis_paged_write_kv(C.byref(c), A, A, 128, 128, 4, None, A, 4, None, 1e6, A, 1 << 20, None)
    assert lib.STATUS[st] == want
    st = L.mis_tree_attention_fwd(C.byref(d), C.byref(c), A, A, A, A, None, 128, 128, 128, 128, A, 4, 4,
                                  A, A, None, A, 1 << 30, None)
    assert lib.STATUS[st] == want


def test_cache_layouts_are_accepted(L):
    d = lib.mis_tree_desc(1, 1, 2, 1, 0.0)
    for kw in (dict(), dict(head_stride=16 * 64, row_stride=64), dict(page_stride=2 * 16 * 128),
               dict(Hkv=1, head_stride=3), dict(n_pages=1, page_stride=0)):
        c = _cache(**kw)
        assert L.mis_tree_attention_workspace_size(C.byref(d), C.byref(c)) > 0, kw


EXTEND = dict(B=3, T=8, page_size=16, n_pages=100, new_len=A, cache_len=A, cache_len_out=A,
              block_table=A, max_pages=4, stride=4, free_pages=A, n_free=50, free_head=A,
              free_head_out=A, cu_new=A, slot_map=A, position_ids=A, ws=A, ws_bytes=1 << 20, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(B=0), "MIS_ERR_INVALID_ARG"), (dict(T=-1), "MIS_ERR_INVALID_ARG"),
    (dict(n_pages=0), "MIS_ERR_INVALID_ARG"), (dict(max_pages=0), "MIS_ERR_INVALID_ARG"),
    (dict(n_free=-1), "MIS_ERR_INVALID_ARG"), (dict(page_size=48), "MIS_ERR_UNSUPPORTED"),
    (dict(n_pages=1 << 27), "MIS_ERR_SHAPE"), (dict(max_pages=1 << 27, stride=1 << 27), "MIS_ERR_SHAPE"),
    (dict(stride=3), "MIS_ERR_SHAPE"), (dict(new_len=None), "MIS_ERR_INVALID_ARG"),
    (dict(cache_len=A + 2), "MIS_ERR_INVALID_ARG"), (dict(slot_map=None), "MIS_ERR_INVALID_ARG"),
    (dict(free_pages=None), "MIS_ERR_INVALID_ARG"), (dict(position_ids=A + 1), "MIS_ERR_INVALID_ARG"),
    (dict(cu_new=None), "MIS_ERR_INVALID_ARG"), (dict(ws=None), "MIS_ERR_WORKSPACE"),
    (dict(ws=A + 16), "MIS_ERR_WORKSPACE"), (dict(ws_bytes=256), "MIS_ERR_WORKSPACE")])
def test_extend_refusals(L, kw, want):
    a = dict(EXTEND)
    a.update(kw)
    assert lib.STATUS[L.mis_paged_extend(*a.values())] == want


WRITE = dict(k=A, v=A, ks=128, vs=128, T=4, src=None, slot=A, n=4, pos=A, base=1e6, ws=A, ws_bytes=256,
             stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), "MIS_ERR_INVALID_ARG"), (dict(n=-1), "MIS_ERR_INVALID_ARG"),
    (dict(n=5), "MIS_ERR_SHAPE"), (dict(ks=120), "MIS_ERR_SHAPE"), (dict(vs=132), "MIS_ERR_SHAPE"),
    (dict(base=1.0), "MIS_ERR_INVALID_ARG"), (dict(base=float("nan")), "MIS_ERR_INVALID_ARG"),
    (dict(slot=None), "MIS_ERR_INVALID_ARG"), (dict(k=None), "MIS_ERR_INVALID_ARG"),
    (dict(v=A + 2), "MIS_ERR_INVALID_ARG"), (dict(src=A + 1), "MIS_ERR_INVALID_ARG"),
    (dict(ws=None), "MIS_ERR_WORKSPACE"), (dict(ws_bytes=128), "MIS_ERR_WORKSPACE")])
def test_write_refusals(L, kw, want):
    a = dict(WRITE)
    a.update(kw)
    c = _cache()
    assert lib.STATUS[L.mis_paged_write_kv(C.byref(c), *a.values())] == want


def test_write_of_nothing_is_accepted(L):
    a = dict(WRITE, n=0, k=None, v=None, slot=None)
    c = _cache()
    assert L.mis_paged_write_kv(C.byref(c), *a.values()) == lib.MIS_OK


TREE = dict(q=A, k=A, v=A, o=A, lse=A, qs=256, ks=128, vs=128, os=256, table=A, max_pages=4, stride=4,
            cache_len=A, cu=A, parents=A, ws=A, ws_bytes=1 << 40, stream=None)


@pytest.mark.parametrize("desc,kw,want", [
    (dict(B=0), {}, "MIS_ERR_INVALID_ARG"), (dict(T=-1), {}, "MIS_ERR_INVALID_ARG"),
    (dict(Hq=0), {}, "MIS_ERR_INVALID_ARG"), (dict(Hq=3), {}, "MIS_ERR_SHAPE"),
    (dict(max_nodes=0), {}, "MIS_ERR_INVALID_ARG"), (dict(max_nodes=257), {}, "MIS_ERR_UNSUPPORTED"),
    (dict(Hq=2 * 129), dict(qs=2 * 129 * 64, os=2 * 129 * 64), "MIS_ERR_UNSUPPORTED"),
    (dict(B=1 << 20), dict(max_pages=1 << 20, stride=1 << 20), "MIS_ERR_UNSUPPORTED"),   # steps pass 32 bits
    (dict(scale=float("inf")), {}, "MIS_ERR_INVALID_ARG"), (dict(scale=float("nan")), {}, "MIS_ERR_INVALID_ARG"),
    (dict(scale=1e-30), {}, "MIS_ERR_INVALID_ARG"),
    ({}, dict(q=None), "MIS_ERR_INVALID_ARG"), ({}, dict(o=A + 8), "MIS_ERR_INVALID_ARG"),
    ({}, dict(lse=A + 2), "MIS_ERR_INVALID_ARG"), ({}, dict(qs=248), "MIS_ERR_SHAPE"),
    ({}, dict(ks=132), "MIS_ERR_SHAPE"), ({}, dict(table=None), "MIS_ERR_INVALID_ARG"),
    ({}, dict(max_pages=0), "MIS_ERR_INVALID_ARG"), ({}, dict(stride=3), "MIS_ERR_SHAPE"),
    ({}, dict(max_pages=1 << 28, stride=1 << 28), "MIS_ERR_SHAPE"),
    ({}, dict(cache_len=None), "MIS_ERR_INVALID_ARG"), ({}, dict(cu=A + 1), "MIS_ERR_INVALID_ARG"),
    ({}, dict(parents=A + 2), "MIS_ERR_INVALID_ARG"), ({}, dict(ws=None), "MIS_ERR_WORKSPACE"),
    ({}, dict(ws=A + 128), "MIS_ERR_WORKSPACE"), ({}, dict(ws_bytes=8), "MIS_ERR_WORKSPACE")])
def test_tree_attention_refusals(L, desc, kw, want):
    d = dict(B=2, T=8, Hq=4, max_nodes=4, scale=0.0)
    d.update(desc)
    a = dict(TREE)
    a.update(kw)
    c = _cache()
    st = L.mis_tree_attention_fwd(C.byref(lib.mis_tree_desc(*d.values())), C.byref(c), *a.values())
    assert lib.STATUS[st] == want


def test_null_descriptors(L):
    c, d = _cache(), lib.mis_tree_desc(1, 1, 2, 1, 0.0)
    for dp, cp in ((None, C.byref(c)), (C.byref(d), None)):
        assert L.mis_tree_attention_workspace_size(dp, cp) == 0
        assert L.mis_tree_attention_fwd(dp, cp, *TREE.values()) == lib.MIS_ERR_INVALID_ARG
    assert L.mis_paged_write_kv(None, *WRITE.values()) == lib.MIS_ERR_INVALID_ARG
    assert L.mis_paged_extend_workspace_size(0) == 0


def test_status_string_of_the_page_list():
    assert lib.mis_status_string(lib.MIS_ERR_DEVICE_PAGES) != "unknown status"


def test_python_calls_refuse_tensors_off_the_gpu():
    import torch
    kv = torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16)
    if torch.cuda.is_available():
        pytest.skip("host tensors are refused by the device check either way")
    with pytest.raises(lib.MisError):
        lib.PagedCache(kv.float(), kv.float())
