"""Refusals of the 8-bit cache's calls and of the per-head norms, before any
device work: made-up addresses through the C calls, host tensors through the
binding."""
import ctypes as C
import os

import pytest

torch = pytest.importorskip("torch")

from ranking_prefill_gb300 import lib  # noqa: E402

MB = 1 << 20
ARG, SHAPE, UNSUP, WS = lib.MIS_ERR_INVALID_ARG, lib.MIS_ERR_SHAPE, lib.MIS_ERR_UNSUPPORTED, lib.MIS_ERR_WORKSPACE


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(lib.LIB_PATH):
        from ranking_prefill_gb300 import build
        build.build()
    return lib.load()


# 10 pages of 16 rows, 2 heads of 64: 20480 bytes of codes each, 320 exponents
CACHE = dict(k=64 * MB, v=65 * MB, k_exp=66 * MB, v_exp=67 * MB, n_pages=10, page_size=16, Hkv=2, D=64,
             page_stride=16 * 128, row_stride=128, head_stride=64)
LAYOUTS = {"rows": {}, "heads": dict(head_stride=16 * 64, row_stride=64), "apart": dict(page_stride=3 * 16 * 128),
           "pages inside": dict(page_stride=128, row_stride=1280),
           "k and v in one": dict(row_stride=256, page_stride=16 * 256, head_stride=128, v=64 * MB + 64)}
BAD_CACHES = [
    (dict(k=0), ARG), (dict(v=0), ARG), (dict(k_exp=0), ARG), (dict(v_exp=0), ARG), (dict(k=64 * MB + 8), ARG),
    (dict(v_exp=67 * MB + 4), ARG), (dict(n_pages=0), ARG), (dict(Hkv=0), ARG), (dict(page_size=24), UNSUP),
    (dict(page_size=8), UNSUP), (dict(page_size=512), UNSUP), (dict(D=96), UNSUP), (dict(D=256), UNSUP),
    (dict(row_stride=120), SHAPE), (dict(row_stride=136), SHAPE), (dict(head_stride=32), SHAPE),
    (dict(page_stride=15 * 128), SHAPE), (dict(row_stride=-128), SHAPE), (dict(n_pages=1 << 27), SHAPE),
    (dict(page_stride=1 << 40), SHAPE)]


def cache(**kw):
    d = dict(CACHE)
    d.update(kw)
    return lib.mis_paged_cache_q8(*[d[f] for f, _ in lib.mis_paged_cache_q8._fields_])


WRITE = dict(k=MB, v=2 * MB, ks=128, vs=160, T=4, src=3 * MB, slot=4 * MB, n=4, pos=5 * MB, base=1e6, kw=7 * MB, eps=1e-6,
             ws=6 * MB, ws_bytes=256, stream=None)
READ = dict(slot=4 * MB, n=4, k=MB, v=2 * MB, ks=128, vs=160, ws=6 * MB, ws_bytes=256, stream=None)
ATTN = dict(q=MB, o=2 * MB, lse=3 * MB, qs=256, os=256, table=4 * MB, max_pages=4, stride=4, cache_len=5 * MB, cu=6 * MB,
            ws=128 * MB, ws_bytes=1 << 40, stream=None)
DESC = dict(B=2, T=8, Hq=4, max_rows=4, scale=0.0)
NORM = dict(q=MB, k=2 * MB, qo=3 * MB, ko=4 * MB, qs=256, ks=128, qos=256, kos=128, T=8, Hq=4, Hkv=2, D=64, qw=5 * MB,
            kw=6 * MB, eps=1e-6, pos=7 * MB, base=1e6, stream=None)


def write(L, c=None, **kw):
    return L.mis_paged_write_kv_q8(C.byref(c or cache()), *dict(WRITE, **kw).values())


def read(L, c=None, **kw):
    return L.mis_paged_read_kv_q8(C.byref(c or cache()), *dict(READ, **kw).values())


def attn(L, c=None, d=None, **kw):
    d = lib.mis_paged_attn_desc(*dict(DESC, **(d or {})).values())
    return L.mis_paged_attention_q8_fwd(C.byref(d), C.byref(c or cache()), *dict(ATTN, **kw).values())


def norm(L, **kw):
    return L.mis_qk_norm_rope(*dict(NORM, **kw).values())


@pytest.mark.parametrize("kw,st", BAD_CACHES)
def test_caches(L, kw, st):
    for f in (write, read, attn):
        assert f(L, cache(**kw)) == st
    assert L.mis_paged_write_kv_q8(None, *WRITE.values()) == ARG
    assert L.mis_paged_attention_q8_workspace_size(C.byref(lib.mis_paged_attn_desc(*DESC.values())),
                                                   C.byref(cache(**kw))) == 0


@pytest.mark.parametrize("kw,st", [
    (dict(T=-1), ARG), (dict(n=-1), ARG), (dict(base=1.0), ARG), (dict(base=float("nan")), ARG), (dict(base=float("inf")), ARG),
    (dict(eps=-1e-6), ARG), (dict(eps=float("nan")), ARG), (dict(eps=2.0), ARG), (dict(ws=0), WS), (dict(ws=6 * MB + 128), WS),
    (dict(ws_bytes=255), WS), (dict(src=0, n=5), SHAPE), (dict(ks=120), SHAPE), (dict(vs=130), SHAPE), (dict(slot=0), ARG),
    (dict(slot=4 * MB + 2), ARG), (dict(src=3 * MB + 1), ARG), (dict(pos=5 * MB + 3), ARG), (dict(k=0), ARG), (dict(v=0), ARG),
    (dict(k=MB + 8), ARG), (dict(kw=7 * MB + 2), ARG),
    # overlaps
    (dict(k=CACHE["k"] + 1024), ARG), (dict(v=CACHE["v"] - 512), ARG), (dict(slot=CACHE["k_exp"] + 316), ARG),
    (dict(pos=CACHE["v_exp"]), ARG), (dict(src=6 * MB + 252), ARG), (dict(kw=CACHE["k"] + 20480 - 16), ARG),
    (dict(ws=65 * MB), ARG), (dict(ws=66 * MB), ARG), (dict(ws=7 * MB), ARG)])
def test_writes(L, kw, st):
    assert write(L, **kw) == st


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("at", [0, 64 * 128, 20480 - 16])
def test_writes_over_any_cache(L, layout, at):
    for buffer in ("k", "v"):
        for name in ("k", "v", "slot", "src", "pos", "kw"):
            c = dict(CACHE, **LAYOUTS[layout])
            off = at // 2048 * 6144 + at % 2048 if layout == "apart" else at
            assert write(L, cache(**LAYOUTS[layout]), **{name: c[buffer] + off}) == ARG


@pytest.mark.parametrize("kw", [
    dict(v=64 * MB), dict(v=64 * MB + 20480 - 64), dict(v=64 * MB - 20480 + 16), dict(k_exp=64 * MB), dict(v_exp=66 * MB + 16),
    dict(k_exp=65 * MB + 20480 - 16), dict(v_exp=65 * MB - 304), dict(LAYOUTS["k and v in one"], v=64 * MB + 48),
    dict(LAYOUTS["k and v in one"], v=64 * MB + 128), dict(LAYOUTS["k and v in one"], v=64 * MB + 80),
    dict(LAYOUTS["k and v in one"], v=64 * MB + 256 * 3 - 64 + 16)])
def test_caches_over_themselves(L, kw):
    assert write(L, cache(**kw)) == ARG


@pytest.mark.parametrize("kw,st", [
    (dict(n=-1), ARG), (dict(ws=0), WS), (dict(ws_bytes=10), WS), (dict(ks=127), SHAPE), (dict(vs=132), SHAPE), (dict(slot=0), ARG),
    (dict(slot=4 * MB + 1), ARG), (dict(k=0), ARG), (dict(v=0), ARG), (dict(v=2 * MB + 4), ARG), (dict(k=2 * MB), ARG),
    (dict(k=CACHE["k"]), ARG), (dict(v=CACHE["v_exp"] + 304), ARG), (dict(k=4 * MB - 1008), ARG), (dict(ws=MB), ARG),
    (dict(k=MB, v=MB + 128, ks=256, vs=256), ARG)])
def test_reads(L, kw, st):
    assert read(L, **kw) == st


@pytest.mark.parametrize("d,st", [
    (dict(B=0), ARG), (dict(T=-1), ARG), (dict(Hq=0), ARG), (dict(max_rows=0), ARG), (dict(max_rows=257), UNSUP), (dict(Hq=3), SHAPE),
    (dict(Hq=258), UNSUP), (dict(scale=1e21), ARG), (dict(scale=1e-21), ARG), (dict(scale=float("nan")), ARG)])
def test_attention_sizes(L, d, st):
    assert attn(L, d=d) == st
    assert L.mis_paged_attention_q8_workspace_size(C.byref(lib.mis_paged_attn_desc(*dict(DESC, **d).values())),
                                                   C.byref(cache())) == 0


@pytest.mark.parametrize("kw,st", [
    (dict(max_pages=0), ARG), (dict(max_pages=1 << 27, stride=1 << 27), SHAPE), (dict(stride=3), SHAPE), (dict(table=0), ARG),
    (dict(cache_len=0), ARG), (dict(cu=0), ARG), (dict(table=4 * MB + 2), ARG), (dict(cache_len=5 * MB + 1), ARG),
    (dict(cu=6 * MB + 2), ARG), (dict(lse=3 * MB + 2), ARG), (dict(qs=248), SHAPE), (dict(os=248), SHAPE), (dict(qs=260), SHAPE),
    (dict(q=0), ARG), (dict(o=0), ARG), (dict(q=MB + 8), ARG), (dict(o=2 * MB + 8), ARG), (dict(ws=0), WS), (dict(ws=128 * MB + 64), WS),
    (dict(ws_bytes=1000), WS),
    # overlaps: 8 rows of q and o 4096 bytes, lse 128, table 32, cu 12
    (dict(o=MB), ARG), (dict(o=MB + 4080), ARG), (dict(o=CACHE["k"]), ARG), (dict(o=CACHE["v"] + 20480 - 16), ARG),
    (dict(o=CACHE["k_exp"] + 304), ARG), (dict(o=4 * MB - 4080), ARG), (dict(o=5 * MB), ARG), (dict(o=6 * MB - 4064), ARG),
    (dict(lse=MB + 4092), ARG), (dict(lse=2 * MB + 100), ARG), (dict(lse=CACHE["v_exp"] - 4), ARG), (dict(lse=6 * MB + 8), ARG),
    (dict(ws=MB), ARG), (dict(ws=2 * MB), ARG), (dict(ws=64 * MB), ARG), (dict(q=128 * MB + 1024), ARG),
    (dict(q=MB, o=MB + 2 * 192, qs=640, os=640), ARG), (dict(q=MB, o=MB + 512, qs=1024, os=2048), ARG)])
def test_attention(L, kw, st):
    assert attn(L, **kw) == st


def test_attention_of_more_steps_than_are_counted(L):
    """(16-row pages: 2^27 - 16 of them make 16,777,214 steps of 128 rows, which count 5 each.)"""
    pages = (0x7fffff00 // 16)
    kw = dict(max_pages=pages, stride=pages, table=1 << 44)
    assert attn(L, d=dict(B=13), **kw) == UNSUP            # 13 requests x 2 kv heads
    assert attn(L, d=dict(B=13), **dict(kw, max_pages=pages + 16, stride=pages + 16)) == SHAPE


@pytest.mark.parametrize("kw,st", [
    (dict(T=-1), ARG), (dict(Hq=-1), ARG), (dict(Hq=0, Hkv=0), ARG), (dict(D=32), UNSUP), (dict(Hq=65537, qs=1 << 23, qos=1 << 23), UNSUP),
    (dict(eps=-1.0), ARG), (dict(eps=float("nan")), ARG), (dict(base=0.5), ARG), (dict(base=float("inf")), ARG), (dict(qs=248), SHAPE),
    (dict(qos=260), SHAPE), (dict(ks=64), SHAPE), (dict(kos=132), SHAPE), (dict(q=0), ARG), (dict(ko=0), ARG), (dict(q=MB + 2), ARG),
    (dict(qw=5 * MB + 8), ARG), (dict(pos=7 * MB + 2), ARG),
    # overlaps: q 4096 bytes, k 2048, weights 128, positions 32
    (dict(qo=MB + 16), ARG), (dict(qo=MB, qos=512), ARG), (dict(qo=2 * MB), ARG), (dict(ko=MB), ARG), (dict(ko=3 * MB + 4080), ARG),
    (dict(qo=5 * MB), ARG), (dict(ko=7 * MB - 2032), ARG), (dict(ko=2 * MB + 128), ARG)])
def test_norms(L, kw, st):
    assert norm(L, **kw) == st


def test_calls_of_no_rows(L):
    assert write(L, n=0, slot=0, k=0, v=0) == lib.MIS_OK
    assert read(L, n=0, slot=0, k=0, v=0) == lib.MIS_OK
    assert norm(L, T=0, q=0, k=0, qo=0, ko=0) == lib.MIS_OK


# ------------------------------------------------------------------ host tensors

def refused(f, *a, **kw):
    with pytest.raises(lib.MisError) as e:
        f(*a, **kw)
    assert e.value.status == ARG


def test_host_tensors():
    i = lambda n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    codes, exps = torch.zeros(2, 16, 2, 64, dtype=torch.uint8), torch.zeros(2, 2, 16, dtype=torch.uint8)
    refused(lib.PagedCacheQ8, codes, codes.clone(), exps, exps.clone())
    ws, rows = torch.zeros(1 << 20, dtype=torch.uint8), torch.zeros(4, 2, 64, dtype=torch.bfloat16)

    class Cache:                                              # as PagedCacheQ8 on the current device, made-up addresses
        device = torch.cuda.current_device() if torch.cuda.is_available() else -1
        Hkv, D = 2, 64
        desc = cache()
        ref = C.byref(desc)

    refused(lib.mis_paged_write_kv_q8, Cache, rows, rows, i(4), ws)
    refused(lib.mis_paged_read_kv_q8, Cache, i(4), rows, rows.clone(), ws)
    desc = lib.PagedAttentionDesc(Cache, B=1, T=4, Hq=2, max_rows=4)
    refused(lib.mis_paged_attention_q8_fwd, desc, rows, torch.zeros_like(rows), None, torch.zeros(1, 4, dtype=torch.int32),
            i(1), i(2), ws)
    refused(lib.mis_qk_norm_rope, rows, rows, rows, rows, i(4))
    refused(lib.mis_qk_norm_rope, None, None, None, None)
    refused(lib.mis_qk_norm_rope, rows, None, None, None)


def test_workspace_size_gives_the_reason():
    class Cache:
        desc = cache()
        ref = C.byref(desc)
    for d, st in ((dict(max_rows=300), UNSUP), (dict(Hq=5), SHAPE), (dict(B=0), ARG)):
        with pytest.raises(lib.MisError) as e:
            lib.PagedAttentionDesc(Cache, **dict(DESC, **d)).workspace_size()
        assert e.value.status == st
