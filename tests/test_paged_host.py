"""The binding's paged calls refuse host tensors, with and without a GPU."""
import pytest

torch = pytest.importorskip("torch")

from ranking_prefill_gb300 import lib  # noqa: E402

BF16, I32 = torch.bfloat16, torch.int32


def refused(f, *a, **kw):
    with pytest.raises(lib.MisError) as e:
        f(*a, **kw)
    assert e.value.status == lib.MIS_ERR_INVALID_ARG


def test_cache_of_host_tensors():
    kv = torch.zeros(2, 16, 2, 64, dtype=BF16)
    refused(lib.PagedCache, kv, kv.clone())


def test_calls_on_host_tensors():
    i = lambda n: torch.zeros(n, dtype=I32)  # noqa: E731
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    refused(lib.mis_paged_extend, i(2), i(2), i(2), torch.zeros(2, 4, dtype=I32), i(9), i(1), i(1), i(3), i(8), i(8),
            16, 9, ws)

    class Cache:                                             # as PagedCache on the current device, made-up addresses
        device = torch.cuda.current_device() if torch.cuda.is_available() else -1
        Hkv, D = 2, 64
        desc = lib.mis_paged_cache(1 << 20, 2 << 20, 4, 16, 2, 64, 16 * 128, 128, 64)
        ref = lib.C.byref(desc)

    rows = torch.zeros(4, 2, 64, dtype=BF16)
    refused(lib.mis_paged_write_kv, Cache, rows, rows, i(4), ws)
    desc = lib.TreeDesc(Cache, B=1, T=4, Hq=2, max_nodes=4)
    refused(lib.mis_tree_attention_fwd, desc, rows, rows, rows, torch.zeros_like(rows), None,
            torch.zeros(1, 4, dtype=I32), i(1), i(2), None, ws)
