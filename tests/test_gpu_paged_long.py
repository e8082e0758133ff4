"""Paged-cache calls at sizes and widths that test_gpu_paged.py does not reach:
stores of more rows than one trip of the index check, requests of 65 to 128 rows
a kv head where waits run out."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import test_gpu_paged as T  # noqa: E402
from ranking_prefill_gb300 import lib  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [4096, 4097, 9001, 20000])
def test_write_finds_bad_indices_anywhere(n):
    rng = np.random.default_rng(n)
    H, D, ps, rows = 1, 64, 64, n + 64
    pages = -(-rows // ps)
    k, v = T.randn(1, n, H, D), T.randn(2, n, H, D)
    good = rng.permutation(pages * ps)[:n]
    T.check_write(*T.make_cache(pages, ps, H, D), k, v, good)
    for at in (0, 255, 256, 4095, 4096, n // 2, n - 1):
        if at >= n:
            continue
        for bad in (pages * ps, (1 << 31) - 1):
            slots = good.copy()
            slots[at] = bad
            T.check_write(*T.make_cache(pages, ps, H, D), k, v, slots, status=lib.MIS_ERR_DEVICE_INDEX)
        src = rng.integers(0, n, n)
        for bad in (n, -1):
            src[at] = bad
            T.check_write(*T.make_cache(pages, ps, H, D), k, v, good, src=src, status=lib.MIS_ERR_DEVICE_INDEX)


WIDTHS = [(8, 2, 128, [20, 32]), (3, 1, 64, [30, 42]), (8, 8, 64, [70, 128])]     # one row tile of 65 to 128 rows


@pytest.mark.parametrize("hq,hkv,D,nodes", WIDTHS)
def test_wait_timeout_is_reported_and_the_workspace_survives(hq, hkv, D, nodes):
    T.test_wait_timeout_is_reported_and_the_workspace_survives(hq, hkv, D, nodes)


@pytest.mark.parametrize("hq,hkv,D,nodes", WIDTHS)
def test_waits_that_run_out_anywhere_end_the_call(hq, hkv, D, nodes):
    T.test_waits_that_run_out_anywhere_end_the_call(hq, hkv, D, nodes)


@pytest.mark.parametrize("hq,hkv,D,nodes", WIDTHS)
@pytest.mark.parametrize("layout,ps", [("heads", 16), ("interleaved", 128)])
def test_one_row_tile(hq, hkv, D, nodes, layout, ps):
    rng = np.random.default_rng(hq)
    nodes = nodes + [1, 9]
    T.Tree([400, 0, 1000, 129], nodes, hq, hkv, D, ps, T.random_parents(rng, nodes, 0.05, reach=9), seed=70,
           layout=layout, pad=8).check()
