"""Tree attention by pairs of row tiles (more than 64 rows a kv head) at small
sizes: the cases of test_gpu_paged.py with a max_nodes that asks for it, and
what only two tiles can get wrong."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import test_gpu_paged as T  # noqa: E402
from ranking_prefill_gb300 import lib  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def wide(monkeypatch):
    class Wide(T.Tree):
        def __init__(self, lens, nodes, hq, hkv, *a, max_nodes=None, **kw):
            low = 64 * hkv // hq + 1                      # the first that has more than 64 rows
            super().__init__(lens, nodes, hq, hkv, *a, max_nodes=max(max_nodes or 1, int(max(nodes)), low), **kw)

    monkeypatch.setattr(T, "Tree", Wide)


HEADS = [(16, 8, 128), (12, 4, 64), (6, 6, 128), (20, 4, 128), (7, 1, 64), (100, 1, 128), (128, 1, 64)]


@pytest.mark.parametrize("hq,hkv,D", HEADS)
@pytest.mark.parametrize("ps", [16, 128])
def test_single_tokens(hq, hkv, D, ps):
    T.test_single_tokens(hq, hkv, D, ps)


@pytest.mark.parametrize("hq,hkv,D", HEADS)
@pytest.mark.parametrize("layout,ps", [("heads", 16), ("interleaved", 256)])
def test_ragged_trees(hq, hkv, D, layout, ps):
    T.test_ragged_trees(hq, hkv, D, layout, ps)


@pytest.mark.parametrize("scale", [0.02, 1.0, -0.3])
def test_scales_and_large_scores(scale):
    T.test_scales_and_large_scores(scale)


@pytest.mark.parametrize("hq,hkv,D,n", [(4, 2, 64, 40), (8, 2, 128, 40), (16, 2, 128, 40), (8, 1, 64, 25)])
def test_heads_and_nodes_of_very_different_size(hq, hkv, D, n):
    T.test_heads_and_nodes_of_very_different_size(hq, hkv, D, n)


@pytest.mark.parametrize("kind", ["page", "len", "negative len", "cu", "parent"])
def test_bad_device_values_are_reported(kind):
    T.test_bad_device_values_are_reported(kind)


@pytest.mark.parametrize("name", [
    "test_parents_of_a_chain_equal_no_parents", "test_long_cache_of_one_request",
    "test_long_and_short_caches_together", "test_many_short_requests",
    "test_no_lse_and_more_rows_than_requests_have", "test_requests_share_pages", "test_nothing_masked_leaks",
    "test_infinite_values_reach_the_rows_that_see_them", "test_rows_that_see_nothing",
    "test_minus_infinity_scores", "test_captured_and_replayed_with_other_lengths",
    "test_two_graphs_share_a_workspace_in_turn", "test_infinite_and_nan_queries_stay_in_their_rows",
    "test_nodes_at_the_edges_of_the_last_cache_tile", "test_two_streams_with_their_own_workspaces"])
def test_as_with_few_rows(name):
    getattr(T, name)()


def ancestors(par, cu):
    """sees[i][j]: node i sees new row j (indices over the batch)."""
    sees = np.zeros((len(par), len(par)), bool)
    for b in range(len(cu) - 1):
        for i in range(cu[b], cu[b + 1]):
            j = i - cu[b]
            if par[i] == -2:
                continue
            while j >= 0 and par[cu[b] + j] != -2:
                sees[i, cu[b] + j] = True
                j = par[cu[b] + j]
    return sees


@pytest.mark.parametrize("hq,hkv,D,nodes,lens", [(4, 2, 128, [100, 9, 128], [37, 130, 0]),
                                                 (6, 2, 64, [60, 85], [300, 96]),
                                                 (10, 2, 128, [52, 51, 25], [128, 5, 260]),
                                                 (4, 1, 64, [200, 256, 1], [70, 0, 129])])
def test_values_of_either_tile_reach_the_rows_that_see_them(hq, hkv, D, nodes, lens):
    rng = np.random.default_rng(hq + D)
    par = T.random_parents(rng, nodes, 0.05, reach=12)
    t = T.Tree(lens, nodes, hq, hkv, D, 16, par, seed=30)
    want = [x.copy() for x in t.oracle()]
    # rows behind the last cached one, in its page, hold NaN and infinities
    for b, n in enumerate(lens):
        if n:
            page, off = t.table[b, (n - 1) // 16], (n - 1) % 16 + 1
            t.kc[page, off:], t.vc[page, off:] = float("nan"), float("-inf")
    sees = ancestors(par, t.cu)
    odd = [j for j in rng.choice(t.T, 7, replace=False)] + [int(t.cu[1]) - 1]
    for j in odd:
        t.v[int(j), 0, int(j) % D] = float("inf")
    t.prepare()
    t.call()
    assert lib.mis_get_device_status(t.ws) == lib.MIS_OK
    got = T.f64(t.o)
    G = hq // hkv
    for j in odd:
        j = int(j)
        rows = np.flatnonzero(sees[:, j])
        assert (got[rows][:, :G, j % D] == np.inf).all()
        want[0][rows, :G, j % D] = np.nan
        got[rows, :G, j % D] = 0.0
    assert np.isfinite(got).all()
    fine = ~np.isnan(want[0])
    a = want[2]
    tol = (2.0 ** -8 + 2.0 ** -12) * a + 2.0 ** -8 * (1 + 2.0 ** -8) * np.abs(want[0]) + 2.0 ** -126
    assert (np.abs(got - want[0])[fine] <= np.broadcast_to(tol, got.shape)[fine]).all()


@pytest.mark.parametrize("hq,hkv,D", [(8, 2, 128), (5, 1, 128), (2, 2, 64)])
def test_units_of_one_tile_of_two_and_of_several_together(hq, hkv, D):
    rng = np.random.default_rng(hq)
    nodes = [3, 256, 0, 33, 64, 1, 200, 129, 32, 65]
    lens = [500, 40, 30, 0, 1000, 128, 2000, 255, 16, 3000]
    T.Tree(lens, nodes, hq, hkv, D, 64, T.random_parents(rng, nodes, 0.03, reach=40), seed=31, pad=8).check()


def test_a_long_cache_split_over_many_blocks():
    t = T.Tree([30000], [64], 4, 1, 128, 128, None, seed=32)
    t.check(rows_of=None)
