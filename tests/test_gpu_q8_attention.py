"""Attention of the newest rows over an 8-bit paged cache, against the oracle."""
import threading

import numpy as np
import pytest
import torch

from oracle import q8_oracle as Q
from q8_helpers import Batch, i32
from ranking_prefill_gb300 import lib

pytestmark = pytest.mark.gpu

HEADS = [(16, 8, 128), (4, 1, 64), (3, 3, 128), (12, 4, 64), (8, 1, 128), (10, 2, 128)]


@pytest.mark.parametrize("hq,hkv,D", HEADS)
@pytest.mark.parametrize("page", [16, 64, 256])
def test_decoded_tokens(hq, hkv, D, page):
    lens = [1, 15, 16, 17, 31, 32, 33, 100, 255, 256, 257, 700]
    Batch(lens, [1] * len(lens), hq, hkv, D, page, seed=1).run().check()


@pytest.mark.parametrize("hq,hkv,D", HEADS)
@pytest.mark.parametrize("order", ["rows", "heads", "both"])
def test_chains(hq, hkv, D, order):
    lens, ns = [5, 64, 33, 300, 129, 16, 90], [5, 3, 8, 2, 1, 16, 0]
    Batch(lens, ns, hq, hkv, D, 32, order=order, seed=2).run().check()


# rows a kv head: both sides of the widths of 8 and 16 rows a warp, of the warps that share a unit, of a unit
@pytest.mark.parametrize("G,n", [(8, 1), (3, 3), (4, 4), (17, 1), (16, 2), (3, 11), (4, 16), (13, 5), (64, 1), (32, 4),
                                 (43, 3), (128, 1), (128, 2), (100, 3), (1, 256), (5, 52)])
def test_rows_of_a_kv_head(G, n):
    Batch([n + 70, n, n + 333], [n, n, max(1, n // 2)], 2 * G, 2, 64, 16, seed=G * 1000 + n).run().check()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("hq,hkv,ns", [(8, 4, [1, 2]), (16, 2, [3, 1]), (4, 1, [40, 7])])
def test_long_requests_are_cut_between_blocks(hq, hkv, D, ns):
    Batch([9001, 5003], ns, hq, hkv, D, 64, seed=5).run().check()


def test_many_short_requests():
    r = np.random.default_rng(6)
    lens = r.integers(0, 60, 700)
    ns = np.minimum(lens, r.integers(0, 4, 700))
    Batch(lens, ns, 4, 2, 64, 16, seed=6).run().check()


def test_empty_requests_and_rows_behind_the_last():
    Batch([0, 40, 0, 0, 12, 0], [0, 2, 0, 0, 12, 0], 4, 2, 64, 16, seed=7, extra_T=5).run().check()
    Batch([0, 30], [0, 0], 4, 2, 64, 16, seed=7, extra_T=3).run().check()


def test_strides_of_q_and_o():
    Batch([77, 130], [2, 5], 6, 2, 128, 16, seed=8, pad=64).run().check()


@pytest.mark.parametrize("scale", [-0.2, 1e-4, 3.0])
def test_scales(scale):
    Batch([200, 75], [3, 1], 4, 2, 64, 16, seed=9, scale=scale, spread=0.1).run().check()


def test_no_lse():
    b = Batch([50], [1], 4, 2, 64, seed=10).run().check()
    o = b.o.clone()
    lib.mis_paged_attention_q8_fwd(b.desc, b.dq, b.o, None, b.dt, b.dl, b.dc, b.ws)
    assert torch.equal(o, b.o)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("hkv,ns", [(1, [1, 9]), (2, [1, 1])])
def test_value_scales_far_apart(D, hkv, ns):
    """Rows of large values with small weights beside rows of tiny values with
    large ones: the weighted value counts, not the weight."""
    b = Batch([600, 90], ns, 2 * hkv, hkv, D, 16, seed=11, spread=0.0)
    r = np.random.default_rng(1)
    ve = r.choice([127 - 50, 127 - 20, 127, 127 + 30], b.ve.shape, p=[0.3, 0.3, 0.3, 0.1]).astype(np.uint8)
    b.ve = ve
    b.ke = (b.ke.astype(int) + r.integers(0, 4, b.ke.shape)).astype(np.uint8)
    b.run().check()


def test_exponents_at_their_limits():
    for e in (71, 247):
        b = Batch([100, 33], [1, 2], 4, 2, 64, 16, seed=12, spread=0.0)
        b.ve[:] = e
        b.run().check()
    b = Batch([100, 33], [1, 2], 4, 2, 64, 16, seed=12, spread=0.0)
    b.ke[:] = np.where(np.arange(b.ke.shape[0])[:, None, None] % 2, 0, 71)     # outside counts as the nearest inside
    b.ve[:] = np.where(np.arange(b.ve.shape[0])[:, None, None] % 2, 3, 71)
    b.run().check()


def test_large_scores_move_the_reference_often():
    b = Batch([3000, 500], [2, 1], 4, 2, 128, 16, seed=13, spread=0.0)
    # keys grow along the cache, so the maximum climbs all the way
    for r, l in enumerate(b.lens):
        at = np.arange(l)
        b.ke[b.table[r, at // 16], at % 16] = (120 + at * 9 // l)[:, None]
    b.run().check()


def test_later_rows_do_not_reach_earlier_ones():
    """NaN codes in K or V of a chain's rows: only rows from there on see them."""
    for what in ("kc", "vc"):
        for row in (0, 3, 6):
            for G, D in ((2, 128), (5, 64), (40, 64)):
                b = Batch([50 + row, 7], [7, 7], 2 * G, 2, D, 16, seed=14)
                at = b.lens[0] - 7 + row
                getattr(b, what)[b.table[0, at // 16], at % 16, 1, 3:9] = [0x7F, 0xFF, 0x7F, 0xFF, 0x7F, 0x7F]
                getattr(b, what)[b.table[1, 0], 6, 0, D - 1] = 0xFF
                b.run().check()


def test_nan_deep_in_the_cache_reaches_what_sees_it():
    b = Batch([3000, 200], [1, 4], 4, 2, 64, 16, seed=15)
    b.vc[b.table[0, 60], 3, 1, 5] = 0x7F
    b.kc[b.table[1, 2], 3, 0, 5] = 0x7F
    b.run().check()
    o = b.o[:, :, :].float()
    assert torch.isnan(o[0, 2:, 5]).all() and not torch.isnan(o[0, :2]).any()


def test_a_row_of_q_with_nan_reaches_no_other():
    b = Batch([300, 40], [3, 1], 8, 2, 64, 16, seed=16)
    good = b.run().o.clone()
    b.q[1, 5] = float("nan")
    b.q[1, 6, 3] = float("inf")
    b.run()
    o = b.o
    assert torch.equal(o[0], good[0]) and torch.equal(o[2:], good[2:])
    assert torch.equal(o[1, :5], good[1, :5]) and torch.equal(o[1, 7], good[1, 7])


def test_queries_of_any_size():
    b = Batch([120, 33], [4, 2], 4, 2, 64, 16, seed=17)
    b.q[0] *= 2.0 ** -60
    b.q[1] *= 2.0 ** -130                                      # subnormal
    b.q[2] = 0.0
    b.q[3, 1] = 0.0
    b.q[3, 1, 7] = 40.0
    b.run().check()
    b.q[4] *= 2.0 ** 40
    b.scale = 2.0 ** -42
    b.run().check()


def test_pages_outside_the_cache_hide_their_rows():
    b = Batch([100, 20, 40], [2, 1, 1], 4, 2, 64, 16, seed=18)
    b.table[0, 1], b.table[0, 3] = -1, b.n_pages
    b.table[1, :2] = 10 ** 9
    b.put().call()
    torch.cuda.synchronize()
    assert lib.mis_get_device_status(b.ws) == lib.MIS_ERR_DEVICE_INDEX
    b.check()
    assert (b.o[2] == 0).all() and torch.isneginf(b.lse[:, 2]).all()
    b.call()
    b.dt.copy_(i32(np.where((b.table < 0) | (b.table >= b.n_pages), 0, b.table)))
    b.call()
    assert lib.mis_get_device_status(b.ws) == lib.MIS_OK


@pytest.mark.parametrize("wrong", ["len<n", "len<0", "len>table", "rows>max", "cu<0", "cu>T", "cu decreasing"])
def test_bad_requests_are_skipped(wrong):
    b = Batch([60, 50, 70], [2, 3, 2], 4, 2, 64, 16, seed=19, max_rows=3).put()
    if wrong.startswith("len"):
        b.dl[1] = {"len<n": 2, "len<0": -5, "len>table": 81}[wrong]
        skip = (1,)
    elif wrong == "rows>max":
        b.desc = lib.PagedAttentionDesc(b.c, B=3, T=b.T, Hq=4, max_rows=2)
        skip = (1,)
    elif wrong == "cu<0":
        b.dc[0] = -1
        skip = (0,)
    elif wrong == "cu>T":
        b.dc[3] = b.T + 1
        skip = (2,)
    else:
        b.dc[2] = 1
        skip = (1, 2)                                          # [2, 1) and [1, 7): six rows of at most three
    b.call()
    torch.cuda.synchronize()
    assert lib.mis_get_device_status(b.ws) == lib.MIS_ERR_DEVICE_INDEX
    b.check(skip)


def test_same_bits_each_call_and_on_a_dirty_workspace():
    b = Batch([5000, 40, 999], [2, 7, 1], 8, 2, 128, 16, seed=20).run()
    o, l = b.o.clone(), b.lse.clone()
    for fill in (0, 0xFF, 0x7F):
        b.ws.fill_(fill)
        b.o.fill_(3.0)
        b.call()
        assert torch.equal(o, b.o) and torch.equal(l, b.lse)


def test_a_captured_call_serves_other_lengths():
    b = Batch([200, 300], [2, 3], 4, 2, 64, 16, seed=21).put()
    b.call()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lib.mis_paged_attention_q8_fwd(b.desc, b.dq, b.o, b.lse, b.dt, b.dl, b.dc, b.ws)
    for lens, ns in (([200, 300], [2, 3]), ([7, 280], [1, 2]), ([150, 1], [3, 1])):
        b.lens, b.ns = lens, ns
        b.cu = np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)
        b.dl.copy_(i32(lens))
        b.dc.copy_(i32(b.cu))
        b.o.fill_(7.0)
        b.lse.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        assert lib.mis_get_device_status(b.ws) == lib.MIS_OK
        b.check()


def test_two_streams_at_once():
    jobs = [Batch([2000 + 50 * i, 70], [1, 2], 8, 2, 128, 16, seed=30 + i).put() for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(20):
        for b, s in zip(jobs, streams):
            b.call(stream=s)
    torch.cuda.synchronize()
    for b in jobs:
        b.check()


def test_a_stalled_call_ends_and_the_next_one_is_right():
    b = Batch([3000, 40, 700], [1, 3, 2], 8, 2, 128, 16, seed=40).put()
    limit = lib.mis_set_wait_limit_ns(2_000_000)
    try:
        lib.mis_inject_stall(1)
        b.call()
        assert lib.mis_get_device_status(b.ws) == lib.MIS_ERR_DEVICE_TIMEOUT
        assert (b.o == 7).all()
    finally:
        lib.mis_inject_stall(0)
        lib.mis_set_wait_limit_ns(limit)
    b.call()
    assert lib.mis_get_device_status(b.ws) == lib.MIS_OK
    b.check()


@pytest.mark.parametrize("ns", [[1, 3, 2], [9, 2, 12]])
def test_waits_that_run_out_anywhere_end_the_call(ns):
    b = Batch([20000, 40, 3000], ns, 8, 2, 128, 16, seed=41).put()
    # The limit is looked at between two tries, and a try may itself hold for longer
    # than the limit: whether a given wait runs out is the machine's affair. What holds
    # for each call is that it ends, and that one that reports no timeout is right.
    limit = lib.mis_set_wait_limit_ns(0)
    try:
        for ns_ in [0, 100, 300, 500, 700, 900] + list(range(1000, 9000, 500)):
            lib.mis_set_wait_limit_ns(ns_)
            b.call()
            status = lib.mis_get_device_status(b.ws)
            assert status in (lib.MIS_OK, lib.MIS_ERR_DEVICE_TIMEOUT)
            if status == lib.MIS_OK:
                b.check()
    finally:
        lib.mis_set_wait_limit_ns(limit)
    b.call()
    assert lib.mis_get_device_status(b.ws) == lib.MIS_OK
    b.check()


def test_narrow_and_wide_units_in_turn():
    """Units of up to 16 rows take their steps in two streams, wider ones in one:
    the products' places pass from one to the other."""
    r = np.random.default_rng(42)
    for seed in range(6):
        ns = r.choice([1, 2, 3, 4, 5, 6, 7, 8], 9)
        lens = ns + r.integers(0, 1500, 9)
        Batch(lens, ns, 8, 2, int(r.choice([64, 128])), 32, seed=seed, max_rows=8).run().check()


def test_two_captured_graphs_share_a_workspace():
    """Replayed in turn on one stream: a narrow call and a wide one over one workspace."""
    jobs = [Batch([4000, 70], [1, 2], 8, 2, 128, 16, seed=50).put(), Batch([900, 33, 2000], [9, 2, 12], 8, 2, 128, 16, seed=51).put()]
    ws = max((b.ws for b in jobs), key=lambda w: w.numel())
    graphs = []
    for b in jobs:
        b.ws = ws
        b.call()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            b.call()
        graphs.append(g)
    for _ in range(3):
        for b, g in zip(jobs, graphs):
            b.o.fill_(7.0)
            b.lse.fill_(7.0)
            g.replay()
            assert lib.mis_get_device_status(ws) == lib.MIS_OK
            b.check()


def test_two_host_threads():
    jobs = [Batch([1500 + 70 * i, 60], [1 + 4 * i, 2], 8, 2, 64, 16, seed=60 + i).put() for i in range(2)]
    torch.cuda.synchronize()
    failed = []

    def work(b):
        try:
            st = torch.cuda.Stream()
            for _ in range(50):
                b.call(stream=st)
            st.synchronize()
        except Exception as e:                             # noqa: BLE001
            failed.append(e)
    threads = [threading.Thread(target=work, args=(b,)) for b in jobs]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not failed
    for b in jobs:
        b.check()


@pytest.mark.parametrize("ns", [[1, 1, 2], [5, 9, 3]])
def test_requests_share_pages(ns):
    """A common prefix: the first pages of every request are the same ones."""
    b = Batch([700, 500, 360], ns, 8, 2, 128, 32, seed=70)
    b.table[1:, :10] = b.table[0, :10]
    b.run().check()


def random_batch(r, most=4096):
    hkv = int(r.integers(1, 5))
    G = int(r.choice([1, 1, 2, 3, 4, 5, 8, 16, 20]))
    B = int(r.integers(1, 9))
    lens = np.exp(r.uniform(0, np.log(most), B)).astype(int)
    ns = np.minimum(lens, r.integers(0, int(r.choice([2, 5, 17])), B))
    return dict(lens=lens, ns=ns, hq=G * hkv, hkv=hkv, D=int(r.choice([64, 128])),
                page=int(r.choice([16, 32, 64, 128, 256])), order=str(r.choice(["rows", "heads", "both"])),
                pad=int(r.choice([0, 8, 64])), extra_T=int(r.integers(0, 3)), spread=float(r.choice([0.2, 1.0])))


@pytest.mark.parametrize("seed", range(12))
def test_random_batches(seed):
    r = np.random.default_rng(seed + 100)
    c = random_batch(r)
    b = Batch(seed=seed, **c).run().check()
    o = b.o.clone()
    b.call()
    assert torch.equal(o, b.o), c
