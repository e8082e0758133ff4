"""Paged-cache operators on the GPU against the fp64 oracle: block tables and
slot maps, K/V rows stored at slots, attention of drafted token trees, and a
run of the three together.

Tolerances (rounding to nearest is off by at most half a step: bf16 2^-8, fp32
2^-24, relative):
  * o: the probabilities are rounded to bf16 before the second product, which
    moves o by at most 2^-8 * a, a = sum_j p_j |v_j|; the result's own rounding
    adds 2^-8 |o|. What is left (fp32 scores: see lse; exp2 and sums) moves the
    probabilities by well under 2^-12 relatively: (2^-8 + 2^-12) a + 2^-8 (1 +
    2^-8) |o|, plus the smallest normal step of bf16.
  * lse: a dot product of D terms in fp32, in any order and with truncated
    partial sums, is off by at most 2 D 2^-24 sum |q k|, i.e. 2 D 2^-24 z with z
    = max_j scale sum |q k_j|; scaling, maximum, exp2 and log2 add a few 2^-24
    of the score's size: 2^-20 (1 + |lse| + z).
  * rotated K: half a bf16 step of the result, and 2^-19 (|x| + |y|) for the
    angle's fp32 rounding (pi 2^-24) and the sine's and cosine's 2^-21.
"""
import numpy as np
import pytest
import torch

from oracle import paged_oracle as P
from ranking_prefill_gb300 import lib, synth
from gpu_helpers import f64

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def i32(a):
    return torch.as_tensor(np.asarray(a, np.int32), device="cuda")


def randn(seed, *shape):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(BF16).cuda()


def workspace(n):
    return torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda")      # no call relies on its contents


# ------------------------------------------------------------------- extend

class Extend:
    """One mis_paged_extend call and its oracle."""

    def __init__(self, new_len, cache_len, page_size, max_pages, T, n_pages=None, free=None, head=0,
                 seed=0, pad=0):
        rng = np.random.default_rng(seed)
        self.new, self.len, self.ps, self.T = np.asarray(new_len), np.asarray(cache_len), page_size, T
        B = len(self.new)
        have = np.clip(-(-np.maximum(self.len, 0) // page_size), 0, max_pages)
        total = int(have.sum() + (self.new.clip(0, 1 << 20) // page_size + 2).sum()) + 10
        self.n_pages = n_pages or total
        order = rng.permutation(self.n_pages)
        self.table = np.full((B, max_pages), -7, np.int64)
        at = 0
        for b in range(B):
            self.table[b, :have[b]] = order[at:at + have[b]]
            at += have[b]
        self.free = order[at:] if free is None else np.asarray(free)
        self.head = head
        wide = torch.full((B, max_pages + pad), -9, dtype=torch.int32, device="cuda")
        wide[:, :max_pages] = i32(self.table)
        self.wide, self.d_table = wide, wide[:, :max_pages]
        self.d_new, self.d_len = i32(self.new), i32(self.len)
        self.d_free, self.d_head = i32(self.free), i32([head])
        self.d_len_out, self.d_head_out = torch.empty_like(self.d_len), torch.empty_like(self.d_head)
        self.d_cu = i32(np.full(B + 1, -5))
        self.d_slot, self.d_pos = i32(np.full(T, -5)), i32(np.full(T, -5))
        self.ws = workspace(lib.mis_paged_extend_workspace_size(B))

    def oracle(self):
        return P.extend(self.new, self.len, self.table, self.free, self.head, self.ps, self.n_pages, self.T)

    def call(self, in_place=False, positions=True):
        lib.mis_paged_extend(self.d_new, self.d_len, self.d_len if in_place else self.d_len_out,
                             self.d_table, self.d_free, self.d_head,
                             self.d_head if in_place else self.d_head_out, self.d_cu, self.d_slot,
                             self.d_pos if positions else None, self.ps, self.n_pages, self.ws)

    def check(self, in_place=False, positions=True):
        want = self.oracle()
        before = self.wide.clone()
        self.call(in_place, positions)
        st = lib.mis_get_device_status(self.ws)
        assert st == (lib.MIS_ERR_DEVICE_INDEX if want["bad_index"] else
                      lib.MIS_ERR_DEVICE_PAGES if want["out_of_pages"] else lib.MIS_OK)
        got = dict(table=self.d_table, cu_new=self.d_cu, slot_map=self.d_slot,
                   cache_len=self.d_len if in_place else self.d_len_out)
        if positions:
            got["position_ids"] = self.d_pos
        for name, t in got.items():
            assert np.array_equal(t.cpu().numpy(), want[name]), name
        assert int(self.d_head if in_place else self.d_head_out) == want["free_head"]
        if self.wide.shape[1] > self.d_table.shape[1]:
            n = self.d_table.shape[1]
            assert torch.equal(self.wide[:, n:], before[:, n:])
        return want


@pytest.mark.parametrize("B,ps,len_hi,new_hi,spare,pad", [
    (1, 16, 0, 1, 0, 0), (1, 256, 1000, 5, 3, 0), (5, 32, 100, 1, 2, 5), (33, 64, 700, 300, 1, 3),
    (257, 16, 2000, 90, 40, 0), (1025, 128, 300, 3, 0, 1), (3000, 16, 50, 20, 11, 0)])
@pytest.mark.parametrize("in_place", [False, True])
def test_extend_matches_a_host_allocator(B, ps, len_hi, new_hi, spare, pad, in_place):
    rng = np.random.default_rng(B + ps)
    lens, new = rng.integers(0, len_hi + 1, B), rng.integers(0, new_hi + 1, B)
    if B > 4:
        lens[:4] = [0, min(ps - 1, len_hi), min(ps, len_hi), min(ps + 1, len_hi)]
        new[1] = 1
    max_pages = int(-(-(lens + new) // ps).max()) + 2
    e = Extend(new, lens, ps, max_pages, int(new.sum()) + spare, seed=B, pad=pad)
    e.check(in_place=in_place, positions=B != 33)


def test_extend_large_prompts():
    lens = [0, 5, 70000]
    new = [60000, 131, 9000]
    Extend(new, lens, 64, 1300, sum(new) + 1000).check()


def test_extend_without_rows_or_requests_rows():
    Extend([0, 0], [17, 0], 16, 4, 0).check(positions=False)
    Extend([0, 0], [17, 0], 16, 4, 5).check()


@pytest.mark.parametrize("n_free", [0, 1, 3, 4])
def test_extend_out_of_pages_serves_the_others(n_free):
    # needs: 1, 0, 2, 0, 1 pages; those without need are served whatever is left
    e = Extend([16, 3, 20, 1, 5], [0, 10, 16, 0 + 31, 0], 16, 6, 60, n_pages=40,
               free=list(range(20, 20 + n_free)))
    want = e.check()
    assert want["out_of_pages"] == (n_free < 4)


def test_extend_continues_at_the_head_in_place():
    e = Extend([1, 1], [16, 31], 16, 5, 2, head=0, seed=3)
    for step in range(20):
        want = e.oracle()
        e.call(in_place=True)
        assert lib.mis_get_device_status(e.ws) == lib.MIS_OK
        assert np.array_equal(e.d_slot.cpu().numpy(), want["slot_map"])
        e.table, e.len, e.head = want["table"], want["cache_len"], want["free_head"]
    assert e.d_len.tolist() == [36, 51] and e.head == 4     # 1 -> 3 pages and 2 -> 4


@pytest.mark.parametrize("kind", ["negative length", "negative new", "row of the table", "rows", "head",
                                  "page id", "old page id"])
def test_extend_bad_device_values(kind):
    new, lens, T, head, free = [5, 20, 1], [3, 16, 30], 26, 0, [30, 31, 32, 33, 34, 35]
    if kind == "negative length":
        lens[1] = -4
    if kind == "negative new":
        new[0] = -1
    if kind == "row of the table":
        new[1] = 4 * 16 - 16 + 1
        T = 60
    if kind == "rows":
        T = 25
    if kind == "head":
        head = 7
    if kind == "page id":
        free[0] = 99
    e = Extend(new, lens, 16, 4, T, n_pages=40, free=free, head=head)
    if kind == "old page id":
        e.table[0, 0] = 40
        e.d_table[0, 0] = 40
    want = e.check()
    assert want["bad_index"]
    # the next clean call on the same workspace reads MIS_OK
    f = Extend([1, 2, 3], [3, 16, 30], 16, 4, 6, n_pages=40)
    f.ws = e.ws
    f.check()


def test_extend_captured_and_replayed_in_place():
    lens = np.array([0, 15, 40, 100])
    e = Extend([1, 1, 1, 1], lens, 16, 9, 6, seed=8)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        e.call(in_place=True)                        # a first step outside the capture
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        e.call(in_place=True)
    want = e.oracle()
    for new in ([1, 1, 1, 1], [0, 2, 1, 3], [5, 0, 0, 1], [1, 1, 1, 1]):
        e.table, e.len, e.head = want["table"], want["cache_len"], want["free_head"]
        e.new = np.array(new)
        e.d_new.copy_(i32(new))
        want = e.oracle()
        g.replay()
        torch.cuda.synchronize()
        for name, t in (("table", e.d_table), ("cache_len", e.d_len), ("cu_new", e.d_cu),
                        ("slot_map", e.d_slot), ("position_ids", e.d_pos)):
            assert np.array_equal(t.cpu().numpy(), want[name]), name


# -------------------------------------------------------------------- write

def make_cache(pages, ps, H, D, layout="rows", fill=0.0):
    if layout == "rows":
        k, v = (torch.full((pages, ps, H, D), fill, dtype=BF16, device="cuda") for _ in "kv")
    elif layout == "heads":
        k, v = (torch.full((pages, H, ps, D), fill, dtype=BF16, device="cuda").transpose(1, 2) for _ in "kv")
    elif layout == "interleaved":
        kv = torch.full((pages, 2, ps, H, D), fill, dtype=BF16, device="cuda")
        k, v = kv[:, 0], kv[:, 1]
    else:                                                # "wide": gaps between the rows' heads
        k, v = (torch.full((pages, ps, H + 1, D + 8), fill, dtype=BF16, device="cuda")[:, :, :H, :D]
                for _ in "kv")
    return k, v


def place_rows(t, pad):
    n, H, D = t.shape
    if not pad:
        return t.contiguous()
    buf = torch.full((n, H * D + pad), 3.0, dtype=BF16, device="cuda")
    view = buf.as_strided((n, H, D), (H * D + pad, D, 1))
    view.copy_(t)
    return view


def check_write(kc, vc, k, v, slots, src=None, pos=None, base=1e6, status=lib.MIS_OK):
    k0, v0 = f64(kc), f64(vc)
    want_k, want_v = P.write_kv(k0, v0, f64(k), f64(v), slots, src, pos, base)
    ws = workspace(lib.mis_paged_write_workspace_size())
    lib.mis_paged_write_kv(lib.PagedCache(kc, vc), k, v, i32(slots), ws,
                           position_ids=None if pos is None else i32(pos), base=base,
                           src_rows=None if src is None else i32(src))
    assert lib.mis_get_device_status(ws) == status
    got_k, got_v = f64(kc), f64(vc)
    assert np.array_equal(got_v, want_v)
    if pos is None:
        assert np.array_equal(got_k, want_k)
        return
    touched = np.zeros(k0.shape[:2], bool)
    for i, s in enumerate(slots):
        r = i if src is None else src[i]
        if 0 <= s < touched.size and 0 <= r < k.shape[0]:
            touched[s // k0.shape[1], s % k0.shape[1]] = True
    assert np.array_equal(got_k[~touched], want_k[~touched])
    D = k.shape[2]
    sizes = {}
    for i, s in enumerate(slots):
        r = i if src is None else src[i]
        if 0 <= s < touched.size and 0 <= r < k.shape[0]:
            x = np.abs(f64(k[r]))
            sizes[s] = np.concatenate([x[:, :D // 2] + x[:, D // 2:]] * 2, axis=1)
    for s, size in sizes.items():
        g, w = (t[s // k0.shape[1], s % k0.shape[1]] for t in (got_k, want_k))
        # + 2^-134: half of bf16's smallest (subnormal) step
        assert (np.abs(g - w) <= 2.0 ** -8 * np.abs(w) + (2.0 ** -19) * size + 2.0 ** -134).all()


@pytest.mark.parametrize("n,H,D,ps,layout,pad,rope", [
    (1, 1, 64, 16, "rows", 0, True), (7, 2, 128, 32, "heads", 8, True), (33, 3, 64, 64, "interleaved", 0, False),
    (100, 8, 128, 16, "wide", 16, True), (257, 5, 128, 256, "rows", 24, False),
    (640, 4, 64, 128, "heads", 0, True), (2000, 8, 128, 64, "rows", 0, True)])
def test_write_matches_the_oracle(n, H, D, ps, layout, pad, rope):
    rng = np.random.default_rng(n)
    pages = n // ps + 3
    kc, vc = make_cache(pages, ps, H, D, layout, fill=2.0)
    k, v = place_rows(randn(n, n, H, D), pad), place_rows(randn(n + 1, n, H, D), pad)
    slots = rng.permutation(pages * ps)[:n]
    slots[rng.random(n) < 0.1] = -1
    pos = rng.integers(0, 1 << 20, n) if rope else None
    if rope and n > 3:
        pos[:4] = [0, 1, (1 << 31) - 1, 131071]
    check_write(kc, vc, k, v, slots, pos=pos, base=[1e6, 1e4][n % 2])


@pytest.mark.parametrize("n,T,rope", [(1, 1, False), (50, 20, True), (300, 4099, False)])
def test_write_picks_source_rows_with_repeats(n, T, rope):
    rng = np.random.default_rng(n)
    kc, vc = make_cache(12, 32, 2, 64)
    k, v = randn(1, T, 2, 64), randn(2, T, 2, 64)
    slots = rng.permutation(12 * 32)[:n]
    check_write(kc, vc, k, v, slots, src=rng.integers(0, T, n),
                pos=rng.integers(0, 5000, n) if rope else None)


def test_write_bad_slots_and_rows_store_nothing():
    kc, vc = make_cache(4, 16, 2, 128)
    k, v = randn(1, 6, 2, 128), randn(2, 6, 2, 128)
    check_write(kc, vc, k, v, [3, 64, 5, -1, 70000, 63], status=lib.MIS_ERR_DEVICE_INDEX)
    check_write(kc, vc, k, v, [3, 4], src=[6, 0], status=lib.MIS_ERR_DEVICE_INDEX)
    check_write(kc, vc, k, v, [3, 4], src=[-1, 0], status=lib.MIS_ERR_DEVICE_INDEX)
    check_write(kc, vc, k, v, [-1, 4], src=[-1, 0])                 # a skipped row's source is not read
    check_write(kc, vc, k, v, [-5, -1])


def test_write_keeps_nan_infinity_and_signed_zero():
    kc, vc = make_cache(2, 16, 1, 64)
    k = randn(3, 2, 1, 64)
    k[0, 0, :4] = torch.tensor([float("nan"), float("inf"), -float("inf"), -0.0], dtype=BF16)
    ws = workspace(256)
    lib.mis_paged_write_kv(lib.PagedCache(kc, vc), k, k, i32([17, 2]), ws)
    torch.cuda.synchronize()
    assert torch.equal(kc[1, 1].view(torch.int16), k[0].view(torch.int16))
    assert torch.equal(vc[0, 2].view(torch.int16), k[1].view(torch.int16))


def test_write_agrees_with_the_rotary_pass():
    # the same rotation as mis_rope_qk at positions its fp32 angles resolve
    T, H, D = 300, 8, 128
    k, v = randn(5, T, H, D), randn(6, T, H, D)
    pos = i32(np.random.default_rng(0).integers(0, 500, T))
    rk = torch.empty_like(k)
    lib.mis_rope_qk(None, k, None, rk, pos)
    kc, vc = make_cache(10, 32, H, D)
    ws = workspace(256)
    lib.mis_paged_write_kv(lib.PagedCache(kc, vc), k, v, i32(np.arange(T) + 20), ws, position_ids=pos)
    got = kc.view(-1, H, D)[20:20 + T].float()
    # two roundings to bf16 of values that differ by angle errors of 500 * 2^-23
    size = k.float().abs()
    size = torch.cat([size[..., :64] + size[..., 64:]] * 2, -1)
    assert bool(((got - rk.float()).abs() <= 2.0 ** -7 * rk.float().abs() + 1e-4 * size).all())


# ---------------------------------------------------------------- attention

class Tree:
    """A batch of drafted trees over a paged cache, and its call."""

    def __init__(self, lens, nodes, hq, hkv, D, ps, parents=None, seed=0, layout="rows", scale=0.0,
                 pad=0, max_nodes=None, T=None, extra_cols=0, q_scale=1.0):
        rng = np.random.default_rng(seed)
        self.lens, self.nodes = np.asarray(lens), np.asarray(nodes)
        B = len(lens)
        self.cu = np.concatenate([[0], np.cumsum(nodes)]).astype(int)
        self.T = int(self.cu[-1]) if T is None else T
        self.parents = parents
        self.hq, self.hkv, self.D, self.ps, self.scale = hq, hkv, D, ps, scale
        pages = -(-self.lens // ps)
        n_pages = int(pages.sum()) + 2
        order = rng.permutation(n_pages)
        self.table = np.zeros((B, max(int(pages.max()), 1) + extra_cols), int)
        at = 0
        for b in range(B):
            self.table[b, :pages[b]] = order[at:at + pages[b]]
            at += pages[b]
        self.table[:, pages.max():] = -3                 # columns behind the last page are never read
        self.kc, self.vc = make_cache(n_pages, ps, hkv, D, layout)
        self.kc.copy_(randn(seed + 1, n_pages, ps, hkv, D))
        self.vc.copy_(randn(seed + 2, n_pages, ps, hkv, D))
        n = max(self.T, 1)
        self.q = place_rows(randn(seed + 3, n, hq, D) * q_scale, pad)
        self.k, self.v = place_rows(randn(seed + 4, n, hkv, D), pad), place_rows(randn(seed + 5, n, hkv, D), pad)
        self.max_nodes = max_nodes or max(int(self.nodes.max()), 1)

    def prepare(self):
        self.cache = lib.PagedCache(self.kc, self.vc)
        self.desc = lib.TreeDesc(self.cache, B=len(self.lens), T=self.T, Hq=self.hq,
                                 max_nodes=self.max_nodes, scale=self.scale)
        self.ws = workspace(self.desc.workspace_size())
        self.o = torch.full_like(self.q, 7.0)
        self.lse = torch.full((self.hq, self.T), 7.0, dtype=torch.float32, device="cuda")
        self.d_table, self.d_len, self.d_cu = i32(self.table), i32(self.lens), i32(self.cu)
        self.d_parents = None if self.parents is None else i32(self.parents)
        return self

    def call(self, lse=True, stream=None):
        lib.mis_tree_attention_fwd(self.desc, self.q, self.k, self.v, self.o, self.lse if lse else None,
                                   self.d_table, self.d_len, self.d_cu, self.d_parents, self.ws, stream=stream)

    def oracle(self, rows_of=None):
        return P.tree_attention(f64(self.q), f64(self.k), f64(self.v), f64(self.kc), f64(self.vc), self.table,
                                self.lens, self.cu, self.parents, scale=self.scale, rows_of=rows_of)

    def compare(self, want, lse=True):
        o, ls, a, z = want
        live = ~np.isnan(a).all(axis=(1, 2))
        got = f64(self.o)
        tol = (2.0 ** -8 + 2.0 ** -12) * a + 2.0 ** -8 * (1 + 2.0 ** -8) * np.abs(o) + 2.0 ** -126
        if self.T:
            err = np.abs(got[:self.T] - o)[live]
            assert np.isfinite(got[:self.T][live]).all()
            bad = err > tol[live]
            assert not bad.any(), (err[bad].max(), int(bad.sum()))
        if lse:
            gl = f64(self.lse)
            empty = np.isneginf(ls)
            assert np.isneginf(gl[empty]).all()
            fine = np.isfinite(ls)
            lt = 2.0 * self.D * 2.0 ** -24 * z + 2.0 ** -20 * (1 + np.abs(np.where(fine, ls, 0)) + z)
            e = np.abs(gl[fine] - ls[fine])
            assert (e <= lt[fine]).all(), e.max()
        return got

    def check(self, rows_of=None, status=lib.MIS_OK, lse=True):
        self.prepare()
        self.call(lse)
        assert lib.mis_get_device_status(self.ws) == status
        self.compare(self.oracle(rows_of), lse)
        o, ls = self.o.clone(), self.lse.clone()
        self.o.fill_(5.0)
        self.call(lse)
        torch.cuda.synchronize()
        live = np.concatenate([np.arange(self.cu[b], self.cu[b + 1]) for b in range(len(self.lens))]) \
            if rows_of is None else np.zeros(0, int)
        live = torch.as_tensor(live, device="cuda")
        assert torch.equal(o[live], self.o[live]) and torch.equal(ls, self.lse)      # the same bits again
        return self


def random_parents(rng, nodes, unused=0.0, reach=4):
    out = []
    for n in nodes:
        for i in range(n):
            p = -1 if i == 0 else int(rng.integers(max(-1, i - reach), i))
            out.append(-2 if i and rng.random() < unused else p)
    return np.array(out, int)


HEADS = [(16, 8, 128), (32, 8, 128), (4, 2, 64), (12, 4, 64), (6, 6, 128), (8, 1, 128), (20, 4, 128),
         (7, 1, 64), (3, 3, 64), (40, 1, 128), (128, 1, 64), (100, 1, 128)]


@pytest.mark.parametrize("hq,hkv,D", HEADS)
@pytest.mark.parametrize("ps", [16, 64, 256])
def test_single_tokens(hq, hkv, D, ps):
    lens = [0, 1, 15, 16, 17, 127, 128, 129, 255, 256, 300, 1000]
    Tree(lens, [1] * len(lens), hq, hkv, D, ps, seed=hq + ps).check()


@pytest.mark.parametrize("hq,hkv,D", HEADS)
@pytest.mark.parametrize("layout,ps", [("rows", 32), ("heads", 16), ("interleaved", 128), ("wide", 64)])
def test_ragged_trees(hq, hkv, D, layout, ps):
    rng = np.random.default_rng(hq * 7 + ps)
    nodes = [1, 7, 0, 16, 33, 2]
    lens = [130, 0, 77, 5, 384, ps]
    Tree(lens, nodes, hq, hkv, D, ps, random_parents(rng, nodes, 0.1), seed=ps, layout=layout, pad=16,
         extra_cols=2).check()


@pytest.mark.parametrize("hq,hkv,D,nodes", [(16, 8, 128, [64, 1, 63]), (32, 8, 128, [64, 40]), (28, 4, 128, [64, 9]),
                                            (8, 1, 128, [256, 129]), (4, 2, 64, [256, 200, 3]),
                                            (2, 2, 128, [128, 127, 129, 130])])
@pytest.mark.parametrize("chain", [False, True])
def test_large_trees_and_chains(hq, hkv, D, nodes, chain):
    rng = np.random.default_rng(len(nodes))
    par = None if chain else random_parents(rng, nodes, 0.05, reach=30)
    lens = [200, 0, 129, 64][:len(nodes)]
    Tree(lens, nodes, hq, hkv, D, 16, par, seed=nodes[0]).check()


@pytest.mark.parametrize("seed", range(12))
def test_random_batches(seed):
    rng = np.random.default_rng(100 + seed)
    hq, hkv, D = HEADS[rng.integers(len(HEADS))]
    B = int(rng.integers(2, 7))
    nodes = rng.integers(1, int(2 ** rng.uniform(0, 7)) + 2, B)
    lens = rng.integers(0, int(2 ** rng.uniform(2, 11)), B)
    par = None if seed % 3 == 0 else random_parents(rng, nodes, 0.05, reach=20)
    Tree(lens, nodes, hq, hkv, D, int(rng.choice([16, 32, 64, 128, 256])), par, seed=seed,
         layout=["rows", "heads", "interleaved", "wide"][seed % 4], pad=8 * (seed % 3),
         scale=[0.0, 0.3, -0.1][seed % 3]).check()


def test_parents_of_a_chain_equal_no_parents():
    nodes = [5, 1, 40]
    par = np.concatenate([np.arange(-1, n - 1) for n in nodes])
    a = Tree([100, 3, 260], nodes, 8, 2, 128, 32, None, seed=4).check()
    b = Tree([100, 3, 260], nodes, 8, 2, 128, 32, par, seed=4).check()
    assert torch.equal(a.o, b.o) and torch.equal(a.lse, b.lse)


def test_long_cache_of_one_request():
    Tree([20000], [3], 8, 2, 128, 64, seed=1).check()


def test_long_and_short_caches_together():
    lens = [9000, 1, 4000, 0, 130]
    Tree(lens, [2, 1, 5, 3, 1], 4, 2, 64, 128, None, seed=2).check()


def test_many_short_requests():
    rng = np.random.default_rng(5)
    B = 300
    Tree(rng.integers(0, 200, B), rng.integers(0, 4, B), 4, 2, 64, 16, None, seed=3).check()


@pytest.mark.parametrize("scale", [0.02, 1.0, -0.3])
def test_scales_and_large_scores(scale):
    Tree([300, 20], [9, 4], 4, 2, 64, 32, None, seed=6, scale=scale, q_scale=4.0).check()


@pytest.mark.parametrize("hq,hkv,D,n", [(4, 2, 64, 9), (8, 2, 128, 13), (16, 2, 128, 40), (8, 1, 64, 7)])
def test_heads_and_nodes_of_very_different_size(hq, hkv, D, n):
    # rows whose scores differ by hundreds share a tile, and scores that grow along
    # the cache move the reference again and again
    t = Tree([700, 90], [n, 3], hq, hkv, D, 16, None, seed=19, max_nodes=n)
    size = torch.linspace(-4, 7, t.q.shape[0] * hq, device="cuda").exp2().view(t.q.shape[0], hq, 1)
    t.q.copy_((t.q.float() * size).to(BF16))
    grow = torch.linspace(0.2, 3, 700, device="cuda")
    for j in range(700):
        page, off = int(t.table[0, j // 16]), j % 16
        t.kc[page, off] = (t.kc[page, off].float() * grow[j]).to(BF16)
    t.check()


def test_no_lse_and_more_rows_than_requests_have():
    t = Tree([50, 300], [3, 2], 4, 2, 64, 16, None, seed=7, T=11, max_nodes=8)
    t.check(lse=False)
    t.prepare()
    t.call()
    assert bool((t.o[5:] == 7.0).all()) and bool((t.lse[:, 5:] == 7.0).all())
    assert bool((t.o[:5] != 7.0).any())


def test_requests_share_pages():
    t = Tree([64, 64, 40], [2, 1, 3], 4, 2, 128, 16, None, seed=8)
    t.table[1] = t.table[0]
    t.table[2, :2] = t.table[0, :2]
    t.check()


def test_nothing_masked_leaks():
    # NaN and infinities in unused cache rows, in rows of other requests' nodes and in
    # other branches of the tree must not reach a row that does not see them
    nodes = [6, 5]
    par = np.array([-1, 0, 0, 1, 2, -2, -1, 0, 1, 2, -2])
    for D, ps in ((128, 16), (64, 64)):
        t = Tree([37, 130], nodes, 4, 2, D, ps, par, seed=9)
        clean = t.oracle()
        bad = float("nan")
        for b in range(2):
            last = t.table[b, (t.lens[b] - 1) // ps]
            off = (t.lens[b] - 1) % ps + 1
            t.kc[last, off:] = bad
            t.vc[last, off:] = float("inf")
        used = set(t.table[0, :-(-37 // ps)]) | set(t.table[1, :-(-130 // ps)])
        for p in set(range(t.kc.shape[0])) - used:
            t.kc[p], t.vc[p] = float("-inf"), bad
        # node 2's branch (2, 4) of request 0 is poisoned, and the unused node 5 of request 0
        t.k[2], t.v[2, 0], t.v[2, 1] = bad, float("inf"), bad
        t.k[5], t.v[5] = float("inf"), bad
        t.v[4, :, 3] = float("-inf")
        t.prepare()
        t.call()
        assert lib.mis_get_device_status(t.ws) == lib.MIS_OK
        o, ls, a, z = (x.copy() for x in clean)
        poisoned = [2, 4]
        got, gl = f64(t.o), f64(t.lse)
        assert np.isnan(got[poisoned]).all() and np.isnan(gl[:, poisoned]).all()
        for x in (o, a):
            x[poisoned] = np.nan
        ls[:, poisoned] = np.nan
        t.compare((o, ls, a, z))


def test_infinite_values_reach_the_rows_that_see_them():
    par = np.array([-1, 0, 0, 1])
    t = Tree([20], [4], 2, 2, 64, 16, par, seed=10)
    t.v[1, 0, 5] = float("inf")
    t.v[1, 1, 6] = float("-inf")
    t.v[3, 0, 5] = float("-inf")
    t.prepare()
    t.call()
    got = f64(t.o)
    assert got[1, 0, 5] == np.inf and got[1, 1, 6] == -np.inf
    assert np.isnan(got[3, 0, 5]) and got[3, 1, 6] == -np.inf           # inf - inf below node 1
    assert np.isfinite(got[[0, 2]]).all()
    keep = np.ones((4, 2, 64), bool)
    keep[1, 0, 5] = keep[1, 1, 6] = keep[3, 0, 5] = keep[3, 1, 6] = False
    assert np.isfinite(got[keep]).all()


def test_rows_that_see_nothing():
    t = Tree([50, 0], [3, 2], 4, 4, 64, 16, np.array([-2, -1, -2, -2, -1]), seed=11).check()
    got, gl = f64(t.o), f64(t.lse)
    assert (got[[0, 2, 3]] == 0).all() and np.isneginf(gl[:, [0, 2, 3]]).all()


def test_minus_infinity_scores():
    # a row whose every visible score is -inf: o = 0, lse = -inf; one visible key left: that key
    t = Tree([0], [2], 2, 2, 64, 16, None, seed=12)
    t.q[:] = 1.0
    t.k[0] = 0.0
    t.k[0, :, 0] = float("-inf")
    t.prepare()
    t.call()
    got, gl = f64(t.o), f64(t.lse)
    assert (got[0] == 0).all() and np.isneginf(gl[:, 0]).all()
    assert np.allclose(got[1], f64(t.v)[1], rtol=2.0 ** -7, atol=0) and np.isfinite(gl[:, 1]).all()


@pytest.mark.parametrize("kind", ["page", "len", "negative len", "nodes", "cu", "parent"])
def test_bad_device_values_are_reported(kind):
    nodes = [3, 4, 2]
    par = np.array([-1, 0, 0, -1, 0, 1, 2, -1, 0])
    t = Tree([40, 150, 33], nodes, 4, 2, 64, 16, par, seed=13, max_nodes=4)
    skipped = []
    if kind == "page":
        t.table[1, 2], t.table[1, 9] = 10 ** 6, -1
    t.prepare()
    want = list(t.oracle())
    if kind == "len":
        t.d_len[1] = t.table.shape[1] * 16 + 1
        skipped = [1]
    if kind == "negative len":
        t.d_len[0] = -1
        skipped = [0]
    if kind == "nodes":
        t.desc = lib.TreeDesc(t.cache, B=3, T=9, Hq=4, max_nodes=3)
        t.ws = workspace(t.desc.workspace_size())
        skipped = [1]
    if kind == "cu":
        t.d_cu[3] = 10 ** 6
        skipped = [2]
    if kind == "parent":
        t.d_parents[4], t.d_parents[8] = 3, -9           # become roots
        t.parents = par.copy()
        t.parents[4] = t.parents[8] = -1
        want = list(t.oracle())
    t.call()
    assert lib.mis_get_device_status(t.ws) == lib.MIS_ERR_DEVICE_INDEX
    for b in skipped:
        r = slice(t.cu[b], t.cu[b + 1])
        assert bool((t.o[r] == 7.0).all()) and bool((t.lse[:, r] == 7.0).all())
        want[0][r], want[2][r], want[1][:, r] = np.nan, np.nan, np.nan
    t.compare(want)
    # the next clean call on the workspace reads MIS_OK
    u = Tree([40, 150, 33], nodes, 4, 2, 64, 16, par, seed=13, max_nodes=4).prepare()
    if u.ws.numel() <= t.ws.numel():
        u.ws = t.ws
    u.call()
    assert lib.mis_get_device_status(u.ws) == lib.MIS_OK


def test_captured_and_replayed_with_other_lengths():
    nodes, hq, hkv, D, ps = [4, 4, 4], 8, 2, 128, 16
    par = random_parents(np.random.default_rng(0), nodes)
    t = Tree([300, 500, 40], nodes, hq, hkv, D, ps, par, seed=14, max_nodes=8).prepare()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        t.call()
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        t.call()
    for lens, nn in (([300, 500, 40], nodes), ([17, 0, 39], [1, 8, 3]), ([299, 512, 0], [8, 0, 4])):
        t.lens, t.nodes = np.array(lens), np.array(nn)
        t.cu = np.concatenate([[0], np.cumsum(nn)])
        t.parents = np.concatenate([random_parents(np.random.default_rng(1), nn),
                                    np.full(12 - sum(nn), -1)]).astype(int)
        t.d_len.copy_(i32(lens)); t.d_cu.copy_(i32(t.cu)); t.d_parents.copy_(i32(t.parents))
        g.replay()
        torch.cuda.synchronize()
        t.compare(t.oracle())


def test_two_graphs_share_a_workspace_in_turn():
    a = Tree([700, 300], [8, 3], 8, 2, 128, 32, None, seed=20).prepare()
    b = Tree([90, 1000, 3], [20, 5, 1], 16, 2, 128, 16, None, seed=21).prepare()
    shared = torch.empty(max(a.ws.numel(), b.ws.numel()), dtype=torch.uint8, device="cuda").fill_(0x5A)
    graphs = []
    for t in (a, b):
        t.ws = shared
        t.call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            t.call()
        graphs.append(g)
    for _ in range(5):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    a.compare(a.oracle())
    b.compare(b.oracle())


def test_infinite_and_nan_queries_stay_in_their_rows():
    # rows of other requests fill up a tile's columns; whatever they hold, this
    # request's rows come out as without them
    t = Tree([300, 200, 40], [2, 3, 1], 8, 2, 128, 16, None, seed=22).prepare()
    want = t.oracle()
    t.q[2] = float("inf")
    t.q[4, :, ::2] = float("nan")
    t.call()
    assert lib.mis_get_device_status(t.ws) == lib.MIS_OK
    want = [x.copy() for x in want]
    for x in (want[0], want[2]):
        x[[2, 4]] = np.nan
    want[1][:, [2, 4]] = np.nan
    t.compare(want)


def test_nodes_at_the_edges_of_the_last_cache_tile():
    # the new rows share the last cache tile when they fit behind it (from a
    # multiple of 8 rows): both sides of that edge, for a few and for many nodes
    lens, nodes = [], []
    for n in (1, 2, 7, 8, 9, 56, 64):
        for off in (0, 1, 7, 8, 9, 120 - n, 127 - n, 128 - n, 121, 127):
            if off >= 0:
                lens.append(128 + off)
                nodes.append(n)
    for hq, hkv, D in ((2, 2, 64), (4, 1, 128)):
        rng = np.random.default_rng(hq)
        Tree(lens, nodes, hq, hkv, D, 16, random_parents(rng, nodes), seed=23).check()


def test_two_streams_with_their_own_workspaces():
    a = Tree([700, 300], [8, 3], 8, 2, 128, 32, None, seed=15).prepare()
    b = Tree([900, 100], [2, 5], 8, 2, 128, 32, None, seed=16).prepare()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        a.call(stream=sa)
        b.call(stream=sb)
    torch.cuda.synchronize()
    a.compare(a.oracle())
    b.compare(b.oracle())


def test_two_host_threads_with_their_own_workspaces():
    import threading
    trees = [Tree([700, 300], [8, 3], 8, 2, 128, 32, None, seed=40).prepare(),
             Tree([90, 500, 3], [70, 5, 30], 8, 2, 64, 16, None, seed=41).prepare()]
    rows = [(randn(42, 300, 2, 64), randn(43, 300, 2, 64), 1e4), (randn(44, 300, 3, 128), randn(45, 300, 3, 128), 1e6)]
    caches = [make_cache(20, 16, k.shape[1], k.shape[2]) for k, _, _ in rows]
    slots = [np.random.default_rng(i).permutation(320)[:300] for i in range(2)]
    d_slots, pos = [i32(s) for s in slots], i32(np.arange(300) * 7)
    wws = [workspace(256) for _ in range(2)]
    torch.cuda.synchronize()
    failed = []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            cache = lib.PagedCache(*caches[i])
            for _ in range(40):
                trees[i].call(stream=stream)
                lib.mis_paged_write_kv(cache, rows[i][0], rows[i][1], d_slots[i], wws[i], position_ids=pos,
                                       base=rows[i][2], stream=stream)
            stream.synchronize()
        except BaseException as e:                       # reported by the test, not by the thread
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    for i in range(2):
        trees[i].compare(trees[i].oracle())
        k, v, base = rows[i]
        kc, vc = (c.clone() for c in caches[i])
        check_write(kc, vc, k, v, slots[i], pos=np.arange(300) * 7, base=base)       # the same again, alone
        assert torch.equal(kc, caches[i][0]) and torch.equal(vc, caches[i][1])


def test_rows_beyond_32_bit_element_offsets():
    # 2.3M cache rows of 1024 elements: offsets past 2^31 elements (and 2^32 bytes)
    H, D, ps = 8, 128, 64
    n_pages = 36000
    kc = torch.empty(n_pages, ps, H, D, dtype=BF16, device="cuda")
    vc = torch.empty_like(kc)
    L, n = 200, 4
    table = np.array([[35999, 33001, 2, 35500]])
    k, v = randn(20, L + n, H, D), randn(21, L + n, H, D)
    slots = np.concatenate([np.arange(ps) + table[0, c] * ps for c in range(4)])[:L]
    ws = workspace(256)
    cache = lib.PagedCache(kc, vc)
    lib.mis_paged_write_kv(cache, k, v, i32(slots), ws)
    assert lib.mis_get_device_status(ws) == lib.MIS_OK
    q = randn(22, n, 16, D)
    o, lse = torch.empty_like(q), torch.empty(16, n, dtype=torch.float32, device="cuda")
    desc = lib.TreeDesc(cache, B=1, T=n, Hq=16, max_nodes=n)
    tws = workspace(desc.workspace_size())
    lib.mis_tree_attention_fwd(desc, q, k[L:], v[L:], o, lse, i32(table), i32([L]), i32([0, n]), None, tws)
    assert lib.mis_get_device_status(tws) == lib.MIS_OK
    t = Tree([L], [n], 16, H, D, ps)
    pk, pv = np.zeros((4, ps, H, D)), np.zeros((4, ps, H, D))
    pk.reshape(-1, H, D)[:L], pv.reshape(-1, H, D)[:L] = f64(k[:L]), f64(v[:L])
    t.o, t.lse = o, lse
    t.compare(P.tree_attention(f64(q), f64(k[L:]), f64(v[L:]), pk, pv, np.arange(4)[None], [L], [0, n], None))
    del kc, vc, cache, desc
    torch.cuda.empty_cache()


WIDTHS = [(8, 2, 128, [4, 2]), (8, 2, 64, [8, 3]), (16, 8, 128, [32, 5]), (8, 1, 128, [33, 40]),
          (4, 2, 64, [64, 130])]          # 16, 32, 64, 128 and 2 x 128 rows a kv head


@pytest.mark.parametrize("hq,hkv,D,nodes", WIDTHS)
def test_wait_timeout_is_reported_and_the_workspace_survives(hq, hkv, D, nodes):
    par = random_parents(np.random.default_rng(2), nodes)
    t = Tree([300, 20], nodes, hq, hkv, D, 16, par, seed=17).prepare()
    old = lib.mis_set_wait_limit_ns(2_000_000)
    lib.mis_inject_stall(1)
    try:
        t.call()
        torch.cuda.synchronize()
        assert lib.mis_get_device_status(t.ws) == lib.MIS_ERR_DEVICE_TIMEOUT
        assert bool((t.o == 7.0).all())
    finally:
        lib.mis_inject_stall(0)
        lib.mis_set_wait_limit_ns(old)
    t.call()
    assert lib.mis_get_device_status(t.ws) == lib.MIS_OK
    t.compare(t.oracle())


@pytest.mark.parametrize("hq,hkv,D,nodes", WIDTHS)
def test_waits_that_run_out_anywhere_end_the_call(hq, hkv, D, nodes):
    # a limit far below the time of a copy: waits give up in whatever role comes first,
    # and every block still ends
    par = random_parents(np.random.default_rng(3), nodes)
    t = Tree([3000, 700], nodes, hq, hkv, D, 16, par, seed=18).prepare()
    for limit in (0, 300, 1000, 3000, 10000):
        old = lib.mis_set_wait_limit_ns(limit)
        try:
            for _ in range(3):
                t.call()
            torch.cuda.synchronize()
            assert lib.mis_get_device_status(t.ws) in (lib.MIS_OK, lib.MIS_ERR_DEVICE_TIMEOUT)
        finally:
            lib.mis_set_wait_limit_ns(old)
    t.call()
    assert lib.mis_get_device_status(t.ws) == lib.MIS_OK
    t.compare(t.oracle())


def test_python_refusals():
    t = Tree([30], [2], 4, 2, 64, 16, None, seed=18).prepare()
    ok = dict(q=t.q, k=t.k, v=t.v, o=t.o, lse=t.lse, table=t.d_table, n=t.d_len, cu=t.d_cu, par=None, ws=t.ws)
    for bad in (dict(q=t.q.float()), dict(k=t.k.cpu()), dict(o=t.o[:, :2]), dict(lse=t.lse.double()),
                dict(cu=t.d_cu[:1]), dict(n=t.d_len.long()), dict(par=t.d_len[:0]), dict(ws=t.ws[:128]),
                dict(q=t.q.transpose(0, 1).contiguous().transpose(0, 1)), dict(table=t.d_table.t()[:1])):
        a = dict(ok)
        a.update(bad)
        if bad.keys() == {"table"} and t.d_table.shape[1] > 1:
            a["table"] = t.d_table[:0]
        with pytest.raises(lib.MisError):
            lib.mis_tree_attention_fwd(t.desc, *a.values())
    with pytest.raises(lib.MisError):
        lib.PagedCache(t.kc, t.vc.transpose(1, 2))
    with pytest.raises(lib.MisError):
        lib.TreeDesc(t.cache, B=1, T=1, Hq=3, max_nodes=1).workspace_size()


# ----------------------------------------------------- the operators together

def test_python_refuses_outputs_over_inputs():
    t = Tree([40], [3], 2, 2, 64, 16, None, seed=24).prepare()
    for o in (t.q, t.k, t.v):
        with pytest.raises(lib.MisError) as e:
            lib.mis_tree_attention_fwd(t.desc, t.q, t.k, t.v, o, t.lse, t.d_table, t.d_len, t.d_cu, None, t.ws)
        assert e.value.status == lib.MIS_ERR_INVALID_ARG
    rows = t.kc.view(-1, 2, 64)                              # the cache's own rows as the source
    other = torch.zeros_like(rows)
    ws = workspace(256)
    for k, v in ((rows, other), (other, t.vc.view(-1, 2, 64)), (other, rows)):
        with pytest.raises(lib.MisError) as e:
            lib.mis_paged_write_kv(t.cache, k, v, i32([1, 2]), ws)
        assert e.value.status == lib.MIS_ERR_INVALID_ARG


def test_prompt_draft_accept_decode():
    """A serving loop: prompts enter the cache, trees are drafted and attended,
    one path of each is accepted into the cache, then one token is decoded.
    Every step equals attention over the whole rotated history."""
    rng = np.random.default_rng(30)
    hq, hkv, D, ps, base = 8, 2, 128, 16, 1e6
    B, n_pages, max_pages = 3, 64, 12
    kc, vc = make_cache(n_pages, ps, hkv, D, "heads")
    cache = lib.PagedCache(kc, vc)
    free = i32(rng.permutation(n_pages))
    head, lens = i32([0]), i32([0] * B)
    table = torch.full((B, max_pages), -1, dtype=torch.int32, device="cuda")
    ews, wws = workspace(lib.mis_paged_extend_workspace_size(B)), workspace(256)
    hist_k, hist_v = [[] for _ in range(B)], [[] for _ in range(B)]       # unrotated rows, fp64

    def extend(new, T):
        cu, slots, pos = i32([0] * (B + 1)), i32([0] * T), i32([0] * T)
        lib.mis_paged_extend(i32(new), lens, lens, table, free, head, head, cu, slots, pos, ps, n_pages, ews)
        return cu, slots, pos

    def rotated(b):
        x = np.array(hist_k[b])
        return P.rotate(x, np.arange(len(x)), base)

    # prompts, rotated while they are stored
    prompt = [37, 16, 90]
    T = sum(prompt) + 5
    k, v = randn(31, T, hkv, D), randn(32, T, hkv, D)
    cu, slots, pos = extend(prompt, T)
    lib.mis_paged_write_kv(cache, k, v, slots, wws, position_ids=pos, base=base)
    at = 0
    for b, n in enumerate(prompt):
        hist_k[b] += list(f64(k[at:at + n])); hist_v[b] += list(f64(v[at:at + n]))
        at += n
    for step in range(3):
        nodes = [5, 9, 1] if step < 2 else [1, 1, 1]
        par = random_parents(rng, nodes)
        T = sum(nodes)
        q, k, v = randn(40 + step, T, hq, D), randn(50 + step, T, hkv, D), randn(60 + step, T, hkv, D)
        n0 = np.concatenate([[0], np.cumsum(nodes)])
        depth = np.zeros(T, int)
        for b in range(B):
            for i in range(nodes[b]):
                p = par[n0[b] + i]
                depth[n0[b] + i] = 0 if p < 0 else depth[n0[b] + p] + 1
        now = np.array([len(h) for h in hist_k])
        assert lens.tolist() == now.tolist()
        where = np.repeat(now, nodes) + depth
        qr, kr = torch.empty_like(q), torch.empty_like(k)
        lib.mis_rope_qk(q, k, qr, kr, i32(where), base)
        desc = lib.TreeDesc(cache, B=B, T=T, Hq=hq, max_nodes=max(nodes))
        ws = workspace(desc.workspace_size())
        o, lse = torch.empty_like(q), torch.empty(hq, T, dtype=torch.float32, device="cuda")
        lib.mis_tree_attention_fwd(desc, qr, kr, v, o, lse, table, lens, i32(n0), i32(par), ws)
        for w in (ews, wws, ws):
            assert lib.mis_get_device_status(w) == lib.MIS_OK
        got = f64(o)
        accept, src = [], []
        for b in range(B):
            for i in range(nodes[b]):
                path = [i]
                while par[n0[b] + path[0]] >= 0:
                    path.insert(0, int(par[n0[b] + path[0]]))
                rows = [n0[b] + j for j in path]
                kk = np.concatenate([rotated(b), f64(kr)[rows]])
                vv = np.concatenate([np.array(hist_v[b]), f64(v)[rows]])
                for g in range(hq):
                    s = kk[:, g // 4] @ f64(qr)[rows[-1], g] / np.sqrt(D)
                    p = np.exp(s - s.max()); p /= p.sum()
                    w, a = p @ vv[:, g // 4], p @ np.abs(vv[:, g // 4])
                    # as above, and the cached K's rounding to bf16: a score moves by at
                    # most 2^-8 scale sum |q k|, a probability by twice that relatively
                    zz = (np.abs(kk[:, g // 4]) @ np.abs(f64(qr)[rows[-1], g])).max() / np.sqrt(D)
                    tol = (2.0 ** -8 * (1 + 2 * zz) + 2.0 ** -11) * a + 2.0 ** -7 * np.abs(w)
                    assert (np.abs(got[rows[-1], g] - w) <= tol).all()
            last = int(rng.integers(0, nodes[b]))
            path = [last]
            while par[n0[b] + path[0]] >= 0:
                path.insert(0, int(par[n0[b] + path[0]]))
            accept.append(len(path))
            src += [int(n0[b] + j) for j in path]
        pad = 4
        cu, slots, pos = extend(accept, sum(accept) + pad)
        lib.mis_paged_write_kv(cache, kr, v, slots, wws, src_rows=i32(src + [0] * pad))
        assert pos.tolist()[:len(src)] == where[src].tolist()
        j = 0
        for b in range(B):
            for _ in range(accept[b]):
                hist_k[b].append(f64(k[src[j]])); hist_v[b].append(f64(v[src[j]]))
                j += 1
    assert lens.tolist() == [len(h) for h in hist_k]


def test_agrees_with_cached_attention_over_the_same_rows():
    """Items over a cached prefix are chains over a paged cache: both calls
    compute the same rows."""
    hq, hkv, D, ps = 16, 8, 128, 32
    S, item = [300, 77], [[5, 20], [9]]
    cl_lens = [[n + 1 for n in row] for row in item]         # an item set ends with its delimiter
    flat = [n for row in cl_lens for n in row]
    T, cache_T = sum(flat), sum(S)
    q, k, v = randn(70, T, hq, D), randn(71, T, hkv, D), randn(72, T, hkv, D)
    ck, cv = randn(73, cache_T, hkv, D), randn(74, cache_T, hkv, D)
    offs = np.concatenate([[0], np.cumsum(flat)])
    plan = lib.CachedPlan([0, sum(cl_lens[0]), T], [0, 2, 3], offs[:-1], [0, S[0]], S, cache_T, hq, hkv, D)
    pws = torch.zeros(plan.workspace_size(), dtype=torch.uint8, device="cuda")
    plan.create(pws)
    o1 = torch.empty_like(q)
    lib.mis_attention_fwd_cached(plan, q, k, v, ck, cv, o1)
    # the items as three requests; the two of request 0 share its pages
    pages = [-(-s // ps) for s in S]
    kc, vc = make_cache(sum(pages), ps, hkv, D)
    slots = np.concatenate([np.arange(S[0]), np.arange(S[1]) + pages[0] * ps])
    ws = workspace(256)
    cache = lib.PagedCache(kc, vc)
    lib.mis_paged_write_kv(cache, ck, cv, i32(slots), ws)
    table = np.zeros((3, max(pages)), int)
    table[0, :pages[0]] = table[1, :pages[0]] = np.arange(pages[0])
    table[2, :pages[1]] = np.arange(pages[1]) + pages[0]
    desc = lib.TreeDesc(cache, B=3, T=T, Hq=hq, max_nodes=max(flat))
    tws = workspace(desc.workspace_size())
    o2 = torch.empty_like(q)
    lib.mis_tree_attention_fwd(desc, q, k, v, o2, None, i32(table), i32([S[0], S[0], S[1]]), i32(offs), None, tws)
    torch.cuda.synchronize()
    assert lib.mis_get_device_status(tws) == lib.MIS_OK
    # each side is off by at most (2^-8 + 2^-12) a + 2^-8 |o|, and a <= max |v|
    tol = 2 * (2.0 ** -8 + 2.0 ** -12) * float(torch.cat([v, cv]).float().abs().max())
    diff = (o1.float() - o2.float()).abs()
    assert bool((diff <= tol + 2.0 ** -7 * o1.float().abs()).all())
