"""Per-head norms with rotation, and rows stored into and read from the 8-bit
cache, against the oracle; then the operators together as a server runs them."""
import math

import numpy as np
import pytest
import torch

from oracle import q8_oracle as Q
from q8_helpers import BF16, f64, i32
from ranking_prefill_gb300 import lib

pytestmark = pytest.mark.gpu

BASE, EPS = 1.0e6, 1.0e-6
FAR = [0, 1, 2, 3, 100, 4095, 131071, 1 << 20, 2 ** 31 - 1, -1, -12345, -2 ** 31]


def draw(r, *shape, spread=1.0):
    return torch.as_tensor(r.standard_normal(shape) * np.exp(spread * r.standard_normal(shape[:-1] + (1,)))).to(BF16)


def positions(r, n):
    return np.where(r.random(n) < 0.5, r.choice(FAR, n), r.integers(0, 200000, n)).astype(np.int64)


def transform(x, weight, pos):
    """fp64 result, and the size that fp32 errors go by: a mean of D squares is
    good to 2^-19 of itself (at most 20 roundings, halved by the root), three
    products and the sine's 2^-22 for each of a pair."""
    x = f64(x)
    y = Q.norm(x, f64(weight), EPS) if weight is not None else x
    size = np.abs(y)
    if pos is not None:
        y, size = Q.rope(y, pos, BASE)
    return y, size * 2.0 ** -18


def near_bf16(got, ref, err):
    assert (np.abs(f64(got) - ref) <= 2.0 ** -8 * np.abs(ref) + err + 1e-38).all()


# ------------------------------------------------------------- norm and rotation

@pytest.mark.parametrize("T", [1, 7, 64, 1000])
@pytest.mark.parametrize("hq,hkv,D", [(16, 8, 128), (12, 4, 64), (1, 1, 128), (5, 3, 64), (40, 1, 128)])
def test_norm_rope(T, hq, hkv, D):
    r = np.random.default_rng(T + hq)
    qkv = draw(r, T, hq + 2 * hkv, D).cuda()
    q, k = qkv[:, :hq], qkv[:, hq:hq + hkv]
    qw, kw = draw(r, D).cuda(), draw(r, D).cuda()
    pos = positions(r, T)
    for w, ps in (((qw, kw), pos), ((qw, None), pos), ((None, kw), None), ((None, None), pos)):
        qo, ko = torch.full((T, hq, D), 7.0, dtype=BF16).cuda(), torch.full((T, hkv, D), 7.0, dtype=BF16).cuda()
        lib.mis_qk_norm_rope(q, k, qo, ko, None if ps is None else i32(ps), q_weight=w[0], k_weight=w[1], eps=EPS, base=BASE)
        near_bf16(qo, *transform(q, w[0], ps))
        near_bf16(ko, *transform(k, w[1], ps))


def test_norm_rope_in_place_and_of_one_tensor():
    r = np.random.default_rng(1)
    T, hq, hkv, D = 50, 6, 2, 128
    qkv = draw(r, T, hq + 2 * hkv, D).cuda()
    was = qkv.clone()
    w, pos = draw(r, D).cuda(), i32(np.arange(T))
    qo, ko = torch.empty(T, hq, D, dtype=BF16).cuda(), torch.empty(T, hkv, D, dtype=BF16).cuda()
    lib.mis_qk_norm_rope(qkv[:, :hq], qkv[:, hq:hq + hkv], qo, ko, pos, w, w)
    q1, k1 = torch.zeros_like(qo), torch.zeros_like(ko)
    lib.mis_qk_norm_rope(qkv[:, :hq], None, q1, None, pos, w)
    lib.mis_qk_norm_rope(None, qkv[:, hq:hq + hkv], None, k1, pos, k_weight=w)
    assert torch.equal(q1, qo) and torch.equal(k1, ko)
    lib.mis_qk_norm_rope(qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, :hq], qkv[:, hq:hq + hkv], pos, w, w)
    assert torch.equal(qkv[:, :hq], qo) and torch.equal(qkv[:, hq:hq + hkv], ko)
    assert torch.equal(qkv[:, hq + hkv:], was[:, hq + hkv:])
    lib.mis_qk_norm_rope(qkv[:0, :hq], None, q1[:0], None, pos, w)


def test_norm_of_rows_of_zeros_and_of_any_size():
    x = torch.zeros(6, 1, 128, dtype=BF16).cuda()
    x[1] = 2.0 ** -70
    x[2] = 2.0 ** 60
    x[3, 0, 5] = float("inf")
    x[4, 0, 5] = float("nan")
    x[5] = 3.0
    w, o = torch.ones(128, dtype=BF16).cuda(), torch.empty(6, 1, 128, dtype=BF16).cuda()
    lib.mis_qk_norm_rope(x, None, o, None, None, w, eps=1e-6)
    o = o[:, 0].float().cpu()
    assert (o[0] == 0).all() and (o[2] == 1).all() and (o[5] == 1).all()
    assert torch.allclose(o[1], torch.full((128,), 2.0 ** -70 * 1000.0), rtol=2.0 ** -8)
    assert torch.isnan(o[4]).all() and torch.isnan(o[3, 5]) and (o[3, :5] == 0).all()


def test_norm_rope_of_far_positions_is_a_turn_by_the_angle():
    """Position p and base b: rotating (1, 0) gives the cosine and sine of p b^(-2i/D) taken in 64 bits."""
    D = 128
    x = torch.zeros(len(FAR), 1, D, dtype=BF16).cuda()
    x[..., :D // 2] = 1.0
    o = torch.empty_like(x)
    lib.mis_qk_norm_rope(x, None, o, None, i32(FAR), base=1e4)
    a = np.asarray(FAR, np.float64)[:, None] * 1e4 ** (-np.arange(D // 2) * 2 / D)
    ref = np.concatenate([np.cos(a), np.sin(a)], -1)
    far = np.abs(np.asarray(FAR, np.float64))[:, None] * 2.0 ** -50 + 2.0 ** -22     # of the frequency, and the sine's
    assert (np.abs(f64(o)[:, 0] - ref) <= 2.0 ** -8 * np.abs(ref) + far).all()


def test_norm_rope_agrees_with_the_plain_rotation():
    r = np.random.default_rng(3)
    q, k, pos = draw(r, 300, 4, 128).cuda(), draw(r, 300, 2, 128).cuda(), i32(np.arange(300))
    a, b, c, d = (torch.empty_like(t) for t in (q, k, q, k))
    lib.mis_rope_qk(q, k, a, b, pos, BASE)
    lib.mis_qk_norm_rope(q, k, c, d, pos, base=BASE)
    for x, y, src in ((a, c, q), (b, d, k)):
        size = Q.rope(f64(src), np.arange(300), BASE)[1]
        assert (np.abs(f64(x) - f64(y)) <= 2.0 ** -7 * np.abs(f64(y)) + size * 2.0 ** -14).all()


# -------------------------------------------------------------- store and read

class Cache:
    def __init__(self, n_pages, page, hkv, D, order="rows"):
        self.n_pages, self.page, self.hkv, self.D = n_pages, page, hkv, D
        shape = (n_pages, page, hkv, D)
        if order == "rows":
            self.k, self.v = (torch.full(shape, 0x55, dtype=torch.uint8).cuda() for _ in range(2))
        elif order == "heads":
            self.k, self.v = (torch.full((n_pages, hkv, page, D), 0x55, dtype=torch.uint8).cuda().transpose(1, 2)
                              for _ in range(2))
        else:
            kv = torch.full((n_pages, page, hkv, 2, D), 0x55, dtype=torch.uint8).cuda()
            self.k, self.v = kv[:, :, :, 0], kv[:, :, :, 1]
        self.ke, self.ve = (torch.full((n_pages, hkv, page), 0x66, dtype=torch.uint8).cuda() for _ in range(2))
        self.c = lib.PagedCacheQ8(self.k, self.v, self.ke, self.ve)

    def rows(self):
        """Codes [slots, hkv, D] and exponents [slots, hkv] of K and V, on the host."""
        n = lambda t: t.cpu().numpy()  # noqa: E731
        flat = lambda t: n(t).reshape(-1, self.hkv, self.D)  # noqa: E731
        exps = lambda t: n(t).transpose(0, 2, 1).reshape(-1, self.hkv)  # noqa: E731
        return flat(self.k), exps(self.ke), flat(self.v), exps(self.ve)


def ws():
    return torch.full((lib.mis_paged_write_workspace_size(),), 0xA5, dtype=torch.uint8, device="cuda")


def check_exact(c, e, x):
    """Codes and exponents of rows that were stored as they are."""
    assert np.array_equal(e.astype(int) - 127, Q.exponent(x))
    want = Q.codes(x, Q.exponent(x))
    assert np.array_equal(c & 0x7F, want & 0x7F) and np.array_equal(c, want)


def check_near(c, e, x, err):
    """Rows that went through fp32 first: the exponent of a maximum within its
    error, and codes within half a step of it plus that error."""
    ex = e.astype(int) - 127
    err_row = err.max(axis=-1)
    a = np.abs(x).max(axis=-1)
    assert (a - err_row <= 448.0 * 2.0 ** ex).all()
    assert ((a + err_row > 448.0 * 2.0 ** (ex - 1)) | (ex == Q.E_LO)).all()
    unit = 2.0 ** ex[..., None].astype(float)
    off = np.abs(Q.values(c, e) - x)
    assert (off <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * unit) * (1 + 2.0 ** -17) + err).all()


@pytest.mark.parametrize("n", [1, 5, 100, 3000, 9001])
@pytest.mark.parametrize("hkv,D,page,order", [(8, 128, 16, "rows"), (3, 64, 32, "heads"), (2, 128, 256, "both"),
                                              (1, 64, 64, "rows")])
def test_store_and_read(n, hkv, D, page, order):
    r = np.random.default_rng(n + hkv)
    src_T = n + 50
    k, v = draw(r, src_T, hkv, D), draw(r, src_T, hkv, D)
    n_pages = n // page + 3
    slots = r.permutation(n_pages * page)[:n].astype(np.int32)
    slots[r.random(n) < 0.1] = -1
    rows = r.integers(0, src_T, n)
    pos, w = positions(r, n), draw(r, D).cuda()
    keep = slots >= 0
    for norm, rot, gather in ((None, None, True), (None, None, False), (w, pos, False), (w, None, True), (None, pos, True)):
        ca, s = Cache(n_pages, page, hkv, D, order), ws()
        lib.mis_paged_write_kv_q8(ca.c, k.cuda(), v.cuda(), i32(slots), s, None if rot is None else i32(rot), BASE,
                                  i32(rows) if gather else None, norm, EPS)
        torch.cuda.synchronize()
        assert lib.mis_get_device_status(s) == lib.MIS_OK
        at = rows if gather else np.arange(n)
        kc, ke, vc, ve = ca.rows()
        check_exact(vc[slots[keep]], ve[slots[keep]], f64(v)[at[keep]])
        if norm is None and rot is None:
            check_exact(kc[slots[keep]], ke[slots[keep]], f64(k)[at[keep]])
        else:
            x, err = transform(k[at[keep]], norm, None if rot is None else rot[keep])
            check_near(kc[slots[keep]], ke[slots[keep]], x, err)
        other = np.setdiff1d(np.arange(n_pages * page), slots[keep])
        assert (kc[other] == 0x55).all() and (vc[other] == 0x55).all()
        assert (ke[other] == 0x66).all() and (ve[other] == 0x66).all()
        # and back, into rows of a wider buffer
        buf = torch.full((n, 2 * hkv * D + 8), 7.0, dtype=BF16).cuda()
        ko, vo = buf[:, :hkv * D].unflatten(1, (hkv, D)), buf[:, hkv * D:2 * hkv * D].unflatten(1, (hkv, D))
        lib.mis_paged_read_kv_q8(ca.c, i32(slots), ko, vo, s)
        torch.cuda.synchronize()
        assert lib.mis_get_device_status(s) == lib.MIS_OK
        for out, c, e in ((ko, kc, ke), (vo, vc, ve)):
            assert np.array_equal(f64(out)[keep], Q.values(c[slots[keep]], e[slots[keep]]))
            assert (f64(out)[~keep] == 7).all()
        assert (buf[:, 2 * hkv * D:] == 7).all()


def test_store_of_zeros_infinities_and_any_size():
    x = torch.zeros(9, 2, 64, dtype=BF16)
    x[1] = 2.0 ** -75
    x[2, :, 3] = 2.0 ** -60
    x[3] = torch.finfo(BF16).max
    x[4, 0, 5], x[4, 0, 6], x[4, 0, 7] = float("inf"), -900.0, 3.0
    x[5, 1, 5], x[5, 1, 6] = float("nan"), 1.0
    x[6] = float("-inf")
    x[7] = torch.linspace(-448, 448, 64)
    x[8] = torch.finfo(BF16).tiny
    ca, s = Cache(2, 16, 2, 64), ws()
    lib.mis_paged_write_kv_q8(ca.c, x.cuda(), x.cuda(), i32(np.arange(9)), s)
    for c, e in (ca.rows()[:2], ca.rows()[2:]):
        check_exact(c[:9], e[:9], f64(x))
    ko, vo = torch.empty_like(x).cuda(), torch.empty_like(x).cuda()
    lib.mis_paged_read_kv_q8(ca.c, i32(np.arange(9)), ko, vo, s)
    assert torch.isnan(ko[6]).all() and torch.isnan(vo[4, 0, 5]) and not torch.isnan(ko[4, 1]).any()
    # a rotation that passes fp32's range keeps NaN there, and the row's other elements
    y = torch.zeros(1, 2, 64, dtype=BF16)
    y[0, 0, 0] = y[0, 0, 32] = torch.finfo(BF16).max
    y[0, 0, 1] = 2.0 ** 110
    lib.mis_paged_write_kv_q8(ca.c, y.cuda(), y.cuda(), i32([20]), s, i32([100]), BASE)
    lib.mis_paged_read_kv_q8(ca.c, i32([20]), ko[:1], vo[:1], s)
    ref = Q.rope(f64(y), [100], BASE)[0][0, 0]
    got = f64(ko)[0, 0]
    assert (np.isnan(got) | (np.abs(got - ref) <= 2.0 ** -4 * np.abs(ref) + 1e38 * 2.0 ** -10)).all() and not np.isnan(got[1])


def test_every_code_and_exponent_reads_back():
    ca, s = Cache(16, 16, 2, 64), ws()
    codes = torch.arange(256, dtype=torch.uint8).cuda()
    ca.k.copy_(codes.repeat(16 * 16 * 2 * 64 // 256).view(16, 16, 2, 64))
    ca.v.copy_(codes.flip(0).repeat(16 * 16 * 2 * 64 // 256).view(16, 16, 2, 64))
    e = torch.arange(256, dtype=torch.uint8).cuda().view(16, 1, 16).expand(16, 2, 16)
    ca.ke.copy_(e)
    ca.ve.copy_(e.flip(0))
    ko, vo = (torch.empty(256, 2, 64, dtype=BF16).cuda() for _ in range(2))
    lib.mis_paged_read_kv_q8(ca.c, i32(np.arange(256)), ko, vo, s)
    kc, ke, vc, ve = ca.rows()
    for out, c, e in ((ko, kc, ke), (vo, vc, ve)):
        want = Q.values(c, e)
        want = np.where(np.abs(want) >= 2.0 ** 128, np.copysign(np.inf, want), want)      # past bf16's range
        assert np.array_equal(f64(out), want, equal_nan=True)


@pytest.mark.parametrize("n", [40, 9000])
def test_bad_slots_and_rows(n):
    """On both sides of the number of rows from which their own threads report them."""
    r = np.random.default_rng(5)
    n_pages = n // 16 + 2
    k = draw(r, n, 2, 64).cuda()
    for bad_slot, bad_row in ((n_pages * 16, None), (2 ** 31 - 1, None), (None, n), (None, -1)):
        ca, s = Cache(n_pages, 16, 2, 64), ws()
        slots, rows = np.arange(n), np.arange(n)[::-1].copy()
        i = n - 3
        if bad_slot is not None:
            slots[i] = bad_slot
        else:
            rows[i] = bad_row
        lib.mis_paged_write_kv_q8(ca.c, k, k, i32(slots), s, src_rows=i32(rows))
        assert lib.mis_get_device_status(s) == lib.MIS_ERR_DEVICE_INDEX
        kc, ke, _, _ = ca.rows()
        good = np.delete(np.arange(n), i)
        check_exact(kc[good], ke[good], f64(k)[rows[good]])
        assert (kc[i] == 0x55).all()
        out = torch.full((n, 2, 64), 7.0, dtype=BF16).cuda()
        lib.mis_paged_read_kv_q8(ca.c, i32(slots), out, out.clone(), s)
        assert lib.mis_get_device_status(s) == (lib.MIS_ERR_DEVICE_INDEX if bad_slot is not None else lib.MIS_OK)
        if bad_slot is not None:
            assert (out[i] == 7).all()
        # a row that is skipped may name any source; the next call's status is its own
        if bad_row is not None:
            slots[i] = -4
            lib.mis_paged_write_kv_q8(ca.c, k, k, i32(slots), s, src_rows=i32(rows))
        else:
            lib.mis_paged_write_kv_q8(ca.c, k, k, i32(np.arange(n)), s)
        assert lib.mis_get_device_status(s) == lib.MIS_OK


@pytest.mark.parametrize("n", [40, 9000])
@pytest.mark.parametrize("bad", ["slot", "row"])
def test_bad_indices_of_wide_rows(n, bad):
    """Rows wide enough that one block looks over the indices of any number of them."""
    n_pages = n // 256 + 2
    r = np.random.default_rng(6)
    k = draw(r, n, 4, 128).cuda()
    for i in (0, n // 2, n - 1):
        ca, s = Cache(n_pages, 256, 4, 128), ws()
        slots, rows = np.arange(n), np.arange(n)[::-1].copy()
        (slots if bad == "slot" else rows)[i] = n_pages * 256 if bad == "slot" else n
        lib.mis_paged_write_kv_q8(ca.c, k, k, i32(slots), s, src_rows=i32(rows))
        assert lib.mis_get_device_status(s) == lib.MIS_ERR_DEVICE_INDEX
        kc, ke, _, _ = ca.rows()
        good = np.delete(np.arange(n), i)
        check_exact(kc[good], ke[good], f64(k)[rows[good]])
        assert (kc[i] == 0x55).all()
        if bad == "slot":
            out = torch.full((n, 4, 128), 7.0, dtype=BF16).cuda()
            lib.mis_paged_read_kv_q8(ca.c, i32(slots), out, out.clone(), s)
            assert lib.mis_get_device_status(s) == lib.MIS_ERR_DEVICE_INDEX
            assert (out[i] == 7).all()


def test_repeated_rows_and_slots():
    """One source row at many slots, one slot read many times."""
    r = np.random.default_rng(7)
    x, ca, s = draw(r, 5, 3, 64), Cache(8, 16, 3, 64), ws()
    rows = r.integers(0, 5, 100)
    lib.mis_paged_write_kv_q8(ca.c, x.cuda(), x.cuda(), i32(np.arange(100)), s, src_rows=i32(rows))
    slots = r.integers(0, 100, 500)
    k, v = (torch.empty(500, 3, 64, dtype=BF16, device="cuda") for _ in range(2))
    lib.mis_paged_read_kv_q8(ca.c, i32(slots), k, v, s)
    assert lib.mis_get_device_status(s) == lib.MIS_OK
    e = Q.exponent(f64(x))
    held = Q.values(Q.codes(f64(x), e), e + 127)[rows][slots]
    assert np.array_equal(f64(k), held) and np.array_equal(f64(v), held)


def test_slots_past_four_gigabytes():
    """A cache whose byte offsets pass 32 bits: rows at its far end, stored, read and attended."""
    n_pages, page, hkv, D = 1100, 256, 128, 128                  # 4.6 GB a buffer
    k, v = (torch.empty(n_pages, page, hkv, D, dtype=torch.uint8, device="cuda") for _ in range(2))
    ke, ve = (torch.full((n_pages, hkv, page), 127, dtype=torch.uint8, device="cuda") for _ in range(2))
    c, s = lib.PagedCacheQ8(k, v, ke, ve), ws()
    r = np.random.default_rng(9)
    x = draw(r, 40, hkv, D, spread=0.3)
    slots = np.concatenate([np.arange(20), n_pages * page - 20 + np.arange(20)])
    lib.mis_paged_write_kv_q8(c, x.cuda(), x.cuda(), i32(slots), s)
    ko, vo = (torch.empty(40, hkv, D, dtype=BF16, device="cuda") for _ in range(2))
    lib.mis_paged_read_kv_q8(c, i32(slots), ko, vo, s)
    e = Q.exponent(f64(x))
    held = Q.values(Q.codes(f64(x), e), e + 127)
    assert np.array_equal(f64(ko), held) and np.array_equal(f64(vo), held)
    # one request over the last page, whose last 20 rows are these: 256 rows, so fill the others with zeros
    k[-1, :page - 20] = 0
    v[-1, :page - 20] = 0
    q = draw(r, 1, hkv, D, spread=0.3)
    desc = lib.PagedAttentionDesc(c, B=1, T=1, Hq=hkv, max_rows=1)
    w2 = torch.empty(desc.workspace_size(), dtype=torch.uint8, device="cuda")
    o, lse = torch.empty(1, hkv, D, dtype=BF16, device="cuda"), torch.empty(hkv, 1, device="cuda")
    lib.mis_paged_attention_q8_fwd(desc, q.cuda(), o, lse, i32([[n_pages - 1]]), i32([page]), i32([0, 1]), w2)
    rows = np.concatenate([np.zeros((page - 20, hkv, D)), held[20:]])
    ro, rl, av, big = Q.attention(f64(q), rows, rows, 1, 1 / math.sqrt(D))
    assert (np.abs(f64(o) - ro) <= 2.0 ** -8 * np.abs(ro) + av * 2.0 ** -10).all()
    assert np.abs(f64(lse).T - rl).max() < 1e-4


# ------------------------------------------------------------------- together

@pytest.mark.parametrize("D,hq,hkv", [(128, 8, 4), (64, 6, 2)])
def test_prompt_decode_and_items_over_a_cached_prefix(D, hq, hkv):
    """A server's run: prompts normed, rotated and stored; tokens decoded one by
    one and three at a time, a graph of the step replayed as lengths grow; then a
    prefix read back for items scored over it by the cached attention."""
    r = np.random.default_rng(4)
    B, page, n_pages, cols = 3, 16, 64, 20
    lens0 = [70, 16, 33]
    table = torch.full((B, cols), -1, dtype=torch.int32).cuda()
    free, head = i32(r.permutation(n_pages)), i32([0])
    cache_len = i32([0] * B)
    shape = (n_pages, hkv, page, D)
    c = lib.PagedCacheQ8(*(torch.zeros(shape, dtype=torch.float8_e4m3fn, device="cuda").transpose(1, 2) for _ in range(2)),
                         *(torch.zeros(n_pages, hkv, page, dtype=torch.uint8, device="cuda") for _ in range(2)))
    qw, kw = draw(r, D, spread=0.1).cuda(), draw(r, D, spread=0.1).cuda()
    hist_k, hist_v = [[] for _ in range(B)], [[] for _ in range(B)]

    def keep(qkv, ns, at):
        """The oracle's own record of what the cache should hold."""
        row = 0
        for b, n in enumerate(ns):
            x = qkv[row:row + n, hq:hq + hkv].cpu()
            hist_k[b].append(transform(x, kw, np.arange(at[b], at[b] + n))[0])
            hist_v[b].append(f64(qkv[row:row + n, hq + hkv:]))
            row += n

    class Step:
        def __init__(self, T, max_rows):
            self.T = T
            self.qkv = torch.zeros(T, hq + 2 * hkv, D, dtype=BF16, device="cuda")
            self.new = i32([0] * B)
            self.cu = i32([0] * (B + 1))
            self.slots, self.pos = i32([0] * T), i32([0] * T)
            self.q, self.o = (torch.zeros(T, hq, D, dtype=BF16, device="cuda") for _ in range(2))
            self.desc = lib.PagedAttentionDesc(c, B=B, T=T, Hq=hq, max_rows=max_rows)
            self.ws = torch.empty(self.desc.workspace_size(), dtype=torch.uint8, device="cuda")
            self.ews = torch.empty(lib.mis_paged_extend_workspace_size(B), dtype=torch.uint8, device="cuda")
            self.wws = ws()

        def call(self):
            lib.mis_paged_extend(self.new, cache_len, cache_len, table, free, head, head, self.cu, self.slots, self.pos,
                                 page, n_pages, self.ews)
            lib.mis_paged_write_kv_q8(c, self.qkv[:, hq:hq + hkv], self.qkv[:, hq + hkv:], self.slots, self.wws, self.pos,
                                      BASE, k_weight=kw, eps=EPS)
            lib.mis_qk_norm_rope(self.qkv[:, :hq], None, self.q, None, self.pos, qw, eps=EPS, base=BASE)
            lib.mis_paged_attention_q8_fwd(self.desc, self.q, self.o, None, table, cache_len, self.cu, self.ws)

        def check(self, ns, at):
            torch.cuda.synchronize()
            for w in (self.ws, self.ews, self.wws):
                assert lib.mis_get_device_status(w) == lib.MIS_OK
            row = 0
            for b, n in enumerate(ns):
                k, v = np.concatenate(hist_k[b]), np.concatenate(hist_v[b])
                q = transform(self.qkv[row:row + n, :hq].cpu(), qw, np.arange(at[b], at[b] + n))[0]
                ro, _, av, big = Q.attention(q, k, v, n, 1 / math.sqrt(D))
                # K, V are held to 2^-4 of themselves, q to 2^-8: scores off by at most big * (2^-4 + 2^-8),
                # weights by twice that in size, values by 2^-4
                tol = 2.0 ** -8 * np.abs(ro) + av * (np.expm1(2 * big * (2.0 ** -4 + 2.0 ** -8))[..., None] * 1.0625 + 2.0 ** -4 + 2.0 ** -10)
                # and the cache as it is held, exactly: read back
                assert (np.abs(f64(self.o[row:row + n]) - ro) <= tol).all()
                row += n

    def fill(step, ns):
        step.qkv.copy_(draw(r, step.T, hq + 2 * hkv, D, spread=0.2))
        step.new.copy_(i32(ns))

    prompt = Step(sum(lens0), max(lens0))
    fill(prompt, lens0)
    keep(prompt.qkv, lens0, [0] * B)
    prompt.call()
    prompt.check(lens0, [0] * B)
    at = list(lens0)
    step = Step(9, 3)
    saved = [t.clone() for t in (cache_len, head, table)]
    fill(step, [1, 1, 1])
    step.call()                                               # before the capture, then undone
    for t, s in zip((cache_len, head, table), saved):
        t.copy_(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step.call()
    for t, s in zip((cache_len, head, table), saved):
        t.copy_(s)
    for ns in ([1, 1, 1], [3, 1, 2], [1, 0, 1], [3, 3, 3], [1, 1, 1]):
        fill(step, ns)
        keep(step.qkv, ns, at)
        g.replay()
        step.check(ns, at)
        at = [a + n for a, n in zip(at, ns)]
    # items over request 0's cached rows
    S = at[0]
    pos = np.arange(S)
    slots = table[0].cpu().numpy()[pos // page] * page + pos % page
    kd, vd = (torch.empty(S, hkv, D, dtype=BF16, device="cuda") for _ in range(2))
    rws = ws()
    lib.mis_paged_read_kv_q8(c, i32(slots), kd, vd, rws)
    want_k, want_v = np.concatenate(hist_k[0]), np.concatenate(hist_v[0])
    check_near(*held(c, slots, 0), want_k, np.abs(want_k) * 2.0 ** -17 + 2.0 ** -17)
    assert np.array_equal(f64(vd), Q.values(Q.codes(want_v, Q.exponent(want_v)), Q.exponent(want_v) + 127))
    items = [4, 7, 1]
    T = sum(items)
    offs = np.concatenate([[0], np.cumsum(items)])
    plan = lib.CachedPlan([0, T], [0, 3], offs[:3], [0], [S], S, hq, hkv, D)
    pws = torch.zeros(plan.workspace_size(), dtype=torch.uint8, device="cuda")
    plan.create(pws)
    iq, ik, iv = draw(r, T, hq, D, spread=0.1).cuda(), draw(r, T, hkv, D, spread=0.1).cuda(), draw(r, T, hkv, D, spread=0.1).cuda()
    o = torch.empty_like(iq)
    lib.mis_attention_fwd_cached(plan, iq, ik, iv, kd, vd, o)
    torch.cuda.synchronize()
    for i, n in enumerate(items):
        s = slice(int(offs[i]), int(offs[i]) + n)
        k, v = np.concatenate([f64(kd), f64(ik[s])]), np.concatenate([f64(vd), f64(iv[s])])
        ro, _, av, _ = Q.attention(f64(iq[s]), k, v, n, 1 / math.sqrt(D))
        assert (np.abs(f64(o[s]) - ro) <= 2.0 ** -8 * np.abs(ro) + av * 2.0 ** -6).all()


def held(c, slots, which):
    codes = (c.k, c.v)[which].view(torch.uint8).cpu().numpy().reshape(-1, c.Hkv, c.D)
    exps = (c.k_exp, c.v_exp)[which].cpu().numpy().transpose(0, 2, 1).reshape(-1, c.Hkv)
    return codes[slots], exps[slots]


def test_layers_back_to_back_are_the_same_as_one_call_at_a_time():
    """Norms, store and attention of 12 layers over reused buffers, each layer's
    output the next one's queries: every call starts before the one before has ended."""
    r = np.random.default_rng(11)
    B, hq, hkv, D, page = 5, 8, 4, 128, 32
    lens = [300, 77, 1500, 33, 640]
    pages = [-(-n // page) for n in lens]
    table = np.full((B, max(pages)), -1, np.int32)
    perm, at = r.permutation(sum(pages)), 0
    for b, n in enumerate(pages):
        table[b, :n] = perm[at:at + n]
        at += n
    shape = (sum(pages), page, hkv, D)
    start = [torch.as_tensor(r.integers(0, 0x7E, shape, dtype=np.uint8)).cuda() for _ in range(2)]
    exps = torch.full((shape[0], hkv, page), 127 - 6, dtype=torch.uint8).cuda()
    caches = [lib.PagedCacheQ8(*(x.clone() for x in start), exps.clone(), exps.clone()) for _ in range(12)]
    pos = i32([n - 1 for n in lens])
    slots = i32([table[b, (n - 1) // page] * page + (n - 1) % page for b, n in enumerate(lens)])
    q0, k, v = (draw(r, B, h, D).cuda() for h in (hq, hkv, hkv))
    w = draw(r, D).cuda()
    desc = lib.PagedAttentionDesc(caches[0], B=B, T=B, Hq=hq, max_rows=1)
    descs = [lib.PagedAttentionDesc(c, B=B, T=B, Hq=hq, max_rows=1) for c in caches]
    w2, s = torch.empty(desc.workspace_size(), dtype=torch.uint8, device="cuda"), ws()
    dt, dl, dc = i32(table), i32(lens), i32(np.arange(B + 1))

    def layers(pause):
        q, o, lse = q0.clone(), torch.empty_like(q0), torch.empty(hq, B, device="cuda")
        torch.cuda.synchronize()
        for c, d in zip(caches, descs):
            lib.mis_qk_norm_rope(q, None, q, None, pos, w)
            pause()
            lib.mis_paged_write_kv_q8(c, k, v, slots, s, pos, BASE, None, w, EPS)
            pause()
            lib.mis_paged_attention_q8_fwd(d, q, o, lse, dt, dl, dc, w2)
            pause()
            q, o = o, q
        torch.cuda.synchronize()
        return q.clone(), lse.clone()
    want = layers(torch.cuda.synchronize)
    assert torch.isfinite(want[0].float()).all()
    for _ in range(10):
        got = layers(lambda: None)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_calls_on_a_stream_of_their_own():
    r = np.random.default_rng(8)
    st = torch.cuda.Stream()
    x, w = draw(r, 2000, 4, 128).cuda(), draw(r, 128).cuda()
    ca, s = Cache(200, 16, 4, 128), ws()
    o, o2 = torch.empty_like(x), torch.empty_like(x)
    torch.cuda.synchronize()
    slots = i32(np.arange(2000))
    torch.cuda.synchronize()
    for _ in range(10):
        lib.mis_qk_norm_rope(x, None, o, None, slots, w, stream=st)
        lib.mis_paged_write_kv_q8(ca.c, x, o, slots, s, stream=st)
        lib.mis_paged_read_kv_q8(ca.c, slots, o2, o, s, stream=st)
    st.synchronize()
    e = Q.exponent(f64(x))
    assert np.array_equal(f64(o2), Q.values(Q.codes(f64(x), e), e + 127))
