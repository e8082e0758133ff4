"""The 8-bit cache's calls at the ends of their ranges: as many indices as 32 bits
count, forms that only long prompts take, values far apart, rows that one key
rules over a long cache."""
import numpy as np
import pytest
import torch

from oracle import q8_oracle as Q
from q8_helpers import BF16, Batch, f64, i32
from ranking_prefill_gb300 import lib
from test_gpu_q8_rows import BASE, Cache, check_exact, check_near, draw, near_bf16, positions, transform, ws

pytestmark = pytest.mark.gpu


def test_as_many_indices_as_32_bits_count():
    """2^31 - 1 rows by index, most of them skipped: the look at the indices ends, and it sees the last ones."""
    n = 2 ** 31 - 1
    x = draw(np.random.default_rng(1), 3, 4, 128)
    slots = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    rows = torch.zeros(n, dtype=torch.int32, device="cuda")
    at = torch.tensor([0, 2 ** 30, n - 2049, n - 2, n - 1], device="cuda")
    src = [0, 1, 2, 1, 2]
    slots[at] = i32([5, 6, 7, 8, 9])
    rows[at] = i32(src)
    ca, s = Cache(1, 16, 4, 128), ws()
    lib.mis_paged_write_kv_q8(ca.c, x.cuda(), x.cuda(), slots, s, src_rows=rows)
    assert lib.mis_get_device_status(s) == lib.MIS_OK
    kc, ke, vc, ve = ca.rows()
    for c, e in ((kc, ke), (vc, ve)):
        check_exact(c[5:10], e[5:10], f64(x)[src])
        assert (c[:5] == 0x55).all() and (c[10:] == 0x55).all() and (e[:5] == 0x66).all()
    for bad, where in ((16, slots), (3, rows)):
        was = where[n - 1].clone()
        where[n - 1] = bad
        lib.mis_paged_write_kv_q8(ca.c, x.cuda(), x.cuda(), slots, s, src_rows=rows)
        assert lib.mis_get_device_status(s) == lib.MIS_ERR_DEVICE_INDEX
        where[n - 1] = was


# ----------------------------------------------------------------------- norms

@pytest.mark.parametrize("hq,hkv", [(13, 3), (10, 6), (5, 6), (8, 8), (3, 9)])
@pytest.mark.parametrize("D", [64, 128])
def test_prompts_normed_four_heads_at_a_time(hq, hkv, D):
    """Tokens so many that a thread takes all heads of one: groups of four that end in a
    tensor, at its end and past it, apart from the input and over it."""
    T = 10000 + hq
    r = np.random.default_rng(hq)
    qkv = draw(r, T, hq + hkv + 1, D).cuda()
    q, k, rest = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:].clone()
    qw, kw, pos = draw(r, D).cuda(), draw(r, D).cuda(), positions(r, T)
    qo, ko = torch.full((T, hq, D), 7.0, dtype=BF16).cuda(), torch.full((T, hkv, D), 7.0, dtype=BF16).cuda()
    lib.mis_qk_norm_rope(q, k, qo, ko, i32(pos), qw, kw, base=BASE)
    near_bf16(qo, *transform(q, qw, pos))
    near_bf16(ko, *transform(k, kw, pos))
    if hkv >= 8:
        k1 = torch.zeros_like(ko)
        lib.mis_qk_norm_rope(None, k, None, k1, i32(pos), k_weight=kw, base=BASE)
        assert torch.equal(k1, ko)
    # one tensor normed, the other turned alone
    q2, k2 = torch.empty_like(qo), torch.empty_like(ko)
    lib.mis_qk_norm_rope(q, k, q2, k2, i32(pos), None, kw, base=BASE)
    near_bf16(q2, *transform(q, None, pos))
    assert torch.equal(k2, ko)
    lib.mis_qk_norm_rope(q, k, q, k, i32(pos), qw, kw, base=BASE)
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(qkv[:, hq + hkv:], rest)


SIZES = [2.0 ** p for p in (0, 40, 61, 63, 64, 90, 124, -30, -55, -60, -74, -90, -110)]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T", [len(SIZES), 1000 * len(SIZES)])
@pytest.mark.parametrize("eps", [0.0, 1e-37, 1e-30, 1e-6])
def test_norms_of_rows_whose_squares_leave_fp32(D, T, eps):
    """Every size beside every other one in a row's heads; normed in both forms and on the way
    to the cache. Errors as in the ordinary range (2^-18); elements 2^60 below their
    row's size may lose bits at fp32's least ones."""
    r = np.random.default_rng(D)
    hq, hkv = 7, 4
    x = draw(r, T, hq + hkv, D, spread=0.0).double()
    size = np.stack([np.roll(SIZES, h)[np.arange(T) % len(SIZES)] for h in range(hq + hkv)], axis=1)
    x = (x.clamp(-8, 8) * torch.as_tensor(size)[..., None]).to(BF16)
    x[:, 1, ::3] = 0.0
    qw, kw = draw(r, D, spread=0.0), draw(r, D, spread=0.0)
    pos = positions(r, T)
    qo, ko = torch.empty(T, hq, D, dtype=BF16).cuda(), torch.empty(T, hkv, D, dtype=BF16).cuda()
    d = x.cuda()
    lib.mis_qk_norm_rope(d[:, :hq], d[:, hq:], qo, ko, i32(pos), qw.cuda(), kw.cuda(), eps=eps, base=BASE)
    for got, rows, w in ((qo, x[:, :hq], qw), (ko, x[:, hq:], kw)):
        ref, pair = Q.rope(Q.norm(f64(rows), f64(w), eps), pos, BASE)
        near_bf16(got, ref, pair * 2.0 ** -18)
    ca, s = Cache(T // 16 + 1, 16, hkv, D), ws()
    k = d[:, hq:].contiguous()
    lib.mis_paged_write_kv_q8(ca.c, k, k, i32(np.arange(T)), s, i32(pos), BASE, k_weight=kw.cuda(), eps=eps)
    kc, ke, vc, ve = ca.rows()
    check_near(kc[:T], ke[:T], ref, pair * 2.0 ** -18 + 1e-38)
    check_exact(vc[:T], ve[:T], f64(k))


def test_norms_without_eps_of_rows_of_zeros_and_infinities():
    """0 / 0 and inf / inf are NaN, what stands beside an infinity is zero, and no other row is touched."""
    x = torch.full((4, 8, 128), 3.0, dtype=BF16)
    x[0, 2] = 0.0
    x[1, 3, 7] = float("inf")
    x[2, 4, 100] = float("nan")
    x[3, 5] = torch.finfo(BF16).max
    w, o = torch.ones(128, dtype=BF16).cuda(), torch.empty(4, 8, 128, dtype=BF16).cuda()
    lib.mis_qk_norm_rope(x.cuda(), None, o, None, None, w, eps=0.0)
    want = torch.ones(4, 8, 128)
    want[0, 2], want[1, 3], want[2, 4] = float("nan"), 0.0, float("nan")
    want[1, 3, 7] = float("nan")
    assert np.array_equal(f64(o), f64(want), equal_nan=True)


@pytest.mark.parametrize("left_out", ["q", "k"])
def test_nothing_of_a_tensor_without_heads_is_looked_at(left_out):
    """Its addresses, its weight's and its strides may be anything."""
    r = np.random.default_rng(3)
    x, w, pos = draw(r, 33, 3, 64).cuda(), draw(r, 64).cuda(), i32(np.arange(33))
    want, got = torch.empty_like(x), torch.full_like(x, 7.0)
    lib.mis_qk_norm_rope(x, None, want, None, pos, w)
    live = (x.data_ptr(), got.data_ptr(), 3 * 64, 3 * 64, 3, w.data_ptr())
    none = (0x1002, 0x2001, -5, 3, 0, 0x3004)
    q, k = (none, live) if left_out == "q" else (live, none)
    st = lib.load().mis_qk_norm_rope(q[0], k[0], q[1], k[1], q[2], k[2], q[3], k[3], 33, q[4], k[4], 64, q[5], k[5], 1e-6,
                                     pos.data_ptr(), BASE, None)
    torch.cuda.synchronize()
    assert st == lib.MIS_OK and torch.equal(got, want)


# ------------------------------------------------------------------- attention

def shared(kc, ke, vc, ve, q, lens, ns, scale):
    """Requests whose tables name the same pages. Returns o and lse."""
    c = lib.PagedCacheQ8(kc, vc, ke, ve)
    B, T, hq = len(lens), int(sum(ns)), q.shape[1]
    desc = lib.PagedAttentionDesc(c, B=B, T=T, Hq=hq, max_rows=max(ns), scale=scale)
    w = torch.full((desc.workspace_size(),), 0xA5, dtype=torch.uint8, device="cuda")
    o, lse = torch.full_like(q, 7.0), torch.full((hq, T), 7.0, device="cuda")
    lib.mis_paged_attention_q8_fwd(desc, q, o, lse, i32(np.tile(np.arange(c.n_pages), (B, 1))), i32(lens),
                                   i32(np.concatenate([[0], np.cumsum(ns)])), w)
    assert lib.mis_get_device_status(w) == lib.MIS_OK
    return f64(o), f64(lse)


@pytest.mark.parametrize("hq,D", [(8, 128), (8, 64), (160, 128), (160, 64)])
@pytest.mark.parametrize("at", [5, 70000, 131071])
def test_a_key_that_rules_a_long_cache(hq, D, at):
    """One key 2^24 to 2^26 above 131,071 others: these weigh half a percent together,
    with values that share a mean. More units than blocks, so that a block takes a
    unit whole. Off by: o's rounding; the weights' (2^-11 of their size) and their
    arguments' (2^-17); the sum of weights, of which a thread adds up to 1,024 (2^-14);
    131,071 products that the tensor core may cut at 2^-24 of a sum of at most 2^-3.5:
    2^-10.5, whatever the weights. So no error that grows with their number is let by."""
    L, hkv, B, page = 131072, 8, 20, 256
    g = torch.Generator(device="cuda").manual_seed(at)
    lut = torch.tensor([0x30, 0x38, 0x3C, 0x38], dtype=torch.uint8, device="cuda")       # 0.5, 1, 1.5, 1
    vc = lut[torch.randint(0, 4, (L // page, page, hkv, D), generator=g, device="cuda")]
    v0 = torch.tensor([0x00, 0x08, 0x10, 0x18, 0x88, 0x94], dtype=torch.uint8, device="cuda").repeat(D)[:D]   # |v| <= 2^-4
    vc[at // page, at % page] = v0
    kc = torch.zeros_like(vc)
    kc[at // page, at % page, :, 0] = 0x38
    ke, ve = (torch.full((L // page, hkv, page), 127, dtype=torch.uint8, device="cuda") for _ in range(2))
    v = vc.view(torch.float8_e4m3fn).float()
    first = f64(v0.view(torch.float8_e4m3fn).float())
    others = np.repeat(f64(v.double().sum(dim=(0, 1))) - first, hq // hkv, axis=0)
    q = torch.zeros(B, hq, D, dtype=BF16, device="cuda")
    q[..., 0] = 1.0
    for p in (24.2, 24.6, 25.3, 26.0):
        scale = float(np.float32(p * np.log(2.0)))
        o, lse = shared(kc, ke, vc, ve, q, [L] * B, [1] * B, scale)
        w = np.exp(-scale)
        total = 1 + w * (L - 1)
        ref, av = (first + w * others) / total, (np.abs(first) + w * others) / total
        tol = 2.0 ** -8 * np.abs(ref) + av * (2.0 ** -11 + 2.0 ** -17 + 2.0 ** -14) + 2.0 ** -10.5
        assert (np.abs(o - ref) <= tol).all(), (p, np.abs(o - ref).max(), tol.min())
        assert np.abs(lse - (scale + np.log(total))).max() <= 2.0 ** -13


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("hq,hkv,B", [(2, 2, 1), (1, 1, 1), (8, 8, 20), (160, 8, 20), (24, 1, 1)])
@pytest.mark.parametrize("L", [2, 130, 300, 2001, 20001])
def test_values_at_both_ends_of_the_exponents(hq, hkv, B, D, L):
    """Rows of tiny or no values, then one of far larger ones, all with the same score:
    every key has a share in the sum, in streams, steps, blocks and their join. Off by:
    the weights and o, each rounded; L roundings of the sum at most."""
    page = 64
    n_pages = -(-L // page)
    kc = torch.zeros(n_pages, page, hkv, D, dtype=torch.uint8, device="cuda")
    ke = torch.full((n_pages, hkv, page), 127, dtype=torch.uint8, device="cuda")
    q = torch.zeros(B, hq, D, dtype=BF16, device="cuda")
    for low, high, code in ((71, 207, 0x00), (71, 247, 0x38), (71, 198, 0x00), (100, 247, 0x38)):
        for at in sorted({0, L // 2, L - 1}):
            vc = torch.full_like(kc, code)
            ve = torch.full_like(ke, low)
            vc[at // page, at % page] = 0x38
            ve[at // page, :, at % page] = high
            o, lse = shared(kc, ke, vc, ve, q, [L] * B, [1] * B, 1.0)
            ref = (2.0 ** (high - 127) + (L - 1) * (2.0 ** (low - 127) if code else 0.0)) / L
            slack = 2.0 ** -8 + 2.0 ** -11 + L * 2.0 ** -24
            assert (np.abs(o - ref) <= slack * ref).all(), (low, high, at, o.ravel()[0] / ref)
            assert np.abs(lse - np.log(L)).max() <= L * 2.0 ** -24 + 2.0 ** -17, (low, high, at)


@pytest.mark.parametrize("ns", [[1, 3, 2, 1], [9, 2, 12, 5]])
def test_what_is_written_beside_waits_that_run_out_is_right(ns):
    """Limits of 0 to 9 us: every element of o and lse is either as it was or as in a
    call whose waits last, to the bit, whatever the status."""
    b = Batch([20000, 40, 3000, 500], ns, 8, 2, 128, 16, seed=80).run().check()
    o, lse = b.o.clone(), b.lse.clone()
    assert not o.isnan().any() and not lse.isnan().any()
    limit = lib.mis_set_wait_limit_ns(0)
    try:
        for t in list(range(0, 2000, 50)) + list(range(2000, 9000, 250)):
            lib.mis_set_wait_limit_ns(t)
            b.o.fill_(float("nan"))
            b.lse.fill_(float("nan"))
            b.call()
            status = lib.mis_get_device_status(b.ws)
            assert status in (lib.MIS_OK, lib.MIS_ERR_DEVICE_TIMEOUT)
            for got, want in ((b.o, o), (b.lse, lse)):
                there = ~got.isnan()
                assert torch.equal(got[there], want[there])
                assert status != lib.MIS_OK or there.all()
    finally:
        lib.mis_set_wait_limit_ns(limit)
