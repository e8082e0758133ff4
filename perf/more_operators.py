"""Measured cases of the operators around an 8-bit paged K/V cache: per-head
norms of queries and keys with the rotary embedding in the same pass, K/V rows
quantised as they are stored, rows read back, and attention of the newest
tokens over the quantised rows.

A cached (row, kv head) is D codes in e4m3 and one exponent byte e + 127; it
stands for code * 2^e, which bfloat16 holds exactly. Stores are compared by
the rows that are read back after them.

A case is a dict of plain values. Its lengths come from the case's own
``shape`` number, its values from the seed, so the work of a case is fixed.
The plain forms are elementary torch operations in 32 bits (64 for rotary
angles); ``exact`` restates the definitions in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

ROPE_BASE = 1.0e6
EPS = 1.0e-6
E_LO, E_HI = -56, 120            # range of a row's exponent


# --------------------------------------------------------------------- cases

def listed():
    return [
        # q and k of one decoding step of 32 requests, columns of the projection's output: latency
        dict(name="norm-decode-32", op="norm", T=32, hq=16, hkv=8, D=128, far=4096),
        # q and k of a prefill batch of 128K tokens
        dict(name="norm-prefill-128k", op="norm", T=131072, hq=16, hkv=8, D=128, far=16384),
        # 3 query heads a kv head, 64 wide, an odd number of rows at far positions
        dict(name="norm-odd-4099", op="norm", T=4099, hq=12, hkv=4, D=64, far=1 << 20),
        # one decoding step of 32 requests stores a row each, K normed and rotated on the way
        dict(name="store-decode-32", op="store", rows=32, src=32, hkv=8, D=128, page=16, pages=4096,
             rope=True, norm=True, gather=False, skip=0.0),
        # 128K prompt rows enter the cache and are read back
        dict(name="store-prompt-128k", op="store", rows=131072, src=131072, hkv=8, D=128, page=64,
             pages=2200, rope=True, norm=True, gather=False, skip=0.0),
        # rows picked by index, already rotated, 64-wide heads, some slots skipped
        dict(name="store-picked-777", op="store", rows=777, src=4099, hkv=4, D=64, page=32, pages=512,
             rope=False, norm=False, gather=True, skip=0.1),
        # a shared prefix of 1025 rows comes back as bf16 rows, for items scored over it
        dict(name="read-prefix-1025", op="read", rows=1025, hkv=8, D=128, page=16, pages=300, skip=0.0),
        # the prefixes of 16 requests, 64K rows
        dict(name="read-prefixes-64k", op="read", rows=65536, hkv=8, D=128, page=64, pages=1100, skip=0.0),
        # a few requests of the decision workload's size decode one token: latency
        dict(name="attn-decode-4", op="attn", shape=7, B=4, hq=16, hkv=8, D=128, page=16, len_lo=100,
             len_hi=300, n_lo=1, n_hi=1),
        # a running batch decodes one token each over prefixes of 512 to 4096
        dict(name="attn-decode-64", op="attn", shape=8, B=64, hq=16, hkv=8, D=128, page=64, len_lo=512,
             len_hi=4096, n_lo=1, n_hi=1),
        # long contexts, 1 to 8 new tokens: the K/V stream
        dict(name="attn-long-4", op="attn", shape=11, B=4, hq=32, hkv=8, D=128, page=64, len_lo=65536,
             len_hi=131072, n_lo=1, n_hi=8),
        # odd everything: 3 query heads a kv head, 64-wide, short caches
        dict(name="attn-odd-5", op="attn", shape=12, B=5, hq=12, hkv=4, D=64, page=32, len_lo=1,
             len_hi=777, n_lo=1, n_hi=13),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "store", "read", "attn", "attn"])
    if op == "norm":
        hq, hkv = rng.choice([(16, 8), (32, 8), (4, 2), (12, 4), (6, 6), (8, 1), (20, 4)])
        D = rng.choice([64, 128])
        return dict(op=op, T=_log(rng, 1, 131072 * 24 * 128 // ((hq + hkv) * D)), hq=hq, hkv=hkv, D=D,
                    far=_log(rng, 16, 1 << 20))
    page = rng.choice([16, 32, 64, 128, 256])
    if op in ("store", "read"):
        rows = _log(rng, 1, 131072 if op == "store" else 65536)
        c = dict(op=op, rows=rows, hkv=rng.choice([1, 2, 3, 4, 8]), D=rng.choice([64, 128]), page=page,
                 pages=rows // page + rng.randrange(1, 50), skip=rng.choice([0.0, 0.0, 0.2]))
        if op == "store":
            c["gather"] = rng.random() < 0.4
            c["src"] = rows + (rng.randrange(500) if c["gather"] else 0)
            c["norm"], c["rope"] = rng.choice([(False, False), (False, True), (True, True), (True, True)])
        return c
    hq, hkv, D = rng.choice([(16, 8, 128), (32, 8, 128), (4, 2, 64), (12, 4, 64), (6, 6, 128),
                             (8, 1, 128), (20, 4, 128)])
    n_hi = _log(rng, 1, 32)
    n_lo = rng.choice([1, n_hi])
    len_hi = _log(rng, 1, 131072)
    # no more key rows in all than the largest listed case, nor many more products
    most = min(400000 // len_hi, 8000000 // (len_hi * n_hi * hq // 32 + 1), 2000 // n_hi)
    return dict(op=op, shape=rng.randrange(1000, 1 << 30), B=_log(rng, 1, max(1, min(128, most))), hq=hq,
                hkv=hkv, D=D, page=page, len_lo=rng.choice([1, max(1, len_hi // 8), len_hi]), len_hi=len_hi,
                n_lo=n_lo, n_hi=n_hi)


def _attn_lengths(c):
    """Cached rows (the new ones among them) and new rows of every request."""
    r = random.Random(c["shape"])
    lens = [r.randint(c["len_lo"], c["len_hi"]) for _ in range(c["B"])]
    n = [min(l, r.randint(c["n_lo"], c["n_hi"])) for l in lens]
    return lens, n


def work(case):
    c = case
    if c["op"] == "norm":
        cells = c["T"] * (c["hq"] + c["hkv"]) * c["D"]
        return {"bytes": 4 * cells + 4 * c["T"] + 4 * c["D"], "flops": 7.0 * cells}
    if c["op"] in ("store", "read"):
        kept = c["rows"] * (1.0 - c["skip"])
        cells = 2 * c["hkv"] * kept * c["D"]                        # of K and V
        back = 3 * cells + 2 * c["hkv"] * kept + 4 * c["rows"]      # codes and scales in, bf16 out, a slot a row
        if c["op"] == "read":
            return {"bytes": back, "flops": cells}
        return {"bytes": 3 * cells + 2 * c["hkv"] * kept + 4 * c["rows"] * (1 + c["rope"] + c["gather"]) + back,
                "flops": cells * (4.0 + 2.0 * c["norm"] + 1.5 * c["rope"])}
    lens, n = _attn_lengths(c)
    pairs = sum(l * m - m * (m - 1) // 2 for l, m in zip(lens, n))
    return {"bytes": sum(lens) * c["hkv"] * (2 * c["D"] + 2) + sum(n) * c["hq"] * (4 * c["D"] + 4) +
            4 * sum(-(-l // c["page"]) for l in lens),
            "flops": 4.0 * c["D"] * c["hq"] * pairs}


# -------------------------------------------------------------------- inputs

def _gen(seed, dev="cuda"):
    return torch.Generator(device=dev).manual_seed(int(seed))


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _rows(g, *shape):
    """Projected rows: normal, of a size of its own each."""
    size = torch.exp(0.4 * torch.randn(*shape[:-1], 1, generator=g, device="cuda"))
    return (torch.randn(shape, generator=g, device="cuda") * size).to(torch.bfloat16)


def _pool(g, c, n_pages, filled):
    """Codes [page, row, kv head, D] and exponent bytes [page, kv head, row] of a cache."""
    shape = (n_pages, c["page"], c["hkv"], c["D"])
    codes = torch.zeros(shape, dtype=torch.uint8, device="cuda")
    scale = torch.full((n_pages, c["hkv"], c["page"]), E_LO + 127, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 25) // (c["page"] * c["hkv"] * c["D"]))
    for p in range(0, n_pages if filled else 0, step):
        x = _rows(g, min(step, n_pages - p), *shape[1:])
        codes[p:p + step], e = _plain_quantise(x.float())
        scale[p:p + step] = e.transpose(1, 2)
    return codes, scale


def prepare(case, seed):
    c = case
    s = {"op": c["op"], "case": c}
    g = _gen(seed)
    hkv, D = c["hkv"], c["D"]

    def weight():
        return (1.0 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(torch.bfloat16)

    if c["op"] == "norm":
        T, hq = c["T"], c["hq"]
        qkv = _rows(g, T, hq + 2 * hkv, D)                  # the projection's output
        s.update(q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], q_weight=weight(), k_weight=weight(),
                 position_ids=torch.randint(0, c["far"], (T,), generator=g, device="cuda", dtype=torch.int32))
    elif c["op"] in ("store", "read"):
        n, p = c["rows"], c["page"]
        s["k_codes"], s["k_scale"] = _pool(g, c, c["pages"], c["op"] == "read")
        s["v_codes"], s["v_scale"] = _pool(g, c, c["pages"], c["op"] == "read")
        slots = torch.randperm(c["pages"] * p, generator=g, device="cuda")[:n].to(torch.int32)
        if n > 1000 and not c.get("gather"):
            # a prompt's rows go page by page: runs of consecutive slots
            pages = torch.randperm(c["pages"], generator=g, device="cuda").to(torch.int32)
            t = torch.arange(n, device="cuda")
            slots = pages[t // p] * p + (t % p).to(torch.int32)
        if c["skip"]:
            off = torch.rand(n, generator=g, device="cuda") < c["skip"]
            slots = torch.where(off, torch.full_like(slots, -1), slots)
        s["slot_map"] = slots
        s["k_out"] = torch.zeros(n, hkv, D, dtype=torch.bfloat16, device="cuda")
        s["v_out"] = torch.zeros(n, hkv, D, dtype=torch.bfloat16, device="cuda")
        if c["op"] == "store":
            s["k"], s["v"] = _rows(g, c["src"], hkv, D), _rows(g, c["src"], hkv, D)
            s["k_weight"] = weight() if c["norm"] else None
            s["position_ids"] = torch.randint(0, 131072, (n,), generator=g, device="cuda",
                                              dtype=torch.int32) if c["rope"] else None
            s["src_rows"] = torch.randint(0, c["src"], (n,), generator=g, device="cuda",
                                          dtype=torch.int32) if c["gather"] else None
    else:
        lens, n = _attn_lengths(c)
        p, B, T = c["page"], c["B"], sum(n)
        pages = [-(-l // p) for l in lens]
        n_pages = sum(pages) + 3
        order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
        table = torch.zeros((B, max(pages)), dtype=torch.int32, device="cuda")
        at = 0
        for b in range(B):
            table[b, :pages[b]] = order[at:at + pages[b]]
            at += pages[b]
        s["k_codes"], s["k_scale"] = _pool(g, c, n_pages, True)
        s["v_codes"], s["v_scale"] = _pool(g, c, n_pages, True)
        s.update(q=torch.randn(T, c["hq"], D, generator=g, device="cuda", dtype=torch.bfloat16),
                 block_table=table, cache_len=_i32(lens), cu_rows=_i32([0] + np.cumsum(n).tolist()),
                 max_rows=max(n), max_len=max(lens))
    if own:
        _own_prepare(s)
    return s


def _own_prepare(s):
    """What a serving program keeps between calls: the cache's handle, a
    workspace, and the outputs' buffers."""
    from ranking_prefill_gb300 import lib
    s["lib"] = lib
    if s["op"] == "norm":
        s["q_out"] = torch.empty(s["q"].shape, dtype=torch.bfloat16, device="cuda")
        s["k_out"] = torch.empty(s["k"].shape, dtype=torch.bfloat16, device="cuda")
        return
    s["cache"] = lib.PagedCacheQ8(s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"])
    size = lib.mis_paged_write_workspace_size()
    if s["op"] == "attn":
        s["desc"] = lib.PagedAttentionDesc(s["cache"], B=int(s["cache_len"].numel()), T=int(s["q"].shape[0]),
                                           Hq=int(s["q"].shape[1]), max_rows=s["max_rows"])
        size = s["desc"].workspace_size()
        s["o"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(s["q"].shape[1], s["q"].shape[0], dtype=torch.float32, device="cuda")
    s["workspace"] = torch.zeros(size, dtype=torch.uint8, device="cuda")


# ----------------------------------------------------------------------- run

def run(state):
    s = state
    if s["op"] == "norm":
        if not own:
            return {"q": _plain_norm_rope(s["q"], s["q_weight"], s["position_ids"]).to(torch.bfloat16),
                    "k": _plain_norm_rope(s["k"], s["k_weight"], s["position_ids"]).to(torch.bfloat16)}
        s["lib"].mis_qk_norm_rope(s["q"], s["k"], s["q_out"], s["k_out"], s["position_ids"],
                                  q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS, base=ROPE_BASE)
        return {"q": s["q_out"], "k": s["k_out"]}
    if s["op"] == "attn":
        if not own:
            return _plain_attention(s)
        s["lib"].mis_paged_attention_q8_fwd(s["desc"], s["q"], s["o"], s["lse"], s["block_table"],
                                            s["cache_len"], s["cu_rows"], s["workspace"])
        return {"o": s["o"], "lse": s["lse"]}
    if own:
        if s["op"] == "store":
            s["lib"].mis_paged_write_kv_q8(s["cache"], s["k"], s["v"], s["slot_map"], s["workspace"],
                                           position_ids=s["position_ids"], base=ROPE_BASE,
                                           src_rows=s["src_rows"], k_weight=s["k_weight"], eps=EPS)
        s["lib"].mis_paged_read_kv_q8(s["cache"], s["slot_map"], s["k_out"], s["v_out"], s["workspace"])
    else:
        if s["op"] == "store":
            _plain_store(s)
        _plain_read(s)
    return {"k": s["k_out"], "v": s["v_out"]}


def _plain_norm_rope(x, weight, positions):
    """[rows, heads, D] in 32 bits: root mean square norm of each head, then the rotation."""
    D = x.shape[-1]
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(dim=-1, keepdim=True) + EPS) * weight.float()
    if positions is None:
        return x
    f = ROPE_BASE ** (-2.0 * torch.arange(D // 2, device=x.device, dtype=torch.float64) / D)
    a = positions.double()[:, None] * f
    cos, sin = a.cos().float()[:, None, :], a.sin().float()[:, None, :]
    x, y = x[..., :D // 2], x[..., D // 2:]
    return torch.cat([x * cos - y * sin, y * cos + x * sin], dim=-1)


def _plain_quantise(x):
    """Codes (as bytes) and exponent bytes of rows in 32 bits: the least power
    of two that brings a row's largest value to 448 at most."""
    m, e = torch.frexp(x.abs().amax(dim=-1))                  # |x| = m 2^e, m in [0.5, 1); 448 = 0.875 2^9
    e = (e - 9 + (m > 0.875)).clamp(E_LO, E_HI)
    codes = (x * torch.exp2(-e.float())[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, (e + 127).to(torch.uint8)


def _power(e):
    """2^(e - 127) of exponent bytes, in 32 bits."""
    return (e.to(torch.int32) << 23).view(torch.float32)


def _plain_store(s):
    hkv, D = s["k"].shape[1:]
    keep = (s["slot_map"] >= 0).nonzero().flatten()
    slots = s["slot_map"][keep].long()
    page, row = slots // s["k_codes"].shape[1], slots % s["k_codes"].shape[1]
    rows = keep if s["src_rows"] is None else s["src_rows"][keep].long()
    pos = None if s["position_ids"] is None else s["position_ids"][keep]
    for x, codes, scale in ((_plain_norm_rope(s["k"][rows], s["k_weight"], pos), s["k_codes"], s["k_scale"]),
                            (s["v"][rows].float(), s["v_codes"], s["v_scale"])):
        q, e = _plain_quantise(x)
        codes.view(-1, hkv, D)[slots] = q
        scale[page, :, row] = e


def _plain_read(s):
    p, hkv, D = s["k_codes"].shape[1:]
    keep = (s["slot_map"] >= 0).nonzero().flatten()
    slots = s["slot_map"][keep].long()
    for codes, scale, out in ((s["k_codes"], s["k_scale"], s["k_out"]), (s["v_codes"], s["v_scale"], s["v_out"])):
        x = codes.view(-1, hkv, D)[slots].view(torch.float8_e4m3fn).float()
        out[keep] = (x * _power(scale[slots // p, :, slots % p])[..., None]).to(torch.bfloat16)


def _plain_gather(codes, scale, page, row):
    """[B, L, hkv, D] values in 32 bits of the rows at (page, row) [B, L]."""
    return codes[page, row].view(torch.float8_e4m3fn).float() * _power(scale[page, :, row])[..., None]


def _plain_attention(s):
    q, dev = s["q"], s["q"].device
    T, hq, D = q.shape
    p, hkv = s["k_codes"].shape[1:3]
    n, L, G = s["max_rows"], s["max_len"], hq // hkv
    lens, cu = s["cache_len"].long(), s["cu_rows"].long()
    B = lens.numel()
    i, at = torch.arange(n, device=dev), torch.arange(L, device=dev)
    row = cu[:-1, None] + i                                             # [B, n] packed rows
    live = row < cu[1:, None]
    row = row.clamp(max=T - 1)
    page = s["block_table"].long()[:, at // p]
    off = (at % p).expand(B, L)
    K = _plain_gather(s["k_codes"], s["k_scale"], page, off).transpose(1, 2)
    V = _plain_gather(s["v_codes"], s["v_scale"], page, off).transpose(1, 2)
    # row i of n_b sees the cached rows up to its own
    seen = lens[:, None] - (cu[1:] - cu[:-1])[:, None] + i + 1          # [B, n]
    see = at < seen[:, :, None]
    see = see.repeat_interleave(G, dim=1)[:, None]                      # rows: token-major, then head of the group
    Q = q[row].float().view(B, n, hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, hkv, n * G, D)
    S = (Q @ K.transpose(2, 3)) * (1.0 / math.sqrt(D))
    S = torch.where(see, S, torch.full_like(S, -math.inf))
    m = S.amax(dim=-1, keepdim=True)
    P = torch.exp(S - m)
    l = P.sum(dim=-1, keepdim=True)
    O = (P @ V) / l
    lse = (m + torch.log(l))[..., 0]
    O = O.view(B, hkv, n, G, D).permute(0, 2, 1, 3, 4).reshape(B, n, hq, D)
    lse = lse.view(B, hkv, n, G).permute(0, 2, 1, 3).reshape(B, n, hq)
    o = torch.empty_like(q)
    out = torch.empty(hq, T, dtype=torch.float32, device=dev)
    o[row[live]] = O[live].to(q.dtype)
    out.t()[row[live]] = lse[live]
    return {"o": o, "lse": out}


# --------------------------------------------------------------------- exact

def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "norm":
        return {"q": _exact_norm_rope(s["q"], s["q_weight"], s["position_ids"]),
                "k": _exact_norm_rope(s["k"], s["k_weight"], s["position_ids"])}
    if s["op"] == "attn":
        return _exact_attention(s)
    out = {"k": s["k_out"].double(), "v": s["v_out"].double()}
    keep = (s["slot_map"] >= 0).nonzero().flatten()
    if s["op"] == "store":
        rows = keep if s["src_rows"] is None else s["src_rows"][keep].long()
        pos = None if s["position_ids"] is None else s["position_ids"][keep]
        out["k"][keep] = _exact_stored(_exact_norm_rope(s["k"][rows], s["k_weight"], pos))
        out["v"][keep] = _exact_stored(s["v"][rows].double())
    else:
        slots = s["slot_map"][keep].long()
        p = case["page"]
        for name in ("k", "v"):
            codes = s[name + "_codes"][slots // p, slots % p]
            e = s[name + "_scale"].transpose(1, 2)[slots // p, slots % p].double() - 127.0
            out[name][keep] = _exact_code(codes) * torch.exp2(e)[..., None]
    return out


def _exact_norm_rope(x, weight, positions):
    """Complex rotation of the pairs in 64 bits."""
    x, D = x.double(), x.shape[-1]
    if weight is not None:
        x = weight.double() * x / torch.sqrt((x * x).sum(dim=-1, keepdim=True) / D + EPS)
    if positions is None:
        return x
    turn = torch.pow(torch.tensor(ROPE_BASE, dtype=torch.float64, device=x.device),
                     torch.arange(0, D, 2, device=x.device, dtype=torch.float64) / -D)
    angle = torch.outer(positions.double(), turn)[:, None, :]
    z = torch.complex(x[..., :D // 2].contiguous(), x[..., D // 2:].contiguous())
    z = z * torch.polar(torch.ones_like(angle), angle)
    return torch.cat([z.real, z.imag], dim=-1)


def _exact_stored(x):
    """What rows in 64 bits are held as: multiples of a step that goes by the
    value's own power of two (3 bits behind the leading one, steps of 2^-9 at
    the small end), in units of the row's scale."""
    a = x.abs().amax(dim=-1, keepdim=True)
    e = torch.ceil(torch.log2(a / 448.0))
    e = torch.where(a > 448.0 * torch.exp2(e), e + 1, torch.where(a <= 224.0 * torch.exp2(e), e - 1, e))
    unit = torch.exp2(torch.where(a > 0, e, torch.full_like(e, E_LO)).clamp(E_LO, E_HI))
    y = x / unit
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3.0)
    return torch.round(y / step) * step * unit


def _exact_code(codes):
    """e4m3: sign, 4 bits of exponent (bias 7), 3 of fraction."""
    c = codes.long()
    e, f = (c >> 3) & 15, (c & 7).double()
    mag = torch.where(e > 0, (8.0 + f) * torch.exp2((e - 10).double()), f * 2.0 ** -9)
    return torch.where(c >= 128, -mag, mag)


def _exact_attention(s):
    """One request and query head at a time."""
    c = s["case"]
    lens, n = _attn_lengths(c)
    q, p, hkv = s["q"].double(), c["page"], c["hkv"]
    T, hq, D = q.shape
    G = hq // hkv
    o = torch.zeros_like(q)
    lse = torch.full((hq, T), -math.inf, dtype=torch.float64, device=q.device)
    r0 = 0
    for L, nb, pages in zip(lens, n, s["block_table"]):
        pages = pages[:-(-L // p)].long()
        last = torch.arange(L - nb, L, device=q.device)
        hide = torch.arange(L, device=q.device)[None, :] > last[:, None]
        for h in range(hkv):
            k, v = ((_exact_code(s[x + "_codes"][pages, :, h]) *
                     torch.exp2(s[x + "_scale"][pages, h].double() - 127.0)[..., None]).reshape(-1, D)[:L]
                    for x in "kv")
            for g in range(h * G, h * G + G):
                z = (q[r0:r0 + nb, g] @ k.T / math.sqrt(D)).masked_fill(hide, -math.inf)
                lse[g, r0:r0 + nb] = torch.logsumexp(z, dim=1)
                o[r0:r0 + nb, g] = torch.softmax(z, dim=1) @ v
        r0 += nb
    return {"o": o, "lse": lse}
