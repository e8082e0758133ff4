"""Measured cases of the paged K/V cache operators: GPU-built block tables and
slot maps, rows written into the cache (rotary embedding of K on the way), and
attention of drafted token trees (or single tokens) over the cache.

A case is a dict of plain values. Its lengths come from the case's own
``shape`` number, its values from the seed, so the work of a case is fixed.
The plain forms are elementary torch operations in 32 bits (64 for rotary
angles); ``exact`` restates the definitions in 64 bits, request by request.
"""
import math
import random

import numpy as np
import torch

own = False

ROPE_BASE = 1.0e6


# --------------------------------------------------------------------- cases

def listed():
    return [
        # one decoding step of 32 running requests: a new slot each, a page now and then
        dict(name="extend-decode-32", op="extend", shape=1, B=32, page=16, len_lo=100, len_hi=3000,
             new_lo=1, new_hi=1, spare=0),
        # 16 prompts of 201K tokens in all enter an empty cache (the varlen-16 batch's size)
        dict(name="extend-prompts-16", op="extend", shape=2, B=16, page=64, len_lo=0, len_hi=0,
             new_lo=9000, new_hi=16137, spare=129),
        # 256 requests grow by chunks of up to 8K tokens: about a million slots, odd starts
        dict(name="extend-chunks-256", op="extend", shape=3, B=256, page=16, len_lo=0, len_hi=5000,
             new_lo=1, new_hi=8191, spare=7),
        # one decoding step of 32 requests: rotate and store one row each
        dict(name="write-decode-32", op="write", shape=4, rows=32, src=32, hkv=8, D=128, page=16,
             pages=4096, rope=True, gather=False, skip=0.0),
        # 128K prompt rows rotated into the cache
        dict(name="write-prompt-128k", op="write", shape=5, rows=131072, src=131072, hkv=8, D=128,
             page=64, pages=2200, rope=True, gather=False, skip=0.0),
        # accepted rows of drafted trees, picked by index, 64-wide heads, some slots skipped
        dict(name="write-accepted-777", op="write", shape=6, rows=777, src=4099, hkv=4, D=64, page=32,
             pages=512, rope=False, gather=True, skip=0.1),
        # a few requests of the decision workload's size decode one token: latency
        dict(name="attn-decode-4", op="attn", shape=7, B=4, hq=16, hkv=8, D=128, page=16, len_lo=100,
             len_hi=300, n_lo=1, n_hi=1, tree=False, unused=0.0),
        # a running batch decodes one token each over prefixes of 512 to 4096
        dict(name="attn-decode-64", op="attn", shape=8, B=64, hq=16, hkv=8, D=128, page=64,
             len_lo=512, len_hi=4096, n_lo=1, n_hi=1, tree=False, unused=0.0),
        # drafted trees of 8 to 32 tokens, ragged, a few nodes pruned
        dict(name="attn-tree-8", op="attn", shape=9, B=8, hq=16, hkv=8, D=128, page=16, len_lo=512,
             len_hi=4096, n_lo=8, n_hi=32, tree=True, unused=0.05),
        # full trees of 64 tokens, 4 query heads a kv head: 256 rows share each key, tensor work
        dict(name="attn-tree-64x16", op="attn", shape=10, B=16, hq=32, hkv=8, D=128, page=128,
             len_lo=2000, len_hi=8000, n_lo=64, n_hi=64, tree=True, unused=0.0),
        # long contexts, short chains of drafted tokens: the K/V stream
        dict(name="attn-long-4", op="attn", shape=11, B=4, hq=32, hkv=8, D=128, page=64,
             len_lo=65536, len_hi=131072, n_lo=1, n_hi=8, tree=False, unused=0.0),
        # odd everything: 3 query heads a kv head, 64-wide, short caches (one of them may be empty)
        dict(name="attn-odd-5", op="attn", shape=12, B=5, hq=12, hkv=4, D=64, page=32, len_lo=0,
             len_hi=777, n_lo=1, n_hi=13, tree=True, unused=0.1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["extend", "write", "attn", "attn"])
    page = rng.choice([16, 32, 64, 128, 256])
    shape = rng.randrange(1000, 1 << 30)
    if op == "extend":
        B = _log(rng, 1, 256)
        hi = _log(rng, 1, 8191)
        return dict(op=op, shape=shape, B=B, page=page, len_lo=0, len_hi=_log(rng, 1, 5000),
                    new_lo=rng.choice([0, 1, hi]), new_hi=hi, spare=rng.randrange(200))
    if op == "write":
        rows = _log(rng, 1, 131072)
        gather = rng.random() < 0.4
        return dict(op=op, shape=shape, rows=rows, src=rows + (rng.randrange(500) if gather else 0),
                    hkv=rng.choice([1, 2, 3, 4, 8]), D=rng.choice([64, 128]), page=page,
                    pages=rows // page + rng.randrange(1, 50), rope=rng.random() < 0.6, gather=gather,
                    skip=rng.choice([0.0, 0.0, 0.2]))
    hq, hkv, D = rng.choice([(16, 8, 128), (32, 8, 128), (4, 2, 64), (12, 4, 64), (6, 6, 128),
                             (8, 1, 128), (20, 4, 128)])
    n_hi = _log(rng, 1, 64)
    n_lo = rng.choice([1, n_hi])
    len_hi = _log(rng, 1, 131072)
    # no more key rows in all than the largest listed case, nor more products than the tree case
    most = min(400000 // len_hi, 8000000 // (len_hi * n_hi * hq // 32 + 1), 2000 // n_hi)
    B = _log(rng, 1, max(1, min(128, most)))
    return dict(op=op, shape=shape, B=B, hq=hq, hkv=hkv, D=D, page=page,
                len_lo=rng.choice([0, len_hi // 8, len_hi]), len_hi=len_hi, n_lo=n_lo, n_hi=n_hi,
                tree=n_hi > 1 and rng.random() < 0.7, unused=rng.choice([0.0, 0.0, 0.1]) if n_hi > 1 else 0.0)


def _extend_lengths(c):
    r = random.Random(c["shape"])
    lens = [r.randint(c["len_lo"], c["len_hi"]) for _ in range(c["B"])]
    new = [r.randint(c["new_lo"], c["new_hi"]) for _ in range(c["B"])]
    return lens, new


def _attn_lengths(c):
    r = random.Random(c["shape"])
    lens = [r.randint(c["len_lo"], c["len_hi"]) for _ in range(c["B"])]
    n = [r.randint(c["n_lo"], c["n_hi"]) for _ in range(c["B"])]
    return lens, n


def _attn_parents(c, n):
    """Parents of every request's nodes (index inside the request, -1 a root,
    -2 an unused node), or None for chains."""
    if not c["tree"] and not c["unused"]:
        return None
    r = random.Random(c["shape"] + 1)
    out = []
    for nb in n:
        for i in range(nb):
            p = max(-1, i - 1 - (r.randrange(4) if c["tree"] else 0))
            out.append(-2 if i > 0 and r.random() < c["unused"] else p)
    return out


def work(case):
    c = case
    if c["op"] == "extend":
        lens, new = _extend_lengths(c)
        T, p = sum(new), c["page"]
        fresh = sum(-(-(l + n) // p) - (-(-l // p)) for l, n in zip(lens, new))
        # lengths in and out, page ids in and table entries out, a slot and a position a token
        return {"bytes": 4 * (4 * c["B"] + 2 + 2 * fresh) + 8 * (T + c["spare"]), "flops": 0}
    if c["op"] == "write":
        # kept rows read and written once, K and V
        row = 2 * 2 * c["hkv"] * c["D"]
        kept = c["rows"] * (1.0 - c["skip"])
        return {"bytes": 2 * row * kept + c["rows"] * (4 + 4 * c["rope"] + 4 * c["gather"]),
                "flops": 3.0 * c["hkv"] * c["D"] * kept * c["rope"]}
    lens, n = _attn_lengths(c)
    kv = 4 * c["hkv"] * c["D"]
    keys = sum(lens) + sum(n)
    pairs = sum(l * m for l, m in zip(lens, n)) + sum(m * (m + 1) // 2 for m in n) * (0.3 if c["tree"] else 1.0)
    return {"bytes": kv * keys + sum(n) * c["hq"] * (4 * c["D"] + 4) + 4 * sum(-(-l // c["page"]) for l in lens),
            "flops": 4.0 * c["D"] * c["hq"] * pairs}


# -------------------------------------------------------------------- inputs

def _gen(seed, dev="cuda"):
    return torch.Generator(device=dev).manual_seed(int(seed))


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    c = case
    s = {"op": c["op"], "case": c}
    g = _gen(seed)
    if c["op"] == "extend":
        lens, new = _extend_lengths(c)
        p, B = c["page"], c["B"]
        have = [-(-l // p) for l in lens]
        need = [-(-(l + n) // p) for l, n in zip(lens, new)]
        n_pages = sum(need) + 5
        order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
        cols = max(max(need), 1)
        table = torch.full((B, cols), -1, dtype=torch.int32, device="cuda")
        first = np.concatenate([[0], np.cumsum(have)])
        for b in range(B):
            table[b, :have[b]] = order[int(first[b]):int(first[b]) + have[b]]
        T = sum(new) + c["spare"]
        s.update(n_pages=n_pages, page=p, new_len=_i32(new), cache_len=_i32(lens), block_table=table,
                 free_pages=order, free_head=_i32([int(first[-1])]), T=T,
                 cache_len_out=torch.empty(B, dtype=torch.int32, device="cuda"),
                 free_head_out=torch.empty(1, dtype=torch.int32, device="cuda"),
                 cu_new=torch.empty(B + 1, dtype=torch.int32, device="cuda"),
                 slot_map=torch.empty(T, dtype=torch.int32, device="cuda"),
                 position_ids=torch.empty(T, dtype=torch.int32, device="cuda"))
    elif c["op"] == "write":
        shape = (c["src"], c["hkv"], c["D"])
        s["k"] = torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)
        s["v"] = torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)
        pool = (c["pages"], c["page"], c["hkv"], c["D"])
        s["k_cache"] = torch.zeros(pool, dtype=torch.bfloat16, device="cuda")
        s["v_cache"] = torch.zeros(pool, dtype=torch.bfloat16, device="cuda")
        slots = torch.randperm(c["pages"] * c["page"], generator=g, device="cuda")[:c["rows"]].to(torch.int32)
        if c["rows"] > 1000 and not c["gather"]:
            # a prompt's rows go page by page: runs of consecutive slots
            pages = torch.randperm(c["pages"], generator=g, device="cuda").to(torch.int32)
            t = torch.arange(c["rows"], device="cuda")
            slots = pages[t // c["page"]] * c["page"] + (t % c["page"]).to(torch.int32)
        if c["skip"]:
            off = torch.rand(c["rows"], generator=g, device="cuda") < c["skip"]
            slots = torch.where(off, torch.full_like(slots, -1), slots)
        s["slot_map"] = slots
        s["position_ids"] = torch.randint(0, 131072, (c["rows"],), generator=g, device="cuda",
                                          dtype=torch.int32) if c["rope"] else None
        s["src_rows"] = torch.randint(0, c["src"], (c["rows"],), generator=g, device="cuda",
                                      dtype=torch.int32) if c["gather"] else None
    else:
        lens, n = _attn_lengths(c)
        p, B, T = c["page"], c["B"], sum(n)
        pages = [-(-l // p) for l in lens]
        n_pages = sum(pages) + 3
        order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
        table = torch.zeros((B, max(max(pages), 1)), dtype=torch.int32, device="cuda")
        at = 0
        for b in range(B):
            table[b, :pages[b]] = order[at:at + pages[b]]
            at += pages[b]

        def rand(*shape):
            return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)

        parents = _attn_parents(c, n)
        s.update(q=rand(T, c["hq"], c["D"]), k=rand(T, c["hkv"], c["D"]), v=rand(T, c["hkv"], c["D"]),
                 k_cache=rand(n_pages, p, c["hkv"], c["D"]), v_cache=rand(n_pages, p, c["hkv"], c["D"]),
                 block_table=table, cache_len=_i32(lens),
                 cu_nodes=_i32([0] + np.cumsum(n).tolist()), max_nodes=max(n), max_len=max(lens),
                 parents=None if parents is None else _i32(parents))
    if own:
        _own_prepare(s)
    return s


def _own_prepare(s):
    """What a serving program keeps between calls: the cache's handle, a
    workspace, and the outputs' buffers."""
    from ranking_prefill_gb300 import lib
    s["lib"] = lib
    if s["op"] == "extend":
        size = lib.mis_paged_extend_workspace_size(int(s["new_len"].numel()))
    elif s["op"] == "write":
        s["cache"] = lib.PagedCache(s["k_cache"], s["v_cache"])
        size = lib.mis_paged_write_workspace_size()
    else:
        s["cache"] = lib.PagedCache(s["k_cache"], s["v_cache"])
        s["desc"] = lib.TreeDesc(s["cache"], B=int(s["cache_len"].numel()), T=int(s["q"].shape[0]),
                                 Hq=int(s["q"].shape[1]), max_nodes=s["max_nodes"])
        size = s["desc"].workspace_size()
        s["o"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(s["q"].shape[1], s["q"].shape[0], dtype=torch.float32, device="cuda")
    s["workspace"] = torch.zeros(size, dtype=torch.uint8, device="cuda")


# ----------------------------------------------------------------------- run

def run(state):
    s = state
    if s["op"] == "extend":
        if own:
            s["lib"].mis_paged_extend(s["new_len"], s["cache_len"], s["cache_len_out"], s["block_table"],
                                      s["free_pages"], s["free_head"], s["free_head_out"], s["cu_new"],
                                      s["slot_map"], s["position_ids"], s["page"], s["n_pages"],
                                      s["workspace"])
        else:
            _plain_extend(s)
        return {k: s[k] for k in ("block_table", "cache_len_out", "free_head_out", "cu_new", "slot_map",
                                  "position_ids")}
    if s["op"] == "write":
        if own:
            s["lib"].mis_paged_write_kv(s["cache"], s["k"], s["v"], s["slot_map"], s["workspace"],
                                        position_ids=s["position_ids"], base=ROPE_BASE,
                                        src_rows=s["src_rows"])
        else:
            _plain_write(s)
        return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if own:
        s["lib"].mis_tree_attention_fwd(s["desc"], s["q"], s["k"], s["v"], s["o"], s["lse"],
                                        s["block_table"], s["cache_len"], s["cu_nodes"], s["parents"],
                                        s["workspace"])
        return {"o": s["o"], "lse": s["lse"]}
    return _plain_attention(s)


def _plain_extend(s):
    p = s["page"]
    new, lens, table = s["new_len"].long(), s["cache_len"].long(), s["block_table"]
    B, cols = table.shape
    have = (lens + p - 1) // p
    need = (lens + new + p - 1) // p - have
    first = s["free_head"].long() + torch.cumsum(need, 0) - need
    cu = torch.zeros(B + 1, dtype=torch.long, device=table.device)
    cu[1:] = torch.cumsum(new, 0)
    # table: the columns behind the old pages take the request's run of the free list
    col = torch.arange(cols, device=table.device)[None, :]
    fresh = col - have[:, None]
    take = (fresh >= 0) & (fresh < need[:, None])
    last = s["free_pages"].numel() - 1
    table.copy_(torch.where(take, s["free_pages"][(first[:, None] + fresh).clamp(0, last)], table))
    # tokens: the request whose run of rows holds them, their position, their page's slot
    t = torch.arange(s["T"], device=table.device)
    b = torch.searchsorted(cu[1:], t, right=True)
    live = b < B
    b = b.clamp(max=B - 1)
    pos = lens[b] + t - cu[b]
    page = table[b, (pos // p).clamp(0, cols - 1)].long()
    s["slot_map"].copy_(torch.where(live, page * p + pos % p, torch.full_like(pos, -1)))
    s["position_ids"].copy_(torch.where(live, pos, torch.zeros_like(pos)))
    s["cu_new"].copy_(cu)
    s["cache_len_out"].copy_(lens + new)
    s["free_head_out"].copy_(s["free_head"] + need.sum())


def _plain_write(s):
    H, D = s["k"].shape[1:]
    keep = (s["slot_map"] >= 0).nonzero().flatten()
    slots = s["slot_map"][keep].long()
    rows = keep if s["src_rows"] is None else s["src_rows"][keep].long()
    k, v = s["k"][rows], s["v"][rows]
    if s["position_ids"] is not None:
        f = ROPE_BASE ** (-2.0 * torch.arange(D // 2, device=k.device, dtype=torch.float64) / D)
        a = s["position_ids"][keep].double()[:, None] * f
        cos, sin = a.cos().float()[:, None, :], a.sin().float()[:, None, :]
        x, y = k[..., :D // 2].float(), k[..., D // 2:].float()
        k = torch.cat([x * cos - y * sin, y * cos + x * sin], dim=-1).to(torch.bfloat16)
    s["k_cache"].view(-1, H, D)[slots] = k
    s["v_cache"].view(-1, H, D)[slots] = v


def _twice(a):
    return (a @ a).clamp(max=1.0)


def _plain_attention(s):
    q, k, v = s["q"], s["k"], s["v"]
    T, hq, D = q.shape
    hkv, p, n, dev = k.shape[1], s["k_cache"].shape[1], s["max_nodes"], q.device
    G, L = hq // hkv, s["max_len"]
    lens, cu = s["cache_len"].long(), s["cu_nodes"].long()
    B = lens.numel()
    i = torch.arange(n, device=dev)
    row = cu[:-1, None] + i                                             # [B, n] packed rows
    live = row < cu[1:, None]
    row = row.clamp(max=T - 1)
    # ancestors of every node: the parent relation, closed (trees of up to 256 levels)
    par = i - 1 if s["parents"] is None else s["parents"][row].long()
    par = par.expand(B, n)
    used = live & (par > -2)
    up = (par[:, :, None] == i) & used[:, :, None] & used[:, None, :]
    eye = torch.eye(n, device=dev, dtype=torch.bool) & used[:, :, None]
    anc = (up | eye).float()
    anc = _twice(_twice(_twice(_twice(_twice(_twice(_twice(_twice(anc)))))))) > 0
    # the cache's rows by block table, then the request's own rows
    at = torch.arange(L, device=dev)
    slot = s["block_table"].long()[:, at // p] * p + at % p if L else torch.zeros(B, 0, dtype=torch.long, device=dev)
    K = torch.cat([s["k_cache"].view(-1, hkv, D)[slot], k[row]], dim=1).float().transpose(1, 2)
    V = torch.cat([s["v_cache"].view(-1, hkv, D)[slot], v[row]], dim=1).float().transpose(1, 2)
    see = torch.cat([(at < lens[:, None])[:, None, :] & used[:, :, None], anc], dim=2)     # [B, n, L + n]
    see = see.repeat_interleave(G, dim=1)[:, None]                      # rows: node-major, then head of the group
    Q = q[row].float().view(B, n, hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, hkv, n * G, D)
    S = (Q @ K.transpose(2, 3)) * (1.0 / math.sqrt(D))
    S = torch.where(see, S, torch.full_like(S, -math.inf))
    m = S.amax(dim=-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    P = torch.exp(S - m)
    l = P.sum(dim=-1, keepdim=True)
    O = torch.where(l > 0, (P @ V) / l, torch.zeros_like(l))
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
    if s["op"] == "extend":
        return _exact_extend(s)
    if s["op"] == "write":
        return _exact_write(s)
    return _exact_attention(s)


def _exact_extend(s):
    """Request by request, as a host allocator would."""
    new, lens = s["new_len"].tolist(), s["cache_len"].tolist()
    free, head, p = s["free_pages"].tolist(), int(s["free_head"]), s["page"]
    table = s["block_table"].cpu().numpy().copy()
    slots, positions, cu = [], [], [0]
    for b, (l, n) in enumerate(zip(lens, new)):
        for c in range(-(-l // p), -(-(l + n) // p)):
            table[b, c] = free[head]
            head += 1
        pos = np.arange(l, l + n)
        slots.append(table[b, pos // p].astype(np.int64) * p + pos % p)
        positions.append(pos)
        cu.append(cu[-1] + n)
    pad = s["T"] - cu[-1]
    slots.append(np.full(pad, -1, np.int64))
    positions.append(np.zeros(pad, np.int64))
    return {"block_table": table, "cache_len_out": np.array(lens) + np.array(new),
            "free_head_out": np.array([head]), "cu_new": np.array(cu),
            "slot_map": np.concatenate(slots), "position_ids": np.concatenate(positions)}


def _exact_write(s):
    """Complex rotation of the pairs in 64 bits, scattered row by row."""
    H, D = s["k"].shape[1:]
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    slots = s["slot_map"].long()
    src = torch.arange(slots.numel(), device=slots.device) if s["src_rows"] is None else s["src_rows"].long()
    k = s["k"].double()[src]
    if s["position_ids"] is not None:
        turn = torch.pow(torch.tensor(ROPE_BASE, dtype=torch.float64, device=k.device),
                         torch.arange(0, D, 2, device=k.device, dtype=torch.float64) / -D)
        angle = torch.outer(s["position_ids"].double(), turn)[:, None, :]
        z = torch.complex(k[..., :D // 2].contiguous(), k[..., D // 2:].contiguous()) * torch.polar(torch.ones_like(angle), angle)
        k = torch.cat([z.real, z.imag], dim=-1)
    ok = slots >= 0
    kc.view(-1, H, D).index_copy_(0, slots[ok], k[ok])
    vc.view(-1, H, D).index_copy_(0, slots[ok], s["v"].double()[src[ok]])
    return {"k_cache": kc, "v_cache": vc}


def _exact_attention(s):
    """One request and kv head at a time, ancestors found by walking up."""
    c = s["case"]
    lens, n = _attn_lengths(c)
    parents = _attn_parents(c, n)
    q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
    T, hq, D = q.shape
    hkv, p = k.shape[1], c["page"]
    G = hq // hkv
    o = torch.zeros_like(q)
    lse = torch.full((hq, T), -math.inf, dtype=torch.float64, device=q.device)
    r0 = 0
    for b in range(c["B"]):
        nb, L = n[b], lens[b]
        tree = np.zeros((nb, nb), bool)
        par = list(range(-1, nb - 1)) if parents is None else parents[r0:r0 + nb]
        for i in range(nb):
            j = i if par[i] > -2 else -1
            while j >= 0 and par[j] > -2:
                tree[i, j] = True
                j = par[j]
        rows = [i for i in range(nb) if par[i] > -2]
        hide = ~torch.as_tensor(tree[rows], device=q.device)
        pages = s["block_table"][b, :-(-L // p)].long() if L else None
        R = torch.as_tensor(rows, device=q.device) + r0
        for h in range(hkv):
            kk, vv = k[r0:r0 + nb, h], v[r0:r0 + nb, h]
            if L:
                kk = torch.cat([s["k_cache"][pages, :, h].reshape(-1, D)[:L].double(), kk])
                vv = torch.cat([s["v_cache"][pages, :, h].reshape(-1, D)[:L].double(), vv])
            for g in range(h * G, h * G + G):
                z = q[R, g] @ kk.T / math.sqrt(D)
                z[:, L:].masked_fill_(hide, -math.inf)
                lse[g, R] = torch.logsumexp(z, dim=1)
                o[R, g] = torch.softmax(z, dim=1) @ vv
        r0 += nb
    return {"o": o, "lse": lse}
