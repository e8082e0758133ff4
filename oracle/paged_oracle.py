"""Plain fp64 reference of the paged K/V cache operators, from their
definitions: a host allocator, a row-by-row store with rotary embedding, and
softmax attention of tree nodes over gathered rows. No code is shared with the
CUDA path. Next to each attention result it gives the two sums that an error
bound needs (see ``tree_attention``).
"""
from __future__ import annotations

import numpy as np

ROOT, UNUSED = -1, -2


def extend(new_len, cache_len, table, free_pages, free_head, page_size, n_pages, T):
    """Allocate pages for every request's new rows, in request order.

    Returns a dict with table, cache_len, free_head, cu_new, slot_map,
    position_ids and the two status findings (bad_index, out_of_pages).
    """
    B, max_pages = table.shape
    table = table.copy()
    out_len = np.array(cache_len, np.int64)
    ps = page_size
    bad_index = out_of_pages = False
    head_ok = 0 <= free_head <= len(free_pages)
    bad_index |= not head_ok
    avail = len(free_pages) - free_head if head_ok else 0
    asked_pages = asked_rows = taken = 0
    cu, slots, pos = [0], [], []
    for b in range(B):
        L, n = int(cache_len[b]), int(new_len[b])
        got = 0
        if L < 0 or n < 0 or L + n > max_pages * ps:
            bad_index = True
        else:
            have, want = -(-L // ps), -(-(L + n) // ps)
            first = asked_pages
            asked_pages += want - have
            asked_rows += n
            ok = True
            if want > have and asked_pages > avail:
                out_of_pages, ok = True, False
            if n > 0 and asked_rows > T:
                bad_index, ok = True, False
            if ok:
                got = n
                for c in range(have, want):
                    page = int(free_pages[free_head + first + c - have])
                    if not 0 <= page < n_pages:
                        bad_index, page = True, -1
                    table[b, c] = page
                if want > have:
                    taken = asked_pages
                for p in range(L, L + n):
                    page = int(table[b, p // ps])
                    if not 0 <= page < n_pages:
                        bad_index = True
                        slots.append(-1)
                    else:
                        slots.append(page * ps + p % ps)
                    pos.append(p)
        out_len[b] += got
        cu.append(cu[-1] + got)
    pad = T - cu[-1]
    return {"table": table, "cache_len": out_len, "free_head": free_head + taken,
            "cu_new": np.array(cu), "slot_map": np.array(slots + [-1] * pad, np.int64),
            "position_ids": np.array(pos + [0] * pad, np.int64),
            "bad_index": bad_index, "out_of_pages": out_of_pages}


def rotate(x, positions, base):
    """Rotate-half rotary embedding of x [n, H, D] at integer positions [n]."""
    D = x.shape[-1]
    f = float(base) ** (-2.0 * np.arange(D // 2) / D)
    a = np.asarray(positions, np.float64)[:, None] * f
    c, s = np.cos(a)[:, None, :], np.sin(a)[:, None, :]
    lo, hi = x[..., :D // 2], x[..., D // 2:]
    return np.concatenate([lo * c - hi * s, hi * c + lo * s], axis=-1)


def write_kv(k_cache, v_cache, k, v, slot_map, src_rows=None, position_ids=None, base=1e6):
    """New (k_cache, v_cache) with the kept rows stored; caches [pages, ps, H, D]."""
    kc, vc = k_cache.copy(), v_cache.copy()
    ps = kc.shape[1]
    for i, s in enumerate(slot_map):
        r = i if src_rows is None else int(src_rows[i])
        if s < 0 or s >= kc.shape[0] * ps or not 0 <= r < len(k):
            continue
        row = k[r:r + 1]
        if position_ids is not None:
            row = rotate(row, [position_ids[i]], base)
        kc[s // ps, s % ps], vc[s // ps, s % ps] = row[0], v[r]
    return kc, vc


def ancestors(parents):
    """bool [n, n]: node i sees node j (the path from i to its root; an unused
    node sees nothing and is seen by none)."""
    n = len(parents)
    see = np.zeros((n, n), bool)
    for i in range(n):
        j = i if parents[i] != UNUSED else -1
        while j >= 0:
            see[i, j] = True
            up = int(parents[j])
            if not 0 <= up < j or parents[up] == UNUSED:
                up = ROOT
            j = up
    return see


def tree_attention(q, k, v, k_cache, v_cache, table, cache_len, cu_nodes, parents, scale=None,
                   rows_of=None):
    """(o [T, Hq, D], lse [Hq, T], a [T, Hq, D], z [Hq, T]) in fp64. Rows outside
    the requests stay NaN. a = sum_j p_j |v_j| and z = max_j scale sum |q k_j|
    bound what rounding the probabilities and the dot products can do.
    rows_of: requests to compute (all by default)."""
    T, Hq, D = q.shape
    H = k.shape[1]
    G = Hq // H
    scale = 1.0 / np.sqrt(D) if not scale else scale
    n_pages, ps = k_cache.shape[:2]
    o = np.full((T, Hq, D), np.nan)
    a = np.full((T, Hq, D), np.nan)
    lse, z = np.full((Hq, T), np.nan), np.full((Hq, T), np.nan)
    for b in range(len(cache_len)) if rows_of is None else rows_of:
        r0, r1, L = int(cu_nodes[b]), int(cu_nodes[b + 1]), int(cache_len[b])
        n = r1 - r0
        if n == 0:
            continue
        par = np.arange(-1, n - 1) if parents is None else np.asarray(parents[r0:r1])
        see_new = ancestors(par)
        pos = np.arange(L)
        page = np.asarray(table[b])[pos // ps].astype(np.int64) if L else pos
        good = (page >= 0) & (page < n_pages)
        pos, page = pos[good], page[good]
        see = np.concatenate([np.repeat((par != UNUSED)[:, None], len(pos), 1), see_new], axis=1)
        for h in range(H):
            kk = np.concatenate([k_cache[page, pos % ps, h], k[r0:r1, h]])
            vv = np.concatenate([v_cache[page, pos % ps, h], v[r0:r1, h]])
            for g in range(h * G, h * G + G):
                for i in range(n):
                    w = see[i]
                    if not w.any():
                        o[r0 + i, g], a[r0 + i, g] = 0.0, 0.0
                        lse[g, r0 + i], z[g, r0 + i] = -np.inf, 0.0
                        continue
                    s = scale * (kk[w] @ q[r0 + i, g])
                    m = s.max()
                    e = np.exp(s - m)
                    p = e / e.sum()
                    lse[g, r0 + i] = m + np.log(e.sum())
                    o[r0 + i, g] = p @ vv[w]
                    a[r0 + i, g] = p @ np.abs(vv[w])
                    z[g, r0 + i] = abs(scale) * (np.abs(kk[w]) @ np.abs(q[r0 + i, g])).max()
    return o, lse, a, z
