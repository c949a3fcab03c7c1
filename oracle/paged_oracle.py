"""64-bit oracle of the paged-cache calls (numpy; test infrastructure only).

Restates each definition with plain loops over requests, sequences, heads and
pages; nothing here shares code with the library.
"""

from __future__ import annotations

import numpy as np


def pages_of(n: int, page: int) -> int:
    return -(-n // page)


def tables(cached, new, free_pages, free_count, block_table, page, num_pages, slot_capacity):
    """-> (block_table, slot_map, seqlens, cu_new, free_left, bad_len, no_pages, bad_index)."""
    table = np.array(block_table, dtype=np.int64)
    cap = table.shape[1] * page
    slots = np.full(slot_capacity, -1, dtype=np.int64)
    cu, lens = [0], []
    free_pages = list(free_pages)
    bad_len = no_pages = bad_index = False
    avail = free_count
    if not 0 <= free_count <= len(free_pages):
        avail, bad_index = 0, True
    wanted, left = 0, avail
    for b, (c, w) in enumerate(zip(cached, new)):
        start = cu[-1]
        cu.append(min(start + max(w, 0), 2**31 - 1))
        fits = not (w > 0 and start + w > slot_capacity)
        if c < 0 or w < 0 or c + w > cap or not fits:
            bad_len = True
            lens.append(c)
            continue
        have = pages_of(c, page)
        need = pages_of(c + w, page) - have
        wanted += need
        if need and wanted > avail:
            no_pages = True
            lens.append(c)
            continue
        for i in range(need):
            p = free_pages[avail - 1 - (wanted - need + i)]
            if not 0 <= p < num_pages:
                p, bad_index = -1, True
            table[b, have + i] = p
        left -= need
        lens.append(c + w)
        for i in range(w):
            p = table[b, (c + i) // page]
            if not 0 <= p < num_pages:
                bad_index = True
                continue
            slots[start + i] = p * page + (c + i) % page
    return table, slots, np.array(lens), np.array(cu), left, bad_len, no_pages, bad_index


def append(keys, vals, means, k_new, v_new, slots, page):
    """keys, vals [P, H, page, d] (changed in place), means [P, H, d] (changed in place)."""
    for t, s in enumerate(slots):
        if s < 0 or s >= keys.shape[0] * page:
            continue
        keys[s // page, :, s % page] = k_new[t]
        vals[s // page, :, s % page] = v_new[t]
    for s in slots:
        if 0 <= s < keys.shape[0] * page and s % page == page - 1 and means is not None:
            means[s // page] = keys[s // page].mean(1)


def attention(q, k, v, scale):
    """q [r, d], k and v [n, d] -> (out [r, d], lse [r])."""
    if len(k) == 0:
        return np.zeros_like(q), np.full(len(q), -np.inf)
    x = (q @ k.T) * scale
    m = x.max(-1, keepdims=True)
    p = np.exp(x - m)
    z = p.sum(-1, keepdims=True)
    return (p @ v) / z, (m + np.log(z))[:, 0]


def gather(pool, table_row, h, pages, n, page):
    """Rows of the listed pages (in list order) of one sequence and head; pages outside the pool
    and rows past the end left out."""
    rows = [np.zeros((0, pool.shape[-1]))]
    for j in pages:
        p = table_row[j]
        if 0 <= p < pool.shape[0]:
            rows.append(pool[p, h, : min(page, n - j * page)])
    return np.concatenate(rows)


def decode(q, keys, vals, table, lens, page, scale, lists=None):
    """q [B, Hq, d], keys and vals [P, Hkv, page, d] -> (out [B, Hq, d], lse [B, Hq]).
    lists: int [B, Hkv, k] page lists, or None for every page."""
    B, Hq, d = q.shape
    H = keys.shape[1]
    r = Hq // H
    out, lse = np.zeros((B, Hq, d)), np.full((B, Hq), -np.inf)
    for b in range(B):
        n = int(lens[b])
        nb = pages_of(n, page)
        for h in range(H):
            pages = range(nb)
            if lists is not None:
                pages = [int(j) for j in lists[b, h][: min(lists.shape[2], nb)] if 0 <= j < nb]
            k = gather(keys, table[b], h, pages, n, page)
            v = gather(vals, table[b], h, pages, n, page)
            at = slice(h * r, h * r + r)
            out[b, at], lse[b, at] = attention(q[b, at], k, v, scale)
    return out, lse


def select(q, means, table, lens, page, scale, topk, sink, recent):
    """-> (page_idx int [B, Hkv, topk], scores list of (first ranked page, fp32 scores))."""
    B, Hq, d = q.shape
    H = means.shape[1]
    r = Hq // H
    idx = np.full((B, H, topk), -1, dtype=np.int64)
    scores = {}
    for b in range(B):
        nb = pages_of(int(lens[b]), page)
        c0 = min(sink, nb)
        c1 = max(c0, nb - recent)
        forced = list(range(c0)) + list(range(c1, nb))
        for h in range(H):
            s = np.zeros(c1 - c0, dtype=np.float32)
            if c1 > c0:
                m = means[table[b, c0:c1], h]
                x = (q[b, h * r:h * r + r] @ m.T) * scale
                e = np.exp(x - x.max(-1, keepdims=True))
                s = (e / e.sum(-1, keepdims=True)).sum(0).astype(np.float32)
            order = sorted(range(c1 - c0), key=lambda j: (-s[j], j))
            take = (forced + [c0 + j for j in order])[:topk]
            idx[b, h, : len(take)] = take
            scores[b, h] = (c0, s)
    return idx, scores
