"""CPU oracle for the paged key/value cache: block tables and slot maps, the write of new rows,
and decode through a block table.

TEST INFRASTRUCTURE ONLY.  Nothing on the product path may import, call or execute this
module.  It shares no code with the CUDA path and imports nothing from the package.

A pool holds ``P`` pages of ``page`` tokens; token x of sequence b is row x % page of page
table[b][x // page].  An entry outside [0, P) is a hole: its tokens are not written and its
keys are hidden.  ``tables`` walks the tokens one by one (a token that opens a page takes the
next page of the free list); the decode gathers the visible rows and is the plain definition of
``decode.py`` on them.
"""
from __future__ import annotations

import numpy as np

from .attention import forward_head


def tables(cache_len, new_len, free_pages, table, page: int, num_pages: int, num_slots: int):
    """Returns (table, total_len, token_start, slots, pages_taken)."""
    table = np.array(table)
    B, M = table.shape
    total, start, slots, taken = [], [0], [], 0
    for b in range(B):
        o = min(max(int(cache_len[b]), 0), M * page)
        n = min(max(int(new_len[b]), 0), M * page - o)
        for x in range(o, o + n):
            if x % page == 0:
                table[b, x // page] = free_pages[taken] if taken < len(free_pages) else -1
                taken += 1
            e = int(table[b, x // page])
            slots.append(e * page + x % page if 0 <= e < num_pages else -1)
        total.append(o + n)
        start.append(start[-1] + n)
    slots = (slots + [-1] * num_slots)[:num_slots]
    return table, np.array(total), np.array(start), np.array(slots, dtype=np.int64), taken


def append(cache, rows, slots):
    """Rows [T, ...] into a pool [P, ..., page, d]; head axes, if any, lie before the page's."""
    cache = np.array(cache)
    page = cache.shape[-2]
    for t, s in enumerate(slots):
        if 0 <= s < cache.shape[0] * page:
            cache[s // page, ..., s % page, :] = rows[t]
    return cache


def visible(table_row, length: int, page: int, num_pages: int, max_len: int):
    """(page, row) of each token of a sequence that a query sees."""
    L = max(0, min(int(length), max_len))
    x = np.arange(L)
    p = np.asarray(table_row)[x // page]
    keep = (p >= 0) & (p < num_pages)
    return p[keep], (x % page)[keep]


def decode(q, k, v, table, cache_len, scale: float):
    """q [B, Hq, d]; k [P, Hkv, page, d], v [P, Hkv, page, e].  Returns (o, lse, spread): spread is
    sum_j p_j |v_j|, what a relative error of the weights is measured against."""
    q = np.asarray(q, np.float64)
    B, Hq, _ = q.shape
    P, Hkv, page, e = v.shape
    o, lse = np.zeros((B, Hq, e)), np.full((B, Hq), -np.inf)
    spread = np.zeros((B, Hq, e))
    for b in range(B):
        p, r = visible(table[b], cache_len[b], page, P, table.shape[1] * page)
        if p.size == 0:
            continue
        for h in range(Hq):
            g = h // (Hq // Hkv)
            keep = np.ones((1, p.size), dtype=bool)
            vv = np.asarray(v[p, g, r], np.float64)
            ob, lb, w = forward_head(q[b, h][None], k[p, g, r], vv, scale, keep)
            o[b, h], lse[b, h], spread[b, h] = ob[0], lb[0], w[0] @ np.abs(vv)
    return o, lse, spread
