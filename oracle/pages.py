"""CPU oracle for the pages of a paged cache: requests forked, freed and compacted, pages copied.

TEST INFRASTRUCTURE ONLY.  Nothing on the product path may import, call or execute this module.
It shares no code with the CUDA path and imports nothing from the package.

Everything goes page by page and pair by pair, as the definitions read; a request's live entries are
the first ceil(length / page) of its row, and an entry outside [0, P) is a hole.
"""
from __future__ import annotations

import numpy as np


def _length(n, M, page):
    return min(max(int(n), 0), M * page)


def fork(cache_len, table, free_pages, src, dst, page: int, P: int):
    """Returns (cache_len, table, copies [(from, to, rows)], pages_taken)."""
    lens, table = np.array(cache_len), np.array(table)
    B, M = table.shape

    def inside(a, b):
        return 0 <= a < B and 0 <= b < B

    named = [b for a, b in zip(src, dst) if inside(a, b)]
    seen, copies, taken = set(), [], 0
    for a, b in zip(src, dst):
        move = (-1, -1, 0)
        if inside(a, b) and b not in seen and a not in named:
            n = _length(lens[a], M, page)
            full, part = divmod(n, page)
            table[b, :full] = table[a, :full]
            if part:
                old, new = int(table[a, full]), -1
                if 0 <= old < P:
                    if taken < len(free_pages):
                        new = int(free_pages[taken])
                    taken += 1
                    if 0 <= new < P:
                        move = (old, new, part)
                table[b, full] = new
            lens[b] = n
        if inside(a, b):
            seen.add(b)
        copies.append(move)
    return lens, table, copies, taken


def live(table, cache_len, page: int, P: int):
    """(row, column, page) of every live entry that names a page."""
    B, M = table.shape
    for b in range(B):
        for c in range(-(-_length(cache_len[b], M, page) // page)):
            if 0 <= table[b, c] < P:
                yield b, c, int(table[b, c])


def free(cache_len, table, rows, page: int, P: int):
    """Returns (cache_len, table, refs, free pages)."""
    lens, table = np.array(cache_len), np.array(table)
    for b in rows:
        if 0 <= b < len(lens):
            lens[b], table[b] = 0, -1
    refs = np.zeros(P, dtype=np.int64)
    for _, _, p in live(table, lens, page, P):
        refs[p] += 1
    return lens, table, refs, [p for p in range(P) if refs[p] == 0]


def compact(cache_len, table, page: int, P: int):
    """Returns (table, moved, copies [(from, to)], pages in use)."""
    table = np.array(table)
    used = sorted({p for _, _, p in live(table, cache_len, page, P)})
    U = len(used)
    room = [p for p in range(U) if p not in set(used)]
    copies = list(zip([p for p in used if p >= U], room))
    new = dict(copies)
    moved = np.full(P, -1)
    for p in used:
        moved[p] = new.get(p, p)
    for b, c, p in list(live(table, cache_len, page, P)):
        table[b, c] = moved[p]
    return table, moved, copies, U


def copy(pool, src, dst, rows=None):
    """pool [P, ..., page, d]."""
    pool = np.array(pool)
    P, page = pool.shape[0], pool.shape[-2]
    for i, (a, b) in enumerate(zip(src, dst)):
        if 0 <= a < P and 0 <= b < P and a != b:
            n = page if rows is None else min(max(int(rows[i]), 0), page)
            pool[b, ..., :n, :] = pool[a, ..., :n, :]
    return pool
