"""Oracle of the life of a cache's pages (numpy, one row after the other): forks, frees,
compactions.

Parity status (pins live in tests/test_oracle_pages.py): examples by hand; over random lives of a
cache every page is free, or named by 1 + shares rows.
"""
from __future__ import annotations

import numpy as np

BAD_INDEX, BAD_SEQLENS, NO_PAGES = 1, 2, 8


def fork(table, lens, parents, children, page, shares, free, head, fork_lens=None):
    """table, lens, shares (copies), copy_src, copy_dst, head_out and the error bits."""
    old, had = table, lens
    table, lens, shares = table.copy(), lens.copy(), shares.copy()
    b, width = table.shape
    n = len(parents)
    src, dst = np.full(n, -1, np.int32), np.full(n, -1, np.int32)
    bits, avail = 0, len(free) - head
    if not 0 <= head <= len(free):
        bits, avail = NO_PAGES, 0
    parent_rows = set(int(x) for x in parents)
    seen, used, taken = set(), 0, 0
    for i in range(n):
        p, c = int(parents[i]), int(children[i])
        ok = 0 <= p < b and 0 <= c < b and c not in seen and c not in parent_rows
        if 0 <= c < b:
            seen.add(c)
        if not ok:
            bits |= BAD_INDEX
            continue
        m = int(had[p]) if fork_lens is None else int(fork_lens[i])
        if m < 0 or m > had[p] or had[p] > width * page:
            bits |= BAD_SEQLENS
            continue
        full, rest = divmod(m, page)
        if rest:
            used += 1
            if used > avail:
                bits |= NO_PAGES
                continue
            taken = used
        for j in range(full):
            pg = int(old[p, j])
            if 0 <= pg < len(shares):
                shares[pg] += 1
                table[c, j] = pg
            else:
                bits |= BAD_INDEX
                table[c, j] = -1
        if rest:
            a, f = int(old[p, full]), int(free[head + used - 1])
            good = 0 <= f < len(shares)
            table[c, full] = f if good else -1
            if good and 0 <= a < len(shares):
                src[i], dst[i] = a, f
            else:
                bits |= BAD_INDEX
        lens[c] = m
    return table, lens, shares, src, dst, head + taken, bits


def release(table, lens, rows, page, shares, free, head):
    """table, lens, shares, free (copies), head_out and the error bits of a free."""
    table, lens, shares, free = table.copy(), lens.copy(), shares.copy(), free.copy()
    b, width = table.shape
    bits, seen, gone = 0, set(), set()
    for r in (int(x) for x in rows):
        if not 0 <= r < b or r in seen:
            bits |= BAD_INDEX
            continue
        seen.add(r)
        if not 0 <= lens[r] <= width * page:
            bits |= BAD_SEQLENS
            continue
        for j in range(-(-int(lens[r]) // page)):
            pg = int(table[r, j])
            table[r, j] = -1
            if not 0 <= pg < len(shares) or pg in gone:
                bits |= BAD_INDEX
            elif shares[pg]:
                shares[pg] -= 1
            else:
                gone.add(pg)
        lens[r] = 0
    pages = sorted(gone)
    if not 0 <= head <= len(free):
        return table, lens, shares, free, head, bits | (NO_PAGES if pages else 0)
    if len(pages) > head:
        bits |= NO_PAGES
        pages = pages[len(pages) - head:]
    free[head - len(pages):head] = pages
    return table, lens, shares, free, head - len(pages), bits


def compact(table, lens, page, shares, free, count):
    """table, shares, free (copies), copy_src, copy_dst, head_out (None: left alone) and the bits."""
    table, shares, free = table.copy(), shares.copy(), free.copy()
    b, width = table.shape
    total, bits, live = len(shares), 0, set()
    src, dst = np.full(count, -1, np.int32), np.full(count, -1, np.int32)
    have = []
    for r in range(b):
        if not 0 <= lens[r] <= width * page:
            bits |= BAD_SEQLENS
        have.append(-(-min(max(int(lens[r]), 0), width * page) // page))
        for j in range(have[r]):
            pg = int(table[r, j])
            if 0 <= pg < total:
                live.add(pg)
            else:
                bits |= BAD_INDEX
    n = len(live)
    movers = sorted(x for x in live if x >= n)
    holes = [x for x in range(n) if x not in live]
    if len(movers) > count or total - n > len(free):
        return table, shares, free, src, dst, None, bits | NO_PAGES
    to = dict(zip(movers, holes))
    for r in range(b):
        for j in range(have[r]):
            table[r, j] = to.get(int(table[r, j]), table[r, j])
    was = shares.copy()
    shares[n:] = 0
    for a, z in to.items():
        shares[z] = was[a]
    src[:len(movers)], dst[:len(movers)] = movers, holes
    head = len(free) - (total - n)
    free[head:] = np.arange(n, total)
    return table, shares, free, src, dst, head, bits
