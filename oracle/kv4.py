"""Oracle of the 4-bit paged KV cache (numpy, fp64): plans, rows, attention over the pages.

Parity status (pins live in tests/test_oracle_kv4.py):
  plan / slots     -- pinned: hand-written examples, slots distinct and inside their pages.
  quantise / pack  -- pinned: hand-packed rows, the worst rounding distance, idempotence.
  attend           -- pinned: torch SDPA in fp64, oracle.fwd_rows on the same values.
"""
from __future__ import annotations

import numpy as np

HALF_MAX = np.float32(65504.0)
BAD_INDEX, BAD_SEQLENS, NO_PAGES = 1, 2, 8


# ---- block tables and slot maps -------------------------------------------------------
def plan(ctx, new, free, head, table, page, num_pages, max_slots):
    """table (copied), slots, seq_lens, cu, head_out and the error bits of nsa_page_plan."""
    table, slots = table.copy(), np.full(max_slots, -1, np.int32)
    b, width = table.shape
    seq, cu = np.zeros(b, np.int32), np.zeros(b + 1, np.int32)
    bits, tok, used = 0, 0, 0
    avail = len(free) - head
    if not 0 <= head <= len(free):
        bits, avail = NO_PAGES, 0
    taken = 0
    for i in range(b):
        c, n = int(ctx[i]), int(new[i])
        ok = c >= 0 and n >= 0 and c + n <= width * page
        need = -(-(c + n) // page) - -(-c // page) if ok else 0
        n = max(n, 0)
        first = tok
        tok, used = tok + n, used + need
        cu[i + 1] = min(tok, max_slots)
        seq[i] = min(max(c, 0), width * page)
        if not ok:
            bits |= BAD_SEQLENS
            continue
        if (n and tok > max_slots) or (need and used > avail):
            bits |= NO_PAGES
            continue
        if need:
            taken = used
        seq[i] = c + n
        have = -(-c // page)
        for t in range(n):
            j, r = divmod(c + t, page)
            fresh = j >= have
            pg = int(free[head + used - need + j - have]) if fresh else int(table[i, j])
            good = 0 <= pg < num_pages
            if fresh and r == 0:
                table[i, j] = pg if good else -1
            if good:
                slots[first + t] = pg * page + r
            else:
                bits |= BAD_INDEX
    return table, slots, seq, cu, head + taken, bits


def slots(table, start, count, page, num_pages, max_slots):
    """slots, cu and the error bits of nsa_page_slots."""
    b, width = table.shape
    out, cu, bits, tok = np.full(max_slots, -1, np.int32), np.zeros(b + 1, np.int32), 0, 0
    for i in range(b):
        c, n = int(start[i]), int(count[i])
        ok = c >= 0 and n >= 0 and c + n <= width * page
        n = max(n, 0)
        first, tok = tok, tok + n
        cu[i + 1] = min(tok, max_slots)
        if not ok:
            bits |= BAD_SEQLENS
        elif n and tok > max_slots:
            bits |= NO_PAGES
        else:
            for t in range(n):
                pg = int(table[i, (c + t) // page])
                if 0 <= pg < num_pages:
                    out[first + t] = pg * page + (c + t) % page
                else:
                    bits |= BAD_INDEX
    return out, cu, bits


# ---- rows -----------------------------------------------------------------------------
def quantise(x):
    """fp32 [..., d] -> codes uint8 [..., d], scale and zero fp16 [..., d / 64]."""
    x = np.asarray(x, np.float32)
    g = x.reshape(*x.shape[:-1], -1, 64)
    nan = np.isnan(g).any(-1)
    g = np.clip(np.where(nan[..., None], np.float32(0), g), -HALF_MAX, HALF_MAX)
    zero = g.min(-1).astype(np.float16)
    z32 = zero.astype(np.float32)
    scale = ((g.max(-1) - z32) / np.float32(15)).astype(np.float16)
    step = scale.astype(np.float64)[..., None]
    t = (g - z32[..., None]).astype(np.float64)
    code = np.where(step > 0, np.rint(t / np.where(step > 0, step, 1)), 0).clip(0, 15)
    zero, scale = np.where(nan, np.float16("nan"), zero), np.where(nan, np.float16(0), scale)
    code = np.where(nan[..., None], 0, code)
    return code.astype(np.uint8).reshape(x.shape), scale, zero


def dequantise(code, scale, zero):
    g = code.reshape(*code.shape[:-1], -1, 64).astype(np.float64)
    x = g * scale.astype(np.float64)[..., None] + zero.astype(np.float64)[..., None]
    return x.reshape(code.shape)


def tile_bytes(d):
    return 32 * (d + d // 8)


def put_row(pool, page, d, slot, head, which, code, scale, zero):
    """Stores a row's codes [d], scale and zero [d / 64]; which: 0 for K, 1 for V."""
    ng = d // 64
    pg, at = divmod(int(slot), page)
    tile, r = divmod(at, 32)
    rec = pool[pg, head, tile * tile_bytes(d):(tile + 1) * tile_bytes(d)]
    row = np.zeros(d // 2, np.uint8)
    for dim in range(d):
        i, j, n = dim // 64, dim % 64 // 8, dim % 8
        row[4 * (j * ng + i) + n // 2] |= int(code[dim]) << (4 * (n % 2))
    rec[(which * 32 + r) * (d // 2):(which * 32 + r + 1) * (d // 2)] = row
    par = rec[32 * d:].view(np.float16).reshape(4, 32, ng)
    par[2 * which, r], par[2 * which + 1, r] = scale, zero


def get_row(pool, page, d, slot, head, which):
    """codes [d], scale and zero [d / 64] of a stored row."""
    ng = d // 64
    pg, at = divmod(int(slot), page)
    tile, r = divmod(at, 32)
    rec = pool[pg, head, tile * tile_bytes(d):(tile + 1) * tile_bytes(d)]
    row = rec[(which * 32 + r) * (d // 2):(which * 32 + r + 1) * (d // 2)]
    code = np.empty(d, np.uint8)
    for dim in range(d):
        i, j, n = dim // 64, dim % 64 // 8, dim % 8
        code[dim] = row[4 * (j * ng + i) + n // 2] >> (4 * (n % 2)) & 15
    par = rec[32 * d:].view(np.float16).reshape(4, 32, ng)
    return code, par[2 * which, r].copy(), par[2 * which + 1, r].copy()


def pack(code, scale, zero):
    """The pool of unpack's arrays."""
    pages, h, _, page, d = code.shape
    ng, nt = d // 64, page // 32
    b = code.reshape(pages, h, 2, nt, 32, ng, 8, 8).swapaxes(2, 3).swapaxes(-3, -2)
    b = (b[..., 0::2] | b[..., 1::2] << 4).astype(np.uint8).reshape(pages, h, nt, 32 * d)
    par = np.stack([scale, zero], 0).astype(np.float16).reshape(2, pages, h, 2, nt, 32, ng)
    par = np.ascontiguousarray(par.transpose(1, 2, 4, 3, 0, 5, 6)).reshape(pages, h, nt, -1)
    return np.concatenate([b, par.view(np.uint8)], -1).reshape(pages, h, -1)


def unpack(pool, page, d):
    """All rows of a pool uint8 [pages, h, bytes]: codes uint8 [pages, h, 2, P, d], scale and
    zero fp16 [pages, h, 2, P, d / 64] (K first, then V)."""
    ng, (pages, h, _) = d // 64, pool.shape
    t = pool.reshape(pages, h, page // 32, tile_bytes(d))
    b = t[..., :32 * d].reshape(pages, h, page // 32, 2, 32, 8, ng, 4)
    code = np.stack([b & 15, b >> 4], -1).reshape(pages, h, page // 32, 2, 32, 8, ng, 8)
    code = code.swapaxes(-3, -2).reshape(pages, h, page // 32, 2, 32, d)
    code = code.swapaxes(2, 3).reshape(pages, h, 2, page, d)
    par = np.ascontiguousarray(t[..., 32 * d:]).view(np.float16)
    par = par.reshape(pages, h, page // 32, 2, 2, 32, ng).transpose(4, 0, 1, 3, 2, 5, 6)
    scale, zero = par.reshape(2, pages, h, 2, page, ng)
    return code, scale, zero


# ---- attention ------------------------------------------------------------------------
def kept_keys(n, page, sel=None, window=0):
    """Positions that the last of n cached tokens attends to, in order."""
    see = np.ones(n, bool)
    if sel is not None:
        see[:] = False
        for blk in map(int, sel):
            if 0 <= blk * page < n:
                see[blk * page:(blk + 1) * page] = True
    if window:
        see[:max(0, n - window)] = False
    return np.flatnonzero(see)


def attend(q, pool, table, lens, page, scale, sel=None, window=0):
    """out fp64 [B, h_q, d], lse [h_q, B], and for each row what error bounds are made of:
    the largest scale * sum |q| |k| of its keys, sum p |v|, and sum p * 8 * (step of v)."""
    bsz, h_q, d = q.shape
    h_k = pool.shape[1]
    g = h_q // h_k
    code, st, ze = unpack(pool, page, d)
    out, lse = np.zeros((bsz, h_q, d)), np.full((h_q, bsz), -np.inf)
    big = np.zeros((bsz, h_q))
    pv, ps = np.zeros((bsz, h_q, d)), np.zeros((bsz, h_q, d))
    for b in range(bsz):
        n = min(max(int(lens[b]), 0), table.shape[1] * page)
        for h in range(h_k):
            keys = kept_keys(n, page, None if sel is None else sel[h, b], window)
            pg = table[b, keys // page]
            live = (pg >= 0) & (pg < pool.shape[0])
            keys, pg = keys[live], pg[live]
            if not len(keys):
                continue
            at = keys % page
            kv = [dequantise(code[pg, h, w, at], st[pg, h, w, at], ze[pg, h, w, at])
                  for w in (0, 1)]
            step = np.repeat(st[pg, h, 1, at].astype(np.float64), 64, -1)
            # what the fp32 sums of q . k are made of: codes up to 15 steps, and the zero
            mag = (np.repeat(st[pg, h, 0, at].astype(np.float64), 64, -1) * 15 +
                   np.abs(np.repeat(ze[pg, h, 0, at].astype(np.float64), 64, -1)))
            for hq in range(h * g, (h + 1) * g):
                s = kv[0] @ q[b, hq] * scale
                m = s.max()
                p = np.exp(s - m)
                tot = p.sum()
                p /= tot
                out[b, hq], lse[hq, b] = p @ kv[1], m + np.log(tot)
                big[b, hq] = abs(scale) * (mag @ np.abs(q[b, hq])).max()
                pv[b, hq], ps[b, hq] = p @ np.abs(kv[1]), p @ step * 8
    return out, lse, big, pv, ps
