"""Pins of the 4-bit paged cache's oracle: hand-made examples, brute force, torch SDPA."""
import numpy as np
import pytest
import torch

import oracle
from oracle import kv4


def test_plan_by_hand():
    # P = 4: request 0 has 3 of 4 places of page 9 used and brings 6; request 1 idles; 2 is new
    table = np.array([[9, -1, -1], [5, 6, -1], [-1, -1, -1]], np.int32)
    t, s, seq, cu, head, bits = kv4.plan([3, 8, 0], [6, 0, 2], [7, 1, 2, 3, 4], 1, table, 4, 10, 10)
    np.testing.assert_array_equal(t, [[9, 1, 2], [5, 6, -1], [3, -1, -1]])
    np.testing.assert_array_equal(s, [39, 4, 5, 6, 7, 8, 12, 13, -1, -1])
    np.testing.assert_array_equal(seq, [9, 8, 2])
    np.testing.assert_array_equal(cu, [0, 6, 6, 8])
    assert (head, bits) == (4, 0)
    # two free pages fewer: the third request is refused
    t, s, seq, cu, head, bits = kv4.plan([3, 8, 0], [6, 0, 2], [7, 1, 2], 1, table, 4, 10, 10)
    np.testing.assert_array_equal(t[2], [-1, -1, -1])
    np.testing.assert_array_equal(s[6:], [-1] * 4)
    assert (list(seq), head, bits) == ([9, 8, 0], 3, kv4.NO_PAGES)


def test_slots_by_hand():
    table = np.array([[3, 1], [0, -1]], np.int32)
    s, cu, bits = kv4.slots(table, [2, 0], [4, 5], 4, 4, 10)
    np.testing.assert_array_equal(s, [14, 15, 4, 5, 0, 1, 2, 3, -1, -1])
    np.testing.assert_array_equal(cu, [0, 4, 9])
    assert bits == kv4.BAD_INDEX


@pytest.mark.parametrize("d", [64, 128])
def test_rows_by_hand(d):
    pool = np.zeros((2, 2, 64 * (d + d // 8)), np.uint8)
    code = np.arange(d, dtype=np.uint8) % 16
    kv4.put_row(pool, 64, d, 64 + 33, 1, 1, code, np.arange(1, d // 64 + 1), np.full(d // 64, -1.))
    tile = pool[1, 1, kv4.tile_bytes(d):]
    row = tile[(32 + 1) * (d // 2):(32 + 2) * (d // 2)]
    # word 0: dimensions 0 ... 7 of group 0, lowest nibble first
    assert row[:4].view("<u4")[0] == 0x76543210
    # the second word is group 1's first at d = 128, the next eight dimensions at d = 64
    assert row[4:8].view("<u4")[0] == (0x76543210 if d == 128 else 0xfedcba98)
    got = kv4.get_row(pool, 64, d, 64 + 33, 1, 1)
    np.testing.assert_array_equal(got[0], code)
    c, s, z = kv4.unpack(pool, 64, d)
    np.testing.assert_array_equal(c[1, 1, 1, 33], code)
    np.testing.assert_array_equal(s[1, 1, 1, 33], got[1])
    np.testing.assert_array_equal(z[1, 1, 1, 33], got[2])
    assert (c.sum(), s.astype(float).sum()) == (code.sum(), got[1].astype(float).sum())


@pytest.mark.parametrize("d,page", [(64, 128), (128, 32)])
def test_pack_is_unpack_reversed(d, page):
    rng = np.random.default_rng(d)
    pool = rng.integers(0, 256, (3, 2, page * (d + d // 8)), dtype=np.uint8)
    np.testing.assert_array_equal(kv4.pack(*kv4.unpack(pool, page, d)), pool)


def test_quantise():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((200, 128)).astype(np.float32)
    x[:, 7] *= 20
    c, s, z = kv4.quantise(x)
    y = kv4.dequantise(c, s, z)
    # half a step, and what the fp16 rounding of scale and zero moves the ends by
    step = np.repeat(s.astype(np.float64), 64, -1)
    assert (np.abs(y - x) <= step * (0.5 + 15 * 2.0 ** -10) + 2.0 ** -10 * np.abs(x).max()).all()
    assert c.reshape(200, 2, 64).max() == 15 and c.min() == 0
    flat, fs, fz = kv4.quantise(np.full((1, 64), 0.25, np.float32))
    assert flat.max() == 0 and fs[0, 0] == 0 and fz[0, 0] == 0.25
    odd, os_, oz = kv4.quantise(np.where(np.arange(64) == 3, np.nan, x[0, :64]))
    assert np.isnan(kv4.dequantise(odd, os_, oz)).all()
    inf = kv4.dequantise(*kv4.quantise(np.where(np.arange(64) < 2, [np.inf], -np.inf)))
    # 15 steps of fp16((65504 + 65504) / 15), off by at most half of fp16's spacing there (8 / 2)
    assert (inf[2:] == -65504).all() and np.abs(inf[:2] - 65504).max() <= 15 * 4


@pytest.mark.parametrize("d,page", [(64, 32), (128, 64)])
def test_attend_matches_sdpa_and_oracle(d, page):
    rng = np.random.default_rng(d)
    lens, h_k, g, width = [200, 1, 0, 77], 2, 3, 8
    per = [-(-n // page) for n in lens]
    pages = sum(per)
    pool = np.zeros((pages, h_k, page * (d + d // 8)), np.uint8)
    table, order, at = np.full((4, width), -1, np.int32), rng.permutation(pages), 0
    for b, n in enumerate(per):
        table[b, :n] = order[at:at + n]
        at += n
    kv = rng.standard_normal((2, sum(lens), h_k, d)).astype(np.float32)
    code, st, ze = kv4.quantise(kv)
    val = kv4.dequantise(code, st, ze)
    base = 0
    for b, n in enumerate(lens):
        for t in range(n):
            slot = table[b, t // page] * page + t % page
            for h in range(h_k):
                for w in (0, 1):
                    kv4.put_row(pool, page, d, slot, h, w, code[w, base + t, h], st[w, base + t, h],
                                ze[w, base + t, h])
        base += n
    q = rng.standard_normal((4, h_k * g, d))
    out, lse, *_ = kv4.attend(q, pool, table, lens, page, 0.1)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    for b, n in enumerate(lens):
        if not n:
            assert (out[b] == 0).all() and np.isneginf(lse[:, b]).all()
            continue
        k, v = (torch.from_numpy(val[w, cu[b]:cu[b + 1]]).transpose(0, 1) for w in (0, 1))
        ref = torch.nn.functional.scaled_dot_product_attention(
            torch.from_numpy(q[b]).unsqueeze(1), k.repeat_interleave(g, 0),
            v.repeat_interleave(g, 0), scale=0.1)
        np.testing.assert_allclose(out[b], ref[:, 0].numpy(), rtol=1e-10, atol=1e-12)
    # a selection: the rows of the last tokens in the selected-attention oracle
    sel = np.array([[[0, 2, -1], [0, 0, -1], [-1, -1, -1], [1, 1, 5]],
                    [[3, 0, 1], [-1, 0, -1], [-1, -1, -1], [0, 9, 0]]], np.int32)
    out, lse, *_ = kv4.attend(q, pool, table, lens, page, 0.1, sel=sel)
    full = np.full((h_k, cu[-1], 3), -1, np.int32)
    qf = np.zeros((cu[-1], h_k * g, d))
    live = [b for b, n in enumerate(lens) if n]
    for b in live:
        full[:, cu[b + 1] - 1], qf[cu[b + 1] - 1] = sel[:, b], q[b]
    rows = np.array([[cu[b + 1] - 1, hq] for b in live for hq in range(h_k * g)])
    ro, rl = oracle.fwd_rows(cu, page, full, qf, val[0], val[1], 0.1, rows)
    np.testing.assert_allclose(out[live].reshape(-1, d), ro, rtol=1e-9, atol=1e-12)
    np.testing.assert_allclose(lse.T[live].reshape(-1), rl, rtol=1e-9)
    # a window leaves the newest keys
    np.testing.assert_array_equal(kv4.kept_keys(77, page, None, 5), np.arange(72, 77))
    np.testing.assert_array_equal(kv4.kept_keys(77, page, [0], 70), np.arange(7, min(page, 77)))
