"""Pins of the page oracle: examples by hand, and books that stay in order over random lives."""
import numpy as np

from oracle import pages
from pages_helpers import check_books, make_state

i32 = lambda *x: np.array(x, np.int32)


def test_fork_and_free_by_hand():
    table = np.array([[3, 5, -1], [-1, -1, -1], [-1, -1, -1]], np.int32)
    lens, shares, free = i32(6, 0, 0), np.zeros(8, np.int32), i32(-1, -1, 0, 1, 2, 4, 6, 7)
    t, n, sh, src, dst, head, bits = pages.fork(table, lens, i32(0, 0), i32(2, 1), 4, shares, free, 2)
    assert bits == 0 and head == 4
    assert t.tolist() == [[3, 5, -1], [3, 1, -1], [3, 0, -1]] and n.tolist() == [6, 6, 6]
    assert sh[3] == 2 and sh.sum() == 2 and src.tolist() == [5, 5] and dst.tolist() == [0, 1]
    t, n, sh, fr, head, bits = pages.release(t, n, i32(2, 0), 4, sh, free, head)
    assert bits == 0 and head == 2 and fr[2:].tolist() == [0, 5, 2, 4, 6, 7]
    assert sh.sum() == 0 and n.tolist() == [0, 6, 0] and t.tolist() == [[-1] * 3, [3, 1, -1], [-1] * 3]
    # forked at a page's end: nothing to copy
    t, n, sh, src, dst, head, bits = pages.fork(t, n, i32(1), i32(0), 4, sh, fr, head, i32(4))
    assert bits == 0 and head == 2 and src[0] == dst[0] == -1 and t[0].tolist() == [3, -1, -1]


def test_compact_by_hand():
    table = np.array([[6, 1, 4], [6, 2, -1]], np.int32)
    shares = i32(0, 0, 0, 0, 0, 0, 1, 0)
    free = np.full(8, -1, np.int32)
    t, sh, fr, src, dst, head, bits = pages.compact(table, i32(9, 8), 4, shares, free, 4)
    assert bits == 0 and head == 4 and src.tolist() == [4, 6, -1, -1] and dst.tolist() == [0, 3, -1, -1]
    assert t.tolist() == [[3, 1, 0], [3, 2, -1]] and sh.tolist() == [0, 0, 0, 1, 0, 0, 0, 0]
    assert fr[4:].tolist() == [4, 5, 6, 7]
    assert pages.compact(table, i32(9, 8), 4, shares, free, 1)[-2:] == (None, pages.NO_PAGES)


def test_books_over_random_lives():
    rng = np.random.default_rng(3)
    for seed in range(30):
        page = int(rng.choice([1, 3, 16]))
        lens = rng.integers(0, 5 * page, 6)
        s = make_state(14, 6, page, lens, seed, spare=40)
        check_books(s)
        for _ in range(12):
            used = np.flatnonzero(s["lens"])
            idle = np.flatnonzero(s["lens"] == 0)
            k = min(len(idle), 3)
            if rng.random() < 0.5 and len(used) and k:
                p = rng.choice(used, k).astype(np.int32)
                n = rng.integers(0, s["lens"][p] + 1).astype(np.int32)
                s["table"], s["lens"], s["shares"], src, dst, s["head"], bits = pages.fork(
                    s["table"], s["lens"], p, rng.permutation(idle)[:k].astype(np.int32), page,
                    s["shares"], s["free"], s["head"], n)
                assert bits in (0, pages.NO_PAGES)
            elif len(used):
                rows = rng.permutation(used)[:rng.integers(1, len(used) + 1)]
                s["table"], s["lens"], s["shares"], s["free"], s["head"], bits = pages.release(
                    s["table"], s["lens"], rows, page, s["shares"], s["free"], s["head"])
                assert bits == 0
            check_books(s)
        s["table"], s["shares"], s["free"], src, dst, s["head"], bits = pages.compact(
            s["table"], s["lens"], page, s["shares"], s["free"], len(s["shares"]) // 2)
        assert bits == 0
        check_books(s)
        live = len(s["shares"]) - (len(s["free"]) - s["head"])
        assert (s["table"][s["table"] >= 0] < live).all()
