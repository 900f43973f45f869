"""States of a cache's pages for the tests."""
import numpy as np

from oracle import pages


def make_state(rows, width, page, lens, seed, spare=10, forks=()):
    """A table whose rows hold pages in random order, and what goes with it; forks: (parent, child)
    pairs made at once.  The free list is as long as the pool."""
    rng = np.random.default_rng(seed)
    per = [-(-n // page) for n in lens]
    total = sum(per) + spare
    order = rng.permutation(total).astype(np.int32)
    table = np.full((rows, width), -1, np.int32)
    at = 0
    for r, n in enumerate(per):
        table[r, :n] = order[at:at + n]
        at += n
    all_lens = np.zeros(rows, np.int32)
    all_lens[:len(lens)] = lens
    free = np.full(total, -7, np.int32)
    free[at:] = order[at:]
    s = dict(table=table, lens=all_lens, shares=np.zeros(total, np.int32), free=free, head=at,
             page=page)
    if forks:
        p, c = np.array(forks, np.int32).T
        s["table"], s["lens"], s["shares"], _, _, s["head"], bits = pages.fork(
            s["table"], s["lens"], p, c, page, s["shares"], s["free"], s["head"])
        assert bits == 0
    return s


def check_books(s):
    """Every page is free, or named by 1 + shares rows."""
    named = np.zeros(len(s["shares"]), int)
    for r, n in enumerate(s["lens"]):
        for j in range(-(-int(n) // s["page"])):
            named[s["table"][r, j]] += 1
    free = s["free"][s["head"]:]
    assert len(set(free.tolist())) == len(free)
    is_free = np.zeros(len(named), bool)
    is_free[free] = True
    assert (is_free == (named == 0)).all()
    assert (s["shares"] == np.maximum(named - 1, 0)).all()
