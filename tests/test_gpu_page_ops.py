"""Forks, frees, compactions and copies of pages on the GPU against the oracle: whole numbers, equal."""
import numpy as np
import pytest
import torch

from oracle import kv4, pages
from pages_helpers import check_books, make_state

pytestmark = pytest.mark.gpu


def _dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def _np(*ts):
    return [t.cpu().numpy() for t in ts]


def _eq(got, want):
    for a, b in zip(got, want):
        np.testing.assert_array_equal(a.cpu().numpy().reshape(-1), np.asarray(b).reshape(-1))


def _state(s):
    return (_dev(s["table"]), _dev(s["lens"]), _dev(s["shares"]), _dev(s["free"]),
            _dev(np.int32([s["head"]])), torch.zeros(1, dtype=torch.int32, device="cuda"))


def _fork(s, parents, children, fork_lens=None):
    import block_sparse_attention_nsa_gb300 as nsa
    table, lens, shares, free, head, status = _state(s)
    p, c = np.int32(parents), np.int32(children)
    src, dst, out = nsa.page_fork(table, lens, _dev(p), _dev(c), s["page"], shares, free, head,
                                  None if fork_lens is None else _dev(np.int32(fork_lens)),
                                  head_out=head, device_status=status)
    want = pages.fork(s["table"], s["lens"], p, c, s["page"], s["shares"], s["free"], s["head"],
                      fork_lens)
    _eq((table, lens, shares, src, dst, out, status), want)
    _eq((free,), (s["free"],))
    return want


def _free(s, rows):
    import block_sparse_attention_nsa_gb300 as nsa
    table, lens, shares, free, head, status = _state(s)
    r = np.int32(rows)
    out = nsa.page_free(table, lens, _dev(r), s["page"], shares, free, head, device_status=status)
    want = pages.release(s["table"], s["lens"], r, s["page"], s["shares"], s["free"], s["head"])
    _eq((table, lens, shares, free, out, status), want)
    return want


def _compact(s, count=None, free=None, in_place=True):
    import block_sparse_attention_nsa_gb300 as nsa
    table, lens, shares, fr, head, status = _state(s)
    if free is not None:
        fr = _dev(free)
    n = len(s["shares"]) // 2 if count is None else count
    src = torch.empty(n, dtype=torch.int32, device="cuda")
    outs = {}
    if not in_place:
        outs = dict(table_out=torch.full_like(table, 99), shares_out=torch.full_like(shares, 99),
                    free_out=fr.clone())
    src, dst, out = nsa.page_compact(table, lens, s["page"], shares, fr, copy_src=src, head_out=head,
                                     device_status=status, **outs)
    want = pages.compact(s["table"], s["lens"], s["page"], s["shares"], s["free"] if free is None else
                         free, n)
    got = (outs["table_out"], outs["shares_out"], outs["free_out"]) if outs else (table, shares, fr)
    left = s["head"] if want[5] is None else want[5]
    _eq(got + (src, dst, out, status), want[:5] + (left, want[6]))
    if outs:
        _eq((table, shares), (s["table"], s["shares"]))
    return want


# ---- orderly calls ---------------------------------------------------------------------
SHAPES = [  # rows, width, page, lens, spare: one CTA; many rows; a wide table; a large pool
    (8, 5, 4, (17, 3, 0, 8), 9), (300, 9, 64, tuple(range(0, 560, 7)), 500),
    (40, 700, 2, (1399, 5, 1, 600), 30), (6, 12, 1, (12, 0, 7), 70000), (1, 1, 1, (1,), 0)]


@pytest.mark.parametrize("rows,width,page,lens,spare", SHAPES)
def test_forks(rows, width, page, lens, spare):
    s = make_state(rows, width, page, lens, rows, spare)
    rng = np.random.default_rng(rows)
    idle = np.arange(len(lens), rows)
    k = min(len(idle), spare)
    children = rng.permutation(idle)[:k]
    parents = rng.integers(0, len(lens), k)
    assert _fork(s, parents, children)[-1] == 0
    part = rng.integers(0, s["lens"][parents] + 1) if k else None
    if k:
        assert _fork(s, parents, children, part.astype(np.int32))[-1] == 0
    _fork(s, [], [])


@pytest.mark.parametrize("rows,width,page,lens,spare", SHAPES)
def test_frees(rows, width, page, lens, spare):
    s = make_state(rows, width, page, lens, rows + 1, spare)
    rng = np.random.default_rng(rows)
    idle = np.arange(len(lens), rows)
    k = min(len(idle), spare)
    if k:
        p, c = rng.integers(0, len(lens), k), rng.permutation(idle)[:k]
        s["table"], s["lens"], s["shares"], _, _, s["head"], bits = pages.fork(
            s["table"], s["lens"], p, c, page, s["shares"], s["free"], s["head"])
        assert bits == 0
    for n in {0, 1, rows // 2, rows}:
        assert _free(s, rng.permutation(rows)[:n])[-1] == 0


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("rows,width,page,lens,spare", SHAPES)
def test_compactions(rows, width, page, lens, spare, in_place):
    forks = [(0, len(lens))] if rows > len(lens) and spare else []
    s = make_state(rows, width, page, lens, rows + 2, spare, forks)
    assert _compact(s, in_place=in_place)[-1] == 0
    # a full pool, and one that is compact already
    s = make_state(rows, width, page, lens, rows + 3, 0)
    s["table"], s["shares"], s["free"], _, _, s["head"], bits = _compact(s, in_place=in_place)
    assert bits == 0
    _compact(s, in_place=in_place)
    s["lens"][:] = 0                       # nothing in use
    _compact(s, in_place=in_place)


def test_long_life():
    """Plans, forks, frees and compactions in turn, in place, without a host in between."""
    import block_sparse_attention_nsa_gb300 as nsa
    rng = np.random.default_rng(5)
    s = make_state(40, 20, 16, tuple(rng.integers(0, 200, 20)), 6, spare=300)
    table, lens, shares, free, head, status = _state(s)
    total = len(s["shares"])
    for turn in range(25):
        new = np.where((s["lens"] > 0) & (s["lens"] < 280), rng.integers(0, 9, 40), 0).astype(np.int32)
        want = kv4.plan(s["lens"], new, s["free"], s["head"], s["table"], 16, total, int(new.sum()))
        s["table"], s["lens"], s["head"] = want[0], want[2], want[4]
        assert want[5] == 0
        nsa.page_plan(lens, _dev(new), free, head, table, 16, total, int(new.sum()), seq_lens=lens,
                      head_out=head, device_status=status)
        used, idle = np.flatnonzero(s["lens"]), np.flatnonzero(s["lens"] == 0)
        k = min(len(idle), 6)
        if k and len(used):
            p, c = rng.choice(used, k).astype(np.int32), rng.permutation(idle)[:k].astype(np.int32)
            s["table"], s["lens"], s["shares"], _, _, s["head"], bits = pages.fork(
                s["table"], s["lens"], p, c, 16, s["shares"], s["free"], s["head"])
            assert bits == 0
            nsa.page_fork(table, lens, _dev(p), _dev(c), 16, shares, free, head, head_out=head,
                          device_status=status)
        used = np.flatnonzero(s["lens"])
        rows = rng.permutation(used)[:5].astype(np.int32)
        s["table"], s["lens"], s["shares"], s["free"], s["head"], bits = pages.release(
            s["table"], s["lens"], rows, 16, s["shares"], s["free"], s["head"])
        nsa.page_free(table, lens, _dev(rows), 16, shares, free, head, head_out=head,
                      device_status=status)
        if turn % 8 == 7:
            s["table"], s["shares"], s["free"], _, _, s["head"], bits = pages.compact(
                s["table"], s["lens"], 16, s["shares"], s["free"], total // 2)
            nsa.page_compact(table, lens, 16, shares, free, head_out=head, device_status=status)
        check_books(s)
    _eq((table, lens, shares, free, head, status),
        (s["table"], s["lens"], s["shares"], s["free"], s["head"], 0))


# ---- what is refused on the device -------------------------------------------------------
def test_refused_forks():
    s = make_state(12, 6, 4, (22, 9, 16, 0), 1, spare=2)
    B, L, N = pages.BAD_INDEX, pages.BAD_SEQLENS, pages.NO_PAGES
    # rows outside, a child named twice, a child that is a parent, a fork onto itself
    assert _fork(s, [0, -1, 1, 1, 2, 12, 3], [5, 6, 5, -3, 1, 7, 3])[-1] == B
    # lengths
    assert _fork(s, [0, 1, 2], [5, 6, 7], np.int32([23, -1, 16]))[-1] == L
    # two pages for three forks that need one; those that need none go on
    assert _fork(s, [0, 0, 1, 2], [5, 6, 7, 8])[-1] == N
    for head in (-1, len(s["free"]) + 1):
        assert _fork({**s, "head": head}, [0, 2], [5, 6])[-1] == N
    # page ids that are none: in full entries, in the last, in the list
    t = s["table"].copy()
    t[0, 2], t[0, 5], t[1, 0] = 999, -5, -1
    assert _fork({**s, "table": t}, [0, 1, 2], [5, 6, 7])[-1] == B
    f = s["free"].copy()
    f[s["head"]] = 1000
    assert _fork({**s, "free": f}, [0, 1], [5, 6])[-1] == B
    n = s["lens"].copy()
    n[0], n[1] = 25, -2
    assert _fork({**s, "lens": n}, [0, 1, 2], [5, 6, 7])[-1] == L


def test_refused_frees():
    s = make_state(12, 6, 4, (22, 9, 16, 4), 2, spare=4, forks=[(0, 5), (2, 6)])
    B, L, N = pages.BAD_INDEX, pages.BAD_SEQLENS, pages.NO_PAGES
    assert _free(s, [0, 0, -1, 12, 5, 0])[-1] == B
    n = s["lens"].copy()
    n[1], n[3] = -4, 25
    assert _free({**s, "lens": n}, [0, 1, 3])[-1] == L
    t = s["table"].copy()
    t[0, 1], t[1, 2], t[2, 0] = -1, 10 ** 6, t[1, 0]      # no ids; a page that its count does not know
    assert _free({**s, "table": t}, [0, 1, 2, 5, 6])[-1] == B
    for head, bits in ((3, N), (0, N), (-1, N), (len(s["free"]) + 1, N)):
        assert _free({**s, "head": head}, [0, 5, 1])[-1] == bits
    assert _free({**s, "head": -1}, [4])[-1] == 0          # nothing to put there


def test_refused_compactions():
    s = make_state(9, 6, 4, (22, 9, 16, 4), 3, spare=20)
    B, L, N = pages.BAD_INDEX, pages.BAD_SEQLENS, pages.NO_PAGES
    moves = int((_compact(s)[3] >= 0).sum())
    assert moves > 1
    for in_place in (True, False):
        assert _compact(s, count=moves, in_place=in_place)[-1] == 0
        assert _compact(s, count=moves - 1, in_place=in_place)[-1] == N
        assert _compact(s, count=0, in_place=in_place)[-1] == N
        assert _compact(s, free=s["free"][:19], in_place=in_place)[-1] == N
        assert _compact(s, free=np.concatenate([s["free"], s["free"]]), in_place=in_place)[-1] == 0
        t, n = s["table"].copy(), s["lens"].copy()
        t[0, 0], t[1, 1] = -1, 5000
        assert _compact({**s, "table": t}, in_place=in_place)[-1] == B
        n[2], n[3] = -1, 100
        t[3, 1:] = t[0, 1:]
        assert _compact({**s, "lens": n, "table": t}, in_place=in_place)[-1] == B | L


# ---- copies ----------------------------------------------------------------------------
@pytest.mark.parametrize("pages_,shape,n", [(5, (16,), 2), (40, (3, 48), 9), (300, (2, 9216), 140),
                                            (7, (1, 100003 * 16), 3), (3000, (4, 32), 1500)])
def test_copies(pages_, shape, n):
    import block_sparse_attention_nsa_gb300 as nsa
    rng = np.random.default_rng(n)
    pool = rng.integers(0, 256, (pages_,) + shape, dtype=np.uint8)
    order = rng.permutation(pages_).astype(np.int32)
    src, dst = rng.choice(order[n:], n).astype(np.int32), order[:n].copy()
    src[n // 2] = dst[n // 2] = -1
    want = pool.copy()
    real = dst >= 0
    want[dst[real]] = pool[src[real]]
    got = _dev(pool)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert nsa.page_copy(got, _dev(src), _dev(dst), device_status=status) is got
    assert int(status.item()) == 0
    np.testing.assert_array_equal(got.cpu().numpy(), want)
    # ids outside the pool, and half a pair, are skipped and reported
    src[0], dst[n - 1] = pages_, -1
    want = pool.copy()
    for a, b in zip(src, dst):
        if 0 <= a < pages_ and 0 <= b < pages_:
            want[b] = pool[a]
    got = _dev(pool)
    nsa.page_copy(got.view(torch.int64), _dev(src), _dev(dst), device_status=status)
    assert int(status.item()) == pages.BAD_INDEX
    np.testing.assert_array_equal(got.cpu().numpy(), want)


def test_copies_past_32_bit_offsets():
    import block_sparse_attention_nsa_gb300 as nsa
    n, size = 2200, 2 << 20                                 # 4.6 GB
    pool = torch.zeros((n, size // 8), dtype=torch.int64, device="cuda")
    pool[1], pool[2150] = 7, torch.arange(size // 8, device="cuda")
    nsa.page_copy(pool, _dev(np.int32([1, 2150])), _dev(np.int32([2199, 0])))
    assert (pool[2199] == 7).all() and torch.equal(pool[0], pool[2150])


def test_refusals_of_python():
    import block_sparse_attention_nsa_gb300 as nsa
    s = make_state(4, 3, 4, (5, 2), 1)
    table, lens, shares, free, head, _ = _state(s)
    rows = _dev(np.int32([0]))
    with pytest.raises(ValueError):
        nsa.page_fork(table, lens.long(), rows, rows, 4, shares, free, head)
    with pytest.raises(ValueError):
        nsa.page_fork(table, lens, rows, _dev(np.int32([0, 1])), 4, shares, free, head)
    with pytest.raises(ValueError):
        nsa.page_free(table.t(), lens, rows, 4, shares, free, head)
    with pytest.raises(nsa.NsaError):
        nsa.page_free(table, lens, rows, 0, shares, free, head)
    pool = torch.zeros((4, 24), dtype=torch.uint8, device="cuda")
    with pytest.raises(nsa.NsaError):
        nsa.page_copy(pool, rows, rows)                     # 24 bytes a page
    with pytest.raises(ValueError):
        nsa.page_copy(pool.t(), rows, rows)


def test_beam_step_in_a_graph():
    """Free, fork and copy, captured and replayed: the same as calls one after the other."""
    import block_sparse_attention_nsa_gb300 as nsa
    s = make_state(30, 8, 32, (100, 33, 64, 7, 250), 9, spare=60,
                   forks=[(i % 5, 5 + i) for i in range(25)])
    pool = np.random.default_rng(1).integers(0, 256, (len(s["shares"]), 2, 64), dtype=np.uint8)
    a, b = (list(_state(s)) + [_dev(pool)] for _ in range(2))
    parents, children = _dev(np.int32([i % 5 for i in range(25)])), _dev(np.arange(5, 30, dtype=np.int32))

    def step(table, lens, shares, free, head, status, pool):
        nsa.page_free(table, lens, children, 32, shares, free, head, head_out=head, device_status=status)
        src, dst, _ = nsa.page_fork(table, lens, parents, children, 32, shares, free, head,
                                    head_out=head, device_status=status)
        nsa.page_copy(pool, src, dst, device_status=status)
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            step(*a)
    for _ in range(3):
        parents.copy_(parents.roll(1))
        graph.replay()
        step(*b)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(a, b))
        check_books(dict(table=a[0].cpu().numpy(), lens=a[1].cpu().numpy(), shares=a[2].cpu().numpy(),
                         free=a[3].cpu().numpy(), head=int(a[4].item()), page=32))
