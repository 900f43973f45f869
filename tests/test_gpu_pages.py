"""Block tables and slot maps built on the GPU, equal to the oracle's in every entry."""
import numpy as np
import pytest
import torch

from oracle import kv4

pytestmark = pytest.mark.gpu


def _dev(x):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(x, np.int32))).cuda()


def _step(rng, ctx, new, page, width, pages, num_free, head, max_slots, spoil=None):
    """Runs a plan, and the slots of what is cached then, both against the oracle."""
    import block_sparse_attention_nsa_gb300 as nsa
    b = len(ctx)
    order = rng.permutation(pages).astype(np.int32)
    table, at = np.full((b, width), -1, np.int32), 0
    for i in range(b):
        n = min(max(0, -(-int(ctx[i]) // page)), width, max(0, pages - num_free - at))
        table[i, :n] = order[at:at + n]
        at += n
    free = order[pages - num_free:] if num_free else order[:0]
    if spoil is not None:
        spoil(table, free)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dt = _dev(table)
    slots, seq, cu, out = nsa.page_plan(_dev(ctx), _dev(new), _dev(free), _dev([head]), dt, page,
                                        pages, max_slots, device_status=status)
    want = kv4.plan(ctx, new, free, head, table, page, pages, max_slots)
    for got, ref, name in zip((dt, slots, seq, cu), want, ("table", "slots", "seq_lens", "cu")):
        np.testing.assert_array_equal(got.cpu().numpy(), ref, err_msg=name)
    assert int(out.item()) == want[4] and int(status.item()) == want[5]
    # in place: lengths and the free list's head advance
    lens, hd, dt2 = _dev(ctx), _dev([head]), _dev(table)
    s2, _, _, _ = nsa.page_plan(lens, _dev(new), _dev(free), hd, dt2, page, pages, max_slots,
                                seq_lens=lens, head_out=hd)
    assert torch.equal(s2, slots) and torch.equal(lens, seq) and torch.equal(dt2, dt)
    assert torch.equal(hd, out)
    start = np.minimum(rng.integers(0, 50, b), np.maximum(want[2], 0)).astype(np.int32)
    count = want[2] - start
    got, gcu = nsa.page_slots(dt, _dev(start), _dev(count), page, pages, max_slots,
                              device_status=status.zero_())
    ref = kv4.slots(want[0], start, count, page, pages, max_slots)
    np.testing.assert_array_equal(got.cpu().numpy(), ref[0])
    np.testing.assert_array_equal(gcu.cpu().numpy(), ref[1])
    assert int(status.item()) == ref[2]
    return want[5]


@pytest.mark.parametrize("b,page,hi", [(1, 64, 1), (1, 32, 5000), (64, 64, 1), (7, 128, 300),
                                       (1000, 32, 20), (1024, 64, 2), (1025, 16, 3), (3000, 1, 4),
                                       (2, 100, 4000)])
def test_plan_and_slots(b, page, hi):
    rng = np.random.default_rng(b + page)
    ctx = rng.integers(0, 400, b)
    new = rng.integers(0, hi + 1, b)
    width = int(-(-(ctx + new).max() // page)) + 1
    need = int((-(-(ctx + new) // page) - -(-ctx // page)).sum())
    pages = int((-(-ctx // page)).sum()) + need + 5
    for pad in (0, 3, 1001):
        assert _step(rng, ctx, new, page, width, pages, need + 5, 2, int(new.sum()) + pad) == 0


def test_plan_largest_batch():
    rng = np.random.default_rng(5)
    b = 16384
    ctx, new = rng.integers(0, 100, b), rng.integers(0, 2, b)
    assert _step(rng, ctx, new, 32, 5, 6 * b, 2 * b, 0, b) == 0


def test_plan_refuses_requests():
    rng = np.random.default_rng(6)
    ctx, new = np.array([10, 60, 0, 64, 5, 30]), np.array([40, 5, 70, 0, 1, 40])
    # pages needed: 0, 1, 2, 0, 0, 1 (page 64)
    base = dict(page=64, width=4, pages=20, head=0)
    total = int(new.sum())
    for num_free in range(6):
        bits = _step(rng, ctx, new, num_free=num_free, max_slots=total, **base)
        assert bits == (0 if num_free >= 4 else kv4.NO_PAGES)
    for room in (0, 39, 40, 45, 115, 116, 155, 156):
        bits = _step(rng, ctx, new, num_free=8, max_slots=room, **base)
        assert bits == (0 if room >= total else kv4.NO_PAGES)
    assert _step(rng, ctx, new, num_free=8, max_slots=total, page=64, width=1, pages=20,
                 head=0) == kv4.BAD_SEQLENS
    for c, n in ((-1, 4), (3, -2), (1 << 30, 1 << 30), (200, 57), (257, 0)):
        ctx2, new2 = ctx.copy(), new.copy()
        ctx2[2], new2[2] = c, n
        bits = _step(rng, ctx2, new2, num_free=8, max_slots=200, **base)
        assert bits & kv4.BAD_SEQLENS
    for head in (-1, 9):
        bits = _step(rng, ctx, new, num_free=8, max_slots=total, page=64, width=4, pages=20,
                     head=head)
        assert bits == kv4.NO_PAGES


def test_plan_bad_page_ids():
    rng = np.random.default_rng(7)
    ctx, new = np.array([10, 60, 0, 64, 5, 30]), np.array([40, 5, 70, 0, 1, 40])

    def in_free(table, free):
        free[1] = 20

    def in_table(table, free):
        table[0, 0] = -1
        table[4, 0] = 1 << 30
    for spoil in (in_free, in_table):
        assert _step(rng, ctx, new, 64, 4, 20, 8, 0, 160, spoil) == kv4.BAD_INDEX


def test_unaligned_slot_map_and_rows_behind():
    import block_sparse_attention_nsa_gb300 as nsa
    table = _dev([[3, 1], [0, 2]])
    buf = torch.full((12,), 77, dtype=torch.int32, device="cuda")
    s, cu = nsa.page_slots(table, _dev([2, 0]), _dev([3, 4]), 4, 4, buf[1:10])
    assert buf.tolist() == [77, 14, 15, 4, 0, 1, 2, 3, -1, -1, 77, 77]
    assert cu.tolist() == [0, 3, 7]


def test_plan_in_a_graph():
    """A captured step that advances its own lengths and free list."""
    import block_sparse_attention_nsa_gb300 as nsa
    b, page, pages = 5, 32, 40
    free = torch.arange(pages, dtype=torch.int32, device="cuda")
    lens, head, one = _dev([0, 31, 32, 5, 60]), _dev([8]), _dev([1] * b)
    table = torch.full((b, 6), -1, dtype=torch.int32, device="cuda")
    table[1:, 0] = torch.arange(4)
    table[4, 1] = 4
    want_t, want_l, want_h = table.cpu().numpy(), lens.tolist(), 8
    slots = torch.empty(b, dtype=torch.int32, device="cuda")
    cu = torch.empty(b + 1, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nsa.page_plan(lens, one, free, head, table, page, pages, slots, lens, cu, head)
    for _ in range(40):
        graph.replay()
        want_t, s, want_l, _, want_h, bits = kv4.plan(want_l, [1] * b, free.tolist(), want_h, want_t,
                                                      page, pages, b)
        assert bits == 0
        np.testing.assert_array_equal(slots.cpu().numpy(), s)
    np.testing.assert_array_equal(table.cpu().numpy(), want_t)
    np.testing.assert_array_equal(lens.cpu().numpy(), want_l)
    assert int(head.item()) == want_h


def test_plan_rejects():
    import block_sparse_attention_nsa_gb300 as nsa
    a, t = _dev([1, 2]), _dev([[0, 1], [2, 3]])
    with pytest.raises(ValueError):
        nsa.page_slots(t, a.long(), a, 4, 4, 8)
    with pytest.raises(ValueError):
        nsa.page_slots(t.t(), a, a, 4, 4, 8)
    with pytest.raises(ValueError):
        nsa.page_plan(a, a[:1], a, a[:1], t, 4, 4, 8)
    with pytest.raises(nsa.NsaError) as e:
        nsa.page_slots(t, a, a, 0, 4, 8)
    assert e.value.code == 1
    with pytest.raises(nsa.NsaError) as e:
        nsa.page_slots(t, a, a, 1 << 30, 4, 8)
    assert e.value.code == 2
