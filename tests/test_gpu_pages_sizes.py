"""Slot maps of the sizes at which more CTAs share them, against the oracle."""
import numpy as np
import pytest
import torch

from oracle import kv4

pytestmark = pytest.mark.gpu


def _dev(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()


@pytest.mark.parametrize("pad", [0, 5])
@pytest.mark.parametrize("total", [4095, 4096, 4097, 32763, 32764, 32768, 32769, 65537, 131075])
def test_maps_around_their_cluster_sizes(total, pad):
    import block_sparse_attention_nsa_gb300 as nsa
    b, page = 130, 32
    rng = np.random.default_rng(total + pad)
    cuts = np.sort(rng.integers(0, total + 1, b - 1))
    new = np.diff(np.concatenate([[0], cuts, [total]])).astype(np.int32)
    ctx = rng.integers(0, 300, b).astype(np.int32)
    width = int((-(-(ctx + new) // page)).max())
    have = -(-ctx // page)
    need = int((-(-(ctx + new) // page) - have).sum())
    pages = int(have.sum()) + need + 3
    order = rng.permutation(pages).astype(np.int32)
    table, at = np.full((b, width), -1, np.int32), 0
    for i in range(b):
        table[i, :have[i]] = order[at:at + have[i]]
        at += have[i]
    free, slots = order[at:], total + pad
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    t = _dev(table)
    got = nsa.page_plan(_dev(ctx), _dev(new), _dev(free), _dev([0]), t, page, pages, slots, device_status=status)
    want = kv4.plan(ctx, new, free, 0, table, page, pages, slots)
    assert int(status.item()) == want[5] == 0
    for x, y in zip((t, *got), want):
        np.testing.assert_array_equal(x.cpu().numpy().reshape(np.shape(y)), y)
    back, cu = nsa.page_slots(t, _dev(ctx), _dev(new), page, pages, slots, device_status=status)
    assert int(status.item()) == 0
    np.testing.assert_array_equal(back.cpu().numpy(), want[1])
    np.testing.assert_array_equal(cu.cpu().numpy(), want[3])
