"""A prefill chunk over cached tokens: pages read back as 16-bit rows, attended to by the
framework's forward."""
import numpy as np
import pytest
import torch

import oracle
from gpu_helpers import check_forward

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page,d,dtype", [(64, 128, torch.bfloat16), (32, 64, torch.float16)])
def test_chunk_over_cached_tokens(page, d, dtype):
    """Requests with cached and new tokens.  The forward takes q, k and v of one length: q has a
    row for each cached token too, whose selection is empty, so that its output is zero."""
    import block_sparse_attention_nsa_gb300 as nsa
    h_k, g, topk, pages = 2, 4, 5, 60
    cached, new = [300, 0, 65, 1], [90, 130, 1, 64]
    b, total = len(new), sum(cached) + sum(new)
    gen = torch.Generator().manual_seed(11)
    i32 = dict(dtype=torch.int32, device="cuda")
    pool = nsa.kv4_pool(pages, page, h_k, d)
    table = torch.full((b, 16), -1, **i32)
    free, head = torch.randperm(pages, generator=gen).int().cuda(), torch.zeros(1, **i32)
    lens, status = torch.zeros(b, **i32), torch.zeros(1, **i32)
    for step in (cached, new):
        n = sum(step)
        k, v = (torch.randn(n, h_k, d, generator=gen).to(dtype).cuda() for _ in range(2))
        slots, _, _, _ = nsa.page_plan(lens, torch.tensor(step, **i32), free, head, table, page, pages,
                                       n, seq_lens=lens, head_out=head, device_status=status)
        nsa.kv4_append(pool, k, v, slots, device_status=status)
    slots, cu = nsa.page_slots(table, torch.zeros_like(lens), lens, page, pages, total,
                               device_status=status)
    kr, vr = nsa.kv4_read(pool, slots, d, dtype=dtype, device_status=status)
    assert int(status.item()) == 0
    q = torch.randn(total, h_k * g, d, generator=gen).to(dtype)
    rng, cu_h = np.random.default_rng(12), cu.cpu().numpy()
    sel = np.full((h_k, total, topk), -1, np.int32)
    fresh = np.zeros(total, bool)
    for r in range(b):
        for t in range(cached[r], cached[r] + new[r]):
            blocks = t // page + 1
            fresh[cu_h[r] + t] = True
            for h in range(h_k):
                pick = np.concatenate([[blocks - 1, 0], rng.integers(0, blocks, topk - 2)])
                sel[h, cu_h[r] + t] = rng.permutation(pick)
    out, lse = nsa.fwd(q.cuda(), kr, vr, torch.from_numpy(sel).cuda(), cu, page, d ** -0.5)
    ref = oracle.fwd(cu_h, page, sel, q, kr, vr, d ** -0.5)
    check_forward(out, lse, *ref)
    old = torch.from_numpy(~fresh).cuda()
    assert (out[old] == 0).all() and torch.isneginf(lse[:, old]).all()
    # the last tokens of the chunks, decoded from the pages themselves
    last = cu[1:].long() - 1
    o4, l4 = nsa.kv4_decode(q[last.cpu()].cuda(), pool, table, lens, d ** -0.5,
                            sel_idx=torch.from_numpy(sel).cuda()[:, last].contiguous())
    torch.testing.assert_close(o4.float(), out[last].float(), rtol=2e-2, atol=2e-2)
    torch.testing.assert_close(l4, lse[:, last], rtol=0, atol=2e-2)   # keys rounded to 16 bits
