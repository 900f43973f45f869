"""Serving steps on the 4-bit cache as they follow one another: rotary positions, pages planned, rows
appended, a prompt forked, pages copied, freed and compacted, and the decode over the shared prefix."""
import numpy as np
import pytest
import torch

from kv4_helpers import DTYPES
from oracle import kv4
from oracle import rope as oracle_rope
from shared_helpers import check_shared

pytestmark = pytest.mark.gpu


def _dev(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device="cuda")


def _cache(tokens, page, h_k, d):
    """A pool and table that hold each row's own copy of its tokens."""
    per = [-(-len(t) // page) for t in tokens]
    x = np.zeros((sum(per) + 1, h_k, 2, page, d), np.float32)
    table = np.full((len(tokens), max(per)), -1, np.int32)
    at = 0
    for b, t in enumerate(tokens):
        table[b, :per[b]] = np.arange(at, at + per[b])
        for i, kv in enumerate(t):
            x[at + i // page, :, :, i % page] = kv.transpose(1, 0, 2)
        at += per[b]
    return kv4.pack(*kv4.quantise(x)), table


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("d,page,dtype", [(128, 64, "bf16"), (64, 32, "fp16")])
def test_steps_together(d, page, dtype, graph):
    import block_sparse_attention_nsa_gb300 as nsa
    dt, rows, h_k, g, prompt, pages = DTYPES[dtype], 40, 2, 4, 301, 150
    gen = torch.Generator().manual_seed(d)
    width = max(1100, 16000 // (rows * h_k)) * 32 // page       # room for far longer sequences
    pool = nsa.kv4_pool(pages, page, h_k, d)
    table = torch.full((rows, width), -1, dtype=torch.int32, device="cuda")
    lens, shares = _dev([0] * rows), _dev([0] * pages)
    free, head, status = _dev(range(pages)), _dev([0]), _dev([0])
    freqs = nsa.rope_freqs(d, scaling="linear", factor=4.0)
    w = oracle_rope.freqs(d, scaling="linear", factor=4.0)
    one, cu = _dev([1] * rows), _dev(range(rows + 1))
    cu_groups, prefix = _dev([0, rows]), _dev([prompt])
    q = torch.empty(rows, h_k * g, d, dtype=dt, device="cuda")
    k, v = (torch.empty(rows, h_k, d, dtype=dt, device="cuda") for _ in range(2))
    q_at, k_at = torch.empty_like(q), torch.empty_like(k)
    out, lse = torch.empty_like(q), torch.empty(h_k * g, rows, device="cuda")
    slots = _dev([0] * rows)

    def step():
        nsa.rope(q, k, freqs, cu_seqlens=cu, start=lens, q_out=q_at, k_out=k_at, device_status=status)
        nsa.page_plan(lens, one, free, head, table, page, pages, slots, seq_lens=lens, head_out=head,
                      device_status=status)
        nsa.kv4_append(pool, k_at, v, slots, device_status=status)
        nsa.kv4_decode_shared(q_at, pool, table, lens, d ** -0.5, cu_groups, prefix, out=out, lse=lse,
                              device_status=status)

    def kv_of(a, b):
        return [np.stack(x) for x in zip(a.float().cpu().numpy(), b.float().cpu().numpy())]

    # the prompt, in row 0
    k0, v0 = (torch.randn(prompt, h_k, d, generator=gen).to(dt).cuda() for _ in range(2))
    _, k0_at = nsa.rope(None, k0, freqs, positions=_dev(range(prompt)))
    new = _dev([prompt] + [0] * (rows - 1))
    s0 = nsa.page_plan(lens, new, free, head, table, page, pages, prompt, seq_lens=lens, head_out=head,
                       device_status=status)[0]
    nsa.kv4_append(pool, k0_at, v0, s0, device_status=status)
    tokens = [kv_of(k0_at, v0)] + [None] * (rows - 1)

    def fork(parents, children, fork_lens=None):
        src, dst, _ = nsa.page_fork(table, lens, _dev(parents), _dev(children), page, shares, free, head,
                                    fork_lens=None if fork_lens is None else _dev(fork_lens),
                                    head_out=head, device_status=status)
        nsa.page_copy(pool, src, dst, device_status=status)
        for i, (a, b) in enumerate(zip(parents, children)):
            tokens[b] = tokens[a][:None if fork_lens is None else fork_lens[i]]

    fork([0] * (rows - 1), range(1, rows))
    captured = None
    if graph:
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            step()
    for turn in range(5):
        if turn == 2:
            gone = [5, 6, 7, 8, 39]
            nsa.page_free(table, lens, _dev(gone), page, shares, free, head, head_out=head,
                          device_status=status)
            fork([3, 3, 0, 11, 11], gone, [prompt, prompt + 1, prompt + 2, prompt, prompt + 2])
        if turn == 3:
            src, dst, _ = nsa.page_compact(table, lens, page, shares, free, head_out=head,
                                           device_status=status)
            nsa.page_copy(pool, src, dst, device_status=status)
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, generator=gen).to(dt))
        at = [len(t) for t in tokens]
        captured.replay() if graph else step()
        ref = oracle_rope.rotate(k.double().cpu().numpy(), at, w, False)
        # half a step, and 2^-20 of the values (at most 6) for fp32
        assert (np.abs(k_at.double().cpu().numpy() - ref) <= torch.finfo(dt).eps / 2 * np.abs(ref) + 6 * 2.0 ** -20).all()
        for b, kv in enumerate(kv_of(k_at, v)):
            tokens[b] = tokens[b] + [kv]
        assert status.item() == 0
        assert lens.tolist() == [len(t) for t in tokens]
        own, own_table = _cache(tokens, page, h_k, d)
        ref = kv4.attend(q_at.double().cpu().numpy(), own, own_table, np.int32([len(t) for t in tokens]), page,
                         d ** -0.5)
        check_shared(out, lse, ref, dt)
    # every page is free or named by a row
    named = set()
    for b, n in enumerate(lens.tolist()):
        named |= set(table[b, :-(-n // page)].tolist())
    assert sorted(named | set(free[head.item():].tolist())) == list(range(pages))
    assert len(named) + pages - head.item() == pages
