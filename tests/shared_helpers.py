"""Caches whose sequences share prefixes, and the error bounds of the decode over them."""
import numpy as np
import torch

from kv4_helpers import check_decode
from oracle import kv4


def make_shared(groups, page, h_k, d, seed, alone=(), width=None, mags=(1.0,)):
    """groups: (prefix, lengths of its sequences) pairs, then sequences that are alone.  Members name
    the first one's full prefix pages and have a copy of what the prefix leaves of the next.  Rows
    that belong to nobody hold random codes with NaN scales and zeros."""
    rng = np.random.default_rng(seed)
    lens = [n for _, ns in groups for n in ns] + list(alone)
    per = [-(-n // page) for n in lens]
    pages = sum(per) + 3
    shape = (pages, h_k, 2, page, d)
    x = rng.standard_normal(shape).astype(np.float32) * rng.choice(mags, shape[:4] + (1,))
    x[..., ::29] *= 3
    code, scale, zero = kv4.quantise(x)
    width = width or max(1, max(per))
    table, order, at = np.full((len(lens), width), -1, np.int32), rng.permutation(pages), 0
    for b, n in enumerate(per):
        table[b, :n] = order[at:at + n]
        at += n
    owned = np.zeros((pages, page), bool)
    row = 0
    for prefix, ns in groups:
        full, rest = divmod(prefix, page)
        for b in range(row + 1, row + len(ns)):
            k = min(full, -(-lens[b] // page))
            table[b, :k] = table[row, :k]
            if rest and k == full and lens[b] > full * page:
                a, z = table[row, full], table[b, full]
                for arr in (code, scale, zero):
                    arr[z, :, :, :rest] = arr[a, :, :, :rest]
        row += len(ns)
    for b, n in enumerate(lens):
        for j in range(per[b]):
            owned[table[b, j], :max(0, min(page, n - j * page))] = True
    code = np.where(owned[:, None, None, :, None], code, rng.integers(0, 16, code.shape, np.uint8))
    free = ~np.broadcast_to(owned[:, None, None, :, None], scale.shape)
    scale[free], zero[free] = np.float16("nan"), np.float16("nan")
    cu = np.concatenate([[0], np.cumsum([len(ns) for _, ns in groups])]).astype(np.int32)
    return (kv4.pack(code, scale, zero), table, np.int32(lens), cu,
            np.int32([p for p, _ in groups]))


def check_shared(out, lse, ref, dtype):
    """check_decode's bounds and, for the prefix' weights and values rounded to fp16, half a step
    (2^-11) each of the sum of p |v|, and fp16's smallest half step."""
    r_out, r_lse, big, pv, ps = ref
    extra = 2.0 ** -10 * (1 + 2.0 ** -8) * pv + 2.0 ** -25
    # as far as the extra bound allows, towards the reference; what is left is check_decode's
    got = out.double().cpu()
    ref_t, ex = torch.from_numpy(r_out), torch.from_numpy(extra)
    off = got - ref_t
    moved = ref_t + torch.sign(off) * (off.abs() - ex).clamp(min=0)
    assert got.isfinite().all()

    class _Wide:                                     # keeps the dtype's bounds without rounding again
        def float(self):
            return self

        def cpu(self):
            return self

        def numpy(self):
            return moved.numpy()
    check_decode(_Wide(), lse, ref, dtype)


def wide(table, page, segs):
    """The table with room for far longer sequences than it has: a batch for which, by the sizes that
    the host knows, sharing may pay (segs: sequences times KV heads, twice for more than 8 query
    heads each)."""
    tiles = max(1100, 16000 // segs)
    cols = -(-tiles * 32 // page)
    out = np.full((table.shape[0], max(cols, table.shape[1])), -1, np.int32)
    out[:, :table.shape[1]] = table
    return out
