"""Long runs of the paged decode: a warp's sums over hundreds of tiles."""
import numpy as np
import pytest
import torch

from kv4_helpers import DTYPES, check_decode, make_cache
from oracle import kv4

pytestmark = pytest.mark.gpu


def _dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def _repeated(b, n, page, h_k, d, seed):
    """b sequences of n tokens that share their pages."""
    pool, table, _ = make_cache((n,), page, h_k, d, seed)
    return pool, np.repeat(table, b, 0), np.full(b, n, np.int32)


@pytest.mark.parametrize("d,h_k,b,dtype", [(128, 2, 128, "bf16"), (64, 2, 256, "bf16"),
                                           (128, 2, 128, "fp16"), (64, 2, 256, "fp16"),
                                           (128, 4, 300, "bf16"), (128, 4, 300, "fp16")])
def test_long_runs_lose_little(d, h_k, b, dtype):
    """Sequences of 64K tokens, of which a warp adds up 280 to 1500 tiles.  Values cancel over so
    many keys, and an error of one sign in each product grows with the run.  A result that is
    rounded once is off by the output type's rounding; what the sums add to that may be a third of
    it for bf16 and three quarters for fp16, in the root of the squares' sum: 1.055 and 1.25
    times the rounding."""
    import block_sparse_attention_nsa_gb300 as nsa
    dt, page, g, n = DTYPES[dtype], 64, 2, 65536
    pool, table, lens = _repeated(b, n, page, h_k, d, 90 + d)
    q = torch.randn(b, h_k * g, d, generator=torch.Generator().manual_seed(91)).to(dt)
    out, _ = nsa.kv4_decode(q.cuda(), _dev(pool), _dev(table), _dev(lens), d ** -0.5)
    rows = [0, b // 2, b - 1]
    ref = kv4.attend(q[rows].double().numpy(), pool, table[:3], lens[:3], page, d ** -0.5)[0]
    rounded = torch.from_numpy(ref).to(dt).double().numpy()
    off = np.linalg.norm(out[rows].double().cpu().numpy() - ref)
    assert off <= (1.055 if dt is torch.bfloat16 else 1.25) * np.linalg.norm(rounded - ref)


# ---- equal runs over a batch: kv4_run_kernel and kv4_merge_kernel ----------------------
# A table much wider than the lengths leaves the host no bound on a segment's tiles, and makes the call
# take equal runs of tiles.  A workspace filled with 0xff shows whether it did: runs write it.
def _workspace(nsa, pages, page, h_k, d, b, h_q):
    need = nsa.kv4_decode_workspace_size(pages, page, h_k, d, b, h_q)
    return torch.full((need,), 0xff, dtype=torch.uint8, device="cuda")


def _ragged(page, h_k, d, seed, most, count, last):
    """`count` sequences of up to `most` tokens (some empty) and one of `last`, of random pages that
    they share; and the pool's largest step of V."""
    rng = np.random.default_rng(seed)
    lens = np.concatenate([rng.integers(0, most + 1, count), [last]]).astype(np.int32)
    lens[[3, 77]] = 0
    lens[5] = 1
    lens = lens[rng.permutation(len(lens))]
    pages = 150
    pool, _, _ = make_cache((pages * page,), page, h_k, d, seed, spare=0)
    table = np.full((len(lens), -(-last // page)), -1, np.int32)
    for b, n in enumerate(lens):
        table[b, :-(-n // page)] = rng.integers(0, pages, -(-n // page))
    step = float(np.max(kv4.unpack(pool, page, d)[1][:, :, 1].astype(np.float64)))
    return pool, table, lens, step


@pytest.mark.parametrize("d,page,h_k,g,dtype,most,count,last,window", [
    # counted tiles of a warp on 152 SMs: 25, 50, 37, 37, 134, 18 (d = 64: sixteen warps an SM)
    (128, 64, 2, 4, "bf16", 3000, 400, 40000, 0),
    (128, 128, 2, 12, "fp16", 3000, 400, 40000, 0),
    (64, 32, 4, 1, "fp16", 3000, 400, 40000, 0),
    (64, 64, 2, 9, "bf16", 3000, 400, 40000, 0),
    (128, 64, 4, 5, "fp16", 9000, 400, 60000, 0),
    (128, 64, 2, 3, "bf16", 3000, 400, 40000, 9000),
    (64, 32, 1, 16, "fp16", 1500, 900, 30000, 0)])
def test_runs_with_many_segments(d, page, h_k, g, dtype, most, count, last, window):
    """Segments that begin, end and cross within a warp's run, a first part kept beside the
    tiles behind it, more than 32 tiles of a segment in a warp, and segments over many CTAs: 40
    sequences against the oracle, all of them against the batch in another order, whose runs
    are cut elsewhere."""
    import block_sparse_attention_nsa_gb300 as nsa
    dt = DTYPES[dtype]
    pool, table, lens, step = _ragged(page, h_k, d, d + g, most, count, last)
    b, h_q = len(lens), h_k * g
    q = torch.randn(b, h_q, d, generator=torch.Generator().manual_seed(g)).to(dt)
    ws = _workspace(nsa, pool.shape[0], page, h_k, d, b, h_q)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (_dev(pool), _dev(table), _dev(lens))
    out, lse = nsa.kv4_decode(q.cuda(), *args, d ** -0.5, window=window, workspace=ws,
                              device_status=status)
    assert (ws != 0xff).any(), "not the equal runs that this test is for"
    rows = np.random.default_rng(1).permutation(b)[:36]
    rows = np.unique(np.concatenate([rows, [lens.argmax(), lens.argmin(), 0, b - 1]]))
    ref = kv4.attend(q[rows].double().numpy(), pool, table[rows], lens[rows], page, d ** -0.5,
                     window=window)
    check_decode(out[rows], lse[:, rows], ref, dt)
    again, lse2 = nsa.kv4_decode(q.cuda(), *args, d ** -0.5, window=window, workspace=ws,
                                 device_status=status)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    perm = torch.randperm(b, generator=torch.Generator().manual_seed(2))
    o2, l2 = nsa.kv4_decode(q[perm].cuda(), _dev(pool), _dev(table[perm.numpy()]),
                            _dev(lens[perm.numpy()]), d ** -0.5, window=window, workspace=ws,
                            device_status=status)
    assert int(status.item()) == 0
    a, c = out[perm.cuda()].double(), o2.double()
    # two roundings to the output type, and twice what check_decode allows a weight's rounding
    tol = torch.finfo(dt).eps * torch.maximum(a.abs(), c.abs()) + 2 * 2.0 ** -11 * 8 * step
    assert ((a - c).abs() <= tol).all()
    dead = torch.isneginf(l2)
    assert torch.equal(torch.isneginf(lse)[:, perm.cuda()], dead) and dead.any()
    assert (a[dead.t()] == 0).all() and (c[dead.t()] == 0).all()
    near = (lse[:, perm.cuda()] - l2).abs()
    assert (near[~dead] <= 2.0 ** -16).all()
