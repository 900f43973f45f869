"""Long runs of the paged decode: a warp's sums over hundreds of tiles."""
import numpy as np
import pytest
import torch

from kv4_helpers import DTYPES, make_cache
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
