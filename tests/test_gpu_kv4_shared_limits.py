"""The decode over shared prefixes at its limits: the shortest runs, one call after the other."""
import numpy as np
import pytest
import torch

from kv4_helpers import DTYPES
from oracle import kv4
from shared_helpers import check_shared, make_shared, wide

pytestmark = pytest.mark.gpu


def _dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


@pytest.mark.parametrize("d,g,dtype", [(64, 2, "bf16"), (128, 1, "fp16"), (128, 4, "bf16"), (128, 4, "fp16")])
def test_short_runs_one_after_the_other(d, g, dtype):
    """Runs of a block or two, whose CTAs end as soon as they have begun, while the next call's begin on the same
    SMs: every call returns what it does alone."""
    import block_sparse_attention_nsa_gb300 as nsa
    page, h_k, n = 32, 2, 70
    sets = []
    for seed, prefix in ((1, 40), (2, 200), (3, 128)):
        pool, table, lens, cu, pre = make_shared([(prefix, tuple(prefix + np.arange(n) % 9))], page, h_k, d, seed)
        q = torch.randn(n, h_k * g, d, generator=torch.Generator().manual_seed(seed)).to(DTYPES[dtype])
        sets.append([q.cuda()] + [_dev(x) for x in (pool, wide(table, page, n * h_k), lens)] + [0.1, _dev(cu), _dev(pre)])
    alone = []
    for s in sets:
        alone.append(nsa.kv4_decode_shared(*s))
        torch.cuda.synchronize()
        ref = kv4.attend(s[0].double().cpu().numpy()[:3], s[1].cpu().numpy(), s[2].cpu().numpy()[:3],
                         s[3].cpu().numpy()[:3], page, 0.1)
        check_shared(alone[-1][0][:3], alone[-1][1][:, :3], ref, DTYPES[dtype])
    got = [nsa.kv4_decode_shared(*sets[i % 3]) for i in range(300)]
    torch.cuda.synchronize()
    for i, (out, lse) in enumerate(got):
        assert torch.equal(out, alone[i % 3][0]) and torch.equal(lse, alone[i % 3][1]), i
