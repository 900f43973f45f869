"""The decode over shared prefixes at its limits: the shortest runs, one call after the other, and positions next
to 2^31."""
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


def _planned(work, pool, b, h_q, page, d):
    """Groups that the call has shared."""
    import block_sparse_attention_nsa_gb300 as nsa
    own = nsa.kv4_decode_workspace_size(pool.shape[0], page, pool.shape[1], d, b, h_q)
    at = -(-own // 256) * 256
    return work[at:at + 4].view(torch.int32).item()


def _workspace(pool, b, h_q, groups, page, d):
    import block_sparse_attention_nsa_gb300 as nsa
    return torch.full((nsa.kv4_decode_shared_workspace_size(pool.shape[0], page, pool.shape[1], d, b, h_q, groups),), 255,
                      dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("d,dtype", [(128, "bf16"), (64, "fp16")])
def test_a_prefix_as_long_as_a_table_can_be(d, dtype):
    """A group that claims all of a table of 2^31 - 32 tokens, whose sequences are short, beside one that
    shares."""
    import block_sparse_attention_nsa_gb300 as nsa
    page, b = 32, 15
    pool, table, lens, cu, prefix = make_shared([(20, (100, 20, 77, 131, 99)), (300, tuple(range(300, 310)))], page, 1, d, 5)
    q = torch.randn(b, 1, d, generator=torch.Generator().manual_seed(1)).to(DTYPES[dtype])
    far = torch.full((b, 2 ** 26 - 1), -1, dtype=torch.int32, device="cuda")
    far[:, :table.shape[1]] = _dev(table)
    prefix[0] = page * far.shape[1]
    work, status = _workspace(pool, b, 1, 2, page, d), torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = nsa.kv4_decode_shared(q.cuda(), _dev(pool), far, _dev(lens), 0.1, _dev(cu), _dev(prefix), workspace=work,
                                     device_status=status)
    assert int(status.item()) == 0 and _planned(work, pool, b, 1, page, d) == 2
    check_shared(out, lse, kv4.attend(q.double().numpy(), pool, table, lens, page, 0.1), DTYPES[dtype])


@pytest.mark.parametrize("d,dtype", [(128, "bf16"), (64, "fp16")])
def test_keys_next_to_the_last_position(d, dtype):
    """Five sequences of nearly 2^31 tokens, all of the same page, so that each of its keys counts as often as
    it occurs."""
    import block_sparse_attention_nsa_gb300 as nsa
    page, g, width = 128, 8, 2 ** 24 - 1
    keys = page * (width - 1) - 5
    lens = np.int32([keys, keys + 1, keys + 100, keys + 133, keys + 5])
    b, h_q, scale = len(lens), g, d ** -0.5
    rng = np.random.default_rng(9)
    pool = kv4.pack(*kv4.quantise(rng.standard_normal((1, 1, 2, page, d), np.float32)))
    q = torch.randn(b, g, d, generator=torch.Generator().manual_seed(2)).to(DTYPES[dtype])
    work, status = _workspace(pool, b, h_q, 1, page, d), torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = nsa.kv4_decode_shared(q.cuda(), _dev(pool), torch.zeros(b, width, dtype=torch.int32, device="cuda"), _dev(lens),
                                     scale, _dev(np.int32([0, b])), _dev(lens[:1]), workspace=work, device_status=status)
    assert int(status.item()) == 0 and _planned(work, pool, b, h_q, page, d) == 1
    code, step, zero = kv4.unpack(pool, page, d)
    k, v = (kv4.dequantise(code[0, 0, w], step[0, 0, w], zero[0, 0, w]) for w in (0, 1))
    s = np.einsum("bhd,kd->bhk", q.double().numpy(), k) * scale
    times = np.int64(lens)[:, None] // page + (np.arange(page) < np.int64(lens)[:, None] % page)
    top = s.max(-1, keepdims=True)
    p = np.exp(s - top) * times[:, None]
    r_lse = (top[..., 0] + np.log(p.sum(-1))).T
    p /= p.sum(-1, keepdims=True)
    # scores and fp32's lse as in check_decode; sums of 32 keys, 256 blocks, 432 of those (110K blocks a CTA) and 152 CTAs
    big = kv4.attend(q.double().numpy(), pool, np.zeros((b, 1), np.int32), [page] * b, page, scale)[2]
    ds, sums = d * 2.0 ** -24 * big + 2.0 ** -20, (32 + 256 + 432 + 152) * 2.0 ** -24
    off = np.abs(lse.double().cpu().numpy() - r_lse)
    assert (off <= ds.T + 2.0 ** -22 * np.abs(r_lse) + sums).all()
    # half a step of the output, V's and a weight's rounding, the tensor core's sums (2048 steps), weights and their sums
    ref, pv = p @ v, p @ np.abs(v)
    tol = torch.finfo(DTYPES[dtype]).eps / 2 * np.abs(ref) + (2.0 ** -10 + 2.0 ** -13 + 2 * ds[..., None] + 2 * sums) * pv + 2.0 ** -25
    assert (np.abs(out.double().cpu().numpy() - ref) <= tol).all()
