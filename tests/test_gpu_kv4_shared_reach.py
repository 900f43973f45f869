"""The decode over shared prefixes where a prefix is shared, which every call here looks up in the plan that it
leaves in its workspace."""
import numpy as np
import pytest
import torch

from kv4_helpers import DTYPES
from oracle import kv4
from shared_helpers import check_shared, make_shared, wide
from workloads import CONFIGS, make_inputs

pytestmark = pytest.mark.gpu


def _dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def _call(q, pool, table, lens, scale, cu, prefix, shared, status=None, stream=None):
    """out and lse of a call whose plan shares that many prefixes."""
    import block_sparse_attention_nsa_gb300 as nsa
    (b, h_q, d), (pages, h_k, size), groups = q.shape, pool.shape, prefix.numel()
    page = size // (d + d // 8)
    need = nsa.kv4_decode_shared_workspace_size(pages, page, h_k, d, b, h_q, groups)
    own = nsa.kv4_decode_workspace_size(pages, page, h_k, d, b, h_q)
    work = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    got = nsa.kv4_decode_shared(q, pool, table, lens, scale, cu, prefix, workspace=work, device_status=status,
                                stream=stream)
    torch.cuda.synchronize()
    at = -(-own // 256) * 256                     # the plan's first number: groups that share
    assert work[at:at + 4].view(torch.int32).item() == shared
    return got


def _run(groups, page, h_k, g, d, dtype, seed, shared, some=None, scale=None, alone=(), mags=(1.0,)):
    pool, table, lens, cu, prefix = make_shared(groups, page, h_k, d, seed, alone, None, mags)
    dt = DTYPES[dtype]
    q = torch.randn(len(lens), h_k * g, d, generator=torch.Generator().manual_seed(seed)).to(dt)
    scale = d ** -0.5 if scale is None else scale
    rows = np.arange(len(lens)) if some is None else np.asarray(some)
    out, lse = _call(q.cuda(), _dev(pool), _dev(wide(table, page, len(lens) * h_k)), _dev(lens), scale, _dev(cu),
                     _dev(prefix), shared)
    ref = kv4.attend(q[rows].double().numpy(), pool, table[rows], lens[rows], page, scale)
    check_shared(out[rows], lse[:, rows], ref, dt)
    return out[rows], ref


def _members(n, prefix, seed, most=40):
    own = np.random.default_rng(seed).integers(0, most, n)
    own[::7] = 0
    return tuple(int(prefix + x) for x in own)


@pytest.mark.parametrize("d,page,n,g", [(64, 128, 8, 2), (128, 64, 8, 2), (128, 64, 40, 4)])
def test_long_fp16_loses_little(d, page, n, g):
    """V rounded to fp16 is off by what the output's rounding is, relative to it, and the two are independent: 2^0.5
    of it together.  The rest (weights in two parts, sums) has up to half of it: 1.5^2 - 2 = 0.5^2."""
    out, ref = _run([(30011, tuple(30011 + 13 * i for i in range(n)))], page, 1, g, d, "fp16", 77, 1,
                    some=(0, 1, n // 2, n - 1))
    rounding = np.linalg.norm(ref[0].astype(np.float16) - ref[0])
    off = np.linalg.norm(out.double().cpu().numpy() - ref[0])
    assert off <= 1.5 * rounding, f"{off / rounding:.3f} roundings off"


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,prefix", [(129, 700), (200, 65), (255, 33), (256, 200), (257, 129), (300, 100), (385, 97),
                                         (511, 128), (512, 161), (513, 128), (520, 300)])
def test_more_rows_than_a_tile(rows, prefix, dtype):
    """Tiles of 256 rows, their second half full, partly full or empty, one behind the other; prefixes that leave
    the second half of a block's keys empty."""
    for g in (4, 3 if rows % 2 else 5):
        n = -(-rows // g)
        keys = prefix if g == 4 or g == 3 else prefix + 100      # fewer sequences: a longer one pays
        own = keys + np.random.default_rng(rows).integers(0, 90, n)
        _run([(keys, tuple(own))], 64 if g == 4 else 32, 2, g, 128, dtype, rows, 1,
             some=sorted({0, 1, 31, 32, n // 2, n - 2, n - 1}))


@pytest.mark.parametrize("d,page,h_k,g,dtype", [(64, 32, 2, 2, "fp16"), (128, 64, 2, 1, "bf16"), (128, 32, 2, 5, "fp16")])
def test_groups_that_share_among_others(d, page, h_k, g, dtype):
    """Of five groups two are worth it; prefixes of one key and around a block."""
    a, b = list(_members(75, 300, 4)), list(_members(130, 129, 5))
    a[3], a[4], b[0], b[129] = 299, 0, 129, 64
    _run([(40, (50, 41)), (300, tuple(a)), (77, ()), (129, tuple(b)), (600, (700,))], page, h_k, g, d, dtype, 7 * d + g, 2,
         alone=(5, 0, 333), some=(0, 1, 2, 3, 5, 6, 76, 77, 78, 205, 206, 207, 208, 209, 210))


@pytest.mark.parametrize("prefix", [1, 33, 127, 129, 513])
def test_prefixes_around_blocks(prefix):
    _run([(prefix, _members(70, prefix, 1))], 64, 1, 1, 128, "bf16", prefix, 1, some=(0, 1, 7, 59, 69))
    _run([(prefix, _members(70, prefix, 2))], 32, 2, 1, 64, "fp16", prefix, 1, some=(0, 1, 7, 59, 69))


@pytest.mark.parametrize("d,g", [(64, 1), (128, 1), (128, 4)])
def test_malformed_groups(d, g):
    """A cu_groups out of order shares nothing; a prefix that cannot be leaves its own group alone."""
    import block_sparse_attention_nsa_gb300 as nsa
    page, n = 32, 60
    pool, table, lens, cu, prefix = make_shared([(300, _members(n, 300, 1)), (200, _members(n, 200, 2))], page, 1, d, 51)
    table = wide(table, page, 2 * n)
    q = torch.randn(2 * n, g, d, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    some = [0, 1, 7, n - 1, n, n + 1, 2 * n - 1]
    ref = kv4.attend(q[some].double().numpy(), pool, table[some], lens[some], page, 0.1)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    bad = nsa.DEVERR_BAD_SEQLENS
    for c, p, shared, bits in ((cu, prefix, 2, 0), ((0, n, 2 * n + 1), prefix, 0, bad), ((1, n, 2 * n), prefix, 0, bad),
                               ((0, n, n - 1), prefix, 0, bad), ((0, -1, 2 * n), prefix, 0, bad),
                               ((0, 2 * n, n), prefix, 0, bad), (cu, (-1, 200), 1, bad), (cu, (300, 10 ** 7), 1, bad),
                               (cu, (300, table.shape[1] * page + 1), 1, bad), (cu, (-2 ** 31, 2 ** 31 - 1), 0, bad)):
        out, lse = _call(q.cuda(), _dev(pool), _dev(table), _dev(lens), 0.1, _dev(np.int32(c)), _dev(np.int32(p)), shared,
                         status.zero_())
        assert int(status.item()) == bits, (c, p)
        check_shared(out[some], lse[:, some], ref, torch.bfloat16)


def test_streams_at_once():
    """Prefix kernels of pairs of CTAs and of single ones on four streams, none of which waits for another, and
    training's forward on a fifth: all of them want all of an SM's tensor memory.  Every call returns what it
    does alone."""
    import block_sparse_attention_nsa_gb300 as nsa
    sets, alone = [], []
    for seed, (d, g, n, prefix, dtype) in enumerate(((128, 4, 70, 3000, "bf16"), (128, 4, 66, 2000, "fp16"),
                                                     (128, 1, 60, 2500, "bf16"), (64, 4, 70, 2800, "bf16"))):
        pool, table, lens, cu, pre = make_shared([(prefix, _members(n, prefix, seed))], 64, 2, d, seed)
        q = torch.randn(n, 2 * g, d, generator=torch.Generator().manual_seed(seed)).to(DTYPES[dtype])
        sets.append([q.cuda(), _dev(pool), _dev(wide(table, 64, 2 * n)), _dev(lens), 0.1, _dev(cu), _dev(pre)])
        alone.append(_call(*sets[-1], 1))
        ref = kv4.attend(q[:3].double().numpy(), pool, table[:3], lens[:3], 64, 0.1)
        check_shared(alone[-1][0][:3], alone[-1][1][:, :3], ref, DTYPES[dtype])
    cfg = CONFIGS["fwd8k"]
    inp = make_inputs(cfg)
    train = [inp[k].cuda() for k in ("q", "k", "v")] + [_dev(inp["sel_idx"]), _dev(inp["cu_seqlens"])]
    want = nsa.fwd(*train, cfg.block, cfg.scale)
    torch.cuda.synchronize()
    streams, got, trained = [torch.cuda.Stream() for _ in range(5)], [], []
    for turn in range(40):
        for i, s in enumerate(sets):
            with torch.cuda.stream(streams[i]):
                got.append((i, nsa.kv4_decode_shared(*s)))
        if turn % 8 == 0:
            with torch.cuda.stream(streams[4]):
                trained.append(nsa.fwd(*train, cfg.block, cfg.scale))
    torch.cuda.synchronize()
    for i, (out, lse) in got:
        assert torch.equal(out, alone[i][0]) and torch.equal(lse, alone[i][1]), i
    for out, lse in trained:
        torch.testing.assert_close(out, want[0], rtol=2 ** -7, atol=2 ** -9)
        torch.testing.assert_close(lse, want[1], rtol=1e-5, atol=1e-5)
