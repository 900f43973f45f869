"""The decode over shared prefixes against the fp64 oracle, which knows nothing of sharing."""
import numpy as np
import pytest
import torch

from kv4_helpers import DTYPES
from oracle import kv4
from shared_helpers import check_shared, make_shared, wide

pytestmark = pytest.mark.gpu


def _dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def _run(groups, page, h_k, g, d, dtype, seed, alone=(), scale=None, width=None, mags=(1.0,), q=None,
         some=None):
    import block_sparse_attention_nsa_gb300 as nsa
    pool, table, lens, cu, prefix = make_shared(groups, page, h_k, d, seed, alone, width, mags)
    dt = DTYPES[dtype]
    if q is None:
        q = torch.randn(len(lens), h_k * g, d, generator=torch.Generator().manual_seed(seed)).to(dt)
    scale = d ** -0.5 if scale is None else scale
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    rows = np.arange(len(lens)) if some is None else np.asarray(some)
    ref = kv4.attend(q[rows].double().numpy(), pool, table[rows], lens[rows], page, scale)
    # as it is, and with a table that leaves the choice to the device
    for t in (table, wide(table, page, len(lens) * h_k)):
        out, lse = nsa.kv4_decode_shared(q.cuda(), _dev(pool), _dev(t), _dev(lens), scale, _dev(cu),
                                         _dev(prefix), device_status=status)
        assert int(status.item()) == 0
        check_shared(out[rows], lse[:, rows], ref, dt)
    return out, ref


@pytest.mark.parametrize("d,page,h_k,g,dtype", [(128, 64, 1, 4, "bf16"), (64, 32, 2, 1, "fp16")])
def test_two_of_one_prompt(d, page, h_k, g, dtype):
    _run([(64, (70, 65))], page, h_k, g, d, dtype, 1)


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 191, 193, 257, 511, 513])
def test_prefixes_around_blocks(n):
    _run([(n, (n + 1, n + 40, n))], 64, 1, 4, 128, "bf16", n)
    _run([(n, (n + 3, n))], 32, 2, 1, 64, "fp16", n)
    _run([(n, (n, n + 1, n + 130, n + 64))], 128, 1, 3, 128, "fp16", n)


@pytest.mark.parametrize("d,page,h_k,g,dtype", [(128, 64, 2, 4, "bf16"), (128, 64, 1, 16, "fp16"),
                                                (64, 32, 3, 1, "fp16"), (128, 128, 2, 8, "bf16"),
                                                (64, 128, 1, 7, "bf16"), (128, 32, 1, 12, "fp16"),
                                                (64, 64, 2, 9, "bf16")])
def test_groups_of_all_kinds(d, page, h_k, g, dtype):
    """Groups of one sequence and of none, a prefix of nothing, sequences that end inside the prefix
    or at its end, empty ones, and sequences behind the last group."""
    groups = [(300, (420, 300, 301, 999)), (200, (260,)), (77, ()), (0, (50, 60)),
              (500, (600, 130, 0, 499, 500)), (64, (64, 64))]
    _run(groups, page, h_k, g, d, dtype, 10 * d + page + g, alone=(5, 0, 333))


@pytest.mark.parametrize("n,g,dtype", [(31, 4, "bf16"), (33, 4, "bf16"), (40, 16, "fp16"), (9, 15, "fp16"),
                                       (128, 1, "bf16"), (129, 1, "fp16"), (300, 1, "bf16")])
def test_rows_around_tiles(n, g, dtype):
    rng = np.random.default_rng(n)
    own = rng.integers(0, 50, n)
    some = sorted(set([0, 1, n // 2, n - 2, n - 1]) | set(rng.integers(0, n, 6).tolist()))
    _run([(200, tuple(200 + own))], 64, 2, g, 64, dtype, n, some=some)
    _run([(130, tuple(130 + own))], 32, 1, g, 128, dtype, n + 1, some=some)


def test_long_prefixes():
    """Runs that cross tiles, heads and groups; partial rows of many CTAs to join."""
    own = tuple(20011 + 3 * i for i in range(70))
    _run([(20011, own)], 64, 3, 4, 128, "bf16", 3, some=(0, 1, 31, 32, 69))
    _run([(9000, tuple(9000 + i for i in range(33))), (4001, (4100, 4001, 4050))], 128, 2, 8, 64, "fp16", 4,
         some=(0, 15, 16, 32, 33, 34, 35))
    many = [(int(p), tuple(int(p) + np.arange(k))) for p, k in
            zip(np.random.default_rng(5).integers(1, 900, 60), [2, 3, 5, 1, 9, 2] * 10)]
    _run(many, 32, 2, 2, 64, "bf16", 5, width=200)


@pytest.mark.parametrize("d,page", [(64, 128), (128, 64)])
def test_long_fp16_loses_little(d, page):
    """Weights and values rounded to fp16 add two errors of the output's own size, at most half of
    it together."""
    lens = (30011, 30030, 30500)
    out, ref = _run([(30011, lens)], page, 1, 2, d, "fp16", 77)
    rounding = np.linalg.norm(ref[0].astype(np.float16) - ref[0])
    assert np.linalg.norm(out.double().cpu().numpy() - ref[0]) <= 1.5 * rounding


def test_spread_of_scores_and_magnitudes():
    groups = [(500, (520, 600, 501)), (64, (90, 64))]
    _run(groups, 64, 2, 4, 128, "bf16", 21, scale=2.0)
    _run(groups, 64, 2, 4, 128, "fp16", 22, scale=-0.5)
    _run(groups, 64, 1, 8, 128, "fp16", 23, scale=1e-3, mags=(2.0 ** -9, 0.1, 8.0))
    _run(groups, 32, 1, 2, 64, "bf16", 24, scale=0.0, mags=(2.0 ** -8, 16.0))
    q = torch.randn(5, 6, 128, generator=torch.Generator().manual_seed(0))
    q *= torch.tensor([1.0, 1e-20, 1e4, 0.0, 1e-3, 300.0]).view(1, 6, 1)
    _run(groups, 64, 1, 6, 128, "bf16", 25, scale=1e-4, q=q.to(torch.bfloat16))


def test_rising_scores():
    """Keys that grow along the prefix: the reference is raised again and again."""
    import block_sparse_attention_nsa_gb300 as nsa
    page, d, n = 64, 128, 3000
    rng = np.random.default_rng(1)
    u = rng.standard_normal(d).astype(np.float32)
    pool, table, lens, cu, prefix = make_shared([(n, (n + 9, n, n + 70))], page, 1, d, 2)
    code, scale, zero = kv4.unpack(pool, page, d)
    for t in range(n):
        pg, at = table[0, t // page], t % page
        c, s, z = kv4.quantise(u * (t / n * 8) + 0.1 * rng.standard_normal(d).astype(np.float32))
        code[pg, 0, 0, at], scale[pg, 0, 0, at], zero[pg, 0, 0, at] = c, s, z
    pool2 = kv4.pack(code, scale, zero)
    table[1:, :n // page] = table[0, :n // page]
    if n % page:
        for b in (1, 2):
            a, z_ = table[0, n // page], table[b, n // page]
            for arr in (code, scale, zero):
                arr[z_, :, :, :n % page] = arr[a, :, :, :n % page]
        pool2 = kv4.pack(code, scale, zero)
    table = wide(table, page, 3)
    for dtype, size in ((torch.bfloat16, 0.3), (torch.float16, 3.0)):
        q = (torch.from_numpy(u)[None, None] * size + torch.randn(3, 2, d,
             generator=torch.Generator().manual_seed(3))).to(dtype)
        out, lse = nsa.kv4_decode_shared(q.cuda(), _dev(pool2), _dev(table), _dev(lens), d ** -0.5,
                                         _dev(cu), _dev(prefix))
        check_shared(out, lse, kv4.attend(q.double().numpy(), pool2, table, lens, page, d ** -0.5), dtype)


@pytest.mark.parametrize("size,scale", [(2.0 ** 100, 2.0 ** -101), (2.0 ** -90, 2.0 ** 90), (1.0, 2.0 ** 40),
                                        (2.0 ** 114, 1.0)])
def test_largest_queries_and_scales(size, scale):
    """Factors past fp32's comfort; weights are those of the largest score alone where scores are
    huge."""
    import block_sparse_attention_nsa_gb300 as nsa
    pool, table, lens, cu, prefix = make_shared([(300, (320, 300, 400))], 64, 1, 128, 31)
    table = wide(table, 64, 3)
    q = (torch.randn(3, 2, 128, generator=torch.Generator().manual_seed(1)) * size).to(torch.bfloat16)
    got = nsa.kv4_decode_shared(q.cuda(), _dev(pool), _dev(table), _dev(lens), scale, _dev(cu), _dev(prefix))
    ref = kv4.attend(q.double().numpy(), pool, table, lens, 64, scale)
    assert got[0].isfinite().all()
    if np.abs(ref[1]).max() < 1e30:
        check_shared(*got, ref, torch.bfloat16)
    else:
        tol = 2.0 ** -8 * np.abs(ref[0]) + 2.0 ** -9 * ref[3] + 1e-6
        assert (np.abs(got[0].double().cpu().numpy() - ref[0]) <= tol).all()


def test_bad_pages_and_nan_rows():
    import block_sparse_attention_nsa_gb300 as nsa
    page, h_k, g, d = 32, 2, 4, 128
    pool, table, lens, cu, prefix = make_shared([(300, (320, 300, 400)), (64, (64, 90))], page, h_k, d, 41)
    table = wide(table, page, 5 * h_k)
    q = torch.randn(5, h_k * g, d, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    # pages of the prefix that are none: their keys are left out, for all of the group
    t = table.copy()
    t[:3, 2], t[:3, 5], t[3:, 0] = -1, pool.shape[0], -9
    out, lse = nsa.kv4_decode_shared(q.cuda(), _dev(pool), _dev(t), _dev(lens), 0.1, _dev(cu), _dev(prefix),
                                     device_status=status)
    assert int(status.item()) == nsa.DEVERR_BAD_INDEX
    check_shared(out, lse, kv4.attend(q.double().numpy(), pool, t, lens, page, 0.1), torch.bfloat16)
    # all of a prefix
    t[:3, :9] = -1
    out, lse = nsa.kv4_decode_shared(q.cuda(), _dev(pool), _dev(t), _dev(lens), 0.1, _dev(cu), _dev(prefix))
    check_shared(out, lse, kv4.attend(q.double().numpy(), pool, t, lens, page, 0.1), torch.bfloat16)
    # a NaN query stays in its row
    ref = kv4.attend(q.double().numpy(), pool, table, lens, page, 0.1)
    bad = q.clone()
    bad[1, 5, 3] = float("nan")
    out, lse = nsa.kv4_decode_shared(bad.cuda(), _dev(pool), _dev(table), _dev(lens), 0.1, _dev(cu),
                                     _dev(prefix))
    assert out[1, 5].isnan().all() and lse[5, 1].isnan()
    out[1, 5], lse[5, 1] = torch.from_numpy(ref[0][1, 5]).to(out), float(ref[1][5, 1])
    check_shared(out, lse, ref, torch.bfloat16)


def test_malformed_groups():
    import block_sparse_attention_nsa_gb300 as nsa
    page, d = 32, 64
    pool, table, lens, cu, prefix = make_shared([(100, (120, 100, 130)), (64, (64, 90))], page, 1, d, 51)
    table = wide(table, page, 5)
    q = torch.randn(5, 2, d, generator=torch.Generator().manual_seed(1)).half()
    ref = kv4.attend(q.double().numpy(), pool, table, lens, page, 0.1)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for c, p in (((0, 3, 6), prefix), ((1, 3, 5), prefix), ((0, 3, 2), prefix), ((0, -1, 5), prefix),
                 (cu, (-1, 64)), (cu, (100, 10 ** 7)), (cu, (100, table.shape[1] * page + 1))):
        out, lse = nsa.kv4_decode_shared(q.cuda(), _dev(pool), _dev(table), _dev(lens), 0.1,
                                         _dev(np.int32(c)), _dev(np.int32(p)), device_status=status.zero_())
        assert int(status.item()) == nsa.DEVERR_BAD_SEQLENS, (c, p)
        check_shared(out, lse, ref, torch.float16)
    n = lens.copy()
    n[1], n[4] = -3, 10 ** 7
    out, lse = nsa.kv4_decode_shared(q.cuda(), _dev(pool), _dev(table), _dev(n), 0.1, _dev(cu), _dev(prefix),
                                     device_status=status.zero_())
    assert int(status.item()) & nsa.DEVERR_BAD_SEQLENS
    assert (out[1] == 0).all() and lse[:, 1].isneginf().all()


def test_streams_graphs_and_dirty_workspaces():
    import block_sparse_attention_nsa_gb300 as nsa
    page, h_k, g, d = 64, 2, 4, 128
    sets = []
    for seed in range(3):
        pool, table, lens, cu, prefix = make_shared([(700, (720, 700, 900, 701)), (64, (64, 90))], page, h_k,
                                                    d, 61 + seed, width=40)
        table = wide(table, page, 6 * h_k)
        q = torch.randn(6, h_k * g, d, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)
        sets.append([x.cuda() if torch.is_tensor(x) else _dev(x) for x in (q, pool, table, lens, cu, prefix)])
    def call(s, **kw):
        q, pool, table, lens, cu, prefix = s
        return nsa.kv4_decode_shared(q, pool, table, lens, 0.1, cu, prefix, **kw)
    want = [call(s) for s in sets]
    torch.cuda.synchronize()
    need = nsa.kv4_decode_shared_workspace_size(sets[0][1].shape[0], page, h_k, d, 6, h_k * g, 2)
    dirty = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    for s, w in zip(sets, want):
        got = call(s, workspace=dirty)
        assert torch.equal(got[0], w[0]) and torch.equal(got[1], w[1])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [call(s, stream=st) for s, st in zip(sets, streams)]
    torch.cuda.synchronize()
    assert all(torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) for a, b in zip(got, want))
    inputs = [x.clone() for x in sets[0]]
    out, lse = torch.empty_like(want[0][0]), torch.empty_like(want[0][1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(inputs, out=out, lse=lse, workspace=dirty)
    for i in (1, 2, 0, 1):
        for a, b in zip(inputs, sets[i]):
            if a.shape == b.shape:
                a.copy_(b)
        graph.replay()
        again = call([a if a.shape == b.shape else b for a, b in zip(inputs, sets[i])])
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


def test_refusals_of_python():
    import block_sparse_attention_nsa_gb300 as nsa
    pool, table, lens, cu, prefix = [_dev(x) for x in make_shared([(64, (70, 65))], 64, 1, 128, 1)]
    q = torch.zeros(2, 4, 128, dtype=torch.bfloat16, device="cuda")
    args = (pool, table, lens, 0.1)
    with pytest.raises(ValueError):
        nsa.kv4_decode_shared(q, *args, cu[:-1], prefix)
    with pytest.raises(ValueError):
        nsa.kv4_decode_shared(q, *args, cu, prefix.long())
    with pytest.raises(nsa.NsaError) as e:
        nsa.kv4_decode_shared(q, *args, cu, prefix, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert e.value.code == 3
    with pytest.raises(nsa.NsaError):
        nsa.kv4_decode_shared(q, *args, cu[:1], prefix[:0])
    with pytest.raises(nsa.NsaError):
        nsa.kv4_decode_shared(torch.zeros(2, 17, 128, dtype=torch.bfloat16, device="cuda"), *args, cu, prefix)


# ---- groups that are large enough to be shared whatever their prefix -----------------------
def _members(n, prefix, seed, most=40):
    """n sequences behind a prefix, some of nothing but it."""
    own = np.random.default_rng(seed).integers(0, most, n)
    own[::7] = 0
    return tuple(int(prefix + x) for x in own)


@pytest.mark.parametrize("prefix", [1, 2, 31, 32, 33, 63, 64, 65, 95, 127, 128, 129, 191, 193, 257, 511, 513])
def test_shared_prefixes_around_blocks(prefix):
    some = (0, 1, 7, 30, 59, 69)
    _run([(prefix, _members(70, prefix, 1))], 64, 1, 1, 128, "bf16", prefix, some=some)
    _run([(prefix, _members(70, prefix, 2))], 32, 2, 1, 64, "fp16", prefix, some=some)
    _run([(prefix + 32, _members(70, prefix + 32, 3))], 128, 1, 3, 128, "fp16", prefix, some=some)


@pytest.mark.parametrize("d,page,h_k,g,dtype", [(128, 64, 3, 1, "bf16"), (64, 32, 2, 2, "fp16"),
                                                (128, 128, 1, 16, "fp16"), (64, 64, 2, 9, "bf16"),
                                                (128, 32, 2, 5, "bf16")])
def test_shared_and_unshared_groups_together(d, page, h_k, g, dtype):
    """Large groups between small ones, members that end inside the prefix, empty ones, tiles that
    are partly full, sequences behind the last group."""
    a, b = list(_members(75, 300, 4)), list(_members(130, 129, 5))
    a[3], a[4], b[0], b[129] = 299, 0, 129, 64
    groups = [(40, (50, 41)), (300, tuple(a)), (77, ()), (129, tuple(b)), (600, (700,))]
    _run(groups, page, h_k, g, d, dtype, 7 * d + g, alone=(5, 0, 333),
         some=(0, 1, 2, 3, 5, 6, 40, 76, 77, 78, 140, 205, 206, 207, 208, 209, 210))


def test_shared_more_groups_than_a_cta_plans():
    groups = [(int(p), _members(int(n), int(p), i, 5)) for i, (p, n) in enumerate(zip(
        np.random.default_rng(1).integers(1, 60, 300), np.random.default_rng(2).integers(0, 4, 300)))]
    groups[100], groups[299] = (200, _members(90, 200, 7)), (70, _members(100, 70, 8))
    n = sum(len(g[1]) for g in groups)
    _run(groups, 32, 1, 1, 64, "bf16", 12, alone=(9, 40), some=tuple(range(0, n + 2, 41)) + (n, n + 1))


def test_shared_many_groups():
    groups = [(int(p), _members(60, int(p), i, 9)) for i, p in
              enumerate(np.random.default_rng(1).integers(1, 200, 25))]
    _run(groups, 32, 2, 1, 64, "bf16", 11, some=tuple(range(0, 1500, 53)))


def test_shared_spread_of_scores_and_largest_queries():
    groups = [(200, _members(60, 200, 1))]
    some = (0, 7, 33, 59)
    _run(groups, 64, 2, 1, 128, "bf16", 21, scale=2.0, some=some)
    _run(groups, 64, 1, 2, 128, "fp16", 22, scale=-0.5, some=some)
    _run(groups, 64, 1, 1, 128, "fp16", 23, scale=1e-3, mags=(2.0 ** -9, 0.1, 8.0), some=some)
    _run(groups, 32, 1, 2, 64, "bf16", 24, scale=0.0, mags=(2.0 ** -8, 16.0), some=some)
    q = torch.randn(60, 6, 128, generator=torch.Generator().manual_seed(0))
    q *= torch.tensor([1.0, 1e-20, 1e4, 0.0, 1e-3, 300.0]).view(1, 6, 1)
    _run(groups, 64, 1, 6, 128, "bf16", 25, scale=1e-4, q=q.to(torch.bfloat16), some=some)
    for size, scale in ((2.0 ** 100, 2.0 ** -101), (2.0 ** -90, 2.0 ** 90)):
        q = torch.randn(60, 1, 128, generator=torch.Generator().manual_seed(1)) * size
        _run(groups, 64, 1, 1, 128, "bf16", 26, scale=scale, q=q.to(torch.bfloat16), some=some)


@pytest.mark.parametrize("size,scale", [(1.0, 2.0 ** 25), (1.0, 2.0 ** 40), (2.0 ** 114, 1.0)])
def test_shared_huge_scores(size, scale):
    """Scores whose neighbours in fp32 are further apart than an exponential tells: the largest
    takes it all, unless two are that close."""
    import block_sparse_attention_nsa_gb300 as nsa
    pool, table, lens, cu, prefix = make_shared([(300, _members(60, 300, 1))], 64, 1, 128, 31)
    table = wide(table, 64, 60)
    q = (torch.randn(60, 1, 128, generator=torch.Generator().manual_seed(1)) * size).to(torch.bfloat16)
    out, _ = nsa.kv4_decode_shared(q.cuda(), _dev(pool), _dev(table), _dev(lens), scale, _dev(cu), _dev(prefix))
    ref = kv4.attend(q.double().numpy(), pool, table, lens, 64, scale)
    assert out.isfinite().all()
    tol = 2.0 ** -8 * np.abs(ref[0]) + 2.0 ** -9 * ref[3] + 1e-6
    assert (np.abs(out.double().cpu().numpy() - ref[0]) <= tol).all()


def test_shared_rising_scores():
    """Keys that grow along the prefix: the reference is raised again and again, in both halves."""
    import block_sparse_attention_nsa_gb300 as nsa
    page, d, n = 64, 128, 1984
    rng = np.random.default_rng(1)
    u = rng.standard_normal(d).astype(np.float32)
    pool, table, lens, cu, prefix = make_shared([(n, _members(60, n, 2))], page, 1, d, 2)
    table = wide(table, page, 60)
    code, scale, zero = kv4.unpack(pool, page, d)
    for t in range(n):
        pg, at = table[0, t // page], t % page
        c, s, z = kv4.quantise(u * (t / n * 8) + 0.1 * rng.standard_normal(d).astype(np.float32))
        code[pg, 0, 0, at], scale[pg, 0, 0, at], zero[pg, 0, 0, at] = c, s, z
    pool = kv4.pack(code, scale, zero)
    for dtype, size in ((torch.bfloat16, 0.3), (torch.float16, 3.0)):
        q = (torch.from_numpy(u)[None, None] * size + torch.randn(60, 1, d,
             generator=torch.Generator().manual_seed(3))).to(dtype)
        out, lse = nsa.kv4_decode_shared(q.cuda(), _dev(pool), _dev(table), _dev(lens), d ** -0.5,
                                         _dev(cu), _dev(prefix))
        check_shared(out, lse, kv4.attend(q.double().numpy(), pool, table, lens, page, d ** -0.5), dtype)


def test_shared_bad_pages_and_nan_rows():
    import block_sparse_attention_nsa_gb300 as nsa
    page, h_k, g, d = 32, 1, 2, 128
    pool, table, lens, cu, prefix = make_shared([(300, _members(60, 300, 1)), (64, _members(60, 64, 2))], page,
                                                h_k, d, 41)
    table = wide(table, page, 120)
    q = torch.randn(120, g, d, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    def call(q, t):
        return nsa.kv4_decode_shared(q.cuda(), _dev(pool), _dev(t), _dev(lens), 0.1, _dev(cu), _dev(prefix),
                                     device_status=status.zero_())
    t = table.copy()
    t[:60, 2], t[:60, 5], t[60:, 0] = -1, pool.shape[0], -9
    out, lse = call(q, t)
    assert int(status.item()) == nsa.DEVERR_BAD_INDEX
    check_shared(out, lse, kv4.attend(q.double().numpy(), pool, t, lens, page, 0.1), torch.bfloat16)
    t[:60, :9] = -1
    out, lse = call(q, t)
    check_shared(out, lse, kv4.attend(q.double().numpy(), pool, t, lens, page, 0.1), torch.bfloat16)
    ref = kv4.attend(q.double().numpy(), pool, table, lens, page, 0.1)
    bad = q.clone()
    bad[17, 1, 3], bad[18, 0, 5] = float("nan"), float("inf")
    out, lse = call(bad, table)
    for b, j in ((17, 1), (18, 0)):
        assert out[b, j].isnan().all() and lse[j, b].isnan()
        out[b, j], lse[j, b] = torch.from_numpy(ref[0][b, j]).to(out), float(ref[1][j, b])
    check_shared(out, lse, ref, torch.bfloat16)
    # a NaN in a cached group of the prefix reaches all of its sequences and nothing else
    code, scale, zero = kv4.unpack(pool, page, d)
    zero[table[0, 3], 0, 1, 7, 0] = np.float16("nan")
    out, lse = nsa.kv4_decode_shared(q.cuda(), _dev(kv4.pack(code, scale, zero)), _dev(table), _dev(lens), 0.1,
                                     _dev(cu), _dev(prefix))
    assert out[:60, :, :64].isnan().all() and out[:60, :, 64:].isfinite().all() and out[60:].isfinite().all()


def test_shared_largest_values():
    """Keys and values at fp16's ends, whose scales are the largest there are."""
    import block_sparse_attention_nsa_gb300 as nsa
    page, d, n = 32, 64, 100
    pool, table, lens, cu, prefix = make_shared([(n, _members(60, n, 2))], page, 1, d, 2)
    table = wide(table, page, 60)
    code, scale, zero = kv4.unpack(pool, page, d)
    rng = np.random.default_rng(3)
    for t in range(0, n - 10, 3):
        for w in (0, 1):
            x = rng.choice([-65504.0, 65504.0, 100.0, -3e4], d).astype(np.float32)
            x[:2] = -65504, 65504
            pg, at = table[0, t // page], t % page
            code[pg, 0, w, at], scale[pg, 0, w, at], zero[pg, 0, w, at] = kv4.quantise(x)
    pool = kv4.pack(code, scale, zero)
    q = (torch.randn(60, 1, d, generator=torch.Generator().manual_seed(1)) * 1e-5).half()
    out, lse = nsa.kv4_decode_shared(q.cuda(), _dev(pool), _dev(table), _dev(lens), 1.0, _dev(cu), _dev(prefix))
    r = kv4.attend(q.double().numpy(), pool, table, lens, page, 1.0)
    fits = np.abs(r[0]) < 65000
    got = out.double().cpu().numpy()
    # values past 65504 (by up to 32) are held to it: half a step of fp16
    tol = 2.0 ** -10 * np.abs(r[0]) + 2.0 ** -9 * r[3] + 2.0 ** -16 * r[2][..., None] * r[3]
    assert (np.abs(got - r[0])[fits] <= tol[fits]).all() and np.isfinite(lse.cpu().numpy()).all()


def test_shared_graph_and_dirty_workspace():
    import block_sparse_attention_nsa_gb300 as nsa
    page, h_k, g, d = 64, 2, 2, 128
    sets = []
    for seed in range(3):
        pool, table, lens, cu, prefix = make_shared(
            [(700, _members(60, 700, 9)), (130, _members(40 + 20 * (seed == 1), 130, 9)),
             (64, _members(20 - 20 * (seed == 1), 64, 9))], page, h_k, d, 61 + seed, width=20)
        table = wide(table, page, 120 * h_k)
        q = torch.randn(120, h_k * g, d, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)
        sets.append([x.cuda() if torch.is_tensor(x) else _dev(x) for x in (q, pool, table, lens, cu, prefix)])
    pages = max(s[1].shape[0] for s in sets)
    for s in sets:
        s[1] = torch.cat([s[1], s[1][:1].expand(pages - s[1].shape[0], -1, -1)]).contiguous()
    def call(s, **kw):
        q, pool, table, lens, cu, prefix = s
        return nsa.kv4_decode_shared(q, pool, table, lens, 0.1, cu, prefix, **kw)
    want = [call(s) for s in sets]
    dirty = torch.full((nsa.kv4_decode_shared_workspace_size(pages, page, h_k, d, 120, h_k * g, 3),), 255,
                       dtype=torch.uint8, device="cuda")
    for s, w in zip(sets, want):
        got = call(s, workspace=dirty)
        assert torch.equal(got[0], w[0]) and torch.equal(got[1], w[1])
    inputs = [x.clone() for x in sets[0]]
    out, lse = torch.empty_like(want[0][0]), torch.empty_like(want[0][1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(inputs, out=out, lse=lse, workspace=dirty)
    for i in (1, 2, 0, 1):
        for a, b in zip(inputs, sets[i]):
            a.copy_(b)
        dirty.fill_(254 - i)
        graph.replay()
        assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,prefix", [(129, 700), (200, 40), (256, 64), (257, 65), (300, 1), (385, 129), (520, 300)])
def test_shared_more_rows_than_a_tile(rows, prefix, dtype):
    """Tiles of 256 rows, their second half full, partly full or empty; prefixes that leave the second
    half of a block's keys empty."""
    n = -(-rows // 4)
    rng = np.random.default_rng(rows)
    own = prefix + rng.integers(0, 90, n)
    some = sorted(set([0, 1, 31, 32, n - 2, n - 1]) | set(rng.integers(0, n, 5).tolist()))
    _run([(prefix, tuple(own))], 64, 2, 4, 128, dtype, rows, some=some)
    # 129 or 131 rows and the like: a group size that does not divide a tile
    g = 3 if rows % 2 else 5
    n = -(-rows // g)
    _run([(prefix, tuple(prefix + rng.integers(0, 90, n))), (70, (90, 75))], 32, 1, g, 128, dtype, rows + 1,
         some=sorted({0, 42 % n, n - 1, n, n + 1}))


def test_shared_tiles_of_two_ctas_cross_runs():
    """Tiles of 256 rows whose blocks many CTAs share, with scores that rise along the prefix in some."""
    own = tuple(16000 + i for i in range(75))
    _run([(16000, own)], 64, 3, 4, 128, "bf16", 41, some=(0, 1, 31, 32, 63, 64, 74), mags=(0.5, 1.0, 4.0))
    _run([(9000, own[:70]), (3000, own[:40])], 32, 2, 5, 128, "fp16", 42, some=(0, 25, 26, 51, 69, 70, 109))


@pytest.mark.parametrize("groups", [2, 300])
@pytest.mark.parametrize("d,page,h_k,g,dtype", [(128, 64, 2, 4, "bf16"), (128, 32, 1, 1, "fp16"), (64, 32, 2, 2, "bf16")])
def test_shared_first_sequences_that_ended(d, page, h_k, g, dtype, groups):
    """The rows of a group's first sequences name nothing of the prefix, or only its beginning (their
    requests ended, or are shorter): it is read from a later one's; of a group that has ended all are empty."""
    import block_sparse_attention_nsa_gb300 as nsa
    parts = [(200, _members(70, 200, 1)), (129, _members(80, 129, 2))] + [(20, (21, 20))] * (groups - 2)
    pool, table, lens, cu, prefix = make_shared(parts, page, h_k, d, 71)
    table = wide(table, page, len(lens) * h_k)
    q = torch.randn(len(lens), h_k * g, d, generator=torch.Generator().manual_seed(1)).to(DTYPES[dtype])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def check(some):
        out, lse = nsa.kv4_decode_shared(q.cuda(), _dev(pool), _dev(table), _dev(lens), 0.1, _dev(cu), _dev(prefix),
                                         device_status=status)
        ref = kv4.attend(q[some].double().numpy(), pool, table[some], lens[some], page, 0.1)
        check_shared(out[some], lse[:, some], ref, DTYPES[dtype])
        assert int(status.item()) == 0
    some = [0, 1, 2, 3, 33, 34, 35, 69, 70, 71, 72, 149]
    lens[0], table[0] = 0, -1                               # as page_free leaves a row
    lens[1], table[1, 1:] = 10, -1
    check(some)
    lens[2:34], table[2:34] = 0, -1                         # more than a warp looks at in one step
    lens[70], table[70] = 0, -1
    check(some)
    lens[35:70], table[35:70] = 0, -1                       # one that has it: the 35th
    check(some)
    lens[34], table[34] = 0, -1                             # none
    check(some)


@pytest.mark.parametrize("g", [1, 4])
def test_shared_pages_past_32_bit_offsets(g):
    """Pages behind the first 4 GB of a pool, of the prefix and behind it."""
    import block_sparse_attention_nsa_gb300 as nsa
    page, h_k, d = 64, 2, 128
    pool, table, lens, cu, prefix = make_shared([(200, _members(70, 200, 1))], page, h_k, d, 81)
    at = 2 ** 32 // (pool.size // pool.shape[0]) + 2
    far = torch.zeros(at + pool.shape[0], *pool.shape[1:], dtype=torch.uint8, device="cuda")
    far[at:] = _dev(pool)
    q = torch.randn(70, h_k * g, d, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    t = np.where(table >= 0, table + at, -1).astype(np.int32)
    out, lse = nsa.kv4_decode_shared(q.cuda(), far, _dev(wide(t, page, 70 * h_k)), _dev(lens), 0.1, _dev(cu), _dev(prefix))
    check_shared(out, lse, kv4.attend(q.double().numpy(), pool, table, lens, page, 0.1), torch.bfloat16)
