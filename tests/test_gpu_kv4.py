"""The 4-bit paged cache on the GPU against the fp64 oracle: rows written and read back,
one-step decode over the pages, and both together with the plan of their slots."""
import numpy as np
import pytest
import torch

from kv4_helpers import DTYPES, check_decode, make_cache, make_selection
from oracle import kv4

pytestmark = pytest.mark.gpu


def _dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


# ---- append and read ------------------------------------------------------------------
def _rows(n, h, d, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, h, d, generator=g) * torch.exp(2 * torch.randn(n, h, 1, generator=g))
    x[..., ::31] *= 5
    x = x.to(dtype)
    if n > 8:
        x[1, 0] = 0.5                                  # a flat row: scale 0
        x[2, 0, 5] = float("inf")
        x[3, 0, 7], x[3, 0, 9] = float("-inf"), float("inf")
        x[4, 0, d - 1] = float("nan")
        x[5, 0] = 1e-6 * torch.arange(d).to(dtype)     # scales among fp16's smallest
        x[6, 0] = torch.arange(d).to(dtype) / 2        # ties between two codes
        x[7, 0] = (torch.arange(d) % 31).to(dtype) * 0.5
    return x


@pytest.mark.parametrize("n,h,d,page,dtype", [(1, 1, 64, 32, "bf16"), (33, 3, 128, 64, "fp16"),
                                              (257, 2, 64, 128, "fp16"), (130, 4, 128, 32, "bf16"),
                                              (5, 5, 128, 128, "bf16"), (43, 5, 64, 32, "bf16")])
def test_append_and_read(n, h, d, page, dtype):
    import block_sparse_attention_nsa_gb300 as nsa
    dt = DTYPES[dtype]
    k, v = _rows(n, h, d, dt, n), _rows(n, h, d, dt, n + 1)
    pages = -(-n // page) + 2
    rng = np.random.default_rng(n)
    slots = rng.permutation(pages * page)[:n].astype(np.int32)
    slots[n // 2] = -1
    before = rng.integers(0, 256, (pages, h, page * (d + d // 8)), dtype=np.uint8)
    pool = _dev(before)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    nsa.kv4_append(pool, k.cuda(), v.cuda(), _dev(slots), device_status=status)
    ref = before.copy()
    for t in range(n):
        for hh in range(h):
            for w, x in enumerate((k, v)):
                if slots[t] >= 0:
                    kv4.put_row(ref, page, d, slots[t], hh, w,
                                *kv4.quantise(x[t, hh].float().numpy()))
    got = pool.cpu().numpy()
    # NaN zeros are compared as NaN, all else bit for bit: rows of no slot stay as they were
    c0, s0, z0 = kv4.unpack(ref, page, d)
    c1, s1, z1 = kv4.unpack(got, page, d)
    np.testing.assert_array_equal(c1, c0)
    np.testing.assert_array_equal(s1, s0)
    np.testing.assert_array_equal(z1, z0)
    kr, vr = nsa.kv4_read(pool, _dev(slots), d, dtype=dt, device_status=status)
    for t in range(n):
        for w, x in enumerate((kr, vr)):
            if slots[t] < 0:
                assert (x[t] == 0).all()
                continue
            for hh in range(h):
                want = torch.from_numpy(kv4.dequantise(*kv4.get_row(ref, page, d, slots[t], hh, w)))
                # the fp32 sum rounds once before the output type does
                want, have = want.numpy(), x[t, hh].double().cpu().numpy()
                tol = np.abs(want) * (torch.finfo(dt).eps / 2 + 2.0 ** -24) + 2.0 ** -25
                np.testing.assert_array_equal(np.isnan(have), np.isnan(want))
                live = ~np.isnan(want)
                big = live & (np.abs(want) > 65504) & np.isinf(have)   # past fp16's range
                ok = live & ~big
                assert (np.abs(have - want)[ok] <= tol[ok]).all()
    assert int(status.item()) == 0


def test_append_strided_views_and_bad_slots():
    import block_sparse_attention_nsa_gb300 as nsa
    n, h, d, page = 70, 2, 128, 32
    row = _rows(n, 4 * h, d, torch.bfloat16, 3).cuda()
    k, v = row[:, 2 * h:3 * h], row[:, 3 * h:]
    slots = torch.randperm(4 * page, generator=torch.Generator().manual_seed(1))[:n].int().cuda()
    a, b = (nsa.kv4_pool(4, page, h, d) for _ in range(2))
    nsa.kv4_append(a, k, v, slots)
    nsa.kv4_append(b, k.contiguous(), v.contiguous(), slots)
    assert torch.equal(a, b) and a.any()
    # heads before tokens
    nsa.kv4_append(b.zero_(), k.transpose(0, 1).contiguous().transpose(0, 1), v, slots)
    assert torch.equal(a, b)
    # one key row for every head
    nsa.kv4_append(b.zero_(), k[:, :1].expand(n, h, d), v, slots)
    kr, _ = nsa.kv4_read(b, slots, d)
    ar, _ = nsa.kv4_read(a, slots, d)
    torch.testing.assert_close(kr[:, 1], ar[:, 0], rtol=0, atol=0, equal_nan=True)
    # slots outside the pool are skipped and reported, on both ways
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    bad = slots.clone()
    bad[0], bad[1] = 4 * page, -2
    nsa.kv4_append(b.zero_(), k, v, bad, device_status=status)
    assert int(status.item()) == nsa.DEVERR_BAD_INDEX
    ref = a.clone()
    nsa.kv4_append(ref.zero_(), k[2:], v[2:], slots[2:].contiguous())
    assert torch.equal(b, ref)
    kr, vr = nsa.kv4_read(b, bad, d, device_status=status.zero_())
    assert int(status.item()) == nsa.DEVERR_BAD_INDEX and (kr[:2] == 0).all() and (vr[:2] == 0).all()
    # no rows at all
    none = torch.empty((0, h, d), dtype=torch.bfloat16, device="cuda")
    nsa.kv4_append(b, none, none, slots[:0])
    assert torch.equal(b, ref) and nsa.kv4_read(b, slots[:0], d)[0].shape == (0, h, d)


# ---- decode ---------------------------------------------------------------------------
def _decode(lens, page, h_k, g, d, dtype, seed, topk=0, window=0, scale=None, mags=(1.0,),
            width=None):
    import block_sparse_attention_nsa_gb300 as nsa
    pool, table, _ = make_cache(lens, page, h_k, d, seed, width=width, mags=mags)
    sel = make_selection(lens, page, h_k, topk, seed + 1) if topk else None
    dt = DTYPES[dtype]
    q = torch.randn(len(lens), h_k * g, d, generator=torch.Generator().manual_seed(seed)).to(dt)
    scale = d ** -0.5 if scale is None else scale
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = nsa.kv4_decode(q.cuda(), _dev(pool), _dev(table), _dev(np.int32(lens)), scale,
                              sel_idx=None if sel is None else _dev(sel), window=window,
                              device_status=status)
    ref = kv4.attend(q.double().numpy(), pool, table, lens, page, scale, sel, window)
    check_decode(out, lse, ref, dt)
    assert int(status.item()) == 0
    return out


RAGGED = (1000, 1, 64, 0, 777, 33, 2049)


@pytest.mark.parametrize("d,page,h_k,g,dtype", [(128, 64, 2, 4, "bf16"), (128, 64, 1, 16, "fp16"),
                                                (64, 32, 3, 1, "fp16"), (128, 128, 2, 8, "bf16"),
                                                (64, 128, 1, 7, "bf16"), (128, 32, 1, 12, "fp16"),
                                                (64, 64, 2, 9, "bf16")])
@pytest.mark.parametrize("topk,window", [(16, 0), (0, 0), (0, 100), (5, 90), (32, 0), (1, 0), (0, 1)])
def test_decode_matches_oracle(d, page, h_k, g, dtype, topk, window):
    _decode(RAGGED, page, h_k, g, d, dtype, 10 * d + page + g, topk, window)
    if not topk and not window:      # a table with room for long caches: lengths from the device alone
        _decode(RAGGED, page, h_k, g, d, dtype, 10 * d + page + g, width=300)


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257, 511, 513])
def test_decode_lengths_around_tiles(n):
    _decode((n,), 64, 1, 4, 128, "bf16", n, window=2 ** 40)
    _decode((n,), 64, 1, 4, 128, "bf16", n)
    _decode((n,), 32, 2, 1, 64, "fp16", n, topk=16)
    _decode((n,), 128, 1, 3, 128, "fp16", n, window=32)
    _decode((n, 0, n), 64, 2, 4, 128, "bf16", n, width=200)


@pytest.mark.parametrize("b", [1, 5, 40, 170, 400])
def test_decode_batches_of_selections(b):
    """Batches for which a segment gets 16, 8, 4, 2 warps and one."""
    rng = np.random.default_rng(b)
    lens = tuple(int(x) for x in rng.integers(1, 700, b))
    _decode(lens, 32, 4, 1, 64, "bf16", b, topk=3)
    _decode(lens, 64, 2, 9, 64, "fp16", b, topk=12)
    _decode(lens, 32, 8, 1, 64, "fp16", b, window=20)


@pytest.mark.parametrize("b", [2, 19, 36, 50, 70, 160, 300])
def test_decode_batches_of_selections_at_128(b):
    """Eight KV heads: segments that share an SM by one, two, three, four, six and twelve, and
    clusters of one and of two CTAs an SM; a second call with an empty sequence in the middle."""
    rng = np.random.default_rng(b + 1000)
    lens = [int(x) for x in rng.integers(1, 600, b)]
    _decode(tuple(lens), 32, 8, 2, 128, "bf16", b, topk=16)
    lens[b // 2] = 0
    _decode(tuple(lens), 32, 8, 1, 128, "fp16", b, topk=4)


def test_decode_long_axis_and_many_sequences():
    _decode((20011,), 64, 2, 4, 128, "bf16", 5)
    _decode((9000, 1, 17000), 128, 1, 16, 64, "fp16", 6)
    rng = np.random.default_rng(7)
    many = tuple(int(x) for x in rng.integers(0, 300, 700))
    _decode(many, 32, 1, 2, 64, "bf16", 7)
    _decode(many, 32, 1, 2, 64, "bf16", 7, width=200)
    _decode(many[:300], 64, 2, 12, 128, "fp16", 9, width=100)
    _decode((9000, 5, 7000, 4500), 64, 2, 4, 128, "bf16", 10, window=5000)
    _decode((9000, 5, 7000, 4500), 32, 1, 1, 64, "fp16", 11, window=4200)
    _decode(tuple(int(x) for x in rng.integers(0, 40, 900)), 32, 3, 1, 64, "bf16", 8, window=7)


@pytest.mark.parametrize("d,page", [(64, 128), (128, 64)])
def test_decode_long_fp16_loses_little(d, page):
    """Over a long cache the values cancel, so that an error of one sign in every sum shows: the
    kernel may add at most half of what the output's own rounding to fp16 costs."""
    import block_sparse_attention_nsa_gb300 as nsa
    lens = (60011, 30002)
    pool, table, _ = make_cache(lens, page, 1, d, 77)
    q = torch.randn(2, 2, d, generator=torch.Generator().manual_seed(78)).half()
    out, _ = nsa.kv4_decode(q.cuda(), _dev(pool), _dev(table), _dev(np.int32(lens)), d ** -0.5)
    ref = kv4.attend(q.double().numpy(), pool, table, lens, page, d ** -0.5, None, 0)[0]
    rounding = np.linalg.norm(ref.astype(np.float16) - ref)
    assert np.linalg.norm(out.double().cpu().numpy() - ref) <= 1.5 * rounding


def test_decode_fp16_many_tiles_a_warp():
    """As above, where one warp adds up a whole sequence: 250 sequences that share their pages,
    8 KV heads, all 32 blocks selected (128 tiles of 32 keys)."""
    import block_sparse_attention_nsa_gb300 as nsa
    n, d, page, h_k, b = 4096, 64, 128, 8, 250
    pool, table, _ = make_cache((n,), page, h_k, d, 79)
    table = np.repeat(table, b, 0)
    lens = np.full(b, n, np.int32)
    sel = np.broadcast_to(np.arange(n // page, dtype=np.int32), (h_k, b, n // page)).copy()
    q = torch.randn(b, h_k, d, generator=torch.Generator().manual_seed(80)).half()
    out, _ = nsa.kv4_decode(q.cuda(), _dev(pool), _dev(table), _dev(lens), d ** -0.5,
                            sel_idx=_dev(sel))
    ref = kv4.attend(q[:3].double().numpy(), pool, table[:3], lens[:3], page, d ** -0.5,
                     sel[:, :3], 0)[0]
    rounding = np.linalg.norm(ref.astype(np.float16) - ref)
    assert np.linalg.norm(out[:3].double().cpu().numpy() - ref) <= 1.5 * rounding


def test_decode_spread_of_scores_and_magnitudes():
    # a peaked softmax, a negative scale, and tokens whose K and V differ by 2^12
    _decode(RAGGED, 64, 2, 4, 128, "bf16", 21, scale=2.0)
    _decode(RAGGED, 64, 2, 4, 128, "fp16", 22, scale=-0.5, topk=16)
    _decode(RAGGED, 64, 1, 8, 128, "fp16", 23, scale=1e-3, mags=(2.0 ** -9, 0.1, 8.0))
    _decode(RAGGED, 32, 1, 2, 64, "bf16", 24, scale=0.0, mags=(2.0 ** -8, 16.0))


def test_decode_wide_query_values():
    """Queries whose heads differ by many powers of two, zero heads among them."""
    import block_sparse_attention_nsa_gb300 as nsa
    lens, page, h_k, g, d = (300, 70), 64, 1, 6, 128
    pool, table, _ = make_cache(lens, page, h_k, d, 31)
    q = torch.randn(2, g, d, generator=torch.Generator().manual_seed(0))
    q *= torch.tensor([1.0, 1e-20, 1e4, 0.0, 1e-3, 300.0]).view(1, g, 1)
    q[0, 0, 5] = 2.0 ** -12
    q = q.to(torch.bfloat16)
    scale = 1e-4
    out, lse = nsa.kv4_decode(q.cuda(), _dev(pool), _dev(table), _dev(np.int32(lens)), scale)
    check_decode(out, lse, kv4.attend(q.double().numpy(), pool, table, lens, page, scale),
                 torch.bfloat16)


def test_decode_nan_row_stays_in_its_head():
    import block_sparse_attention_nsa_gb300 as nsa
    lens, page, h_k, g, d = (500, 200), 64, 2, 4, 128
    pool, table, _ = make_cache(lens, page, h_k, d, 32)
    q = torch.randn(2, h_k * g, d, generator=torch.Generator().manual_seed(0)).to(torch.bfloat16)
    ref = kv4.attend(q.double().numpy(), pool, table, lens, page, 0.1)
    bad = q.clone()
    bad[0, 5, 3] = float("nan")
    out, lse = nsa.kv4_decode(bad.cuda(), _dev(pool), _dev(table), _dev(np.int32(lens)), 0.1)
    assert out[0, 5].isnan().all() and lse[5, 0].isnan()
    out[0, 5], lse[5, 0] = torch.from_numpy(ref[0][0, 5]).to(out), float(ref[1][5, 0])
    check_decode(out, lse, ref, torch.bfloat16)


def test_decode_reports_bad_tables_lengths_and_selections():
    import block_sparse_attention_nsa_gb300 as nsa
    lens, page, h_k, g, d = (300, 200, 128), 64, 2, 2, 64
    pool, table, _ = make_cache(lens, page, h_k, d, 33, width=5)
    q = torch.randn(3, h_k * g, d, generator=torch.Generator().manual_seed(0)).to(torch.float16)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call(tab, lengths, sel=None):
        status.zero_()
        out, lse = nsa.kv4_decode(q.cuda(), _dev(pool), _dev(tab), _dev(np.int32(lengths)), 0.1,
                                  sel_idx=None if sel is None else _dev(sel), device_status=status)
        ref = kv4.attend(q.double().numpy(), pool, tab, lengths, page, 0.1, sel)
        check_decode(out, lse, ref, torch.float16)
        return int(status.item())

    assert call(table, lens) == 0
    for bad in (-1, pool.shape[0], 1 << 30):
        tab = table.copy()
        tab[0, 2], tab[2, 0], tab[2, 1] = bad, bad, bad    # a hole, and a sequence without keys
        assert call(tab, lens) == nsa.DEVERR_BAD_INDEX
    assert call(table, (300, -5, 128)) == nsa.DEVERR_BAD_SEQLENS
    # longer than its row: held to the table, whose last pages are not there
    assert call(table, (300, 200, 1 << 30)) == nsa.DEVERR_BAD_SEQLENS | nsa.DEVERR_BAD_INDEX
    sel = make_selection(lens, page, h_k, 4, 3)
    assert call(table, lens, sel) == 0
    for bad in (-2, 5, 1 << 30):
        sel[1, 2, 0] = bad
        assert call(table, lens, sel) == nsa.DEVERR_BAD_INDEX
    # a block that no longer is causal does not exist in a decode: the last one is the newest
    sel[:] = -1
    assert call(table, lens, sel) == 0


def test_decode_rejects():
    import block_sparse_attention_nsa_gb300 as nsa
    pool = nsa.kv4_pool(4, 64, 2, 128)
    q = torch.zeros(2, 4, 128, dtype=torch.bfloat16, device="cuda")
    table = torch.zeros(2, 2, dtype=torch.int32, device="cuda")
    lens = torch.ones(2, dtype=torch.int32, device="cuda")
    with pytest.raises(nsa.NsaError) as e:
        nsa.kv4_decode(q[:, :3].contiguous(), pool, table, lens, 0.1)      # 3 heads on 2
    assert e.value.code == 1
    with pytest.raises(nsa.NsaError) as e:
        nsa.kv4_decode(q.float(), pool, table, lens, 0.1)
    assert e.value.code == 2
    with pytest.raises(nsa.NsaError) as e:
        nsa.kv4_decode(q, pool, table, lens, float("nan"))
    assert e.value.code == 1
    with pytest.raises(nsa.NsaError) as e:
        nsa.kv4_decode(q, pool, table, lens, 0.1, window=-1)
    assert e.value.code == 1
    with pytest.raises(nsa.NsaError) as e:
        nsa.kv4_decode(q, pool, table, lens, 0.1, window=-2 ** 40)
    assert e.value.code == 1
    with pytest.raises(nsa.NsaError) as e:                                  # 33 slots
        nsa.kv4_decode(q, pool, table, lens, 0.1,
                       sel_idx=torch.zeros(2, 2, 33, dtype=torch.int32, device="cuda"))
    assert e.value.code == 2
    with pytest.raises(ValueError):
        nsa.kv4_decode(q.transpose(0, 1), pool, table, lens, 0.1)           # not contiguous
    with pytest.raises(ValueError):
        nsa.kv4_decode(q, pool, table.long(), lens, 0.1)
    with pytest.raises(ValueError):
        nsa.kv4_decode(q, pool, table, lens.cpu(), 0.1)
    with pytest.raises(ValueError):
        nsa.kv4_decode(q[..., :64].contiguous(), pool[:, :, :100].contiguous(), table, lens, 0.1)
    with pytest.raises(ValueError):
        nsa.kv4_append(pool, q, q, lens)                                    # 4 heads into 2
    with pytest.raises(nsa.NsaError) as e:                                  # 8-byte aligned rows
        odd = torch.zeros(2 * 2 * 128 + 4, dtype=torch.bfloat16, device="cuda")[4:].view(2, 2, 128)
        nsa.kv4_append(pool, odd, odd, lens)
    assert e.value.code == 1


def test_decode_other_stream_graph_and_shared_workspace():
    """On a stream of its own, two shapes captured into graphs that share a workspace and are
    replayed in turn, after their inputs have changed in place."""
    import block_sparse_attention_nsa_gb300 as nsa
    page, h_k, g, d = 64, 2, 4, 128
    side = torch.cuda.Stream()
    sets = []
    for seed, lens in ((41, (5000, 3)), (42, (900, 4000, 1))):
        pool, table, _ = make_cache(lens, page, h_k, d, seed, width=80)
        q = torch.randn(len(lens), h_k * g, d, generator=torch.Generator().manual_seed(seed))
        q = q.to(torch.bfloat16)
        sets.append(dict(pool=pool, table=table, q=q, lens=lens, dq=q.cuda(), dpool=_dev(pool),
                         dtab=_dev(table), dlens=_dev(np.int32(lens))))
    need = max(nsa.kv4_decode_workspace_size(s["pool"].shape[0], page, h_k, d, len(s["lens"]),
                                             h_k * g) for s in sets)
    ws = torch.full((max(need, 16),), 0xff, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    for s in sets:
        s["out"], s["lse"] = nsa.kv4_decode(s["dq"], s["dpool"], s["dtab"], s["dlens"], 0.1,
                                            workspace=ws, stream=side)
    side.synchronize()
    for s in sets:
        check_decode(s["out"], s["lse"], kv4.attend(s["q"].double().numpy(), s["pool"], s["table"],
                                                    s["lens"], page, 0.1), torch.bfloat16)
    graphs = []
    for s in sets:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            nsa.kv4_decode(s["dq"], s["dpool"], s["dtab"], s["dlens"], 0.1, out=s["out"],
                           lse=s["lse"], workspace=ws)
        graphs.append(graph)
    for k in range(3):
        for s, graph in zip(sets, graphs):
            s["lens"] = tuple(max(0, n - 700 * k) for n in s["lens"])
            s["dlens"].copy_(_dev(np.int32(s["lens"])))
            graph.replay()
        torch.cuda.synchronize()
        for s in sets:
            ref = kv4.attend(s["q"].double().numpy(), s["pool"], s["table"], s["lens"], page, 0.1)
            check_decode(s["out"], s["lse"], ref, torch.bfloat16)


def test_decode_is_repeatable():
    import block_sparse_attention_nsa_gb300 as nsa
    lens, page, h_k, g, d = (7000, 3000, 12), 64, 2, 8, 128
    pool, table, _ = make_cache(lens, page, h_k, d, 51)
    q = torch.randn(3, h_k * g, d, generator=torch.Generator().manual_seed(1)).half().cuda()
    args = (q, _dev(pool), _dev(table), _dev(np.int32(lens)), 0.1)
    out, lse = nsa.kv4_decode(*args)
    for _ in range(5):
        o, l = nsa.kv4_decode(*args)
        assert torch.equal(o, out) and torch.equal(l, lse)


def test_decode_nan_value_stays_in_its_group_and_sequence():
    """A stored NaN in V reaches its 64 dimensions of the sequence that attends to it; one
    behind a window reaches nothing."""
    import block_sparse_attention_nsa_gb300 as nsa
    lens, page, h_k, g, d = (500, 200), 64, 1, 3, 128
    pool, table, _ = make_cache(lens, page, h_k, d, 34)
    q = torch.randn(2, g, d, generator=torch.Generator().manual_seed(0)).to(torch.bfloat16)
    ref = kv4.attend(q.double().numpy(), pool, table, lens, page, 0.1)
    slot = table[0, 2] * page + 5                       # position 133 of sequence 0
    code, scale, zero = kv4.get_row(pool, page, d, slot, 0, 1)
    zero[1] = np.float16("nan")
    kv4.put_row(pool, page, d, slot, 0, 1, code * 0, scale, zero)
    args = (q.cuda(), _dev(pool), _dev(table), _dev(np.int32(lens)), 0.1)
    out, lse = nsa.kv4_decode(*args)
    assert out[0, :, 64:].isnan().all() and lse.isfinite().all()
    ref[0][0, :, :64] = kv4.attend(q.double().numpy(), pool, table, lens, page, 0.1)[0][0, :, :64]
    out[0, :, 64:] = torch.from_numpy(ref[0][0, :, 64:]).to(out)
    check_decode(out, lse, ref, torch.bfloat16)
    ref = kv4.attend(q.double().numpy(), pool, table, lens, page, 0.1, window=366)   # from 134 on
    out, lse = nsa.kv4_decode(*args, window=366)
    check_decode(out, lse, ref, torch.bfloat16)


def test_pool_beyond_32_bit_offsets():
    """Pages whose bytes lie past 2^32: the same rows in a small pool read and attend alike."""
    import block_sparse_attention_nsa_gb300 as nsa
    page, h_k, g, d, n = 128, 8, 2, 128, 700
    far, near = nsa.kv4_pool(33000, page, h_k, d), nsa.kv4_pool(8, page, h_k, d)
    assert far.numel() > (1 << 32)
    gen = torch.Generator().manual_seed(2)
    k, v = (torch.randn(n, h_k, d, generator=gen).half().cuda() for _ in range(2))
    q = torch.randn(1, h_k * g, d, generator=gen).half().cuda()
    lens, zero = _dev(np.int32([n])), _dev(np.int32([0]))
    got = []
    for pool, first in ((far, 32990), (near, 1)):
        table = torch.arange(first, first + 6, dtype=torch.int32, device="cuda").view(1, 6)
        slots, _ = nsa.page_slots(table, zero, lens, page, pool.shape[0], n)
        nsa.kv4_append(pool, k, v, slots)
        kr, vr = nsa.kv4_read(pool, slots, d, dtype=torch.float16)
        got.append((kr, vr) + tuple(nsa.kv4_decode(q, pool, table, lens, 0.1)))
    for a, b in zip(*got):
        assert torch.equal(a, b)
    # 4 bits keep a normal row to within half a step of about a third
    assert (got[0][0].float() - k.float()).abs().max() < 0.5


def test_steps_in_a_graph_between_streams():
    """Append and decode captured on a forked stream, behind a torch kernel and before one: each
    replay sees what the last one left."""
    import block_sparse_attention_nsa_gb300 as nsa
    page, h_k, g, d, b = 32, 2, 2, 64, 3
    pool = nsa.kv4_pool(12, page, h_k, d)
    table = torch.arange(12, dtype=torch.int32, device="cuda").view(b, 4)
    lens = torch.zeros(b, dtype=torch.int32, device="cuda")
    step = torch.ones(b, dtype=torch.int32, device="cuda")
    k, v = (torch.zeros(b, h_k, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = torch.zeros(b, h_k * g, d, dtype=torch.bfloat16, device="cuda")
    src = torch.zeros(3, b, h_k, d, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(nsa.kv4_decode_workspace_size(12, page, h_k, d, b, h_k * g),
                     dtype=torch.uint8, device="cuda")
    out, total = torch.empty_like(q), torch.zeros_like(q, dtype=torch.float32)
    lse = torch.empty(h_k * g, b, device="cuda")
    slots = torch.empty(b, dtype=torch.int32, device="cuda")
    cu = torch.empty(b + 1, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()

    def body():
        main = torch.cuda.current_stream()
        k.copy_(src[0])
        v.copy_(src[1])
        q.copy_(src[2].repeat_interleave(g, 1))
        side.wait_stream(main)
        with torch.cuda.stream(side):
            nsa.page_slots(table, lens, step, page, 12, slots, cu)
            nsa.kv4_append(pool, k, v, slots)
            lens.add_(step)
            nsa.kv4_decode(q, pool, table, lens, 0.3, out=out, lse=lse, workspace=ws)
        main.wait_stream(side)
        total.add_(out.float())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        body()
    gen = torch.Generator().manual_seed(4)
    want = torch.zeros(b, h_k * g, d, dtype=torch.float64)
    for n in range(1, 41):
        x = torch.randn(3, b, h_k, d, generator=gen).to(torch.bfloat16)
        src.copy_(x)
        graph.replay()
        qn = x[2].repeat_interleave(g, 1)
        ref = kv4.attend(qn.double().numpy(), pool.cpu().numpy(), table.cpu().numpy(), [n] * b,
                         page, 0.3)
        check_decode(out, lse, ref, torch.bfloat16)
        want += out.double().cpu()
    assert lens.tolist() == [40] * b
    torch.testing.assert_close(total.double().cpu(), want, rtol=0, atol=40 * 40 * 2.0 ** -24)


def test_calls_on_two_streams_and_between_torch_kernels():
    """Unsynchronised loops on two streams, each call behind a torch kernel that writes its
    inputs and before one that reads its outputs: the same sums as with a wait after each."""
    import block_sparse_attention_nsa_gb300 as nsa
    page, h_k, g, d = 64, 2, 4, 128
    sets = []
    for seed, lens in ((61, (4000, 5, 900)), (62, (3000,) * 5)):
        pool, table, _ = make_cache(lens, page, h_k, d, seed, width=80)
        gen = torch.Generator().manual_seed(seed)
        qs = torch.randn(12, len(lens), h_k * g, d, generator=gen).to(torch.bfloat16).cuda()
        sel = make_selection(lens, page, h_k, 8, seed)
        need = nsa.kv4_decode_workspace_size(pool.shape[0], page, h_k, d, len(lens), h_k * g)
        sets.append(dict(pool=_dev(pool), table=_dev(table), lens=_dev(np.int32(lens)), qs=qs,
                         q=torch.empty_like(qs[0]), sel=_dev(sel), stream=torch.cuda.Stream(),
                         ws=torch.empty(need, dtype=torch.uint8, device="cuda")))

    def loop(s, wait):
        total = torch.zeros(s["q"].shape, device="cuda")
        for q in s["qs"]:
            for sel in (None, s["sel"]):
                s["q"].copy_(q)
                out, _ = nsa.kv4_decode(s["q"], s["pool"], s["table"], s["lens"], 0.1, sel_idx=sel,
                                        workspace=s["ws"])
                total.add_(out.float())
                if wait:
                    torch.cuda.synchronize()
        return total
    want = [loop(s, True) for s in sets]
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for s in sets:
            with torch.cuda.stream(s["stream"]):
                got.append(loop(s, False))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


# ---- a serving loop -------------------------------------------------------------------
@pytest.mark.parametrize("page,d", [(64, 128), (32, 64)])
def test_serving_steps(page, d):
    """Prompts, then decode steps: plan, append, selected decode; the pages read back equal
    what a 16-bit cache of the same values gives through nsa.decode, and the oracle."""
    import block_sparse_attention_nsa_gb300 as nsa
    h_k, g, steps, topk = 2, 4, 3, 4
    prompts = [150, 1, 0, 333]
    b, width, pages = len(prompts), 16, 40
    gen = torch.Generator().manual_seed(9)
    pool = nsa.kv4_pool(pages, page, h_k, d)
    table = torch.full((b, width), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(pages, generator=gen).int().cuda()
    head = torch.zeros(1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(b, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    have = [0] * b
    for step in range(steps + 1):
        new = prompts if step == 0 else [1] * b
        n = sum(new)
        k, v = (torch.randn(n + 3, h_k, d, generator=gen).to(torch.bfloat16).cuda()
                for _ in range(2))
        slots, _, _, _ = nsa.page_plan(lens, torch.tensor(new, dtype=torch.int32, device="cuda"),
                                       free, head, table, page, pages, n + 3, seq_lens=lens,
                                       head_out=head, device_status=status)
        nsa.kv4_append(pool, k, v, slots, device_status=status)
        have = [x + y for x, y in zip(have, new)]
        assert lens.tolist() == have and (slots[n:] == -1).all()
        assert int(head.item()) == sum(-(-x // page) for x in have)
    q = torch.randn(b, h_k * g, d, generator=gen).to(torch.bfloat16)
    sel = make_selection(have, page, h_k, topk, 3)
    dsel = _dev(sel)
    out, lse = nsa.kv4_decode(q.cuda(), pool, table, lens, d ** -0.5, sel_idx=dsel,
                              device_status=status)
    ref = kv4.attend(q.double().numpy(), pool.cpu().numpy(), table.cpu().numpy(), have, page,
                     d ** -0.5, sel)
    check_decode(out, lse, ref, torch.bfloat16)
    # read back into a packed 16-bit cache
    total = sum(have)
    slots, cu = nsa.page_slots(table, torch.zeros_like(lens), lens, page, pages, total,
                               device_status=status)
    kr, vr = nsa.kv4_read(pool, slots, d, device_status=status)
    o16, l16 = nsa.decode(q.cuda(), kr, vr, dsel, cu, page, d ** -0.5)
    torch.testing.assert_close(o16.float(), out.float(), rtol=2e-2, atol=2e-2)
    torch.testing.assert_close(l16, lse, rtol=0, atol=2e-2)   # keys rounded to bf16
    assert int(status.item()) == 0
