"""Paged decode at the ends of its number ranges: queries, scales and scores as large as the types
hold, where one key takes all of a row's weight."""
import numpy as np
import pytest
import torch

from kv4_helpers import DTYPES
from oracle import kv4

pytestmark = pytest.mark.gpu


def _dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def _caches(lens, page, h_k, d, seed, width=None, k_mag=1.0, k_shift=0.0):
    """A pool with these sequences' rows and its table; K times k_mag, plus k_shift."""
    import block_sparse_attention_nsa_gb300 as nsa
    per = [-(-n // page) for n in lens]
    pages = sum(per) + 1
    table = np.full((len(lens), width or max(per)), -1, np.int32)
    table[:, :max(per)][np.arange(max(per)) < np.array(per)[:, None]] = np.arange(sum(per))
    gen = torch.Generator().manual_seed(seed)
    k, v = (torch.randn(sum(lens), h_k, d, generator=gen) for _ in range(2))
    pool = nsa.kv4_pool(pages, page, h_k, d)
    slots, _ = nsa.page_slots(_dev(table), _dev(np.zeros(len(lens), np.int32)),
                              _dev(np.int32(lens)), page, pages, sum(lens))
    nsa.kv4_append(pool, (k * k_mag + k_shift).clamp(-6e4, 6e4).half().cuda(), v.half().cuda(), slots)
    return pool, table


def _check_one_hot(q, pool, table, lens, page, scale, **kw):
    """out is one key's row, rounded once, and lse its score, where the oracle's weights leave it
    all but 2^-40 with room for the scores' errors: d 2^-24 of a score's largest sum of
    magnitudes, as everywhere, and 2^-22 for the products with scale and log2 e and back."""
    import block_sparse_attention_nsa_gb300 as nsa
    d, dt = q.shape[-1], q.dtype
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = nsa.kv4_decode(q.cuda(), pool, _dev(table), _dev(np.int32(lens)), scale,
                              device_status=status, **kw)
    ref, r_lse, big, pv, ps = kv4.attend(q.double().numpy(), pool.cpu().numpy(), table, lens, page,
                                         scale)
    room = 2.0 * (d * 2.0 ** -24 + 2.0 ** -22) * big
    got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    code, st, ze = kv4.unpack(pool.cpu().numpy(), page, d)
    g = q.shape[1] // pool.shape[1]
    clear = 0
    for b, n in enumerate(lens):
        at = np.arange(n)
        pg = table[b, at // page]
        for hq in range(q.shape[1]):
            h = hq // g
            rows = [kv4.dequantise(code[pg, h, w, at % page], st[pg, h, w, at % page],
                                   ze[pg, h, w, at % page]) for w in (0, 1)]
            s = rows[0] @ q[b, hq].double().numpy() * scale
            tol = room[b, hq] + 2.0 ** -22 * abs(r_lse[hq, b]) + 2.0 ** -19
            assert abs(gl[hq, b] - r_lse[hq, b]) <= tol, (b, hq, gl[hq, b], r_lse[hq, b])
            top = np.sort(s)[::-1]
            if n > 1 and top[0] - top[1] < 28 + 2 * room[b, hq]:
                continue
            clear += 1
            want = rows[1][s.argmax()]
            half = torch.finfo(dt).eps / 2
            # 2^-11 of eight steps: weights of bf16 outputs in fp16; 2^-18: the fp32 sums
            slack = (2.0 ** -11 + 2.0 ** -18) * ps[b, hq] + 2.0 ** -18 * pv[b, hq]
            assert (np.abs(got[b, hq] - want) <= half * np.abs(want) + slack + 2.0 ** -24).all(), (b, hq)
    assert clear >= q.shape[0] * q.shape[1] // 2 and int(status.item()) == 0


@pytest.mark.parametrize("exponent", [100, 118, 120, 121, 122, 123, 125])
@pytest.mark.parametrize("d,shift", [(128, 0.0), (64, 0.0), (128, 3.0)])
def test_queries_up_to_the_largest(exponent, d, shift):
    """bf16 queries of magnitudes up to 2^127, whose scores fp32 holds; with K shifted to positive
    values every score of the second half's heads is negative."""
    lens, page, h_k, g = (300, 1, 70), 64, 2, 4
    pool, table = _caches(lens, page, h_k, d, 3, k_mag=0.05, k_shift=0.05 * shift)
    q = torch.randn(3, h_k * g, d, generator=torch.Generator().manual_seed(4))
    if shift:
        q = q.abs()
        q[:, g:] *= -1
    q = (q.clamp(-3.5, 3.5) * 2.0 ** exponent).to(torch.bfloat16)
    assert q.isfinite().all()
    for width in (None, 2500):        # segments, and runs that leave parts to a merge
        t = table if width is None else np.pad(table, ((0, 0), (0, width - table.shape[1])),
                                               constant_values=-1)
        _check_one_hot(q, pool, t, lens, page, (0.25 if shift else -0.25))


@pytest.mark.parametrize("dtype,scale", [("fp16", 1e32), ("fp16", -3e36), ("fp16", 3.3e38),
                                         ("bf16", 1e30), ("bf16", 2.5e38)])
def test_scales_up_to_the_largest(dtype, scale):
    lens, page, h_k, g, d = (300, 70), 32, 1, 4, 64
    pool, table = _caches(lens, page, h_k, d, 5)
    q = torch.randn(2, g, d, generator=torch.Generator().manual_seed(6)) * min(1.0, 1e36 / abs(scale))
    _check_one_hot(q.to(DTYPES[dtype]), pool, table, lens, page, scale)


@pytest.mark.parametrize("mag", [30.0, 1e3, 2e4])
@pytest.mark.parametrize("d,dtype", [(128, "bf16"), (64, "fp16")])
def test_scores_of_any_size(mag, d, dtype):
    """Scores up to 1e10: each is rounded as fp32 rounds it, and differences from the largest are
    taken from what was rounded, so that no weight exceeds one."""
    lens, page, h_k, g = (500, 33), 64, 2, 4
    pool, table = _caches(lens, page, h_k, d, 7, k_mag=mag)
    q = torch.randn(2, h_k * g, d, generator=torch.Generator().manual_seed(8)) * mag
    q = q.clamp(-6e4, 6e4).to(DTYPES[dtype])
    _check_one_hot(q, pool, table, lens, page, d ** -0.5)


@pytest.mark.parametrize("base", [2.0 ** 22, 2.0 ** 24, 1.2 * 2.0 ** 24, 1.2 * 2.0 ** 25, -1.2 * 2.0 ** 25,
                                  1.2 * 2.0 ** 26, 2.0 ** 30])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_large_scores_that_rise_by_small_steps(base, dtype):
    """Scores of about `base` in units of the exponent's base 2, whose spacing is then a few such units:
    steps of one spacing, in whatever order a warp meets them.  All tokens have one row of V, so that
    the output is that row whatever a rounding does to the weights."""
    import block_sparse_attention_nsa_gb300 as nsa
    d, page, n, dt = 128, 64, 4096, DTYPES[dtype]
    gen = torch.Generator().manual_seed(9)
    q = torch.zeros(1, 2, d, dtype=dt)
    q[..., 0], q[..., 64] = 2.0 ** 15, 2.0
    a = float(torch.tensor(abs(base) / 2.0 ** 15).half())
    step = max(4.0, 2.0 ** (np.floor(np.log2(a * 2.0 ** 15)) - 23)) / 2.0
    k = torch.empty(n, 1, d)
    k[..., :64] = a if base > 0 else -a                # a flat group: its zero alone
    k[..., 64:] = (torch.randint(0, 4, (n // 32,), generator=gen) * step).repeat_interleave(32).view(n, 1, 1)
    v = (torch.arange(d) % 16 * 0.9990234375).expand(n, 1, d)
    pool, slots = nsa.kv4_pool(n // page, page, 1, d), _dev(np.arange(n, dtype=np.int32))
    nsa.kv4_append(pool, k.half().cuda(), v.half().contiguous().cuda(), slots)
    _, vr = nsa.kv4_read(pool, slots[:1], d, dtype=torch.float16)
    want = vr[0, 0].double().cpu()
    scale = 1 / 1.4426950408889634
    for width in (n // page, 2500):
        table = np.full((1, width), -1, np.int32)
        table[0, :n // page] = np.arange(n // page)
        out, lse = nsa.kv4_decode(q.cuda(), pool, _dev(table), _dev(np.int32([n])), scale)
        s = (q[0, 0].double() @ k[:, 0].half().double().t()) * scale
        tol = 2.0 ** -18 * want.abs() + torch.finfo(dt).eps / 2 * want.abs() + 2.0 ** -11 * 8
        assert ((out.double().cpu() - want).abs() <= tol).all()
        # the score's roundings: of the product, of the factor, of log2 e
        assert ((lse.double().cpu() - torch.logsumexp(s, 0)).abs() <= 2.0 ** -21 * s.abs().max() + 1e-5).all()
