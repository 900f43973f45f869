"""Rotary positions on the GPU against the oracle in extended precision."""
import numpy as np
import pytest
import torch

from kv4_helpers import DTYPES
from oracle import rope as oracle_rope

pytestmark = pytest.mark.gpu


def _rows(n, h, d, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, h, d, generator=g) * torch.exp(2 * torch.randn(n, h, 1, generator=g))
    return x.to(dtype)


def _check(got, x, pos, w, inter, mscale, sign, dtype):
    """Half a step of the output; and 2^-21 of the pair's size for fp32 (the sine and cosine: one
    step each of a value below 1 and the argument's rounding, 3 * 2^-24 together; two products and
    a sum) and for what the frequency's two roundings to 53 bits make of a far position."""
    xd = x.double().numpy()
    ref = oracle_rope.rotate(xd, pos, w, inter, mscale, sign)
    half = len(w)
    one = np.ones(len(w))
    size = np.zeros_like(xd)
    a = slice(0, 2 * half, 2) if inter else slice(0, half)
    b = slice(1, 2 * half, 2) if inter else slice(half, 2 * half)
    p = np.array([abs(v or 0) for v in pos], np.float64)[:, None, None]
    both = np.abs(xd[..., a]) + np.abs(xd[..., b])
    size[..., a] = size[..., b] = both * abs(mscale) * (2.0 ** -21 * one + p * w * 2.0 ** -51)
    tiny = 2.0 ** -25 if dtype is torch.float16 else 0.0
    tol = torch.finfo(dtype).eps / 2 * np.abs(ref) * (1 + 2.0 ** -10) + size + tiny
    off = np.abs(got.double().cpu().numpy() - ref)
    assert (off <= tol).all(), f"off by {(off / np.maximum(tol, 1e-300)).max():.2f} of the bound"
    rest = got[..., 2 * half:].cpu()
    assert torch.equal(rest, x[..., 2 * half:])


@pytest.mark.parametrize("n,hq,hk,d,rot,inter,dtype", [
    (1, 1, 1, 64, 64, False, "bf16"), (37, 16, 4, 128, 128, False, "bf16"),
    (37, 6, 3, 64, 32, True, "fp16"), (5, 7, 1, 256, 96, False, "fp16"),
    (300, 2, 0, 128, 16, True, "bf16"), (3, 0, 5, 128, 128, True, "fp16"),
    (2, 40, 8, 512, 512, False, "bf16"), (9, 3, 2, 104, 80, True, "bf16"),
    (4, 3, 1, 72, 48, False, "fp16")])
@pytest.mark.parametrize("far", [0, 1])
def test_positions(n, hq, hk, d, rot, inter, dtype, far):
    import block_sparse_attention_nsa_gb300 as nsa
    dt = DTYPES[dtype]
    rng = np.random.default_rng(n + rot)
    pos = rng.integers(-5, 2 ** 31 if far else 4000, n).astype(np.int32)
    pos[0] = 2 ** 31 - 1 if far else 0
    how = dict(scaling="ramp", factor=8.0, trained=4096) if far else {}
    freqs = nsa.rope_freqs(rot, **how)
    w = oracle_rope.freqs(rot, **{"base": 10000.0, **how})
    q = _rows(n, hq, d, dt, 1) if hq else None
    k = _rows(n, hk, d, dt, 2) if hk else None
    cuda = lambda x: None if x is None else x.cuda()
    p = torch.from_numpy(pos).cuda()
    for call, sign in ((nsa.rope, 1), (nsa.rope_bwd, -1)):
        qo, ko = call(cuda(q), cuda(k), freqs, positions=p, interleaved=inter, mscale=1.25)
        for got, x in ((qo, q), (ko, k)):
            if x is None:
                assert got is None
                continue
            _check(got, x, [int(v) for v in pos], w, inter, 1.25, sign, dt)


@pytest.mark.parametrize("starts", [False, True])
@pytest.mark.parametrize("lens", [(1,), (5, 0, 0, 70, 1), tuple([1] * 65), tuple([3, 0] * 600)])
def test_packed_batches(lens, starts):
    import block_sparse_attention_nsa_gb300 as nsa
    pad = 7
    n = sum(lens) + pad
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    rng = np.random.default_rng(len(lens))
    start = rng.integers(0, 10 ** 6, len(lens)).astype(np.int32) if starts else None
    q, k = _rows(n, 3, 64, torch.bfloat16, 3), _rows(n, 1, 64, torch.bfloat16, 4)
    freqs, w = nsa.rope_freqs(64), oracle_rope.freqs(64)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    # in place; the rows behind the last sequence stay
    qc, kc = q.cuda(), k.cuda()
    qo, ko = nsa.rope(qc, kc, freqs, cu_seqlens=torch.from_numpy(cu).cuda(),
                      start=None if start is None else torch.from_numpy(start).cuda(), q_out=qc,
                      k_out=kc, device_status=status)
    assert qo is qc and ko is kc and int(status.item()) == 0
    pos = oracle_rope.positions(n, cu, start)
    for got, x in ((qc, q), (kc, k)):
        _check(got, x, pos, w, False, 1.0, 1, torch.bfloat16)
        assert torch.equal(got[n - pad:].cpu(), x[n - pad:])
    # the way back, to another tensor: its rows behind the last sequence are left
    back = torch.full_like(qc, 5.0)
    nsa.rope_bwd(qc, None, freqs, cu_seqlens=torch.from_numpy(cu).cuda(),
                 start=None if start is None else torch.from_numpy(start).cuda(), dq_in=back)
    assert (back[n - pad:] == 5).all()
    _check(back[:n - pad], qc[:n - pad].cpu(), pos[:n - pad], w, False, 1.0, -1, torch.bfloat16)


def test_malformed_batches_leave_rows_and_say_so():
    import block_sparse_attention_nsa_gb300 as nsa
    x = _rows(12, 2, 64, torch.float16, 5).cuda()
    freqs = nsa.rope_freqs(64)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full_like(x, 9.0)
    cu = torch.tensor([4, 8], dtype=torch.int32, device="cuda")
    nsa.rope(x, None, freqs, cu_seqlens=cu, q_out=out, device_status=status)
    assert int(status.item()) == nsa.DEVERR_BAD_SEQLENS
    assert (out[:4] == 9).all() and (out[8:] == 9).all()
    want, _ = nsa.rope(x[4:8], None, freqs, positions=torch.arange(4, dtype=torch.int32, device="cuda"))
    assert torch.equal(out[4:8], want)


def test_views_and_broadcast_heads():
    import block_sparse_attention_nsa_gb300 as nsa
    n, hq, hk, d = 70, 4, 2, 128
    row = _rows(n, hq + 2 * hk, d, torch.bfloat16, 6).cuda()
    q, k = row[:, :hq], row[:, hq:hq + hk]
    pos = torch.randint(0, 9999, (n,), device="cuda", dtype=torch.int32)
    freqs = nsa.rope_freqs(64)
    want = nsa.rope(q.contiguous(), k.contiguous(), freqs, positions=pos)
    got = nsa.rope(q, k, freqs, positions=pos)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # heads before tokens, on both sides
    t = lambda x: x.transpose(0, 1).contiguous().transpose(0, 1)
    out = t(torch.zeros_like(want[0]))
    nsa.rope(t(q), None, freqs, positions=pos, q_out=out)
    assert torch.equal(out, want[0])
    # one key row for every head; the last half of the head, through a view
    one = nsa.rope(None, k[:, :1].expand(n, 5, d), freqs, positions=pos)[1]
    assert torch.equal(one, want[1][:, :1].expand(n, 5, d))
    tail = row.clone()
    nsa.rope(tail[:, :hq, 64:], None, freqs, positions=pos, q_out=tail[:, :hq, 64:])
    assert torch.equal(tail[:, :hq, 64:], nsa.rope(q[..., 64:].contiguous(), None, freqs, positions=pos)[0])
    assert torch.equal(tail[..., :64], row[..., :64]) and torch.equal(tail[:, hq:], row[:, hq:])
    # in place on the fused rows
    whole = row.clone()
    nsa.rope(whole[:, :hq], whole[:, hq:hq + hk], freqs, positions=pos, q_out=whole[:, :hq],
             k_out=whole[:, hq:hq + hk])
    assert torch.equal(whole[:, :hq], want[0]) and torch.equal(whole[:, hq + hk:], row[:, hq + hk:])
    with pytest.raises(nsa.NsaError):
        nsa.rope(None, k, freqs, positions=pos, k_out=k[:, :1].expand(n, hk, d))
    with pytest.raises(ValueError):
        nsa.rope(q, k, freqs.int(), positions=pos)
    with pytest.raises(ValueError):
        nsa.rope(q, k, freqs, positions=pos.long())
    with pytest.raises(ValueError):
        nsa.rope(q, k.half(), freqs, positions=pos)
    # no tokens at all
    assert nsa.rope(q[:0], k[:0], freqs, positions=pos[:0])[0].shape == (0, hq, d)


def test_gradient_against_differences():
    import block_sparse_attention_nsa_gb300 as nsa
    n, h, d = 6, 2, 64
    x, g = _rows(n, h, d, torch.float16, 7), _rows(n, h, d, torch.float16, 8)
    pos = torch.arange(100, 100 + n, dtype=torch.int32, device="cuda")
    freqs, w = nsa.rope_freqs(32), oracle_rope.freqs(32)
    grad, _ = nsa.rope_bwd(g.cuda(), None, freqs, positions=pos, interleaved=True, mscale=0.75)
    f = lambda y: (oracle_rope.rotate(y, pos.tolist(), w, True, 0.75) * g.double().numpy()).sum((1, 2))
    rng = np.random.default_rng(0)
    for _ in range(20):
        e = rng.standard_normal(x.shape)
        num = (f(x.double().numpy() + 1e-4 * e) - f(x.double().numpy() - 1e-4 * e)) / 2e-4
        got = (grad.double().cpu().numpy() * e).sum((1, 2))
        bound = (np.abs(grad.double().cpu().numpy() * e).sum((1, 2))) * 2.0 ** -11 + 1e-6
        assert (np.abs(num - got) <= bound).all()


def test_streams_and_graphs():
    import block_sparse_attention_nsa_gb300 as nsa
    n, h, d = 200, 4, 128
    x = [_rows(n, h, d, torch.bfloat16, s).cuda() for s in range(4)]
    freqs = nsa.rope_freqs(d)
    cu = torch.tensor([0, 50, 200], dtype=torch.int32, device="cuda")
    want = [nsa.rope(a, a, freqs, cu_seqlens=cu)[0] for a in x]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in x]
    got = [nsa.rope(a, None, freqs, cu_seqlens=cu, stream=s)[0] for a, s in zip(x, streams)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    buf = x[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nsa.rope(buf, None, freqs, cu_seqlens=cu, q_out=buf)
        nsa.rope_bwd(buf, None, freqs, cu_seqlens=cu, dq_in=buf)
        nsa.rope(buf, None, freqs, cu_seqlens=cu, q_out=buf)
    for a in x[1:]:
        buf.copy_(a)
        graph.replay()
        once, _ = nsa.rope(a, None, freqs, cu_seqlens=cu)
        back, _ = nsa.rope_bwd(once, None, freqs, cu_seqlens=cu)
        assert torch.equal(buf, nsa.rope(back, None, freqs, cu_seqlens=cu)[0])


def test_rows_past_32_bit_offsets():
    """Tokens and heads further apart than 2^31 bytes, in place and not, against the same rows close together."""
    import block_sparse_attention_nsa_gb300 as nsa
    n, h, d = 3, 2, 64
    freqs, pos = nsa.rope_freqs(32), torch.tensor([1, 70000, 5], dtype=torch.int32, device="cuda")
    x = torch.randn(n, h, d, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    want = nsa.rope(x, x, freqs, positions=pos)[0]
    far = 2 ** 31 // (n - 1) + 8
    for strides in ((far, d, 1), (d, 2 ** 31 + 8, 1)):
        buf = torch.zeros(2 ** 31 + 2 ** 12, dtype=torch.bfloat16, device="cuda")
        view = buf.as_strided((n, h, d), strides)
        view.copy_(x)
        got = nsa.rope(view, None, freqs, positions=pos)[0]
        assert torch.equal(got, want)
        nsa.rope(None, view, freqs, positions=pos, k_out=view)
        assert torch.equal(view, want)
