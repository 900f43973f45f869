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


@pytest.mark.parametrize("d,dtype", [(64, "fp16"), (128, "fp16"), (64, "bf16"), (128, "bf16")])
def test_selections_of_a_whole_sequence_by_one_warp(d, dtype):
    """850 sequences of 8 KV heads: 6800 segments of 128 tiles, each one warp's on 148, 152 and 160
    SMs.  The bounds are test_long_runs_lose_little's."""
    import block_sparse_attention_nsa_gb300 as nsa
    dt, n, page, h_k, b = DTYPES[dtype], 4096, 128, 8, 850
    pool, table, lens = _repeated(b, n, page, h_k, d, 79)
    sel = np.broadcast_to(np.arange(n // page, dtype=np.int32), (h_k, b, n // page)).copy()
    q = torch.randn(b, h_k, d, generator=torch.Generator().manual_seed(80)).to(dt)
    out, _ = nsa.kv4_decode(q.cuda(), _dev(pool), _dev(table), _dev(lens), d ** -0.5,
                            sel_idx=_dev(sel))
    rows = [0, 7, 424, 849]
    ref = kv4.attend(q[rows].double().numpy(), pool, table[:4], lens[:4], page, d ** -0.5,
                     sel[:, :4])[0]
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


def _wide(lens, page, h_k, g, d, seed, dtype=torch.bfloat16, width=2000):
    import block_sparse_attention_nsa_gb300 as nsa
    pool, table, _ = make_cache(lens, page, h_k, d, seed, width=width)
    q = torch.randn(len(lens), h_k * g, d, generator=torch.Generator().manual_seed(seed)).to(dtype)
    s = dict(pool=pool, table=table, q=q, lens=lens, dq=q.cuda(), dpool=_dev(pool),
             dtab=_dev(table), dlens=_dev(np.int32(lens)), out=torch.empty_like(q).cuda(),
             lse=torch.empty(h_k * g, len(lens), device="cuda"))
    s["ws"] = _workspace(nsa, pool.shape[0], page, h_k, d, len(lens), h_k * g)
    return s


def _oracle_check(s, page, scale):
    ref = kv4.attend(s["q"].double().numpy(), s["pool"], s["table"], s["lens"], page, scale)
    check_decode(s["out"], s["lse"], ref, s["q"].dtype)


def test_runs_on_another_stream_in_graphs_and_with_a_shared_workspace():
    """Two shapes on a stream of their own, then captured into graphs that share a workspace and are
    replayed in turn, while their lengths change in place."""
    import block_sparse_attention_nsa_gb300 as nsa
    page, h_k, g, d = 64, 2, 4, 128
    side = torch.cuda.Stream()
    sets = [_wide(lens, page, h_k, g, d, seed)
            for seed, lens in ((41, (5000, 3)), (42, (900, 4000, 1)))]
    ws = max((s["ws"] for s in sets), key=torch.numel)
    torch.cuda.synchronize()
    for s in sets:
        nsa.kv4_decode(s["dq"], s["dpool"], s["dtab"], s["dlens"], 0.1, out=s["out"], lse=s["lse"],
                       workspace=ws, stream=side)
    side.synchronize()
    assert (ws != 0xff).any()
    for s in sets:
        _oracle_check(s, page, 0.1)
    graphs = []
    for s in sets:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            nsa.kv4_decode(s["dq"], s["dpool"], s["dtab"], s["dlens"], 0.1, out=s["out"],
                           lse=s["lse"], workspace=ws)
        graphs.append(graph)
    for k in range(4):
        ws.fill_(0xff)                   # nothing is carried over
        for s, graph in zip(sets, graphs):
            s["lens"] = tuple(max(0, n - 700 * k) for n in s["lens"])
            s["dlens"].copy_(_dev(np.int32(s["lens"])))
            graph.replay()
        torch.cuda.synchronize()
        assert (ws != 0xff).any()
        for s in sets:
            _oracle_check(s, page, 0.1)


def test_runs_on_two_streams_and_between_torch_kernels():
    """Unsynchronised loops on two streams, each call behind a torch kernel that writes its query and
    before one that reads its output, several shapes in turn on one workspace: the same sums as
    with a wait after each."""
    import block_sparse_attention_nsa_gb300 as nsa
    page, h_k, g, d = 64, 2, 4, 128
    loops = []
    for seed in (61, 63):
        sets = [_wide(lens, page, h_k, g, d, seed + k, width=1500 + 200 * k)
                for k, lens in enumerate(((4000, 5, 900), (3000,) * 5))]
        qs = [torch.randn((12,) + s["q"].shape, generator=torch.Generator().manual_seed(seed))
              .to(torch.bfloat16).cuda() for s in sets]
        loops.append((sets, qs, max((s["ws"] for s in sets), key=torch.numel), torch.cuda.Stream()))

    def run(sets, qs, ws, wait):
        totals = [torch.zeros(s["q"].shape, device="cuda") for s in sets]
        for k in range(12):
            for s, q, total in zip(sets, qs, totals):
                s["dq"].copy_(q[k])
                nsa.kv4_decode(s["dq"], s["dpool"], s["dtab"], s["dlens"], 0.1, out=s["out"],
                               lse=s["lse"], workspace=ws)
                total.add_(s["out"].float())
                if wait:
                    torch.cuda.synchronize()
        return totals
    want = [run(s, q, w, True) for s, q, w, _ in loops]
    assert all((w != 0xff).any() for _, _, w, _ in loops)
    for _ in range(3):
        got = []
        for s, q, w, stream in loops:
            with torch.cuda.stream(stream):
                stream.wait_stream(torch.cuda.default_stream())
                got.append(run(s, q, w, False))
        torch.cuda.synchronize()
        for a, b in zip(sum(got, []), sum(want, [])):
            assert torch.equal(a, b)


@pytest.mark.parametrize("graphed", [False, True])
def test_steps_of_plan_append_and_runs(graphed):
    """Serving steps back to back, without a wait or as one captured step that is replayed: a plan
    that opens pages, an append into them, a decode over everything cached, each launched while the
    one before it ends, behind a torch kernel that makes the step's rows."""
    import block_sparse_attention_nsa_gb300 as nsa
    page, h_k, g, d, b, steps = 32, 2, 2, 64, 5, 70
    pages, width = 40, 4000
    gen = torch.Generator().manual_seed(4)
    rows = torch.randn(steps, 3, b, h_k, d, generator=gen).to(torch.bfloat16)
    i32 = dict(dtype=torch.int32, device="cuda")
    pool = nsa.kv4_pool(pages, page, h_k, d)
    table = torch.full((b, width), -1, **i32)
    free = torch.randperm(pages, generator=gen).int().cuda()
    head, lens, one = torch.zeros(1, **i32), torch.zeros(b, **i32), torch.ones(b, **i32)
    slots, cu, status = torch.empty(b, **i32), torch.empty(b + 1, **i32), torch.zeros(1, **i32)
    at, drows = torch.zeros((), dtype=torch.int64, device="cuda"), rows.cuda()
    kvq = torch.empty_like(drows[0])
    q = torch.empty(b, h_k * g, d, dtype=torch.bfloat16, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(h_k * g, b, device="cuda")
    outs = torch.zeros((steps,) + out.shape, dtype=out.dtype, device="cuda")
    lses = torch.zeros((steps,) + lse.shape, device="cuda")
    ws = _workspace(nsa, pages, page, h_k, d, b, h_k * g)

    def step():
        kvq.copy_(drows.index_select(0, at.view(1))[0])
        q.copy_(kvq[2].repeat_interleave(g, 1))
        nsa.page_plan(lens, one, free, head, table, page, pages, slots, lens, cu, head, status)
        nsa.kv4_append(pool, kvq[0], kvq[1], slots, status)
        nsa.kv4_decode(q, pool, table, lens, 0.3, out=out, lse=lse, workspace=ws,
                       device_status=status)
        outs.index_copy_(0, at.view(1), out.unsqueeze(0))
        lses.index_copy_(0, at.view(1), lse.unsqueeze(0))
        at.add_(1)
    if graphed:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
    for _ in range(steps):
        graph.replay() if graphed else step()
    torch.cuda.synchronize()
    assert (ws != 0xff).any() and int(status.item()) == 0 and lens.tolist() == [steps] * b
    assert int(head.item()) == b * -(-steps // page)
    hpool, htab = pool.cpu().numpy(), table.cpu().numpy()
    for t in (0, 1, 30, 31, 32, 33, 63, 64, steps - 1):
        ref = kv4.attend(rows[t, 2].repeat_interleave(g, 1).double().numpy(), hpool, htab,
                         [t + 1] * b, page, 0.3)
        check_decode(outs[t], lses[t], ref, torch.bfloat16)
