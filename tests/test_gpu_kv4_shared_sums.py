"""Sums of the decode over shared prefixes that run over thousands of blocks in one CTA."""
import numpy as np
import pytest
import torch

from kv4_helpers import DTYPES
from oracle import kv4
from shared_helpers import check_shared

pytestmark = pytest.mark.gpu

PAGE, G = 128, 16
SOME = [0, 700]                                   # sequences that are compared


def _whole_tiles():
    """Sequences of G query heads whose rows are a tile of 128 (two CTAs: 256) for every SM, so that each
    takes a tile from the prefix' first block to its last."""
    return torch.cuda.get_device_properties(0).multi_processor_count * 128 // G


def _decode(k, v, times, q, scale):
    """A prefix of k and v [pages, PAGE, d], named `times` times over, for all sequences; compared rows of out
    and lse, and the oracle's values (of keys that all occur equally often; `times` shows in lse alone)."""
    import block_sparse_attention_nsa_gb300 as nsa
    d, pages = k.shape[-1], k.shape[0]
    pool = kv4.pack(*kv4.quantise(np.stack([k, v], 1)[:, None]))
    b, n = q.shape[0], pages * times * PAGE
    once = torch.arange(pages, dtype=torch.int32, device="cuda")
    table = once.repeat(times).expand(b, -1).contiguous()
    lens = torch.full((b,), n, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, b], dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    need = nsa.kv4_decode_shared_workspace_size(pages, PAGE, 1, d, b, G, 1)
    work = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    out, lse = nsa.kv4_decode_shared(q.cuda(), torch.from_numpy(pool).cuda(), table, lens, scale, cu, lens[:1],
                                     workspace=work, device_status=status)
    assert int(status.item()) == 0
    own = nsa.kv4_decode_workspace_size(pages, PAGE, 1, d, b, G)
    at = -(-own // 256) * 256                     # the plan: groups that share, first
    assert work[at:at + 4].view(torch.int32).item() == 1
    ref = kv4.attend(q[SOME].double().numpy(), pool, np.tile(np.arange(pages, dtype=np.int32), (len(SOME), 1)),
                     [pages * PAGE] * len(SOME), PAGE, scale)
    return out[SOME].double().cpu().numpy(), lse[:, SOME].double().cpu().numpy(), ref, ref[1] + np.log(times)


def _lse_bound(ref, lse, d):
    """Scores: sums of d products in fp32, the exponential's and logarithm's 2^-20; fp32's rounding of lse; sums
    of weights in steps of at most 32 numbers (a block), 256 (blocks) and 256 (sums of those), each addition off
    by 2^-24 of its sum: 544 * 2^-24."""
    return (d * 2.0 ** -24 * ref[2] + 2.0 ** -20).T + 2.0 ** -22 * np.abs(lse) + 544 * 2.0 ** -24


def _two_keys(d, dtype):
    """Two keys in turn, half a million times: sums whose roundings do not cancel."""
    rng = np.random.default_rng(7)
    two = np.abs(rng.standard_normal((2, 2, d))).astype(np.float32) + np.float32(0.5)
    k, v = (np.tile(x, (PAGE // 2, 1))[None] for x in (two[:, 0], two[:, 1]))
    q = torch.randn(_whole_tiles(), G, d, generator=torch.Generator().manual_seed(8)).to(DTYPES[dtype])
    return _decode(k, v, 4096, q, 0.5 * d ** -0.5)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_sums_of_equal_weights(dtype, d):
    _, lse, ref, ref_lse = _two_keys(d, dtype)
    far = (np.abs(lse - ref_lse) / _lse_bound(ref, ref_lse, d)).max()
    assert far <= 1, f"lse off by {far:.3f} of its bound"


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_products_of_equal_weights(dtype, d):
    """Half a step of the output type, V's rounding to fp16 and a weight's (2^-11 each), sums of weights as in
    lse, and 2048 products of the tensor core's one after the other, each cut by up to 2^-24: 2^-13."""
    out, _, ref, _ = _two_keys(d, dtype)
    bound = (torch.finfo(DTYPES[dtype]).eps / 2 + 2.0 ** -10 + 2.0 ** -13) * np.abs(ref[0]) + ref[3] * (
        2 * (d * 2.0 ** -24 * ref[2] + 2.0 ** -20)[..., None] + 544 * 2.0 ** -24)
    off = (np.abs(out - ref[0]) / bound).max()
    assert off <= 1, f"out off by {off:.3f} of its bound"


@pytest.mark.parametrize("mean", [0.0, 1.0])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_errors_do_not_grow_with_a_run(dtype, d, mean):
    """4096 blocks of a tile in one run.  For fp16 V's rounding is as large as the output's own, so that the
    two are 2^0.5 of it; up to 1.5 is left to what the tensor core cuts off its sums, half of the output's
    rounding (1.5^2 - 2 = 0.5^2).  For bf16, whose rounding is eight times as large, all else is within 1.1."""
    rng = np.random.default_rng(5)
    k = rng.standard_normal((256, PAGE, d), np.float32)
    v = rng.standard_normal((256, PAGE, d), np.float32) + np.float32(mean)
    dt = DTYPES[dtype]
    q = torch.randn(_whole_tiles(), G, d, generator=torch.Generator().manual_seed(6)).to(dt)
    out, lse, ref, ref_lse = _decode(k, v, 16, q, d ** -0.5)
    rounding = np.linalg.norm(torch.from_numpy(ref[0]).to(dt).double().numpy() - ref[0])
    off = np.linalg.norm(out - ref[0])
    far = (np.abs(lse - ref_lse) / _lse_bound(ref, ref_lse, d)).max()
    assert off <= (1.5 if dtype == "fp16" else 1.1) * rounding, f"out off by {off / rounding:.3f} of its rounding"
    assert far <= 1, f"lse off by {far:.3f} of its bound"


@pytest.mark.parametrize("order", ["rising", "falling", "late", "first and last"])
@pytest.mark.parametrize("d,dtype,blocks", [(64, "fp16", 200), (128, "fp16", 193), (64, "bf16", 600), (128, "bf16", 513)])
def test_scores_that_change_from_run_to_run(d, dtype, blocks, order):
    """The reference is raised from one run of sums to the next, or never again; the first runs have no keys at
    all (pages that are none), or all but the first and the last block have none."""
    import block_sparse_attention_nsa_gb300 as nsa
    rng = np.random.default_rng(3)
    u = rng.standard_normal(d).astype(np.float32)
    up = np.linspace(0, 6, blocks * PAGE, dtype=np.float32).reshape(blocks, PAGE, 1)
    k = u * (up[::-1, ::-1] if order == "falling" else up) + 0.1 * rng.standard_normal((blocks, PAGE, d), np.float32)
    v = rng.standard_normal((blocks, PAGE, d), np.float32) + np.float32(0.5)
    pool = kv4.pack(*kv4.quantise(np.stack([k, v], 1)[:, None]))
    table = np.arange(blocks, dtype=np.int32)
    if order == "late":
        table[:blocks // 2 + 3] = -1
    if order == "first and last":
        table[1:-1] = -1
    dt, b, n = DTYPES[dtype], _whole_tiles(), blocks * PAGE - 37
    q = (torch.from_numpy(u) * 0.4 + torch.randn(b, G, d, generator=torch.Generator().manual_seed(4))).to(dt)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    rows = torch.from_numpy(table).cuda().expand(b, -1).contiguous()
    lens = torch.full((b,), n, dtype=torch.int32, device="cuda")
    out, lse = nsa.kv4_decode_shared(q.cuda(), torch.from_numpy(pool).cuda(), rows, lens, d ** -0.5,
                                     torch.tensor([0, b], dtype=torch.int32, device="cuda"), lens[:1], device_status=status)
    assert int(status.item()) == (nsa.DEVERR_BAD_INDEX if (table < 0).any() else 0)
    some = [0, 1, 7, 8, b // 2, b - 1]
    check_shared(out[some], lse[:, some], kv4.attend(q[some].double().numpy(), pool, np.tile(table, (len(some), 1)),
                                                     [n] * len(some), PAGE, d ** -0.5), dt)
