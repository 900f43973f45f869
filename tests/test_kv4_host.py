"""Host-side checks of the 4-bit paged cache's C ABI: refusals before anything is launched
(no GPU needed; the same in the GPU tier)."""
import ctypes

import pytest

FAKE = 1 << 20          # never dereferenced: every call below fails its checks


@pytest.fixture(scope="module", params=["host", pytest.param("gpu-box", marks=pytest.mark.gpu)])
def lib(request):
    from block_sparse_attention_nsa_gb300 import build
    build.build()
    import block_sparse_attention_nsa_gb300 as nsa
    return nsa.load()


def _page(**kw):
    from block_sparse_attention_nsa_gb300.kv4 import PageDims
    base = dict(num_seqs=4, page_size=64, table_width=8, num_pages=100, num_free=10, max_slots=16)
    return PageDims(**{**base, **kw})


def _kv4(**kw):
    from block_sparse_attention_nsa_gb300.kv4 import Kv4Dims
    base = dict(num_pages=100, page_size=64, h_k=2, head_dim=128, dtype=0)
    return Kv4Dims(**{**base, **kw})


def _plan(lib, d, null=None, odd=None):
    a = [FAKE] * 9 + [None]
    if null is not None:
        a[null] = None
    if odd is not None:
        a[odd] = FAKE + 2
    return lib.nsa_page_plan(d, *a, None)


def test_plan_refusals(lib):
    for kw in (dict(num_seqs=0), dict(page_size=0), dict(table_width=0), dict(num_pages=-1),
               dict(num_free=-1), dict(max_slots=-1)):
        assert _plan(lib, _page(**kw)) == 1, kw
    for kw in (dict(num_seqs=16385), dict(table_width=1 << 20, page_size=1 << 11),
               dict(num_pages=1 << 25)):
        assert _plan(lib, _page(**kw)) == 2, kw
    for i in range(9):
        assert _plan(lib, _page(), null=i) == 1, i
    for i in range(10):
        assert _plan(lib, _page(), odd=i) == 1, i
    assert lib.nsa_page_plan(None, *[FAKE] * 10, None) == 1
    for i in range(6):
        a = [FAKE] * 5 + [None, None]
        a[i] = FAKE + 1
        assert lib.nsa_page_slots(_page(), *a) == 1, i
    assert lib.nsa_page_slots(_page(num_seqs=20000), *[FAKE] * 5, None, None) == 2


def test_row_refusals(lib):
    def append(d=None, n=4, k=FAKE, ks=256, v=FAKE, vs=256, slots=FAKE, pool=FAKE, st=None, kh=128):
        return lib.nsa_kv4_append(d or _kv4(), n, k, ks, kh, v, vs, 128, slots, pool, st, None)
    for kw in (dict(n=-1), dict(k=None), dict(v=None), dict(slots=None), dict(pool=None),
               dict(k=FAKE + 8), dict(v=FAKE + 2), dict(ks=260), dict(vs=-4), dict(kh=4),
               dict(slots=FAKE + 2), dict(pool=FAKE + 8), dict(st=FAKE + 1)):
        assert append(**kw) == 1, kw
    for kw in (dict(head_dim=256), dict(head_dim=96), dict(page_size=16), dict(page_size=48),
               dict(dtype=2), dict(num_pages=1 << 25)):
        assert append(_kv4(**kw)) == 2, kw
    assert append(_kv4(h_k=0)) == 1
    assert append(_kv4(num_pages=1 << 24, h_k=128)) == 2         # 2^32 tiles
    assert append(_kv4(h_k=1 << 20), n=1 << 20) == 2
    assert append(n=0, k=None, v=None, slots=None) == 0          # nothing to do

    def read(n=4, pool=FAKE, slots=FAKE, k=FAKE, v=FAKE, st=None):
        return lib.nsa_kv4_read(_kv4(), n, pool, slots, k, v, st, None)
    for kw in (dict(n=-1), dict(k=None), dict(v=None), dict(slots=None), dict(pool=None),
               dict(k=FAKE + 8), dict(st=FAKE + 2)):
        assert read(**kw) == 1, kw
    size = ctypes.c_size_t()
    assert lib.nsa_kv4_page_bytes(_kv4(), ctypes.byref(size)) == 0 and size.value == 64 * 144
    assert lib.nsa_kv4_page_bytes(_kv4(page_size=128, head_dim=64), ctypes.byref(size)) == 0
    assert size.value == 128 * 72
    assert lib.nsa_kv4_page_bytes(_kv4(), None) == 1


def test_decode_refusals(lib):
    def decode(d=None, b=2, h_q=8, width=4, topk=4, window=0, q=FAKE, pool=FAKE, table=FAKE,
               lens=FAKE, sel=FAKE, scale=0.1, out=FAKE, lse=FAKE, st=None, ws=FAKE, size=1 << 40):
        return lib.nsa_kv4_decode(d or _kv4(), b, h_q, width, topk, window, q, pool, table, lens,
                                  sel, scale, out, lse, st, ws, size, None)
    for kw in (dict(b=0), dict(h_q=3), dict(h_q=0), dict(width=0), dict(topk=-1), dict(window=-1),
               dict(scale=float("inf")), dict(scale=float("nan")), dict(q=None), dict(pool=None),
               dict(table=None), dict(lens=None), dict(sel=None), dict(topk=0), dict(out=None),
               dict(lse=None), dict(q=FAKE + 8), dict(out=FAKE + 8), dict(pool=FAKE + 8),
               dict(lse=FAKE + 2), dict(sel=FAKE + 2), dict(ws=FAKE + 8), dict(st=FAKE + 2)):
        assert decode(**kw) == 1, kw
    for kw in (dict(h_q=34), dict(topk=33), dict(width=1 << 26), dict(b=1 << 28),
               dict(b=1 << 10, width=1 << 18)):
        assert decode(**kw) == 2, kw
    size = ctypes.c_size_t()
    assert lib.nsa_kv4_decode_workspace_size(_kv4(), 2, 8, 0, ctypes.byref(size)) == 0
    if size.value:
        assert decode(topk=0, sel=None, size=size.value - 1) == 3
        assert decode(topk=0, sel=None, ws=None, size=0) == 3
    assert lib.nsa_kv4_decode_workspace_size(_kv4(), 2, 7, 0, ctypes.byref(size)) == 1
    assert lib.nsa_kv4_decode_workspace_size(_kv4(), 2, 8, 0, None) == 1


def test_python_refuses_cpu_tensors(lib):
    import torch

    import block_sparse_attention_nsa_gb300 as nsa
    x = torch.zeros(2, 2, dtype=torch.int32)
    with pytest.raises(ValueError):
        nsa.page_slots(x, x[0], x[0], 4, 4, 8)
    with pytest.raises(ValueError):
        nsa.kv4_read(torch.zeros(2, 2, 9216, dtype=torch.uint8), x[0], 128)
    with pytest.raises(nsa.NsaError):
        nsa.kv4_pool(2, 16, 2, 128, device="cpu")
    with pytest.raises(nsa.NsaError) as e:
        nsa.kv4_pool(2 ** 32 + 2, 64, 2, 128, device="cpu")      # would wrap to 2
    assert e.value.code == 2
