"""Host-side checks of the page calls: refusals before anything is launched."""
import pytest

FAKE = 1 << 20          # never dereferenced: every call below fails its checks


@pytest.fixture(scope="module", params=["host", pytest.param("gpu-box", marks=pytest.mark.gpu)])
def lib(request):
    from block_sparse_attention_nsa_gb300 import build
    build.build()
    import block_sparse_attention_nsa_gb300 as nsa
    return nsa.load()


def _dims(**kw):
    from block_sparse_attention_nsa_gb300.pages import PageOpsDims
    base = dict(num_seqs=4, page_size=64, table_width=8, num_pages=100, num_free=10, count=3)
    return PageOpsDims(**{**base, **kw})


CALLS = [("nsa_page_fork", 12, (4,)), ("nsa_page_free", 8, ()), ("nsa_page_compact", 10, ())]


@pytest.mark.parametrize("name,args,optional", CALLS)
def test_refusals(lib, name, args, optional):
    def call(d, at=None, value=None):
        a = [FAKE] * (args - 1) + [None]               # the last: device_status
        if at is not None:
            a[at] = value
        return getattr(lib, name)(d, *a, None)
    for kw in (dict(num_seqs=0), dict(page_size=0), dict(table_width=0), dict(num_pages=-1),
               dict(num_free=-1), dict(count=-1)):
        assert call(_dims(**kw)) == 1, kw
    for kw in (dict(num_seqs=16385), dict(num_pages=(1 << 22) + 1), dict(table_width=1 << 25)):
        assert call(_dims(**kw)) == 2, kw
    if name != "nsa_page_compact":
        assert call(_dims(count=16385)) == 2
    for i in range(args):
        if i not in optional and i != args - 1:
            assert call(_dims(), i, None) == 1, i
        assert call(_dims(), i, FAKE + 2) == 1, i
    assert getattr(lib, name)(None, *[FAKE] * args, None) == 1


def test_copy_refusals(lib):
    def call(pages=10, size=4096, n=3, pool=FAKE, src=FAKE, dst=FAKE, st=None):
        return lib.nsa_page_copy(pages, size, n, pool, src, dst, st, None)
    for kw in (dict(pages=-1), dict(size=0), dict(n=-1), dict(pool=None), dict(pool=FAKE + 8),
               dict(src=None), dict(dst=None), dict(src=FAKE + 1), dict(dst=FAKE + 2),
               dict(st=FAKE + 3)):
        assert call(**kw) == 1, kw
    for kw in (dict(size=4104), dict(size=1 << 40)):
        assert call(**kw) == 2, kw
    assert call(n=0, src=None, dst=None) == 0


def test_python_refuses_cpu_tensors(lib):
    import torch

    import block_sparse_attention_nsa_gb300 as nsa
    x = torch.zeros(2, 2, dtype=torch.int32)
    one = x[0, :1]
    with pytest.raises(ValueError):
        nsa.page_fork(x, x[0], one, one, 4, x[0], x[0], one)
    with pytest.raises(ValueError):
        nsa.page_free(x, x[0], one, 4, x[0], x[0], one)
    with pytest.raises(ValueError):
        nsa.page_compact(x, x[0], 4, x[0], x[0])
    with pytest.raises(ValueError):
        nsa.page_copy(x, one, one)


def test_shared_decode_refusals(lib):
    import ctypes

    from block_sparse_attention_nsa_gb300.kv4 import Kv4Dims
    base = dict(num_pages=100, page_size=64, h_k=2, head_dim=128, dtype=0)

    def call(b=2, h_q=8, width=4, groups=1, q=FAKE, pool=FAKE, table=FAKE, lens=FAKE, cu=FAKE, pre=FAKE,
             scale=0.1, out=FAKE, lse=FAKE, st=None, ws=FAKE, size=1 << 40, **kw):
        return lib.nsa_kv4_decode_shared(Kv4Dims(**{**base, **kw}), b, h_q, width, groups, q, pool, table,
                                         lens, cu, pre, scale, out, lse, st, ws, size, None)
    for kw in (dict(b=0), dict(h_q=3), dict(width=0), dict(groups=0), dict(scale=float("nan")), dict(q=None),
               dict(pool=None), dict(table=None), dict(lens=None), dict(cu=None), dict(pre=None),
               dict(out=None), dict(lse=None), dict(q=FAKE + 8), dict(cu=FAKE + 2), dict(pre=FAKE + 1),
               dict(ws=FAKE + 8), dict(st=FAKE + 2), dict(h_k=0)):
        assert call(**kw) == 1, kw
    for kw in (dict(h_q=34), dict(width=1 << 26), dict(b=1 << 28), dict(groups=(1 << 20) + 1),
               dict(b=1 << 10, width=1 << 18), dict(head_dim=256), dict(page_size=16)):
        assert call(**kw) == 2, kw
    assert call(ws=None, size=0) == 3 and call(size=1024) == 3
    size = ctypes.c_size_t()
    f = lib.nsa_kv4_decode_shared_workspace_size
    assert f(Kv4Dims(**base), 2, 8, 1, ctypes.byref(size)) == 0 and size.value > 0
    assert call(size=size.value - 1) == 3
    assert f(Kv4Dims(**base), 2, 8, 0, ctypes.byref(size)) == 1
    assert f(Kv4Dims(**base), 2, 8, 1, None) == 1
