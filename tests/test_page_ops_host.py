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
