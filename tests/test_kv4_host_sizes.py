"""Sizes whose products pass 64 bits are refused by the paged cache's calls, before any launch."""
import pytest

FAKE = 1 << 20          # never dereferenced: every call below fails its checks


@pytest.fixture(scope="module", params=["host", pytest.param("gpu-box", marks=pytest.mark.gpu)])
def lib(request):
    from block_sparse_attention_nsa_gb300 import build
    build.build()
    import block_sparse_attention_nsa_gb300 as nsa
    return nsa.load()


@pytest.mark.parametrize("n,h_k", [(2 ** 31 - 1, 2 ** 31 - 1), (2 ** 30, 2 ** 30), (2 ** 29, 2 ** 28),
                                   (2 ** 31 - 1, 2 ** 27)])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_times_heads(lib, n, h_k, d):
    from block_sparse_attention_nsa_gb300.kv4 import Kv4Dims
    dims = Kv4Dims(num_pages=1, page_size=32, h_k=h_k, head_dim=d, dtype=0)
    assert lib.nsa_kv4_append(dims, n, FAKE, 0, 0, FAKE, 0, 0, FAKE, FAKE, None, None) == 2
    assert lib.nsa_kv4_read(dims, n, FAKE, FAKE, FAKE, FAKE, None, None) == 2
