"""Host-side checks of the rotary calls: frequencies, and refusals before anything is launched."""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import rope as oracle_rope

FAKE = 1 << 20          # never dereferenced: every call below fails its checks, or has no rows


@pytest.fixture(scope="module", params=["host", pytest.param("gpu-box", marks=pytest.mark.gpu)])
def lib(request):
    from block_sparse_attention_nsa_gb300 import build
    build.build()
    import block_sparse_attention_nsa_gb300 as nsa
    return nsa.load()


@pytest.mark.parametrize("how", [dict(), dict(scaling="linear", factor=8.0), dict(base=500000.0),
                                 dict(scaling="base", factor=4.0), dict(base=0.5),
                                 dict(scaling="ramp", factor=16.0, trained=8192)])
@pytest.mark.parametrize("rot", [16, 64, 128])
def test_freqs(lib, rot, how):
    import block_sparse_attention_nsa_gb300 as nsa
    got = nsa.rope_freqs(rot, device="cpu", **how).numpy().view(np.uint64)
    want = oracle_rope.freqs(rot, **{"base": 10000.0, **how}) / (2 * math.pi)
    part = want - np.floor(want)
    # the library's and the oracle's doubles may differ by a few steps of the frequency, and whole
    # units of 2^-64 leave less than one
    off = np.abs(got.astype(np.float64) / 2.0 ** 64 - part)
    off = np.minimum(off, 1 - off)
    assert (off <= 8 * 2.0 ** -53 * want + 2.0 ** -64).all()


def test_freqs_refusals(lib):
    out = (ctypes.c_uint64 * 8)()
    def call(rot=16, base=1e4, code=0, factor=2.0, trained=100.0, low=1.0, high=32.0, host=out):
        return lib.nsa_rope_freqs(rot, base, code, factor, trained, low, high, host)
    assert call() == 0 and call(code=3) == 0
    inf, nan = float("inf"), float("nan")
    for kw in (dict(rot=0), dict(rot=-2), dict(rot=7), dict(base=0.0), dict(base=-1.0), dict(base=inf),
               dict(base=nan), dict(code=4), dict(code=-1), dict(code=1, factor=0.0),
               dict(code=1, factor=nan), dict(code=2, factor=inf), dict(code=2, rot=2),
               dict(code=2, base=1e300, factor=1e300), dict(code=3, trained=0.0),
               dict(code=3, low=2.0, high=2.0), dict(code=3, high=nan), dict(host=None)):
        assert call(**kw) == 1, kw
    import block_sparse_attention_nsa_gb300 as nsa
    with pytest.raises(ValueError):
        nsa.rope_freqs(16, scaling="other", device="cpu")
    with pytest.raises(nsa.NsaError):
        nsa.rope_freqs(-4, device="cpu")
    with pytest.raises(nsa.NsaError) as e:
        nsa.rope_freqs(2 ** 32 + 16, device="cpu")
    assert e.value.code == 2


def test_refusals(lib):
    from block_sparse_attention_nsa_gb300.rope import RopeDims
    base = dict(num_tokens=4, h_q=4, h_k=2, head_dim=128, rot_dim=64, interleaved=0, num_seqs=0,
                dtype=0)
    def call(q=(FAKE, 512, 128), k=(FAKE, 256, 128), qo=(2 * FAKE, 512, 128), ko=(3 * FAKE, 256, 128),
             freqs=FAKE, pos=FAKE, cu=None, start=None, mscale=1.0, status=None, bwd=False, **kw):
        f = lib.nsa_rope_bwd if bwd else lib.nsa_rope
        return f(RopeDims(**{**base, **kw}), *q, *k, freqs, pos, cu, start, mscale, *qo, *ko, status, None)
    inf = float("inf")
    for bwd in (False, True):
        for kw in (dict(num_tokens=-1), dict(h_q=-1), dict(h_q=0, h_k=0), dict(rot_dim=0),
                   dict(rot_dim=144), dict(interleaved=2), dict(mscale=inf), dict(freqs=None),
                   dict(pos=None), dict(cu=FAKE), dict(num_seqs=1), dict(start=FAKE),
                   dict(pos=None, cu=FAKE), dict(freqs=FAKE + 4), dict(pos=FAKE + 2),
                   dict(status=FAKE + 1), dict(ko=(None, 256, 128)), dict(q=(None, 512, 128)),
                   dict(q=(FAKE + 8, 512, 128)), dict(k=(FAKE, 260, 128)), dict(k=(FAKE, 256, 4)),
                   dict(qo=(2 * FAKE + 2, 512, 128)),
                   # an output's rows overlap
                   dict(qo=(2 * FAKE, 512, 0)), dict(qo=(2 * FAKE, 0, 128)),
                   dict(qo=(2 * FAKE, 504, 128)), dict(qo=(2 * FAKE, 128, 504)),
                   dict(qo=(2 * FAKE, -504, 128)),
                   # an output is its input in another order
                   dict(qo=(FAKE, 128, 512)), dict(ko=(FAKE, 512, 128))):
            assert call(bwd=bwd, **kw) == 1, kw
        for kw in (dict(dtype=2), dict(head_dim=132), dict(head_dim=520), dict(rot_dim=24),
                   dict(num_tokens=1 << 30), dict(q=(FAKE, 1 << 41, 128))):
            assert call(bwd=bwd, **kw) == 2, kw
        # no rows: nothing to do, whatever the pointers
        assert call(bwd=bwd, num_tokens=0) == 0
        assert call(bwd=bwd, num_tokens=0, h_k=0, k=(None, 0, 0), ko=(None, 0, 0)) == 0


def test_python_refusals(lib):
    import block_sparse_attention_nsa_gb300 as nsa
    x = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    f = nsa.rope_freqs(64, device="cpu")
    p = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        nsa.rope(x, x, f, positions=p)                       # CPU tensors
    with pytest.raises(ValueError):
        nsa.rope(None, None, f, positions=p)
