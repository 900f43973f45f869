"""Caches, inputs and error bounds of the 4-bit paged cache's GPU tests."""
import numpy as np
import torch

from oracle import kv4

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def make_cache(lens, page, h_k, d, seed, width=None, spare=3, mags=(1.0,)):
    """A pool whose pages hold normal K and V (each token times one of `mags`) and whose
    unowned rows hold random codes with NaN scales and zeros; the table's free entries are
    -1 where the row has more columns than pages."""
    rng = np.random.default_rng(seed)
    per = [-(-n // page) for n in lens]
    pages = sum(per) + spare
    shape = (pages, h_k, 2, page, d)
    x = rng.standard_normal(shape).astype(np.float32) * rng.choice(mags, shape[:4] + (1,))
    x[..., ::29] *= 3
    code, scale, zero = kv4.quantise(x)
    width = width or max(1, max(per))
    table, order, at = np.full((len(lens), width), -1, np.int32), rng.permutation(pages), 0
    owned = np.zeros((pages, page), bool)
    for b, n in enumerate(per):
        table[b, :n] = order[at:at + n]
        owned[table[b, :n]] = np.arange(n * page).reshape(n, page) < lens[b]
        at += n
    code = np.where(owned[:, None, None, :, None], code, rng.integers(0, 16, code.shape, np.uint8))
    free = ~np.broadcast_to(owned[:, None, None, :, None], scale.shape)
    scale[free], zero[free] = np.float16("nan"), np.float16("nan")
    return kv4.pack(code, scale, zero), table, order[at:].astype(np.int32)


def make_selection(lens, page, h_k, topk, seed, holes=True):
    """int32 [h_k, B, topk]: the newest block, block 0, random ones (repeats allowed), -1."""
    rng = np.random.default_rng(seed)
    sel = np.full((h_k, len(lens), topk), -1, np.int32)
    for h in range(h_k):
        for b, n in enumerate(lens):
            nb = -(-n // page)
            if nb:
                row = [nb - 1, 0] + list(rng.integers(-1 if holes else 0, nb, topk))
                sel[h, b] = rng.permutation(row[:topk])
    return sel


def check_decode(out, lse, ref, dtype):
    """ref: oracle.kv4.attend's values.  The bounds:
    scores   each is a sum of d products in fp32, off by at most d 2^-24 of the sum of their
             magnitudes (`big`), and the exponential and logarithm by 2^-20;
    lse      the scores' bound and fp32's own rounding of lse and its sums;
    out      half a step of the output type; where it is bf16, weights times the step of V
             rounded to fp16: 2^-11 of p * step times a code counted from 8 (at most 8 steps);
             where it is fp16, those weights in two parts (2^-22) and sums of 16 products that
             are cut below 2^-24 of the largest exponent, a code's up to 8 leading zeros
             counted in: 17 * 2^-16 of the largest p * step, 2^-15 of its 8 steps, and less
             than four times that with the sums so far; twice the scores' bound on every
             weight, and 2^-18 for the fp32 sums."""
    r_out, r_lse, big, pv, ps = ref
    d = r_out.shape[-1]
    got, gl = out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    ds = d * 2.0 ** -24 * big + 2.0 ** -20
    fin = np.isfinite(r_lse)
    np.testing.assert_array_equal(np.isneginf(gl), ~fin)
    off = np.abs(np.where(fin, gl, 0) - np.where(fin, r_lse, 0))
    tol = ds.T + 2.0 ** -22 * np.abs(np.where(fin, r_lse, 0)) + 2.0 ** -20
    assert (off <= tol).all(), f"lse off by {(off / tol).max():.2f} of its bound"
    half = torch.finfo(dtype).eps / 2
    tiny = 2.0 ** -25 if dtype is torch.float16 else 0.0
    term = ps * (2.0 ** -2 if dtype is torch.float16 else 1.0)
    tol = half * np.abs(r_out) + tiny + 2.0 ** -11 * term + (2 * ds[..., None] + 2.0 ** -18) * (pv + ps)
    tol[~fin.T] = 0
    off = np.abs(got - r_out)
    assert np.isfinite(got).all()
    assert (off <= tol).all(), f"out off by {np.nanmax(off / np.maximum(tol, 1e-30)):.2f} of its bound"
