"""Binding of the rotary positions (include/nsa_rope.h): queries and keys turned by their
positions, and the gradient.

Argument marshalling only.  q, k and the outputs may be strided views whose last dimension is
contiguous; all tensors live on the current device; outputs that are not given are allocated on
the launching stream.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from .kv4 import _DTYPES, _device, _empty, _fail, _held, _ints, _lib, _raw, _status

__all__ = ["rope_freqs", "rope", "rope_bwd"]

_SCALING = {"none": 0, "linear": 1, "base": 2, "ramp": 3}


class RopeDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("num_tokens", "h_q", "h_k", "head_dim", "rot_dim",
                                              "interleaved", "num_seqs", "dtype")]


def signatures():
    """ctypes result and argument types of the library's functions."""
    vp, i32, f64, st = ctypes.c_void_p, ctypes.c_int32, ctypes.c_double, ctypes.c_int
    rt = [vp, ctypes.c_int64, ctypes.c_int64]
    call = (st, [ctypes.POINTER(RopeDims), *rt, *rt, vp, vp, vp, vp, ctypes.c_float, *rt, *rt, vp, vp])
    return {
        "nsa_rope_freqs": (st, [i32, f64, i32, f64, f64, f64, f64, vp]),
        "nsa_rope": call,
        "nsa_rope_bwd": call,
    }


def rope_freqs(rot_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
               trained: float = 0.0, low: float = 1.0, high: float = 32.0, device="cuda"):
    """Frequencies base^(-2 i / rot_dim), int64 [rot_dim / 2]: the part of a turn that a position
    advances, in 2^-64 (as unsigned numbers).  scaling: "none"; "linear", divided by factor;
    "base", base times factor^(rot_dim / (rot_dim - 2)); "ramp", pairs that make `high` turns or more
    over `trained` positions as they are, those of `low` or fewer divided by factor, a linear ramp
    between (the factor on q and k that goes with it, 0.1 ln(factor) + 1, is rope's mscale)."""
    code = _SCALING.get(scaling)
    if code is None:
        raise ValueError(f"scaling: one of {', '.join(_SCALING)} expected, got {scaling!r}")
    rot_dim, = _held((rot_dim,), "rope_freqs")
    host = torch.empty(max(0, rot_dim) // 2, dtype=torch.int64)
    status = _lib().nsa_rope_freqs(rot_dim, base, code, factor, trained, low, high, host.data_ptr())
    if status:
        _fail(status, "rope_freqs")
    return host.to(device)


@functools.lru_cache(maxsize=4096)
def _rope_dims(*sizes):
    return RopeDims(*_held(sizes, "rope dims"))


def _tensor(name, t, n, heads, d, dtype, dev):
    """Pointer and strides of t [n, heads, d], whose last dimension has to be contiguous."""
    shape, strides = t.shape, t.stride()
    if (len(shape) != 3 or shape[0] != n or shape[1] != heads or shape[2] != d or strides[2] != 1
            or t.dtype is not dtype or t.get_device() != dev):
        raise ValueError(f"{name}: a {dtype} tensor {(n, heads, d)} on device {dev} with a contiguous last "
                         f"dimension expected, got {t.dtype} {tuple(shape)}, strides {strides}, on {t.device}")
    return t.data_ptr(), strides[0], strides[1]


_NONE = (None, 0, 0)
_i64 = torch.int64


def _run(where, call, q, k, freqs, positions, cu_seqlens, start, interleaved, mscale, q_out, k_out,
         device_status, stream):
    first = k if q is None else q
    if first is None:
        raise ValueError("q or k expected")
    if first.dim() != 3:
        raise ValueError("q and k [N, heads, d] expected")
    n, h, d = first.shape
    dtype, dev = first.dtype, _device(first)
    code = _DTYPES.get(dtype)
    if code is None:
        _fail(2, f"{where}: dtype {dtype}")
    h_q = h_k = 0
    q_in = k_in = q_to = k_to = _NONE
    if q is None:
        if q_out is not None:
            raise ValueError("q: an output without its input")
    else:
        h_q = h
        q_in = _tensor("q", q, n, h_q, d, dtype, dev)
        if q_out is None:
            q_out = _empty((n, h_q, d), dtype, dev, stream)
        q_to = _tensor("q's output", q_out, n, h_q, d, dtype, dev)
    if k is None:
        if k_out is not None:
            raise ValueError("k: an output without its input")
    else:
        h_k = k.shape[1] if k.dim() == 3 else -1
        k_in = _tensor("k", k, n, h_k, d, dtype, dev)
        if k_out is None:
            k_out = _empty((n, h_k, d), dtype, dev, stream)
        k_to = _tensor("k's output", k_out, n, h_k, d, dtype, dev)
    if (freqs.dtype is not _i64 or freqs.dim() != 1 or freqs.get_device() != dev
            or not freqs.is_contiguous()):
        raise ValueError("freqs: the int64 tensor that rope_freqs makes expected, on the tensors' device")
    seqs, pos, cu, at = 0, None, None, None
    if positions is not None:
        if cu_seqlens is not None or start is not None:
            raise ValueError("either positions, or cu_seqlens and start")
        _ints("positions", positions, n, dev)
        pos = positions.data_ptr()
    elif cu_seqlens is not None:
        seqs = cu_seqlens.numel() - 1
        if seqs < 1:
            raise ValueError("cu_seqlens: at least two entries expected")
        _ints("cu_seqlens", cu_seqlens, seqs + 1, dev)
        cu = cu_seqlens.data_ptr()
        if start is not None:
            _ints("start", start, seqs, dev)
            at = start.data_ptr()
    else:
        raise ValueError("positions or cu_seqlens expected")
    status = call(
        _rope_dims(n, h_q, h_k, d, 2 * freqs.numel(), 1 if interleaved else 0, seqs, code), *q_in, *k_in,
        freqs.data_ptr(), pos, cu, at, mscale, *q_to, *k_to,
        None if device_status is None else _status(device_status, dev), _raw(stream, dev))
    if status:
        _fail(status, where)
    return q_out, k_out


def rope(q, k, freqs, positions=None, cu_seqlens=None, start=None, interleaved: bool = False,
         mscale: float = 1.0, q_out=None, k_out=None, device_status=None, stream=None):
    """q [N, h_q, d] and k [N, h_k, d] (one may be None) with the pairs of their first 2 *
    freqs.numel() dimensions turned by the tokens' positions and scaled by mscale; the other
    dimensions as they are.  Pairs are (i, i + half), or (2 i, 2 i + 1) where interleaved.
    Positions: int32 [N], or those of a packed batch by cu_seqlens int32 [S + 1], counted from
    start int32 [S] (None: 0) in each sequence; rows behind the last sequence are left as they are.
    q_out and k_out may be q and k.  Returns q_out, k_out."""
    return _run("rope", _lib().nsa_rope, q, k, freqs, positions, cu_seqlens, start, interleaved, mscale,
                q_out, k_out, device_status, stream)


def rope_bwd(dq_out, dk_out, freqs, positions=None, cu_seqlens=None, start=None,
             interleaved: bool = False, mscale: float = 1.0, dq_in=None, dk_in=None,
             device_status=None, stream=None):
    """The gradients of rope's q and k from those of its outputs (dq_in and dk_in may be dq_out and
    dk_out).  Returns dq_in, dk_in."""
    return _run("rope_bwd", _lib().nsa_rope_bwd, dq_out, dk_out, freqs, positions, cu_seqlens, start,
                interleaved, mscale, dq_in, dk_in, device_status, stream)
