"""Binding of the 4-bit paged KV cache (include/nsa_kv4.h): block tables and slot maps,
rows written and read back, one-step decode over the pages.

Argument marshalling only, as in the package's other calls.  All tensors are contiguous
(k and v of kv4_append may be strided) and live on the current device; outputs that are
not given are allocated on the launching stream.  device_status, where given, is an int32
tensor of one element into which the device ORs its error bits.
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional

import torch

__all__ = ["page_plan", "page_slots", "kv4_pool", "kv4_append", "kv4_read", "kv4_decode",
           "kv4_decode_workspace_size", "DEVERR_BAD_INDEX", "DEVERR_BAD_SEQLENS",
           "DEVERR_NO_PAGES"]

DEVERR_BAD_INDEX, DEVERR_BAD_SEQLENS, DEVERR_NO_PAGES = 1, 2, 8
_DTYPES = {torch.bfloat16: 0, torch.float16: 1}


class PageDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("num_seqs", "page_size", "table_width", "num_pages",
                                              "num_free", "max_slots")]


class Kv4Dims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("num_pages", "page_size", "h_k", "head_dim",
                                              "dtype")]


def signatures():
    """ctypes result and argument types of the library's functions."""
    vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    sz, f32, st = ctypes.c_size_t, ctypes.c_float, ctypes.c_int
    pd, kd = ctypes.POINTER(PageDims), ctypes.POINTER(Kv4Dims)
    psz = ctypes.POINTER(sz)
    return {
        "nsa_page_plan": (st, [pd] + [vp] * 11),
        "nsa_page_slots": (st, [pd] + [vp] * 7),
        "nsa_kv4_page_bytes": (st, [kd, psz]),
        "nsa_kv4_append": (st, [kd, i32, vp, i64, i64, vp, i64, i64, vp, vp, vp, vp]),
        "nsa_kv4_read": (st, [kd, i32, vp, vp, vp, vp, vp, vp]),
        "nsa_kv4_decode": (st, [kd, i32, i32, i32, i32, i32, vp, vp, vp, vp, vp, f32, vp, vp, vp,
                                vp, sz, vp]),
        "nsa_kv4_decode_workspace_size": (st, [kd, i32, i32, i32, psz]),
    }


_handle = None


def _lib():
    global _handle
    if _handle is None:
        from . import load
        _handle = load()
    return _handle


def _fail(code: int, where: str):
    from . import NsaError
    raise NsaError(code, where)


def _held(sizes, where):
    """ctypes would wrap what 32 bits do not hold."""
    if not all(-2 ** 31 <= x < 2 ** 31 for x in sizes):
        _fail(2, f"{where}: sizes {sizes} beyond 32 bits")
    return sizes


@functools.lru_cache(maxsize=4096)
def _page_dims(*sizes):
    return PageDims(*_held(sizes, "page dims"))


@functools.lru_cache(maxsize=4096)
def _kv4_dims(*sizes):
    return Kv4Dims(*_held(sizes, "kv4 dims"))


_current_device = torch.cuda.current_device
# The current stream's handle without a Stream object around it; builds of
# torch without CUDA do not have this name.
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                          lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _check(name, t, dtype, shape, dev):
    """A contiguous tensor of this dtype and shape on the current device."""
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.get_device() != dev:
        raise ValueError(f"{name}: a contiguous {dtype} tensor {tuple(shape)} on device {dev} "
                         f"expected, got {t.dtype} {tuple(t.shape)}, strides {t.stride()}, on "
                         f"{t.device}")


_i32 = torch.int32


def _ints(name, t, n, dev):
    """A contiguous int32 tensor of n entries on the current device (cheaper than _check)."""
    if t.dtype is not _i32 or t.numel() != n or t.get_device() != dev or not t.is_contiguous():
        _check(name, t, _i32, (n,), dev)


def _device(t):
    """The index of t's device, which has to be the current one."""
    dev = t.get_device()
    if dev < 0 or dev != _current_device():
        raise ValueError(f"tensors have to be on the current CUDA device, got {t.device}")
    return dev


def _raw(stream, dev):
    return _current_stream(dev) if stream is None else stream.cuda_stream


def _empty(shape, dtype, dev, stream):
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):   # the block belongs to the stream that uses it
        return torch.empty(shape, dtype=dtype, device=dev)


def _status(t, dev):
    if t is None:
        return None
    _ints("device_status", t, 1, dev)
    return t.data_ptr()


def _slot_map(slot_map, dev, stream):
    """slot_map (or a new one of that many entries) and its length."""
    if isinstance(slot_map, int):
        return _empty((slot_map,), _i32, dev, stream), slot_map
    n = slot_map.numel()
    _ints("slot_map", slot_map, n, dev)
    return slot_map, n


def page_plan(ctx_lens, new_lens, free_pages, free_head, block_table, page_size: int,
              num_pages: int, slot_map, seq_lens=None, cu_new=None, head_out=None,
              device_status=None, stream=None):
    """Gives the new tokens of a step their pages and slots.

    ctx_lens, new_lens int32 [B]: tokens cached and tokens brought; free_pages int32 [F],
    used from entry free_head[0] on; block_table int32 [B, W], updated in place; slot_map
    int32 [M] or its length M.  Returns slot_map (packed in request order, -1 behind the
    last token), seq_lens = ctx + new (may be ctx_lens), cu_new [B + 1] and head_out [1]
    (may be free_head)."""
    dev = _device(block_table)
    b, width = block_table.shape
    free = free_pages.numel()
    _ints("block_table", block_table, b * width, dev)
    _ints("ctx_lens", ctx_lens, b, dev)
    _ints("new_lens", new_lens, b, dev)
    _ints("free_pages", free_pages, free, dev)
    _ints("free_head", free_head, 1, dev)
    slot_map, slots = _slot_map(slot_map, dev, stream)
    if seq_lens is None:
        seq_lens = _empty((b,), _i32, dev, stream)
    else:
        _ints("seq_lens", seq_lens, b, dev)
    if cu_new is None:
        cu_new = _empty((b + 1,), _i32, dev, stream)
    else:
        _ints("cu_new", cu_new, b + 1, dev)
    if head_out is None:
        head_out = _empty((1,), _i32, dev, stream)
    else:
        _ints("head_out", head_out, 1, dev)
    code = _lib().nsa_page_plan(
        _page_dims(b, page_size, width, num_pages, free, slots), ctx_lens.data_ptr(),
        new_lens.data_ptr(), free_pages.data_ptr(), free_head.data_ptr(), block_table.data_ptr(),
        slot_map.data_ptr(), seq_lens.data_ptr(), cu_new.data_ptr(), head_out.data_ptr(),
        None if device_status is None else _status(device_status, dev), _raw(stream, dev))
    if code:
        _fail(code, "page_plan")
    return slot_map, seq_lens, cu_new, head_out


def page_slots(block_table, start, count, page_size: int, num_pages: int, slot_map, cu=None,
               device_status=None, stream=None):
    """Slots of cached tokens: positions start[b] ... start[b] + count[b] - 1 of each
    request, packed in request order, -1 behind the last.  slot_map int32 [M] or its length
    M.  Returns slot_map and cu int32 [B + 1], the requests' offsets in it."""
    dev = _device(block_table)
    b, width = block_table.shape
    _ints("block_table", block_table, b * width, dev)
    _ints("start", start, b, dev)
    _ints("count", count, b, dev)
    slot_map, slots = _slot_map(slot_map, dev, stream)
    if cu is None:
        cu = _empty((b + 1,), _i32, dev, stream)
    else:
        _ints("cu", cu, b + 1, dev)
    code = _lib().nsa_page_slots(
        _page_dims(b, page_size, width, num_pages, 0, slots), block_table.data_ptr(),
        start.data_ptr(), count.data_ptr(), slot_map.data_ptr(), cu.data_ptr(),
        None if device_status is None else _status(device_status, dev), _raw(stream, dev))
    if code:
        _fail(code, "page_slots")
    return slot_map, cu


def kv4_pool(num_pages: int, page_size: int, h_k: int, head_dim: int, device="cuda"):
    """A pool of pages, uint8 [num_pages, h_k, page_bytes], zeroed."""
    size = ctypes.c_size_t()
    code = _lib().nsa_kv4_page_bytes(_kv4_dims(num_pages, page_size, h_k, head_dim, 0),
                                     ctypes.byref(size))
    if code:
        _fail(code, "kv4_pool")
    return torch.zeros((num_pages, h_k, size.value), dtype=torch.uint8, device=device)


@functools.lru_cache(maxsize=4096)
def _pool_layout(shape, head_dim, dtype, where):
    """Kv4Dims of a pool's shape: its page size follows from the bytes of a page."""
    pages, h_k, size = shape
    page_size, rest = divmod(size, head_dim + head_dim // 8)
    if rest:
        raise ValueError(f"pool: {size} bytes a page are no whole tokens of head_dim {head_dim}")
    code = _DTYPES.get(dtype)
    if code is None:
        _fail(2, f"{where}: dtype {dtype}")
    return _kv4_dims(pages, page_size, h_k, head_dim, code)


def _pool_dims(pool, head_dim, dtype, where):
    dev = _device(pool)
    shape = pool.shape
    if pool.dtype is not torch.uint8 or len(shape) != 3 or not pool.is_contiguous():
        raise ValueError("pool: a contiguous uint8 tensor [num_pages, h_k, page_bytes] expected")
    return _pool_layout(shape, head_dim, dtype, where), dev


def kv4_append(pool, k, v, slot_map, device_status=None, stream=None):
    """Quantises the rows of k and v [n, h_k, d] into the slots of slot_map int32 [n] (-1: no
    slot).  k and v may be strided views whose last dimension is contiguous.  Each slot at
    most once.  Returns pool."""
    shape, dtype = k.shape, k.dtype
    if len(shape) != 3 or shape != v.shape or dtype is not v.dtype:
        raise ValueError("k and v of one shape [n, h_k, d] and dtype expected")
    n, h_k, d = shape
    dims, dev = _pool_dims(pool, d, dtype, "kv4_append")
    if h_k != dims.h_k:
        raise ValueError(f"k has {h_k} heads, the pool {dims.h_k}")
    (kt, kh, ke), (vt, vh, ve) = k.stride(), v.stride()
    if ke != 1 or ve != 1 or k.get_device() != dev or v.get_device() != dev:
        raise ValueError("k and v need a contiguous last dimension, on the pool's device")
    _ints("slot_map", slot_map, n, dev)
    if n >> 31:
        _fail(2, "kv4_append: rows beyond 32 bits")
    code = _lib().nsa_kv4_append(dims, n, k.data_ptr(), kt, kh, v.data_ptr(), vt, vh,
                                 slot_map.data_ptr(), pool.data_ptr(),
                                 None if device_status is None else _status(device_status, dev),
                                 _raw(stream, dev))
    if code:
        _fail(code, "kv4_append")
    return pool


def kv4_read(pool, slot_map, head_dim: int, k=None, v=None, dtype: torch.dtype = torch.bfloat16,
             device_status=None, stream=None):
    """The cached rows of slot_map int32 [n] as k, v [n, h_k, head_dim] (zeros where the slot
    is -1), in the dtype of k where it is given.  head_dim has to be the one that the pool was
    made for: the pool's bytes do not say (64 tokens of 128 dimensions are as many as 128 of 64)."""
    if k is not None:
        dtype = k.dtype
    dims, dev = _pool_dims(pool, head_dim, dtype, "kv4_read")
    n = slot_map.numel()
    _ints("slot_map", slot_map, n, dev)
    if n >> 31:
        _fail(2, "kv4_read: rows beyond 32 bits")
    shape = (n, dims.h_k, head_dim)
    if k is None:
        k = _empty(shape, dtype, dev, stream)
    else:
        _check("k", k, dtype, shape, dev)
    if v is None:
        v = _empty(shape, dtype, dev, stream)
    else:
        _check("v", v, dtype, shape, dev)
    code = _lib().nsa_kv4_read(dims, n, pool.data_ptr(), slot_map.data_ptr(), k.data_ptr(),
                               v.data_ptr(),
                               None if device_status is None else _status(device_status, dev),
                               _raw(stream, dev))
    if code:
        _fail(code, "kv4_read")
    return k, v


@functools.lru_cache(maxsize=4096)
def _decode_workspace(dims_key, num_seqs, h_q, topk):
    size = ctypes.c_size_t()
    code = _lib().nsa_kv4_decode_workspace_size(_kv4_dims(*dims_key), num_seqs, h_q, topk,
                                                ctypes.byref(size))
    if code:
        _fail(code, "kv4_decode_workspace_size")
    return size.value


def kv4_decode_workspace_size(num_pages: int, page_size: int, h_k: int, head_dim: int,
                              num_seqs: int, h_q: int, topk: int = 0) -> int:
    """Workspace bytes of kv4_decode (topk 0: without a selection)."""
    return _decode_workspace((num_pages, page_size, h_k, head_dim, 0), num_seqs, h_q, topk)


def kv4_decode(q, pool, block_table, seq_lens, scale: float, sel_idx=None, window: int = 0,
               out=None, lse=None, workspace: Optional[torch.Tensor] = None, device_status=None,
               stream=None):
    """One-step decode over the pages: q [B, h_q, d], the last token of each sequence, attends
    to its cached keys: to the blocks (pages) of sel_idx int32 [h_k, B, T], or to all where
    it is None, within the last `window` tokens where that is > 0.  Returns out [B, h_q, d]
    and lse float32 [h_q, B].  workspace: uint8, at least kv4_decode_workspace_size bytes;
    allocated here when None and needed."""
    shape, dtype = q.shape, q.dtype
    if len(shape) != 3:
        raise ValueError("q [B, h_q, d] expected")
    b, h_q, d = shape
    dims, dev = _pool_dims(pool, d, dtype, "kv4_decode")
    h_k = dims.h_k
    if not q.is_contiguous() or q.get_device() != dev:
        _check("q", q, dtype, shape, dev)
    rows, width = block_table.shape
    if rows != b:
        raise ValueError(f"block_table of {rows} rows for {b} sequences")
    _ints("block_table", block_table, b * width, dev)
    _ints("seq_lens", seq_lens, b, dev)
    topk, sel = 0, None
    if sel_idx is not None:
        topk, sel = sel_idx.shape[-1], sel_idx.data_ptr()
        _check("sel_idx", sel_idx, _i32, (h_k, b, topk), dev)
        if topk == 0:
            raise ValueError("sel_idx: at least one slot expected")
    if out is None:
        out = _empty(shape, dtype, dev, stream)
    else:
        _check("out", out, dtype, shape, dev)
    if lse is None:
        lse = _empty((h_q, b), torch.float32, dev, stream)
    else:
        _check("lse", lse, torch.float32, (h_q, b), dev)
    if workspace is None:
        need = _decode_workspace((dims.num_pages, dims.page_size, h_k, d, dims.dtype), b, h_q, topk)
        if need:
            workspace = _empty((need,), torch.uint8, dev, stream)
    else:
        if (workspace.dtype is not torch.uint8 or not workspace.is_contiguous()
                or workspace.get_device() != dev):
            _check("workspace", workspace, torch.uint8, workspace.shape, dev)
    if not -1 < window < 0x7fffffff:      # beyond every length, or negative (refused below)
        window = 0x7fffffff if window > 0 else -1
    if width >> 31 or b >> 31:
        _fail(2, "kv4_decode: sizes beyond 32 bits")
    ws, ws_bytes = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel())
    code = _lib().nsa_kv4_decode(
        dims, b, h_q, width, topk, window, q.data_ptr(), pool.data_ptr(), block_table.data_ptr(),
        seq_lens.data_ptr(), sel, scale, out.data_ptr(), lse.data_ptr(),
        None if device_status is None else _status(device_status, dev), ws, ws_bytes,
        _raw(stream, dev))
    if code:
        _fail(code, "kv4_decode")
    return out, lse
