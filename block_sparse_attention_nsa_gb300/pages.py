"""Binding of the life of a cache's pages (include/nsa_kv4.h): rows of the block table forked and
freed, the pool compacted, pages copied.

Argument marshalling only.  All tensors are contiguous and live on the current device; lists that
are not given are allocated on the launching stream.  seq_lens and the block table are updated in
place, and so are shares (int32 [num_pages], rows that name a page beyond the first; zeros at the
beginning) and the free list.  Its head is read from free_head and written to head_out, which may be
the same tensor.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from .kv4 import _check, _device, _empty, _fail, _held, _i32, _ints, _lib, _raw, _status

__all__ = ["page_fork", "page_free", "page_compact", "page_copy"]


class PageOpsDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("num_seqs", "page_size", "table_width", "num_pages",
                                              "num_free", "count")]


def signatures():
    """ctypes result and argument types of the library's functions."""
    vp, i32, i64, st = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_int
    pd = ctypes.POINTER(PageOpsDims)
    return {
        "nsa_page_fork": (st, [pd] + [vp] * 13),
        "nsa_page_free": (st, [pd] + [vp] * 9),
        "nsa_page_compact": (st, [pd] + [vp] * 11),
        "nsa_page_copy": (st, [i32, i64, i32, vp, vp, vp, vp, vp]),
    }


@functools.lru_cache(maxsize=4096)
def _dims(*sizes):
    return PageOpsDims(*_held(sizes, "page dims"))


def _state(block_table, seq_lens, shares, free_pages):
    """The device and the sizes of a cache's state."""
    dev = _device(block_table)
    b, width = block_table.shape
    pages, free = shares.numel(), free_pages.numel()
    _ints("block_table", block_table, b * width, dev)
    _ints("seq_lens", seq_lens, b, dev)
    _ints("shares", shares, pages, dev)
    _ints("free_pages", free_pages, free, dev)
    return dev, b, width, pages, free


def _list(name, t, n, dev, stream):
    if t is None:
        return _empty((n,), _i32, dev, stream)
    _ints(name, t, n, dev)
    return t


def page_fork(block_table, seq_lens, parents, children, page_size: int, shares, free_pages,
              free_head, fork_lens=None, copy_src=None, copy_dst=None, head_out=None,
              device_status=None, stream=None):
    """Makes rows children int32 [n] continuations of rows parents int32 [n], behind their first
    fork_lens int32 [n] tokens (None: all).  Full pages are shared; a partly full last page gets a
    page of the free list in its place.  Returns copy_src, copy_dst int32 [n], what page_copy then
    has to copy in each pool (-1: nothing), and head_out [1]."""
    dev, b, width, pages, free = _state(block_table, seq_lens, shares, free_pages)
    n = parents.numel()
    _ints("parents", parents, n, dev)
    _ints("children", children, n, dev)
    _ints("free_head", free_head, 1, dev)
    lens = None
    if fork_lens is not None:
        _ints("fork_lens", fork_lens, n, dev)
        lens = fork_lens.data_ptr()
    copy_src = _list("copy_src", copy_src, n, dev, stream)
    copy_dst = _list("copy_dst", copy_dst, n, dev, stream)
    head_out = _list("head_out", head_out, 1, dev, stream)
    code = _lib().nsa_page_fork(
        _dims(b, page_size, width, pages, free, n), block_table.data_ptr(), seq_lens.data_ptr(),
        parents.data_ptr(), children.data_ptr(), lens, shares.data_ptr(), free_pages.data_ptr(),
        free_head.data_ptr(), copy_src.data_ptr(), copy_dst.data_ptr(), head_out.data_ptr(),
        None if device_status is None else _status(device_status, dev), _raw(stream, dev))
    if code:
        _fail(code, "page_fork")
    return copy_src, copy_dst, head_out


def page_free(block_table, seq_lens, rows, page_size: int, shares, free_pages, free_head,
              head_out=None, device_status=None, stream=None):
    """Frees rows int32 [n]: pages that no other row names go to the free list, in ascending order,
    before its head; the rows' entries become -1, their lengths 0.  Returns head_out [1]."""
    dev, b, width, pages, free = _state(block_table, seq_lens, shares, free_pages)
    n = rows.numel()
    _ints("rows", rows, n, dev)
    _ints("free_head", free_head, 1, dev)
    head_out = _list("head_out", head_out, 1, dev, stream)
    code = _lib().nsa_page_free(
        _dims(b, page_size, width, pages, free, n), block_table.data_ptr(), seq_lens.data_ptr(),
        rows.data_ptr(), shares.data_ptr(), free_pages.data_ptr(), free_head.data_ptr(),
        head_out.data_ptr(), None if device_status is None else _status(device_status, dev),
        _raw(stream, dev))
    if code:
        _fail(code, "page_free")
    return head_out


def page_compact(block_table, seq_lens, page_size: int, shares, free_pages, table_out=None,
                 shares_out=None, free_out=None, copy_src=None, copy_dst=None, head_out=None,
                 device_status=None, stream=None):
    """Moves the pages that rows name to the pool's beginning.  table_out, shares_out and free_out
    (None: block_table, shares, free_pages, in place) get the new ids, counts and free list, which
    is rebuilt: pages that no row names count as free.  Returns copy_src, copy_dst (given, or int32
    [num_pages // 2]), the moves that page_copy then has to make in each pool, -1 behind them, and
    head_out [1]."""
    dev, b, width, pages, free = _state(block_table, seq_lens, shares, free_pages)
    if table_out is None:
        table_out = block_table
    else:
        _check("table_out", table_out, _i32, block_table.shape, dev)
    if shares_out is None:
        shares_out = shares
    else:
        _ints("shares_out", shares_out, pages, dev)
    if free_out is None:
        free_out = free_pages
    else:
        _ints("free_out", free_out, free, dev)
    given = copy_src if copy_src is not None else copy_dst
    n = pages // 2 if given is None else given.numel()
    copy_src = _list("copy_src", copy_src, n, dev, stream)
    copy_dst = _list("copy_dst", copy_dst, n, dev, stream)
    head_out = _list("head_out", head_out, 1, dev, stream)
    code = _lib().nsa_page_compact(
        _dims(b, page_size, width, pages, free, n), block_table.data_ptr(), seq_lens.data_ptr(),
        shares.data_ptr(), table_out.data_ptr(), shares_out.data_ptr(), free_out.data_ptr(),
        copy_src.data_ptr(), copy_dst.data_ptr(), head_out.data_ptr(),
        None if device_status is None else _status(device_status, dev), _raw(stream, dev))
    if code:
        _fail(code, "page_compact")
    return copy_src, copy_dst, head_out


def page_copy(pool, copy_src, copy_dst, device_status=None, stream=None):
    """Copies pages of a pool [num_pages, ...] (contiguous, of any dtype; a page is a multiple of 16
    bytes): page copy_src[i] to page copy_dst[i], int32 [n]; pairs of -1 are skipped.  A page is the
    destination of one pair at most, and no source then.  Returns pool."""
    dev = _device(pool)
    if pool.dim() < 2 or not pool.is_contiguous():
        raise ValueError("pool: a contiguous tensor [num_pages, ...] expected")
    n, pages = copy_src.numel(), pool.shape[0]
    _ints("copy_src", copy_src, n, dev)
    _ints("copy_dst", copy_dst, n, dev)
    _held((n, pages), "page_copy")
    size = pool.numel() // pages * pool.element_size() if pages else 16
    code = _lib().nsa_page_copy(pages, size, n, pool.data_ptr(), copy_src.data_ptr(),
                                copy_dst.data_ptr(),
                                None if device_status is None else _status(device_status, dev),
                                _raw(stream, dev))
    if code:
        _fail(code, "page_copy")
    return pool
