"""ctypes binding of include/hb_paged.h: decode attention of rows that share
prefixes in a paged bf16 cache, the attention weight that each cached token
gets, and eviction by it.

Argument marshalling and checks only; every step runs in libhb.so.  Tensors
are used as device memory; work goes to ``stream`` (a torch stream), or to
the current stream of the tensors' device.  A bad call raises HbError (what
the library refuses) or ValueError (what only the tensors show).
"""
from __future__ import annotations

import ctypes
from typing import Sequence

import torch

from . import native
from .cache import _BF16, _I32, _check, _device, _host_pages, _int32, _page_addr, _raw_stream, _refuse, _work


class _Pool(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("num_blocks", ctypes.c_int),
                ("n_kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int)]


class _Weights(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("num_blocks", ctypes.c_int), ("n_kv_heads", ctypes.c_int)]


_bound = None


def _lib():
    global _bound
    if _bound is None:
        L = native.lib()
        vp, ci, ll, cf = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_float
        for name, args, res in (
                ("hb_decode_shared", [vp, vp, ll, vp, ci, vp, ci, ci, ci, vp, vp, ci, vp, ll, vp, ll, vp], ci),
                ("hb_decode_shared_workspace", [ci, ci, ci, ci, ci, vp, vp, ci], ll),
                ("hb_decode_weigh", [vp, vp, ll, vp, ci, vp, ci, ci, ci, ci, vp, vp, ci, cf, vp, ll, vp, ll, vp], ci),
                ("hb_decode_weigh_workspace", [ci, ci, ci, ci, ci, ci], ll),
                ("hb_evict_select", [vp, vp, ci, vp, ci, ci, ci, ci, ci, vp, vp], ci),
                ("hb_evict_move", [vp, vp, ci, vp, ci, vp, ci, ci, vp, vp, ci, vp, ci, vp], ci)):
            f = getattr(L, name)
            f.argtypes = args
            f.restype = res
        _bound = L
    return _bound


class PagedPool:
    """K and V pools, bf16 tensors [num_blocks][n_kv_heads][16][head_dim], whose memory must stay where it is.
    Read-only once made."""
    __slots__ = ("_k", "_v", "_c", "_addr", "_dev", "_kv", "_d")

    def __init__(self, k: torch.Tensor, v: torch.Tensor):
        shape = k.shape
        dev = k.get_device()
        if (len(shape) != 4 or shape[2] != 16 or v.shape != shape or k.dtype not in _BF16 or v.dtype not in _BF16
                or not k.is_contiguous() or not v.is_contiguous() or v.get_device() != dev):
            raise ValueError("the pools are contiguous bf16 tensors [num_blocks][n_kv_heads][16][head_dim] on one device")
        self._kv, self._d = shape[1], shape[3]
        self._k, self._v, self._dev = k, v, dev
        self._c = _Pool(k.data_ptr(), v.data_ptr(), shape[0], self._kv, self._d)
        self._addr = ctypes.addressof(self._c)

    k = property(lambda self: self._k)
    v = property(lambda self: self._v)
    num_blocks = property(lambda self: self._c.num_blocks)
    n_kv_heads = property(lambda self: self._kv)
    head_dim = property(lambda self: self._d)


def _weight_pool(weights, kv: int, dev: int) -> _Weights:
    shape = weights.shape
    if len(shape) != 3 or shape[1] != kv or shape[2] != 16 or weights.dtype != torch.float32 or not weights.is_contiguous():
        raise ValueError(f"weights must be a contiguous fp32 tensor [blocks][{kv}][16]")
    if dev < 0 or weights.get_device() != dev:
        raise ValueError("the tensors must lie on one CUDA device")
    return _Weights(weights.data_ptr(), shape[0], kv)


def _rows_ok(t, shape, d, heads, dev):
    return (t.shape == shape and t.dtype in _BF16 and (s := t.stride())[2] == 1 and (heads == 1 or s[1] == d)
            and t.get_device() == dev)


def _ints_ok(t, dim, n, dev):
    return t.dtype == _I32 and t.dim() == dim and t.shape[0] == n and t.is_contiguous() and t.get_device() == dev


def decode_shared_workspace(n_rows: int, n_heads: int, n_kv_heads: int, head_dim: int, max_ctx: int,
                            group_rows: Sequence[int], prefix_lens: Sequence[int]) -> int:
    r, p = _host_pages(group_rows, "group_rows"), _host_pages(prefix_lens, "prefix_lens")
    if len(r) != len(p):
        raise ValueError("group_rows and prefix_lens must have the same length")
    return _check(
        _lib().hb_decode_shared_workspace(*map(_int32, (n_rows, n_heads, n_kv_heads, head_dim, max_ctx)), _page_addr(r),
                                          _page_addr(p), len(r)), "hb_decode_shared_workspace")


def decode_shared(pool: PagedPool, q, block_tables, ctx_lens, max_ctx: int, group_rows: Sequence[int],
                  prefix_lens: Sequence[int], out, workspace=None, stream=None):
    """hb_decode_shared: q, out [n][n_heads][head_dim] bf16; block_tables int32 [n][stride], ctx_lens int32 [n] on the
    device; group_rows, prefix_lens: host lists or int32 arrays.  workspace: a tensor of at least
    decode_shared_workspace() bytes, or None for a new one (only on the current stream)."""
    if q.dim() != 3:
        raise ValueError("q must be [n][n_heads][head_dim]")
    n, heads, d = shape = q.shape
    dev = pool._dev
    r, p = _host_pages(group_rows, "group_rows"), _host_pages(prefix_lens, "prefix_lens")
    if len(r) != len(p):
        raise ValueError("group_rows and prefix_lens must have the same length")
    if (d != pool._d or dev < 0 or not _rows_ok(q, shape, d, heads, dev) or not _rows_ok(out, shape, d, heads, dev)
            or not _ints_ok(block_tables, 2, n, dev) or not _ints_ok(ctx_lens, 1, n, dev)):
        _refuse(((q, "q", n, heads, pool._d), (out, "out", n, heads, pool._d)),
                ((block_tables, "block_tables", 2, n), (ctx_lens, "ctx_lens", 1, n)))
    if not n:
        if len(r):
            _check(native.HB_EINVAL, "hb_decode_shared")
        return
    if dev != _device():
        with torch.cuda.device(dev):
            return decode_shared(pool, q, block_tables, ctx_lens, max_ctx, r, p, out, workspace, stream)
    ws = _work(workspace, stream, dev, decode_shared_workspace, n, heads, pool._kv, d, max_ctx, r, p)
    rc = _lib().hb_decode_shared(pool._addr, q.data_ptr(), q.stride(0), block_tables.data_ptr(),
                                 _int32(block_tables.shape[1]), ctx_lens.data_ptr(), _int32(n), heads, _int32(max_ctx),
                                 _page_addr(r), _page_addr(p), len(r), out.data_ptr(), out.stride(0), ws.data_ptr(),
                                 ws.nbytes, _raw_stream(dev, stream))
    if rc:
        _check(rc, "hb_decode_shared")


def decode_weigh_workspace(n_seqs: int, n_queries: int, n_heads: int, n_kv_heads: int, head_dim: int,
                           max_ctx: int) -> int:
    return _check(
        _lib().hb_decode_weigh_workspace(*map(_int32, (n_seqs, n_queries, n_heads, n_kv_heads, head_dim, max_ctx))),
        "hb_decode_weigh_workspace")


def decode_weigh(pool: PagedPool, q, block_tables, ctx_lens, max_ctx: int, weights, weight_tables, decay: float, out,
                 workspace=None, stream=None):
    """hb_decode_weigh: q, out [n * n_queries][n_heads][head_dim] bf16, n_queries rows for each of the n entries of
    ctx_lens; weights fp32 [blocks][n_kv_heads][16], updated in place; weight_tables int32 [n][stride].  workspace: as
    for decode_shared, of decode_weigh_workspace() bytes."""
    if q.dim() != 3:
        raise ValueError("q must be [n * n_queries][n_heads][head_dim]")
    rows, heads, d = shape = q.shape
    dev, n = pool._dev, ctx_lens.numel()
    nq = rows // n if n else 1
    if rows != n * nq or (n and not rows):
        raise ValueError(f"q must have a multiple of {n} rows, not {rows}")
    if (d != pool._d or dev < 0 or not _rows_ok(q, shape, d, heads, dev) or not _rows_ok(out, shape, d, heads, dev)
            or not _ints_ok(block_tables, 2, n, dev) or not _ints_ok(ctx_lens, 1, n, dev)
            or not _ints_ok(weight_tables, 2, n, dev)):
        _refuse(((q, "q", rows, heads, pool._d), (out, "out", rows, heads, pool._d)),
                ((block_tables, "block_tables", 2, n), (ctx_lens, "ctx_lens", 1, n),
                 (weight_tables, "weight_tables", 2, n)))
    w = _weight_pool(weights, pool._kv, dev)
    if not n:
        return
    if dev != _device():
        with torch.cuda.device(dev):
            return decode_weigh(pool, q, block_tables, ctx_lens, max_ctx, weights, weight_tables, decay, out, workspace,
                                stream)
    ws = _work(workspace, stream, dev, decode_weigh_workspace, n, nq, heads, pool._kv, d, max_ctx)
    rc = _lib().hb_decode_weigh(pool._addr, q.data_ptr(), q.stride(0), block_tables.data_ptr(),
                                _int32(block_tables.shape[1]), ctx_lens.data_ptr(), _int32(n), _int32(nq), heads,
                                _int32(max_ctx), ctypes.addressof(w), weight_tables.data_ptr(),
                                _int32(weight_tables.shape[1]), decay, out.data_ptr(), out.stride(0), ws.data_ptr(),
                                ws.nbytes, _raw_stream(dev, stream))
    if rc:
        _check(rc, "hb_decode_weigh")


def evict_select(weights, weight_tables, lens, max_len: int, keep: int, n_first: int, n_recent: int, kept, stream=None):
    """hb_evict_select: weights fp32 [blocks][n_kv_heads][16]; weight_tables int32 [n][stride], lens int32 [n] on the
    device; kept int32 [n][n_kv_heads][keep] receives the positions that stay, ascending, then -1."""
    if weights.dim() != 3:
        raise ValueError("weights must be [blocks][n_kv_heads][16]")
    dev, kv, n = weights.get_device(), weights.shape[1], lens.numel()
    w = _weight_pool(weights, kv, dev)
    if not _ints_ok(weight_tables, 2, n, dev) or not _ints_ok(lens, 1, n, dev) or not _ints_ok(kept, 3, n, dev):
        _refuse((), ((weight_tables, "weight_tables", 2, n), (lens, "lens", 1, n), (kept, "kept", 3, n)))
    if kept.shape != (n, kv, keep):
        raise ValueError(f"kept must be [{n}][{kv}][{keep}], not {list(kept.shape)}")
    if dev != _device():
        with torch.cuda.device(dev):
            return evict_select(weights, weight_tables, lens, max_len, keep, n_first, n_recent, kept, stream)
    rc = _lib().hb_evict_select(ctypes.addressof(w), weight_tables.data_ptr(), _int32(weight_tables.shape[1]),
                                lens.data_ptr(), _int32(n), _int32(max_len), _int32(keep), _int32(n_first),
                                _int32(n_recent), kept.data_ptr(), _raw_stream(dev, stream))
    if rc:
        _check(rc, "hb_evict_select")


def evict_move(pool: PagedPool, block_tables, new_tables, kept, weights=None, weight_tables=None,
               new_weight_tables=None, stream=None):
    """hb_evict_move: slot i of new_tables gets K and V (and, with weights, the weight) of slot kept[.., i] of
    block_tables.  Tables int32 [n][stride], kept int32 [n][n_kv_heads][keep] on the device, as evict_select writes
    it."""
    dev, kv = pool._dev, pool._kv
    if kept.dim() != 3 or kept.shape[1] != kv:
        raise ValueError(f"kept must be [n][{kv}][keep]")
    n, _, keep = kept.shape
    if dev < 0 or not _ints_ok(kept, 3, n, dev) or not _ints_ok(block_tables, 2, n, dev) or not _ints_ok(new_tables, 2, n, dev):
        _refuse((), ((kept, "kept", 3, n), (block_tables, "block_tables", 2, n), (new_tables, "new_tables", 2, n)))
    w, args = None, (None, 0, None, 0)
    if weights is not None:
        if weight_tables is None or new_weight_tables is None:
            raise ValueError("weights are moved between weight_tables and new_weight_tables")
        w = _weight_pool(weights, kv, dev)
        if not _ints_ok(weight_tables, 2, n, dev) or not _ints_ok(new_weight_tables, 2, n, dev):
            _refuse((), ((weight_tables, "weight_tables", 2, n), (new_weight_tables, "new_weight_tables", 2, n)))
        args = (weight_tables.data_ptr(), _int32(weight_tables.shape[1]), new_weight_tables.data_ptr(),
                _int32(new_weight_tables.shape[1]))
    elif weight_tables is not None or new_weight_tables is not None:
        raise ValueError("the tables of weights come with the weights")
    if dev != _device():
        with torch.cuda.device(dev):
            return evict_move(pool, block_tables, new_tables, kept, weights, weight_tables, new_weight_tables, stream)
    rc = _lib().hb_evict_move(pool._addr, block_tables.data_ptr(), _int32(block_tables.shape[1]), new_tables.data_ptr(),
                              _int32(new_tables.shape[1]), kept.data_ptr(), _int32(n), _int32(keep),
                              None if w is None else ctypes.addressof(w), *args, _raw_stream(dev, stream))
    if rc:
        _check(rc, "hb_evict_move")
