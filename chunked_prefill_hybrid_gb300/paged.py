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
import struct
from operator import index
from typing import Sequence

import torch

from . import native
from .cache import _BF16, _I32, _check, _device, _host_pages, _int32, _raw_stream, _refuse, _work

_F32 = torch.float32
_MOST = 0x7FFFFFFF
# hb_paged_pool and hb_weight_pool: packed bytes take a third of a ctypes structure's time
_pack_pool = struct.Struct("@PPiii4x").pack
_pack_weights = struct.Struct("@Pii").pack

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
                ("hb_paged_test_lost_block", [], None),
                ("hb_evict_select", [vp, vp, ci, vp, ci, ci, ci, ci, ci, vp, vp], ci),
                ("hb_evict_move", [vp, vp, ci, vp, ci, vp, ci, ci, vp, vp, ci, vp, ci, vp], ci)):
            f = getattr(L, name)
            f.argtypes = args
            f.restype = res
        _bound = L
    return _bound


# As in cache.py, each call looks at its tensors in one expression (most of a
# small call's time is the host's) and says what is wrong in _refuse.  Kernels
# launch on the current device, so a call on tensors of another one makes that
# current first.


class PagedPool:
    """K and V pools, bf16 tensors [num_blocks][n_kv_heads][16][head_dim], whose memory must stay where it is.
    Read-only once made."""
    __slots__ = ("_k", "_v", "_c", "_dev", "_kv", "_d")

    def __init__(self, k: torch.Tensor, v: torch.Tensor):
        shape = k.shape
        self._dev = dev = k.get_device()
        if (len(shape) != 4 or shape[2] != 16 or v.shape != shape or k.dtype not in _BF16 or v.dtype not in _BF16
                or not k.is_contiguous() or not v.is_contiguous() or v.get_device() != dev):
            raise ValueError("the pools are contiguous bf16 tensors [num_blocks][n_kv_heads][16][head_dim] on one device")
        blocks, self._kv, _, self._d = shape
        self._k, self._v = k, v
        self._c = _pack_pool(k.data_ptr(), v.data_ptr(), _int32(blocks), self._kv, self._d)

    k = property(lambda self: self._k)
    v = property(lambda self: self._v)
    num_blocks = property(lambda self: self._k.shape[0])
    n_kv_heads = property(lambda self: self._kv)
    head_dim = property(lambda self: self._d)


def _weight_pool(weights, kv: int, dev: int) -> bytes:
    shape = weights.shape
    if (len(shape) != 3 or shape[1] != kv or shape[2] != 16 or weights.dtype != _F32 or not weights.is_contiguous()
            or dev < 0 or weights.get_device() != dev):
        if dev < 0 or weights.get_device() != dev:
            raise ValueError("the tensors must lie on one CUDA device")
        raise ValueError(f"weights must be a contiguous fp32 tensor [blocks][{kv}][16]")
    return _pack_weights(weights.data_ptr(), _int32(shape[0]), kv)


def _groups(group_rows, prefix_lens):
    r, p = _host_pages(group_rows, "group_rows"), _host_pages(prefix_lens, "prefix_lens")
    n = len(r)
    if n != len(p):
        raise ValueError("group_rows and prefix_lens must have the same length")
    return r.tobytes(), p.tobytes(), n


def _shared_workspace(n, heads, kv, d, max_ctx, rows, prefix, groups) -> int:
    return _check(_lib().hb_decode_shared_workspace(n, heads, kv, d, max_ctx, rows, prefix, groups),
                  "hb_decode_shared_workspace")


def decode_shared_workspace(n_rows: int, n_heads: int, n_kv_heads: int, head_dim: int, max_ctx: int,
                            group_rows: Sequence[int], prefix_lens: Sequence[int]) -> int:
    return _shared_workspace(*map(_int32, (n_rows, n_heads, n_kv_heads, head_dim, max_ctx)),
                             *_groups(group_rows, prefix_lens))


def decode_shared(pool: PagedPool, q, block_tables, ctx_lens, max_ctx: int, group_rows: Sequence[int],
                  prefix_lens: Sequence[int], out, workspace=None, stream=None):
    """hb_decode_shared: q, out [n][n_heads][head_dim] bf16; block_tables int32 [n][stride], ctx_lens int32 [n] on the
    device; group_rows, prefix_lens: host lists or int32 arrays.  workspace: a tensor of at least
    decode_shared_workspace() bytes, or None for a new one (only on the current stream)."""
    shape, tshape = q.shape, block_tables.shape
    if len(shape) != 3:
        raise ValueError("q must be [n][n_heads][head_dim]")
    n, heads, d = shape
    dev = pool._dev
    rows, prefix, groups = _groups(group_rows, prefix_lens)
    if (d != pool._d or out.shape != shape or q.dtype not in _BF16 or out.dtype not in _BF16
            or (qs := q.stride())[2] != 1 or (os_ := out.stride())[2] != 1
            or (heads > 1 and (qs[1] != d or os_[1] != d)) or len(tshape) != 2 or tshape[0] != n
            or ctx_lens.shape != tshape[:1] or block_tables.dtype != _I32 or ctx_lens.dtype != _I32
            or not block_tables.is_contiguous() or not ctx_lens.is_contiguous() or dev < 0 or q.get_device() != dev
            or out.get_device() != dev or block_tables.get_device() != dev or ctx_lens.get_device() != dev):
        _refuse(((q, "q", n, heads, pool._d), (out, "out", n, heads, pool._d)),
                ((block_tables, "block_tables", 2, n), (ctx_lens, "ctx_lens", 1, n)))
    max_ctx = index(max_ctx)
    if tshape[1] > _MOST or n > _MOST or not -_MOST <= max_ctx <= _MOST:
        raise native.HbError(native.HB_ERANGE, "a size does not fit 32 bits")
    if not n:
        if groups:
            _check(native.HB_EINVAL, "hb_decode_shared")
        return
    if dev != _device():
        with torch.cuda.device(dev):
            return decode_shared(pool, q, block_tables, ctx_lens, max_ctx, group_rows, prefix_lens, out, workspace, stream)
    ws = _work(workspace, stream, dev, _shared_workspace, n, heads, pool._kv, d, max_ctx, rows, prefix, groups)
    rc = _lib().hb_decode_shared(pool._c, q.data_ptr(), qs[0], block_tables.data_ptr(), tshape[1], ctx_lens.data_ptr(), n,
                                 heads, max_ctx, rows, prefix, groups, out.data_ptr(), os_[0], ws.data_ptr(), ws.nbytes,
                                 _raw_stream(dev, stream))
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
    shape, tshape, wshape = q.shape, block_tables.shape, weight_tables.shape
    if len(shape) != 3:
        raise ValueError("q must be [n * n_queries][n_heads][head_dim]")
    rows, heads, d = shape
    dev, n = pool._dev, ctx_lens.numel()
    nq = rows // n if n else 1
    if rows != n * nq or (n and not rows):
        raise ValueError(f"q must have a multiple of {n} rows, not {rows}")
    if (d != pool._d or out.shape != shape or q.dtype not in _BF16 or out.dtype not in _BF16
            or (qs := q.stride())[2] != 1 or (os_ := out.stride())[2] != 1
            or (heads > 1 and (qs[1] != d or os_[1] != d)) or len(tshape) != 2 or tshape[0] != n or len(wshape) != 2
            or wshape[0] != n or ctx_lens.dim() != 1 or block_tables.dtype != _I32 or ctx_lens.dtype != _I32
            or weight_tables.dtype != _I32 or not block_tables.is_contiguous() or not ctx_lens.is_contiguous()
            or not weight_tables.is_contiguous() or dev < 0 or q.get_device() != dev or out.get_device() != dev
            or block_tables.get_device() != dev or ctx_lens.get_device() != dev or weight_tables.get_device() != dev):
        _refuse(((q, "q", rows, heads, pool._d), (out, "out", rows, heads, pool._d)),
                ((block_tables, "block_tables", 2, n), (ctx_lens, "ctx_lens", 1, n),
                 (weight_tables, "weight_tables", 2, n)))
    w = _weight_pool(weights, pool._kv, dev)
    max_ctx = index(max_ctx)
    if tshape[1] > _MOST or wshape[1] > _MOST or rows > _MOST or not -_MOST <= max_ctx <= _MOST:
        raise native.HbError(native.HB_ERANGE, "a size does not fit 32 bits")
    if not n:
        return
    if dev != _device():
        with torch.cuda.device(dev):
            return decode_weigh(pool, q, block_tables, ctx_lens, max_ctx, weights, weight_tables, decay, out, workspace,
                                stream)
    ws = _work(workspace, stream, dev, decode_weigh_workspace, n, nq, heads, pool._kv, d, max_ctx)
    rc = _lib().hb_decode_weigh(pool._c, q.data_ptr(), qs[0], block_tables.data_ptr(), tshape[1], ctx_lens.data_ptr(), n,
                                nq, heads, max_ctx, w, weight_tables.data_ptr(), wshape[1], decay, out.data_ptr(),
                                os_[0], ws.data_ptr(), ws.nbytes, _raw_stream(dev, stream))
    if rc:
        _check(rc, "hb_decode_weigh")


def paged_test_lost_block():
    """Test hook: this thread's next decode_shared or decode_weigh that attends keys for several rows at once loses a
    copy, and its waits for it run out."""
    _lib().hb_paged_test_lost_block()


def evict_select(weights, weight_tables, lens, max_len: int, keep: int, n_first: int, n_recent: int, kept, stream=None):
    """hb_evict_select: weights fp32 [blocks][n_kv_heads][16]; weight_tables int32 [n][stride], lens int32 [n] on the
    device; kept int32 [n][n_kv_heads][keep] receives the positions that stay, ascending, then -1."""
    shape, tshape, kshape = weights.shape, weight_tables.shape, kept.shape
    dev, n = weights.get_device(), lens.numel()
    w = _weight_pool(weights, shape[1] if len(shape) == 3 else 0, dev)
    if (len(tshape) != 2 or tshape[0] != n or lens.dim() != 1 or len(kshape) != 3 or kshape[0] != n
            or weight_tables.dtype != _I32 or lens.dtype != _I32 or kept.dtype != _I32
            or not weight_tables.is_contiguous() or not lens.is_contiguous() or not kept.is_contiguous()
            or weight_tables.get_device() != dev or lens.get_device() != dev or kept.get_device() != dev):
        _refuse((), ((weight_tables, "weight_tables", 2, n), (lens, "lens", 1, n), (kept, "kept", 3, n)))
    if kshape[1] != shape[1] or kshape[2] != keep:
        raise ValueError(f"kept must be [{n}][{shape[1]}][{keep}], not {list(kshape)}")
    if dev != _device():
        with torch.cuda.device(dev):
            return evict_select(weights, weight_tables, lens, max_len, keep, n_first, n_recent, kept, stream)
    rc = _lib().hb_evict_select(w, weight_tables.data_ptr(), _int32(tshape[1]), lens.data_ptr(), _int32(n),
                                _int32(max_len), _int32(keep), _int32(n_first), _int32(n_recent), kept.data_ptr(),
                                _raw_stream(dev, stream))
    if rc:
        _check(rc, "hb_evict_select")


def evict_move(pool: PagedPool, block_tables, new_tables, kept, weights=None, weight_tables=None,
               new_weight_tables=None, stream=None):
    """hb_evict_move: slot i of new_tables gets K and V (and, with weights, the weight) of slot kept[.., i] of
    block_tables.  Tables int32 [n][stride], kept int32 [n][n_kv_heads][keep] on the device, as evict_select writes
    it."""
    dev, kv = pool._dev, pool._kv
    kshape, fshape, tshape = kept.shape, block_tables.shape, new_tables.shape
    if len(kshape) != 3 or kshape[1] != kv:
        raise ValueError(f"kept must be [n][{kv}][keep]")
    n, _, keep = kshape
    if (len(fshape) != 2 or fshape[0] != n or len(tshape) != 2 or tshape[0] != n or kept.dtype != _I32
            or block_tables.dtype != _I32 or new_tables.dtype != _I32 or not kept.is_contiguous()
            or not block_tables.is_contiguous() or not new_tables.is_contiguous() or dev < 0 or kept.get_device() != dev
            or block_tables.get_device() != dev or new_tables.get_device() != dev):
        _refuse((), ((kept, "kept", 3, n), (block_tables, "block_tables", 2, n), (new_tables, "new_tables", 2, n)))
    w = from_w = to_w = None
    ws = ns = 0
    if weights is not None:
        if weight_tables is None or new_weight_tables is None:
            raise ValueError("weights are moved between weight_tables and new_weight_tables")
        w = _weight_pool(weights, kv, dev)
        wshape, nshape = weight_tables.shape, new_weight_tables.shape
        if (len(wshape) != 2 or wshape[0] != n or len(nshape) != 2 or nshape[0] != n or weight_tables.dtype != _I32
                or new_weight_tables.dtype != _I32 or not weight_tables.is_contiguous()
                or not new_weight_tables.is_contiguous() or weight_tables.get_device() != dev
                or new_weight_tables.get_device() != dev):
            _refuse((), ((weight_tables, "weight_tables", 2, n), (new_weight_tables, "new_weight_tables", 2, n)))
        from_w, ws, to_w, ns = weight_tables.data_ptr(), wshape[1], new_weight_tables.data_ptr(), nshape[1]
    elif weight_tables is not None or new_weight_tables is not None:
        raise ValueError("the tables of weights come with the weights")
    if fshape[1] > _MOST or tshape[1] > _MOST or ws > _MOST or ns > _MOST or n > _MOST or keep > _MOST:
        raise native.HbError(native.HB_ERANGE, "a size does not fit 32 bits")
    if dev != _device():
        with torch.cuda.device(dev):
            return evict_move(pool, block_tables, new_tables, kept, weights, weight_tables, new_weight_tables, stream)
    rc = _lib().hb_evict_move(pool._c, block_tables.data_ptr(), fshape[1], new_tables.data_ptr(), tshape[1],
                              kept.data_ptr(), n, keep, w, from_w, ws, to_w, ns, _raw_stream(dev, stream))
    if rc:
        _check(rc, "hb_evict_move")
