"""ctypes binding of include/hb_cache.h: the paged KV cache in 4 bits, the
attention over it, and operations on pages.

Argument marshalling and checks only; every step runs in libhb.so.  Tensors
are used as device memory; work goes to ``stream`` (a torch stream), or to
the current stream of the tensors' device.  A bad call raises HbError (what
the library refuses) or ValueError (what only the tensors show).
"""
from __future__ import annotations

import ctypes
from operator import index
from typing import Optional, Sequence, Tuple

import numpy as np
import torch

from . import native
from .native import HbError


class _Pool(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("num_blocks", ctypes.c_int), ("n_kv_heads", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float)]


_bound = None


def _lib():
    global _bound
    if _bound is None:
        L = native.lib()
        vp, ci, ll, P = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.POINTER
        for name, args, res in (
                ("hb_kv4_pool_bytes", [ci, ci, ci], ll),
                ("hb_kv4_append", [vp, vp, ll, vp, ll, vp, ci, vp], ci),
                ("hb_kv4_read", [vp, vp, ci, vp, ll, vp, ll, vp], ci),
                ("hb_kv4_decode", [vp, vp, ll, vp, ci, vp, ci, ci, ci, vp, ll, vp, ll, vp], ci),
                ("hb_kv4_decode_workspace", [ci, ci, ci, ci, ci], ll),
                ("hb_kv4_chunk", [vp, vp, ll, vp, ci, ci, ci, ci, vp, ll, vp, ll, vp], ci),
                ("hb_kv4_chunk_workspace", [ci, ci, ci, ci, ci], ll),
                ("hb_kv4_test_lost_page", [], None),
                ("hb_copy_pages", [vp, ll, ci, ll, ci, vp, vp, ci, vp], ci),
                ("hb_copy_blocks", [vp, vp, vp, ci], ci),
                ("hb_pages_create", [ci, P(vp)], ci),
                ("hb_pages_destroy", [vp], None),
                ("hb_pages_extend", [vp, ci, ci, vp, vp], ci),
                ("hb_pages_fork", [vp, ci, ci, ci], ci),
                ("hb_pages_release", [vp, ci], ci),
                ("hb_pages_compact", [vp, vp, vp, ci], ci),
                ("hb_pages_table", [vp, ci, vp, ci, vp], ci),
                ("hb_pages_num_free", [vp], ci),
                ("hb_pages_refcount", [vp, ci], ci)):
            f = getattr(L, name)
            f.argtypes = args
            f.restype = res
        _bound = L
    return _bound


def _check(rc: int, what: str) -> int:
    if rc < 0:
        raise HbError(int(rc), f"{what} refused its arguments" if rc != native.HB_ECUDA else f"{what}: a CUDA call failed")
    return rc


def _raw_stream(dev: int, stream) -> int:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    if stream.device.index != dev:
        raise ValueError("the stream belongs to another device than the tensors")
    return stream.cuda_stream


def _int32(x) -> int:
    """An integer argument of the library (ctypes would cut it to 32 bits without a word)."""
    x = index(x)
    if not -(1 << 31) <= x < 1 << 31:
        raise HbError(native.HB_ERANGE, f"{x} does not fit 32 bits")
    return x


_device = torch._C._cuda_getDevice  # torch.cuda.current_device, for when a tensor shows that CUDA is up
_BF16 = (torch.bfloat16, torch.int16, torch.uint16)  # bf16, or its bits as elsewhere in the package
_I32 = torch.int32


def _refuse(rows, ints):
    """Say what is wrong with a call's tensors: rows of (tensor, name, n, heads, d), ints of (tensor, name, dim, n)."""
    for t, name, n, heads, d in rows:
        if t.shape != (n, heads, d):
            raise ValueError(f"{name} must be [{n}][{heads}][{d}], not {list(t.shape)}")
        if t.dtype not in _BF16:
            raise ValueError(f"{name} must be bf16, not {t.dtype}")
        if t.stride(2) != 1 or (t.stride(1) != d and heads > 1):
            raise ValueError(f"{name}: the heads of a row must be dense")
    for t, name, dim, n in ints:
        if t.dtype != _I32 or t.dim() != dim or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous int32 tensor of {dim} dimension(s)")
        if n >= 0 and t.shape[0] != n:
            raise ValueError(f"{name} must have {n} rows, not {t.shape[0]}")
    raise ValueError("the tensors must lie on one CUDA device")


# Each call below looks at its tensors in one expression (a call takes some 6 us
# of host time, half of it here), and says what is wrong in _refuse.  Kernels
# launch on the current device, so a call on tensors of another one makes that
# current first.


def kv4_pool_bytes(num_blocks: int, n_kv_heads: int, head_dim: int) -> int:
    return _check(_lib().hb_kv4_pool_bytes(_int32(num_blocks), _int32(n_kv_heads), _int32(head_dim)),
                  "hb_kv4_pool_bytes")


class Kv4Pool:
    """A pool of the 4-bit cache over a uint8 tensor [num_blocks][n_kv_heads][18 head_dim], whose memory must stay
    where it is.  Read-only once made."""
    __slots__ = ("_data", "_c", "_addr", "_dev", "_kv", "_d")

    def __init__(self, data: torch.Tensor, k_scale: float = 1.0, v_scale: float = 1.0):
        shape = data.shape
        if data.dtype != torch.uint8 or len(shape) != 3 or shape[2] % 18 or not data.is_contiguous():
            raise ValueError("a 4-bit pool is a contiguous uint8 tensor [num_blocks][n_kv_heads][18 head_dim]")
        self._kv, self._d = shape[1], shape[2] // 18
        self._data, self._dev = data, data.get_device()
        self._c = _Pool(data.data_ptr(), shape[0], self._kv, self._d, k_scale, v_scale)
        self._addr = ctypes.addressof(self._c)

    data = property(lambda self: self._data)
    num_blocks = property(lambda self: self._c.num_blocks)
    n_kv_heads = property(lambda self: self._kv)
    head_dim = property(lambda self: self._d)
    k_scale = property(lambda self: self._c.k_scale)  # as the library uses it, in 32 bits
    v_scale = property(lambda self: self._c.v_scale)

    @classmethod
    def empty(cls, num_blocks: int, n_kv_heads: int, head_dim: int, k_scale: float = 1.0, v_scale: float = 1.0,
              device="cuda") -> "Kv4Pool":
        """A new pool of zeros."""
        kv4_pool_bytes(num_blocks, n_kv_heads, head_dim)
        return cls(torch.zeros((num_blocks, n_kv_heads, 18 * head_dim), dtype=torch.uint8, device=device), k_scale,
                   v_scale)


def kv4_append(pool: Kv4Pool, k, v, slots, stream=None):
    """Quantise rows k, v [n][n_kv_heads][head_dim] into the pool at slots (device int32 [n]; -1 skips a row)."""
    n, kv, d, dev = slots.numel(), pool._kv, pool._d, pool._dev
    if (k.shape != (n, kv, d) or v.shape != (n, kv, d) or k.dtype not in _BF16 or v.dtype not in _BF16
            or (ks := k.stride())[2] != 1 or (vs := v.stride())[2] != 1 or (kv > 1 and (ks[1] != d or vs[1] != d))
            or slots.dtype != _I32 or slots.dim() != 1 or not slots.is_contiguous() or dev < 0
            or k.get_device() != dev or v.get_device() != dev or slots.get_device() != dev):
        _refuse(((k, "k", n, kv, d), (v, "v", n, kv, d)), ((slots, "slots", 1, n),))
    if not n:
        return
    if dev != _device():
        with torch.cuda.device(dev):
            return kv4_append(pool, k, v, slots, stream)
    rc = _lib().hb_kv4_append(pool._addr, k.data_ptr(), ks[0], v.data_ptr(), vs[0], slots.data_ptr(),
                              _int32(n), _raw_stream(dev, stream))
    if rc:
        _check(rc, "hb_kv4_append")


def kv4_read(pool: Kv4Pool, slots, k_out, v_out, stream=None):
    """The values at slots as bf16 rows, into k_out, v_out [n][n_kv_heads][head_dim]."""
    n, kv, d, dev = slots.numel(), pool._kv, pool._d, pool._dev
    if (k_out.shape != (n, kv, d) or v_out.shape != (n, kv, d) or k_out.dtype not in _BF16 or v_out.dtype not in _BF16
            or (ks := k_out.stride())[2] != 1 or (vs := v_out.stride())[2] != 1
            or (kv > 1 and (ks[1] != d or vs[1] != d))
            or slots.dtype != _I32 or slots.dim() != 1 or not slots.is_contiguous() or dev < 0
            or k_out.get_device() != dev or v_out.get_device() != dev or slots.get_device() != dev):
        _refuse(((k_out, "k_out", n, kv, d), (v_out, "v_out", n, kv, d)), ((slots, "slots", 1, n),))
    if not n:
        return
    if dev != _device():
        with torch.cuda.device(dev):
            return kv4_read(pool, slots, k_out, v_out, stream)
    rc = _lib().hb_kv4_read(pool._addr, slots.data_ptr(), _int32(n), k_out.data_ptr(), ks[0], v_out.data_ptr(), vs[0],
                            _raw_stream(dev, stream))
    if rc:
        _check(rc, "hb_kv4_read")


def kv4_decode_workspace(n_decodes: int, n_heads: int, n_kv_heads: int, head_dim: int, max_ctx: int) -> int:
    return _check(_lib().hb_kv4_decode_workspace(*map(_int32, (n_decodes, n_heads, n_kv_heads, head_dim, max_ctx))),
                  "hb_kv4_decode_workspace")


def kv4_chunk_workspace(chunk_offset: int, chunk_len: int, n_heads: int, n_kv_heads: int, head_dim: int) -> int:
    return _check(
        _lib().hb_kv4_chunk_workspace(*map(_int32, (chunk_offset, chunk_len, n_heads, n_kv_heads, head_dim))),
        "hb_kv4_chunk_workspace")


def _work(workspace, stream, dev: int, need, *args):
    """The caller's workspace, or a new one of need(*args) bytes: torch's allocator orders its reuse on the current
    stream, so a call on a stream of its own wants a workspace of its own."""
    if workspace is None:
        if stream is not None:
            raise ValueError("a call on a stream of its own wants a workspace of its own")
        return torch.empty(need(*args), dtype=torch.uint8, device=torch.device("cuda", dev))
    if not workspace.is_contiguous() or workspace.get_device() != dev:
        raise ValueError("the workspace must be a contiguous tensor on the pool's device")
    return workspace


def kv4_decode(pool: Kv4Pool, q, block_tables, ctx_lens, max_ctx: int, out, workspace=None, stream=None):
    """hb_kv4_decode: q, out [n][n_heads][head_dim] bf16; block_tables int32 [n][stride], ctx_lens int32 [n] on the
    device.  workspace: a tensor of at least kv4_decode_workspace() bytes, or None for a new one (only on the
    current stream)."""
    if q.dim() != 3:
        raise ValueError("q must be [n][n_heads][head_dim]")
    n, heads, d = shape = q.shape
    dev, lens_ok = pool._dev, block_tables.dim() == 2 and ctx_lens.dim() == 1
    if (d != pool._d or out.shape != shape or q.dtype not in _BF16 or out.dtype not in _BF16
            or (qs := q.stride())[2] != 1 or (os_ := out.stride())[2] != 1
            or (heads > 1 and (qs[1] != d or os_[1] != d)) or not lens_ok
            or block_tables.dtype != _I32 or ctx_lens.dtype != _I32 or block_tables.shape[0] != n
            or ctx_lens.shape[0] != n or not block_tables.is_contiguous() or not ctx_lens.is_contiguous() or dev < 0
            or q.get_device() != dev or out.get_device() != dev or block_tables.get_device() != dev
            or ctx_lens.get_device() != dev):
        _refuse(((q, "q", n, heads, pool._d), (out, "out", n, heads, pool._d)),
                ((block_tables, "block_tables", 2, n), (ctx_lens, "ctx_lens", 1, n)))
    if not n:
        return
    if dev != _device():
        with torch.cuda.device(dev):
            return kv4_decode(pool, q, block_tables, ctx_lens, max_ctx, out, workspace, stream)
    ws = _work(workspace, stream, dev, kv4_decode_workspace, n, heads, pool._kv, d, max_ctx)
    rc = _lib().hb_kv4_decode(pool._addr, q.data_ptr(), qs[0], block_tables.data_ptr(), _int32(block_tables.shape[1]),
                              ctx_lens.data_ptr(), _int32(n), heads, _int32(max_ctx), out.data_ptr(), os_[0],
                              ws.data_ptr(), ws.nbytes, _raw_stream(dev, stream))
    if rc:
        _check(rc, "hb_kv4_decode")


def kv4_chunk(pool: Kv4Pool, q, block_table, chunk_offset: int, out, workspace=None, stream=None):
    """hb_kv4_chunk: q, out [chunk_len][n_heads][head_dim] bf16; block_table int32 [blocks] on the device.
    workspace: as for kv4_decode, of kv4_chunk_workspace() bytes."""
    if q.dim() != 3:
        raise ValueError("q must be [chunk_len][n_heads][head_dim]")
    n, heads, d = shape = q.shape
    dev = pool._dev
    if (d != pool._d or out.shape != shape or q.dtype not in _BF16 or out.dtype not in _BF16
            or (qs := q.stride())[2] != 1 or (os_ := out.stride())[2] != 1
            or (heads > 1 and (qs[1] != d or os_[1] != d))
            or block_table.dtype != _I32 or block_table.dim() != 1 or not block_table.is_contiguous() or dev < 0
            or q.get_device() != dev or out.get_device() != dev or block_table.get_device() != dev):
        _refuse(((q, "q", n, heads, pool._d), (out, "out", n, heads, pool._d)), ((block_table, "block_table", 1, -1),))
    if not n:
        return
    if dev != _device():
        with torch.cuda.device(dev):
            return kv4_chunk(pool, q, block_table, chunk_offset, out, workspace, stream)
    ws = _work(workspace, stream, dev, kv4_chunk_workspace, chunk_offset, n, heads, pool._kv, d)
    rc = _lib().hb_kv4_chunk(pool._addr, q.data_ptr(), qs[0], block_table.data_ptr(), _int32(block_table.shape[0]),
                             _int32(chunk_offset), _int32(n), heads, out.data_ptr(), os_[0], ws.data_ptr(), ws.nbytes,
                             _raw_stream(dev, stream))
    if rc:
        _check(rc, "hb_kv4_chunk")


def kv4_test_lost_page():
    """Test hook: the next kv4_decode or kv4_chunk of this thread loses a page, and its waits for it run out."""
    _lib().hb_kv4_test_lost_page()


_NP32 = np.dtype(np.int32)


def _host_pages(a, name: str) -> np.ndarray:
    if type(a) is np.ndarray and a.dtype is _NP32 and a.ndim == 1 and a.flags.c_contiguous:
        return a
    v = np.asarray(a)
    if v.ndim != 1 or (v.size and v.dtype.kind not in "iu"):
        raise ValueError(f"{name} must be a list of page numbers")
    if v.size and (v.min() < -(1 << 31) or v.max() >= 1 << 31):
        raise HbError(native.HB_ERANGE, f"{name}: a page number does not fit 32 bits")
    return np.ascontiguousarray(v, np.int32)


def _page_addr(a: np.ndarray) -> int:
    try:
        return ctypes.addressof(ctypes.c_char.from_buffer(a))  # a third of the time of a.ctypes.data
    except (TypeError, ValueError):                            # read-only or empty
        return a.ctypes.data


def copy_pages(pools, src: Sequence[int], dst: Sequence[int], stream=None):
    """Copy page src[i] to dst[i] in every pool of a tensor [n_pools][num_blocks][...] (any dtype; each pool's pages
    dense).  src, dst: host lists or int32 arrays; a destination may be neither repeated nor a source."""
    s, d = _host_pages(src, "src"), _host_pages(dst, "dst")
    n = len(s)
    if n != len(d):
        raise ValueError("src and dst must have the same length")
    shape = pools.shape
    n_pools, blocks = shape[:2] if len(shape) >= 3 else (0, 0)
    if pools.is_contiguous() and n_pools and blocks:
        page = pools.numel() // (n_pools * blocks)
        stride = page * blocks
    else:
        strides, page, dense = pools.stride(), 1, n_pools > 0 and blocks > 0
        for size, step in zip(shape[:1:-1], strides[:1:-1]):
            dense = dense and (step == page or size == 1)
            page *= size
        if not dense or (strides[1] != page and blocks > 1):
            raise ValueError("pools must be a tensor [n_pools][num_blocks][...] with the pages of each pool dense")
        stride = strides[0] if n_pools > 1 else page * blocks
    dev = pools.get_device()
    if dev < 0:
        raise ValueError("pools must lie on a CUDA device")
    if not n:
        return
    if dev != _device():
        with torch.cuda.device(dev):
            return copy_pages(pools, s, d, stream)
    es = pools.element_size()
    rc = _lib().hb_copy_pages(pools.data_ptr(), stride * es, _int32(n_pools), page * es, _int32(blocks), _page_addr(s),
                              _page_addr(d), _int32(n), _raw_stream(dev, stream))
    if rc:
        _check(rc, "hb_copy_pages")


def copy_blocks(ctx: "native.Context", src: Sequence[int], dst: Sequence[int]):
    """copy_pages over the K and V pools of every layer of a context, on its stream."""
    s, d = _host_pages(src, "src"), _host_pages(dst, "dst")
    if len(s) != len(d):
        raise ValueError("src and dst must have the same length")
    ctx._check(_lib().hb_copy_blocks(ctx.h, s.ctypes.data, d.ctypes.data, _int32(len(s))))


class PageTable:
    """hb_pages: which pages each sequence holds, with copy-on-write forks and compaction (host only)."""

    def __init__(self, num_blocks: int):
        self.num_blocks = num_blocks
        self.L = _lib()
        h = ctypes.c_void_p()
        _check(self.L.hb_pages_create(_int32(num_blocks), ctypes.byref(h)), "hb_pages_create")
        self.h = h

    def extend(self, seq: int, n_tokens: int) -> Optional[Tuple[int, int]]:
        """Grow seq to n_tokens tokens; returns the (source, destination) of the page to copy first, if any."""
        s, d = ctypes.c_int32(), ctypes.c_int32()
        _check(self.L.hb_pages_extend(self.h, _int32(seq), _int32(n_tokens), ctypes.addressof(s), ctypes.addressof(d)),
               "hb_pages_extend")
        return (s.value, d.value) if s.value >= 0 else None

    def fork(self, parent: int, child: int, n_tokens: int = -1):
        """child shares the pages of parent's first n_tokens tokens (all of them by default)."""
        _check(self.L.hb_pages_fork(self.h, _int32(parent), _int32(child), _int32(n_tokens)), "hb_pages_fork")

    def release(self, seq: int):
        _check(self.L.hb_pages_release(self.h, _int32(seq)), "hb_pages_release")

    def compact(self, max_moves: Optional[int] = None) -> Tuple[np.ndarray, np.ndarray]:
        """(src, dst) of the page moves that bring held pages to the front, for copy_pages."""
        m = self.num_blocks if max_moves is None else _int32(min(index(max_moves), self.num_blocks))
        src, dst = np.empty(max(m, 1), np.int32), np.empty(max(m, 1), np.int32)
        n = _check(self.L.hb_pages_compact(self.h, src.ctypes.data, dst.ctypes.data, m), "hb_pages_compact")
        return src[:n], dst[:n]

    def table(self, seq: int) -> np.ndarray:
        n = _check(self.L.hb_pages_table(self.h, _int32(seq), None, 0, None), "hb_pages_table")
        out = np.empty(max(n, 1), np.int32)
        _check(self.L.hb_pages_table(self.h, seq, out.ctypes.data, n, None), "hb_pages_table")
        return out[:n]

    def length(self, seq: int) -> int:
        n = ctypes.c_int()
        _check(self.L.hb_pages_table(self.h, _int32(seq), None, 0, ctypes.addressof(n)), "hb_pages_table")
        return n.value

    @property
    def num_free(self) -> int:
        return _check(self.L.hb_pages_num_free(self.h), "hb_pages_num_free")

    def refcount(self, block: int) -> int:
        return _check(self.L.hb_pages_refcount(self.h, _int32(block)), "hb_pages_refcount")

    def free(self):
        if getattr(self, "h", None):
            self.L.hb_pages_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass
