"""ctypes binding of include/hb_cache.h: the paged KV cache in 4 bits, the
attention over it, and operations on pages.

Argument marshalling and checks only; every step runs in libhb.so.  Tensors
are used as device memory; work goes to ``stream`` (a torch stream), or to
the current stream of the tensors' device.  A bad call raises HbError (what
the library refuses) or ValueError (what only the tensors show).
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass
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


def _launch(dev: int, stream, fn, *args) -> int:
    """fn(*args, stream) with the tensors' device current, where its kernels must launch."""
    if dev != torch.cuda.current_device():
        with torch.cuda.device(dev):
            return _launch(dev, stream, fn, *args)
    if stream is None:
        return fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    if stream.device.index != dev:
        raise ValueError("the stream belongs to another device than the tensors")
    return fn(*args, stream.cuda_stream)


def _same_device(dev: int, *tensors):
    if dev < 0:
        raise ValueError("the tensors must lie on a CUDA device")
    for t in tensors:
        if t.get_device() != dev:
            raise ValueError("the tensors must lie on one CUDA device")


_TWO_BYTES = (torch.bfloat16, torch.int16, torch.uint16)  # bf16, or its bits as elsewhere in the package


def _rows(t, name: str, n: int, heads: int, d: int) -> int:
    """Row stride of a [n][heads][d] operand whose rows are dense inside."""
    if t.shape != (n, heads, d):
        raise ValueError(f"{name} must be [{n}][{heads}][{d}], not {list(t.shape)}")
    if t.dtype not in _TWO_BYTES:
        raise ValueError(f"{name} must be bf16, not {t.dtype}")
    rs, hs, es = t.stride()
    if es != 1 or (hs != d and heads > 1):
        raise ValueError(f"{name}: the heads of a row must be dense")
    return rs if n > 1 else heads * d


def _i32(t, name: str, dim: int):
    if t.dtype != torch.int32 or t.dim() != dim or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor of {dim} dimension(s)")


def kv4_pool_bytes(num_blocks: int, n_kv_heads: int, head_dim: int) -> int:
    return _check(_lib().hb_kv4_pool_bytes(num_blocks, n_kv_heads, head_dim), "hb_kv4_pool_bytes")


@dataclass(frozen=True, eq=False)
class Kv4Pool:
    """A pool of the 4-bit cache over a uint8 tensor [num_blocks][n_kv_heads][18 head_dim], whose memory must stay
    where it is."""
    data: torch.Tensor
    k_scale: float = 1.0
    v_scale: float = 1.0

    def __post_init__(self):
        t = self.data
        if t.dtype != torch.uint8 or t.dim() != 3 or not t.is_contiguous() or t.shape[2] % 18:
            raise ValueError("a 4-bit pool is a contiguous uint8 tensor [num_blocks][n_kv_heads][18 head_dim]")
        blocks, kv, d = int(t.shape[0]), int(t.shape[1]), int(t.shape[2]) // 18
        c = _Pool(t.data_ptr(), blocks, kv, d, self.k_scale, self.v_scale)
        for name, value in (("num_blocks", blocks), ("n_kv_heads", kv), ("head_dim", d), ("c", c),
                            ("c_addr", ctypes.addressof(c))):
            object.__setattr__(self, name, value)

    @classmethod
    def empty(cls, num_blocks: int, n_kv_heads: int, head_dim: int, k_scale: float = 1.0, v_scale: float = 1.0,
              device="cuda") -> "Kv4Pool":
        """A new pool of zeros."""
        kv4_pool_bytes(num_blocks, n_kv_heads, head_dim)
        return cls(torch.zeros((num_blocks, n_kv_heads, 18 * head_dim), dtype=torch.uint8, device=device), k_scale,
                   v_scale)


def kv4_append(pool: Kv4Pool, k, v, slots, stream=None):
    """Quantise rows k, v [n][n_kv_heads][head_dim] into the pool at slots (device int32 [n]; -1 skips a row)."""
    _i32(slots, "slots", 1)
    n = slots.shape[0]
    ks, vs = _rows(k, "k", n, pool.n_kv_heads, pool.head_dim), _rows(v, "v", n, pool.n_kv_heads, pool.head_dim)
    dev = pool.data.get_device()
    _same_device(dev, k, v, slots)
    if n:
        _check(_launch(dev, stream, _lib().hb_kv4_append, pool.c_addr, k.data_ptr(), ks, v.data_ptr(), vs,
                       slots.data_ptr(), n), "hb_kv4_append")


def kv4_read(pool: Kv4Pool, slots, k_out, v_out, stream=None):
    """The values at slots as bf16 rows, into k_out, v_out [n][n_kv_heads][head_dim]."""
    _i32(slots, "slots", 1)
    n = slots.shape[0]
    ks = _rows(k_out, "k_out", n, pool.n_kv_heads, pool.head_dim)
    vs = _rows(v_out, "v_out", n, pool.n_kv_heads, pool.head_dim)
    dev = pool.data.get_device()
    _same_device(dev, k_out, v_out, slots)
    if n:
        _check(_launch(dev, stream, _lib().hb_kv4_read, pool.c_addr, slots.data_ptr(), n, k_out.data_ptr(), ks,
                       v_out.data_ptr(), vs), "hb_kv4_read")


def kv4_decode_workspace(n_decodes: int, n_heads: int, n_kv_heads: int, head_dim: int, max_ctx: int) -> int:
    return _check(_lib().hb_kv4_decode_workspace(n_decodes, n_heads, n_kv_heads, head_dim, max_ctx),
                  "hb_kv4_decode_workspace")


def kv4_chunk_workspace(chunk_offset: int, chunk_len: int, n_heads: int, n_kv_heads: int, head_dim: int) -> int:
    return _check(_lib().hb_kv4_chunk_workspace(chunk_offset, chunk_len, n_heads, n_kv_heads, head_dim),
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
    n, heads, _ = q.shape
    qs, os_ = _rows(q, "q", n, heads, pool.head_dim), _rows(out, "out", n, heads, pool.head_dim)
    _i32(block_tables, "block_tables", 2)
    _i32(ctx_lens, "ctx_lens", 1)
    if block_tables.shape[0] != n or ctx_lens.shape[0] != n:
        raise ValueError("block_tables and ctx_lens must have one row for each row of q")
    dev = pool.data.get_device()
    _same_device(dev, q, block_tables, ctx_lens, out)
    if not n:
        return
    ws = _work(workspace, stream, dev, kv4_decode_workspace, n, heads, pool.n_kv_heads, pool.head_dim, max_ctx)
    _check(_launch(dev, stream, _lib().hb_kv4_decode, pool.c_addr, q.data_ptr(), qs, block_tables.data_ptr(),
                   block_tables.shape[1], ctx_lens.data_ptr(), n, heads, max_ctx, out.data_ptr(), os_, ws.data_ptr(),
                   ws.nbytes), "hb_kv4_decode")


def kv4_chunk(pool: Kv4Pool, q, block_table, chunk_offset: int, out, workspace=None, stream=None):
    """hb_kv4_chunk: q, out [chunk_len][n_heads][head_dim] bf16; block_table int32 [blocks] on the device.
    workspace: as for kv4_decode, of kv4_chunk_workspace() bytes."""
    if q.dim() != 3:
        raise ValueError("q must be [chunk_len][n_heads][head_dim]")
    n, heads, _ = q.shape
    qs, os_ = _rows(q, "q", n, heads, pool.head_dim), _rows(out, "out", n, heads, pool.head_dim)
    _i32(block_table, "block_table", 1)
    dev = pool.data.get_device()
    _same_device(dev, q, block_table, out)
    if not n:
        return
    ws = _work(workspace, stream, dev, kv4_chunk_workspace, chunk_offset, n, heads, pool.n_kv_heads, pool.head_dim)
    _check(_launch(dev, stream, _lib().hb_kv4_chunk, pool.c_addr, q.data_ptr(), qs, block_table.data_ptr(),
                   block_table.shape[0], chunk_offset, n, heads, out.data_ptr(), os_, ws.data_ptr(), ws.nbytes),
           "hb_kv4_chunk")


def _host_pages(a, name: str) -> np.ndarray:
    if type(a) is np.ndarray and a.dtype == np.int32 and a.ndim == 1 and a.flags.c_contiguous:
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
    shape, strides = pools.shape, pools.stride()
    page = 1
    dense = len(shape) >= 3 and shape[0] > 0 and shape[1] > 0
    for size, step in zip(shape[:1:-1], strides[:1:-1]):
        dense = dense and (step == page or size == 1)
        page *= size
    if not dense or (strides[1] != page and shape[1] > 1):
        raise ValueError("pools must be a tensor [n_pools][num_blocks][...] with the pages of each pool dense")
    dev = pools.get_device()
    _same_device(dev)
    if not n:
        return
    page *= pools.element_size()
    stride = strides[0] * pools.element_size() if shape[0] > 1 else page * shape[1]
    _check(_launch(dev, stream, _lib().hb_copy_pages, pools.data_ptr(), stride, shape[0], page, shape[1],
                   _page_addr(s), _page_addr(d), n), "hb_copy_pages")


def copy_blocks(ctx: "native.Context", src: Sequence[int], dst: Sequence[int]):
    """copy_pages over the K and V pools of every layer of a context, on its stream."""
    s, d = _host_pages(src, "src"), _host_pages(dst, "dst")
    if len(s) != len(d):
        raise ValueError("src and dst must have the same length")
    ctx._check(_lib().hb_copy_blocks(ctx.h, s.ctypes.data, d.ctypes.data, len(s)))


class PageTable:
    """hb_pages: which pages each sequence holds, with copy-on-write forks and compaction (host only)."""

    def __init__(self, num_blocks: int):
        self.num_blocks = num_blocks
        self.L = _lib()
        h = ctypes.c_void_p()
        _check(self.L.hb_pages_create(num_blocks, ctypes.byref(h)), "hb_pages_create")
        self.h = h

    def extend(self, seq: int, n_tokens: int) -> Optional[Tuple[int, int]]:
        """Grow seq to n_tokens tokens; returns the (source, destination) of the page to copy first, if any."""
        s, d = ctypes.c_int32(), ctypes.c_int32()
        _check(self.L.hb_pages_extend(self.h, seq, n_tokens, ctypes.addressof(s), ctypes.addressof(d)),
               "hb_pages_extend")
        return (s.value, d.value) if s.value >= 0 else None

    def fork(self, parent: int, child: int, n_tokens: int = -1):
        """child shares the pages of parent's first n_tokens tokens (all of them by default)."""
        _check(self.L.hb_pages_fork(self.h, parent, child, n_tokens), "hb_pages_fork")

    def release(self, seq: int):
        _check(self.L.hb_pages_release(self.h, seq), "hb_pages_release")

    def compact(self, max_moves: Optional[int] = None) -> Tuple[np.ndarray, np.ndarray]:
        """(src, dst) of the page moves that bring held pages to the front, for copy_pages."""
        m = self.num_blocks if max_moves is None else max_moves
        src, dst = np.empty(max(m, 1), np.int32), np.empty(max(m, 1), np.int32)
        n = _check(self.L.hb_pages_compact(self.h, src.ctypes.data, dst.ctypes.data, m), "hb_pages_compact")
        return src[:n], dst[:n]

    def table(self, seq: int) -> np.ndarray:
        n = _check(self.L.hb_pages_table(self.h, seq, None, 0, None), "hb_pages_table")
        out = np.empty(max(n, 1), np.int32)
        _check(self.L.hb_pages_table(self.h, seq, out.ctypes.data, n, None), "hb_pages_table")
        return out[:n]

    def length(self, seq: int) -> int:
        n = ctypes.c_int()
        _check(self.L.hb_pages_table(self.h, seq, None, 0, ctypes.addressof(n)), "hb_pages_table")
        return n.value

    @property
    def num_free(self) -> int:
        return _check(self.L.hb_pages_num_free(self.h), "hb_pages_num_free")

    def refcount(self, block: int) -> int:
        return _check(self.L.hb_pages_refcount(self.h, block), "hb_pages_refcount")

    def free(self):
        if getattr(self, "h", None):
            self.L.hb_pages_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass
