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

from . import native
from .native import HbError


class _Pool(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("num_blocks", ctypes.c_int), ("n_kv_heads", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float)]


_sigs = False


def _lib():
    global _sigs
    L = native.lib()
    if not _sigs:
        vp, ci, ll, P = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.POINTER
        for name, args, res in (
                ("hb_kv4_pool_bytes", [ci, ci, ci], ll),
                ("hb_kv4_append", [P(_Pool), vp, ll, vp, ll, vp, ci, vp], ci),
                ("hb_kv4_read", [P(_Pool), vp, ci, vp, ll, vp, ll, vp], ci),
                ("hb_kv4_decode", [P(_Pool), vp, ll, vp, ci, vp, ci, ci, ci, vp, ll, vp, ll, vp], ci),
                ("hb_kv4_decode_workspace", [ci, ci, ci, ci, ci], ll),
                ("hb_kv4_chunk", [P(_Pool), vp, ll, vp, ci, ci, ci, ci, vp, ll, vp, ll, vp], ci),
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
        _sigs = True
    return L


def _check(rc: int, what: str) -> int:
    if rc < 0:
        raise HbError(int(rc), f"{what} refused its arguments" if rc != native.HB_ECUDA else f"{what}: a CUDA call failed")
    return rc


def _call(device, stream, fn, *args) -> int:
    """fn(*args, stream) with `device` current, where its kernels must launch."""
    import torch
    if stream is not None and stream.device != device:
        raise ValueError("the stream belongs to another device than the tensors")
    if device.index == torch.cuda.current_device():
        return fn(*args, (stream or torch.cuda.current_stream()).cuda_stream)
    with torch.cuda.device(device):
        return fn(*args, (stream or torch.cuda.current_stream()).cuda_stream)


def _same_device(device, *tensors):
    if device.type != "cuda" or any(t.device != device for t in tensors):
        raise ValueError("the tensors must lie on one CUDA device")


_TWO_BYTES = ("torch.bfloat16", "torch.int16", "torch.uint16")  # bf16, or its bits as elsewhere in the package


def _rows(t, name: str, n: int, heads: Optional[int], d: int):
    """Row stride of a [n][heads][d] operand whose rows are dense inside."""
    if t.dim() != 3 or t.shape[0] != n or t.shape[2] != d or (heads is not None and t.shape[1] != heads):
        raise ValueError(f"{name} must be [{n}][{heads if heads is not None else 'heads'}][{d}], not {list(t.shape)}")
    if str(t.dtype) not in _TWO_BYTES:
        raise ValueError(f"{name} must be bf16, not {t.dtype}")
    if n and (t.stride(2) != 1 or (t.shape[1] > 1 and t.stride(1) != d)):
        raise ValueError(f"{name}: the heads of a row must be dense")
    return t.stride(0) if n > 1 else t.shape[1] * d


def _i32(t, name: str, dim: int):
    if str(t.dtype) != "torch.int32" or t.dim() != dim or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor of {dim} dimension(s)")


def kv4_pool_bytes(num_blocks: int, n_kv_heads: int, head_dim: int) -> int:
    return _check(_lib().hb_kv4_pool_bytes(num_blocks, n_kv_heads, head_dim), "hb_kv4_pool_bytes")


@dataclass
class Kv4Pool:
    """A pool of the 4-bit cache over a uint8 tensor [num_blocks][n_kv_heads][18 head_dim]."""
    data: "object"
    k_scale: float = 1.0
    v_scale: float = 1.0

    def __post_init__(self):
        t = self.data
        if str(t.dtype) != "torch.uint8" or t.dim() != 3 or not t.is_contiguous() or t.shape[2] % 18:
            raise ValueError("a 4-bit pool is a contiguous uint8 tensor [num_blocks][n_kv_heads][18 head_dim]")
        self.num_blocks, self.n_kv_heads, self.head_dim = int(t.shape[0]), int(t.shape[1]), int(t.shape[2]) // 18
        self.c = _Pool(t.data_ptr(), self.num_blocks, self.n_kv_heads, self.head_dim, self.k_scale, self.v_scale)

    @classmethod
    def empty(cls, num_blocks: int, n_kv_heads: int, head_dim: int, k_scale: float = 1.0, v_scale: float = 1.0,
              device="cuda") -> "Kv4Pool":
        """A new pool of zeros."""
        import torch
        kv4_pool_bytes(num_blocks, n_kv_heads, head_dim)
        return cls(torch.zeros((num_blocks, n_kv_heads, 18 * head_dim), dtype=torch.uint8, device=device), k_scale,
                   v_scale)


def kv4_append(pool: Kv4Pool, k, v, slots, stream=None):
    """Quantise rows k, v [n][n_kv_heads][head_dim] into the pool at slots (device int32 [n]; -1 skips a row)."""
    n = int(slots.shape[0])
    _i32(slots, "slots", 1)
    ks, vs = _rows(k, "k", n, pool.n_kv_heads, pool.head_dim), _rows(v, "v", n, pool.n_kv_heads, pool.head_dim)
    _same_device(pool.data.device, k, v, slots)
    if n:
        _check(_call(pool.data.device, stream, _lib().hb_kv4_append, ctypes.byref(pool.c), k.data_ptr(), ks,
                     v.data_ptr(), vs, slots.data_ptr(), n), "hb_kv4_append")


def kv4_read(pool: Kv4Pool, slots, k_out, v_out, stream=None):
    """The values at slots as bf16 rows, into k_out, v_out [n][n_kv_heads][head_dim]."""
    n = int(slots.shape[0])
    _i32(slots, "slots", 1)
    ks, vs = _rows(k_out, "k_out", n, pool.n_kv_heads, pool.head_dim), _rows(v_out, "v_out", n, pool.n_kv_heads, pool.head_dim)
    _same_device(pool.data.device, k_out, v_out, slots)
    if n:
        _check(_call(pool.data.device, stream, _lib().hb_kv4_read, ctypes.byref(pool.c), slots.data_ptr(), n,
                     k_out.data_ptr(), ks, v_out.data_ptr(), vs), "hb_kv4_read")


def kv4_decode_workspace(n_decodes: int, n_heads: int, n_kv_heads: int, head_dim: int, max_ctx: int) -> int:
    return _check(_lib().hb_kv4_decode_workspace(n_decodes, n_heads, n_kv_heads, head_dim, max_ctx),
                  "hb_kv4_decode_workspace")


def kv4_chunk_workspace(chunk_offset: int, chunk_len: int, n_heads: int, n_kv_heads: int, head_dim: int) -> int:
    return _check(_lib().hb_kv4_chunk_workspace(chunk_offset, chunk_len, n_heads, n_kv_heads, head_dim),
                  "hb_kv4_chunk_workspace")


def _work(workspace, need: int, device):
    """Pointer and size of the caller's workspace, or of a new one (stream-ordered, from torch's allocator)."""
    import torch
    if workspace is None:
        if need == 0:
            return None, 0, None
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    if not workspace.is_contiguous() or workspace.device != device:
        raise ValueError("the workspace must be a contiguous tensor on the pool's device")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def kv4_decode(pool: Kv4Pool, q, block_tables, ctx_lens, max_ctx: int, out, workspace=None, stream=None):
    """hb_kv4_decode: q, out [n][n_heads][head_dim] bf16; block_tables int32 [n][stride], ctx_lens int32 [n] on the
    device.  workspace: a tensor of at least kv4_decode_workspace() bytes, or None for a new one (only on the
    current stream: torch's allocator orders its reuse there)."""
    n, n_heads = int(q.shape[0]), int(q.shape[1])
    qs, os_ = _rows(q, "q", n, None, pool.head_dim), _rows(out, "out", n, n_heads, pool.head_dim)
    _i32(block_tables, "block_tables", 2)
    _i32(ctx_lens, "ctx_lens", 1)
    if block_tables.shape[0] != n or ctx_lens.shape[0] != n:
        raise ValueError("block_tables and ctx_lens must have one row for each row of q")
    _same_device(pool.data.device, q, block_tables, ctx_lens, out)
    if not n:
        return
    if workspace is None:
        if stream is not None:
            raise ValueError("a call on a stream of its own wants a workspace of its own")
        need = kv4_decode_workspace(n, n_heads, pool.n_kv_heads, pool.head_dim, max_ctx)
    else:
        need = 0
    wp, wn, keep = _work(workspace, need, pool.data.device)
    _check(_call(pool.data.device, stream, _lib().hb_kv4_decode, ctypes.byref(pool.c), q.data_ptr(), qs,
                 block_tables.data_ptr(), int(block_tables.shape[1]), ctx_lens.data_ptr(), n, n_heads, int(max_ctx),
                 out.data_ptr(), os_, wp, wn), "hb_kv4_decode")


def kv4_chunk(pool: Kv4Pool, q, block_table, chunk_offset: int, out, workspace=None, stream=None):
    """hb_kv4_chunk: q, out [chunk_len][n_heads][head_dim] bf16; block_table int32 [blocks] on the device.
    workspace: as for kv4_decode, of kv4_chunk_workspace() bytes."""
    n, n_heads = int(q.shape[0]), int(q.shape[1])
    qs, os_ = _rows(q, "q", n, None, pool.head_dim), _rows(out, "out", n, n_heads, pool.head_dim)
    _i32(block_table, "block_table", 1)
    _same_device(pool.data.device, q, block_table, out)
    if not n:
        return
    if workspace is None:
        if stream is not None:
            raise ValueError("a call on a stream of its own wants a workspace of its own")
        need = kv4_chunk_workspace(chunk_offset, n, n_heads, pool.n_kv_heads, pool.head_dim)
    else:
        need = 0
    wp, wn, keep = _work(workspace, need, pool.data.device)
    _check(_call(pool.data.device, stream, _lib().hb_kv4_chunk, ctypes.byref(pool.c), q.data_ptr(), qs,
                 block_table.data_ptr(), int(block_table.shape[0]), int(chunk_offset), n, n_heads, out.data_ptr(),
                 os_, wp, wn), "hb_kv4_chunk")


def _host_pages(a, name: str) -> np.ndarray:
    v = np.asarray(a)
    if v.ndim != 1 or (v.size and v.dtype.kind not in "iu"):
        raise ValueError(f"{name} must be a list of page numbers")
    if v.size and (v.min() < -(1 << 31) or v.max() >= 1 << 31):
        raise HbError(native.HB_ERANGE, f"{name}: a page number does not fit 32 bits")
    return np.ascontiguousarray(v, np.int32)


def copy_pages(pools, src: Sequence[int], dst: Sequence[int], stream=None):
    """Copy page src[i] to dst[i] in every pool of a tensor [n_pools][num_blocks][...] (any dtype; each pool's pages
    dense).  src, dst: host lists or int32 arrays; a destination may be neither repeated nor a source."""
    s, d = _host_pages(src, "src"), _host_pages(dst, "dst")
    if len(s) != len(d):
        raise ValueError("src and dst must have the same length")
    if pools.dim() < 3 or pools.shape[0] < 1 or pools.shape[1] < 1 or not pools[0].is_contiguous():
        raise ValueError("pools must be a tensor [n_pools][num_blocks][...] with the pages of each pool dense")
    if pools.device.type != "cuda":
        raise ValueError("pools must lie on a CUDA device")
    if not len(s):
        return
    es = pools.element_size()
    page = pools[0, 0].numel() * es
    stride = pools.stride(0) * es if pools.shape[0] > 1 else page * int(pools.shape[1])
    _check(_call(pools.device, stream, _lib().hb_copy_pages, pools.data_ptr(), stride, int(pools.shape[0]), page,
                 int(pools.shape[1]), s.ctypes.data, d.ctypes.data, len(s)), "hb_copy_pages")


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
