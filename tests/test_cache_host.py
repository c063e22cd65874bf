"""The 4-bit cache and the page operations without a GPU: what the calls
refuse, the page table against a plain model of it, the binding's checks."""
import ctypes
import random

import numpy as np
import pytest

from chunked_prefill_hybrid_gb300 import cache, native
from chunked_prefill_hybrid_gb300.native import HB_EINVAL, HB_ENOMEM, HB_ERANGE, HB_OK, HbError


@pytest.fixture(scope="module")
def L():
    import __graft_entry__
    __graft_entry__.build_library()
    return cache._lib()


def _pool(**over):
    a = dict(data=16, num_blocks=8, n_kv_heads=2, head_dim=128, k_scale=1.0, v_scale=1.0)
    a.update(over)
    return cache._Pool(*[a[n] for n, _ in cache._Pool._fields_])


def test_pool_bytes(L):
    assert cache.kv4_pool_bytes(3, 5, 128) == 3 * 5 * 18 * 128
    assert cache.kv4_pool_bytes((1 << 27) - 1, 8, 64) == ((1 << 27) - 1) * 8 * 18 * 64  # past 32 bits
    for bad in ((0, 1, 64), (1, 0, 64), (1, 1, 96), (1 << 27, 1, 64), (-1, 1, 128), (1, 70000, 64)):
        assert L.hb_kv4_pool_bytes(*bad) == HB_EINVAL


@pytest.mark.parametrize("over", [
    dict(data=None), dict(data=8), dict(num_blocks=0), dict(n_kv_heads=0), dict(head_dim=80), dict(k_scale=0.0),
    dict(k_scale=-1.0), dict(v_scale=float("nan")), dict(v_scale=float("inf")), dict(k_scale=1e-30)])
def test_bad_pool_is_refused_by_every_call(L, over):
    p = ctypes.byref(_pool(**over))
    assert L.hb_kv4_append(p, 16, 256, 16, 256, 16, 4, None) == HB_EINVAL
    assert L.hb_kv4_read(p, 16, 4, 16, 256, 16, 256, None) == HB_EINVAL
    assert L.hb_kv4_decode(p, 16, 256, 16, 8, 16, 4, 2, 100, 16, 256, None, 0, None) == HB_EINVAL
    assert L.hb_kv4_chunk(p, 16, 256, 16, 8, 0, 4, 2, 16, 256, None, 0, None) == HB_EINVAL


def _append(L, **over):
    a = dict(k=16, ks=256, v=16, vs=256, slots=16, n=4)
    a.update(over)
    return L.hb_kv4_append(ctypes.byref(_pool()), a["k"], a["ks"], a["v"], a["vs"], a["slots"], a["n"], None)


def test_append_and_read_refusals(L):
    for over in (dict(k=None), dict(v=None), dict(slots=None), dict(k=24), dict(v=8), dict(ks=255), dict(ks=248),
                 dict(vs=260), dict(vs=-256), dict(n=-1)):
        assert _append(L, **over) == HB_EINVAL, over
    assert _append(L, n=0, k=None, v=None, slots=None) == HB_OK
    p = ctypes.byref(_pool())
    assert L.hb_kv4_read(p, 16, 4, 16, 252, 16, 256, None) == HB_EINVAL
    assert L.hb_kv4_read(p, None, 4, 16, 256, 16, 256, None) == HB_EINVAL
    assert L.hb_kv4_read(p, None, 0, None, 0, None, 0, None) == HB_OK
    assert L.hb_kv4_append(None, 16, 256, 16, 256, 16, 4, None) == HB_EINVAL


def _decode(L, **over):
    a = dict(q=16, qs=512, bt=16, stride=64, ctx=16, n=4, heads=4, max_ctx=1000, out=16, os=512, ws=16, wn=1 << 40)
    a.update(over)
    return L.hb_kv4_decode(ctypes.byref(_pool()), a["q"], a["qs"], a["bt"], a["stride"], a["ctx"], a["n"], a["heads"],
                           a["max_ctx"], a["out"], a["os"], a["ws"], a["wn"], None)


def test_decode_refusals(L):
    for over in (dict(q=None), dict(bt=None), dict(ctx=None), dict(out=None), dict(q=8), dict(out=24), dict(qs=504),
                 dict(os=516), dict(n=-1), dict(heads=3), dict(heads=0), dict(max_ctx=-1), dict(ws=None), dict(ws=8)):
        assert _decode(L, **over) == HB_EINVAL, over
    for over in (dict(stride=62), dict(wn=0), dict(n=65536), dict(max_ctx=1 << 27, stride=1 << 24)):
        assert _decode(L, **over) == HB_ERANGE, over
    need = cache.kv4_decode_workspace(4, 4, 2, 128, 1000)
    assert need > 0 and _decode(L, wn=need - 1) == HB_ERANGE
    assert _decode(L, n=0, q=None, out=None, bt=None, ctx=None) == HB_OK
    for bad in ((-1, 4, 2, 128, 10), (4, 3, 2, 128, 10), (4, 4, 2, 96, 10), (4, 4, 2, 64, -1), (65536, 4, 2, 64, 10)):
        assert L.hb_kv4_decode_workspace(*bad) == HB_EINVAL
    assert cache.kv4_decode_workspace(0, 4, 2, 64, 10) == 0


def _chunk(L, **over):
    a = dict(q=16, qs=512, bt=16, nb=64, off=1000, n=24, heads=4, out=16, os=512, ws=16, wn=1 << 40)
    a.update(over)
    return L.hb_kv4_chunk(ctypes.byref(_pool()), a["q"], a["qs"], a["bt"], a["nb"], a["off"], a["n"], a["heads"],
                          a["out"], a["os"], a["ws"], a["wn"], None)


def test_chunk_refusals(L):
    for over in (dict(q=None), dict(bt=None), dict(out=None), dict(q=8), dict(out=24), dict(qs=504), dict(os=516),
                 dict(n=-1), dict(off=-1), dict(heads=3), dict(heads=0)):
        assert _chunk(L, **over) == HB_EINVAL, over
    for over in (dict(nb=63), dict(off=1 << 27, nb=1 << 24)):
        assert _chunk(L, **over) == HB_ERANGE, over
    need = cache.kv4_chunk_workspace(100000, 8, 4, 2, 128)
    assert need > 0 and _chunk(L, off=100000, n=8, nb=7000, wn=need - 1) == HB_ERANGE
    assert _chunk(L, off=100000, n=8, nb=7000, ws=8) == HB_EINVAL
    assert _chunk(L, n=0, q=None, out=None, bt=None) == HB_OK
    for bad in ((-1, 4, 4, 2, 128), (0, -1, 4, 2, 128), (0, 4, 3, 2, 128), (0, 4, 4, 2, 80), (1 << 27, 1, 4, 2, 128)):
        assert L.hb_kv4_chunk_workspace(*bad) == HB_EINVAL


def _i32(*v):
    return np.array(v, np.int32)


def _copy(L, src, dst, **over):
    a = dict(data=16, stride=8 * 256, pools=2, page=256, nb=8)
    a.update(over)
    return L.hb_copy_pages(a["data"], a["stride"], a["pools"], a["page"], a["nb"], src.ctypes.data, dst.ctypes.data,
                           len(src), None)


def test_copy_pages_refusals(L):
    one, two = _i32(1), _i32(2)
    for over in (dict(data=None), dict(data=8), dict(page=24), dict(page=0), dict(stride=8 * 256 - 16),
                 dict(stride=2056), dict(pools=0), dict(nb=0)):
        assert _copy(L, one, two, **over) == HB_EINVAL, over
    for s, d in ((_i32(8), two), (one, _i32(8)), (_i32(-1), two), (one, _i32(-1))):
        assert _copy(L, s, d) == HB_ERANGE
    assert _copy(L, _i32(1, 2), _i32(3, 3)) == HB_EINVAL      # a repeated destination
    assert _copy(L, _i32(1, 2), _i32(2, 3)) == HB_EINVAL      # a destination that is a source
    assert _copy(L, _i32(1), _i32(1)) == HB_EINVAL
    assert _copy(L, _i32(), _i32()) == HB_OK
    assert L.hb_copy_pages(16, 2048, 2, 256, 8, None, None, 1, None) == HB_EINVAL
    assert L.hb_copy_blocks(None, None, None, 0) == HB_EINVAL


class Model:
    """The page table's rules, written plainly."""

    def __init__(self, n):
        self.n, self.seqs = n, {}

    def refs(self, b):
        return sum(pages.count(b) for _, pages in self.seqs.values())

    def free(self):
        held = {b for _, pages in self.seqs.values() for b in pages}
        return [b for b in range(self.n) if b not in held]

    def extend(self, s, n):
        have, pages = self.seqs.get(s, (0, []))
        if n < have:
            return "EINVAL"
        pages, free, copy = list(pages), self.free(), None
        split = n > have and have % 16 and self.refs(pages[-1]) > 1
        if (n + 15) // 16 - len(pages) + bool(split) > len(free):
            return "ENOMEM"
        if split:
            copy = (pages[-1], free.pop(0))
            pages[-1] = copy[1]
        while len(pages) < (n + 15) // 16:
            pages.append(free.pop(0))
        self.seqs[s] = (n, pages)
        return copy

    def fork(self, a, b, n):
        if a not in self.seqs or b in self.seqs or n > self.seqs[a][0] or n < -1:
            return "EINVAL"
        m = self.seqs[a][0] if n < 0 else n
        self.seqs[b] = (m, self.seqs[a][1][:(m + 15) // 16])

    def compact(self, most):
        moves = []
        while len(moves) < most:
            free = [f for f in self.free() if f not in [s for s, _ in moves]]
            held = [b for b in range(self.n) if self.refs(b)]
            if not held or not free or held[-1] < free[0]:
                break
            moves.append((held[-1], free[0]))
            self.seqs = {k: (n, [free[0] if b == held[-1] else b for b in p]) for k, (n, p) in self.seqs.items()}
        return moves


def test_page_table_follows_its_rules(L):
    for seed in range(20):
        rng = random.Random(seed)
        n = rng.choice((1, 5, 40))
        t, m = cache.PageTable(n), Model(n)
        for _ in range(150):
            s, what = rng.randrange(8) - 2, rng.random()
            if what < 0.5:
                tokens = max(0, m.seqs.get(s, (0, []))[0] + rng.choice((-1, 0, 1, 1, 5, 16, 17, 60)))
                want = m.extend(s, tokens)
                if isinstance(want, str):
                    with pytest.raises(HbError) as e:
                        t.extend(s, tokens)
                    assert e.value.code == (HB_EINVAL if want == "EINVAL" else HB_ENOMEM)
                else:
                    assert t.extend(s, tokens) == want
            elif what < 0.7:
                child, cut = rng.randrange(8) - 2, rng.choice((-1, 0, 7, 16, 33))
                if m.fork(s, child, cut) == "EINVAL":
                    with pytest.raises(HbError):
                        t.fork(s, child, cut)
                else:
                    t.fork(s, child, cut)
            elif what < 0.9:
                if s in m.seqs:
                    del m.seqs[s]
                    t.release(s)
                else:
                    with pytest.raises(HbError):
                        t.release(s)
            else:
                most = rng.choice((0, 1, 3, n))
                src, dst = t.compact(most)
                assert list(zip(src.tolist(), dst.tolist())) == m.compact(most)
                assert not set(src.tolist()) & set(dst.tolist())
            assert t.num_free == len(m.free())
            for k, (tokens, pages) in m.seqs.items():
                assert t.table(k).tolist() == pages and t.length(k) == tokens
            for b in range(n):
                assert t.refcount(b) == m.refs(b)


def test_page_table_refusals(L):
    with pytest.raises(HbError):
        cache.PageTable(0)
    t = cache.PageTable(4)
    for bad in (lambda: t.table(3), lambda: t.length(3), lambda: t.release(3), lambda: t.fork(3, 4),
                lambda: t.extend(1, -1), lambda: t.refcount(4), lambda: t.refcount(-1), lambda: t.compact(-1)):
        with pytest.raises(HbError):
            bad()
    with pytest.raises(HbError) as e:
        t.extend(1, 2 ** 31 - 1)
    assert e.value.code == HB_ENOMEM and t.num_free == 4
    assert L.hb_pages_create(4, None) == HB_EINVAL
    assert L.hb_pages_num_free(None) == HB_EINVAL
    t.extend(1, 0)  # a sequence of no tokens holds no page and exists
    assert t.length(1) == 0 and t.table(1).tolist() == [] and t.num_free == 4
    t.fork(1, 2)
    assert t.length(2) == 0


def test_large_tables_cost_little(L):
    """Free pages are a bit each; pairs are checked without a look at the pages that they do not name."""
    with pytest.raises(HbError):
        cache.PageTable(1 << 27)
    t = cache.PageTable((1 << 27) - 1)
    assert t.extend(1, 33) is None and t.table(1).tolist() == [0, 1, 2] and t.num_free == (1 << 27) - 4
    t.free()
    for n in (63, 64, 65, 200):                              # every page, whatever the last word holds
        t = cache.PageTable(n)
        t.extend(1, 16 * n)
        assert t.table(1).tolist() == list(range(n)) and t.num_free == 0
        with pytest.raises(HbError):
            t.extend(2, 1)
        assert t.compact()[0].size == 0
        t.release(1)
        assert t.num_free == n
    assert _copy(L, _i32(1, 5), _i32(2, 1), nb=1 << 20, stride=256 << 20) == HB_EINVAL
    for over in (dict(page=1 << 47), dict(page=1 << 40, nb=1 << 20), dict(stride=1 << 60), dict(stride=1 << 46, pools=4)):
        assert _copy(L, _i32(1), _i32(2), **over) == HB_EINVAL, over


def test_numbers_past_32_bits_are_refused_not_cut(L):
    t = cache.PageTable(4)
    t.extend(1, 20)
    big = 1 << 32
    for bad in (lambda: cache.PageTable(big + 4), lambda: t.extend(big + 1, 30), lambda: t.extend(1, big + 30),
                lambda: t.fork(1, big + 2), lambda: t.fork(big + 1, 2), lambda: t.release(big + 1),
                lambda: t.table(big + 1), lambda: t.length(big + 1), lambda: t.refcount(big),
                lambda: cache.kv4_pool_bytes(big + 3, 5, 128), lambda: cache.kv4_decode_workspace(4, 4, 2, 64, big),
                lambda: cache.kv4_chunk_workspace(big, 4, 4, 2, 64)):
        with pytest.raises(HbError) as e:
            bad()
        assert e.value.code == HB_ERANGE
    assert t.length(np.int64(1)) == 20 and t.table(np.int32(1)).tolist() == [0, 1]
    assert t.compact(1 << 40)[0].size == 0
    with pytest.raises(TypeError):
        t.extend(1, 30.5)


def test_binding_checks_tensors(L):
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError):
        cache.Kv4Pool(torch.zeros(2, 2, 18 * 64))                       # not bytes
    with pytest.raises(ValueError):
        cache.Kv4Pool(torch.zeros(2, 2, 100, dtype=torch.uint8))        # not 18 d
    with pytest.raises(HbError):
        cache.Kv4Pool.empty(2, 2, 80, device="cpu")
    p = cache.Kv4Pool.empty(2, 2, 64, device="cpu")
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    slots = torch.zeros(3, dtype=torch.int32)
    for bad in (dict(k=k.float()), dict(k=k[:2]), dict(k=k[:, :1]), dict(k=k.transpose(0, 1)[:, :2]),
                dict(slots=slots.long()), dict()):                      # the last: tensors not on a GPU
        a = dict(k=k, v=k, slots=slots)
        a.update(bad)
        with pytest.raises(ValueError):
            cache.kv4_append(p, a["k"], a["v"], a["slots"])
        with pytest.raises(ValueError):
            cache.kv4_read(p, a["slots"], a["k"], a["v"])
    bt, ctx = torch.zeros(3, 1, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    for q, o, b, c in ((k, k, bt[:2], ctx), (k, k, bt, ctx[:1]), (k, k[:, :1], bt, ctx), (k, k, bt.long(), ctx),
                       (k, k, bt, ctx)):
        with pytest.raises(ValueError):
            cache.kv4_decode(p, q, b, c, 5, o)
    with pytest.raises(ValueError):
        cache.kv4_chunk(p, k, bt[0], 0, k)
    pools = torch.zeros(2, 4, 16)
    for src, dst in (([0], [1, 2]), ([0.5], [1]), ([[0]], [[1]]), ([0], [1])):
        with pytest.raises(ValueError):
            cache.copy_pages(pools, src, dst)
    with pytest.raises(ValueError):
        cache.copy_pages(pools.transpose(1, 2), [0], [1])


def test_chunks_of_more_work_than_a_cta_can_count_are_refused(L):
    """A CTA counts its pages, eight a key tile, in 32 bits: 2^28 tiles are more than it may have."""
    most, last = 1 << 27, 1 << 24
    assert L.hb_kv4_chunk_workspace(most - last, last, 2, 2, 64) == HB_EINVAL       # some 8.5e8 tiles a CTA
    assert _chunk(L, off=most - last, n=last, heads=2, qs=256, os=256, nb=most // 16) == HB_ERANGE
    assert cache.kv4_chunk_workspace(most - last // 4, last // 4, 2, 2, 64) >= 0    # 2.2e8
    assert L.hb_kv4_chunk_workspace(most - last // 2, last // 2, 2, 2, 64) == HB_EINVAL
    assert cache.kv4_chunk_workspace(most - 512, 512, 64, 8, 128) >= 0


def test_compact_refuses_a_count_past_32_bits(L):
    """-2^32 + 5 is not 5: the arrays for the moves would have room for one."""
    t = cache.PageTable(8)
    t.extend(1, 128)
    for most in (-(1 << 32) + 5, -(1 << 32), -(1 << 40) + 1):
        with pytest.raises(HbError) as e:
            t.compact(most)
        assert e.value.code == HB_ERANGE
    with pytest.raises(HbError) as e:
        t.compact(-1)
    assert e.value.code == HB_EINVAL
    assert t.table(1).tolist() == list(range(8))
