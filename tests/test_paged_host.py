"""The calls of include/hb_paged.h without a GPU: what they refuse, and the
binding's checks."""
import ctypes

import numpy as np
import pytest

from chunked_prefill_hybrid_gb300 import native, paged
from chunked_prefill_hybrid_gb300.native import HB_EINVAL, HB_ERANGE, HB_OK, HbError

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def L():
    import __graft_entry__
    __graft_entry__.build_library()
    return paged._lib()


def _pool(**over):
    a = dict(k=16, v=16, num_blocks=8, n_kv_heads=2, head_dim=128)
    a.update(over)
    return paged._pack_pool(*[a[n] or 0 for n in ("k", "v", "num_blocks", "n_kv_heads", "head_dim")])


def _weights(**over):
    a = dict(data=16, num_blocks=8, n_kv_heads=2)
    a.update(over)
    return paged._pack_weights(*[a[n] or 0 for n in ("data", "num_blocks", "n_kv_heads")])


def _ints(x):
    return None if x is None else np.array(x, np.int32).ctypes.data_as(ctypes.c_void_p)


def _shared(L, pool=None, **over):
    a = dict(q=16, qs=512, bt=16, stride=64, ctx=16, n=4, heads=4, max_ctx=1000, rows=[3, 1], pre=[100, 0], out=16,
             os=512, ws=16, wn=1 << 40)
    a.update(over)
    ng = a.get("ng", len(a["rows"]) if a["rows"] is not None else 0)
    return L.hb_decode_shared(pool or _pool(), a["q"], a["qs"], a["bt"], a["stride"], a["ctx"], a["n"],
                              a["heads"], a["max_ctx"], _ints(a["rows"]), _ints(a["pre"]), ng, a["out"], a["os"],
                              a["ws"], a["wn"], None)


def _weigh(L, pool=None, w=None, **over):
    a = dict(q=16, qs=512, bt=16, stride=64, ctx=16, n=2, nq=2, heads=4, max_ctx=1000, wt=16, wstride=64, decay=1.0,
             out=16, os=512, ws=16, wn=1 << 40)
    a.update(over)
    return L.hb_decode_weigh(pool or _pool(), a["q"], a["qs"], a["bt"], a["stride"], a["ctx"], a["n"],
                             a["nq"], a["heads"], a["max_ctx"], w or _weights(), a["wt"], a["wstride"],
                             a["decay"], a["out"], a["os"], a["ws"], a["wn"], None)


def _select(L, w=None, **over):
    a = dict(wt=16, stride=64, lens=16, n=3, max_len=1000, keep=100, first=4, recent=10, kept=16)
    a.update(over)
    return L.hb_evict_select(w or _weights(), a["wt"], a["stride"], a["lens"], a["n"], a["max_len"],
                             a["keep"], a["first"], a["recent"], a["kept"], None)


def _move(L, pool=None, w=None, **over):
    a = dict(bt=16, stride=64, new=16, nstride=7, kept=16, n=3, keep=100, wt=16, wstride=64, nwt=16, nwstride=7)
    a.update(over)
    return L.hb_evict_move(pool or _pool(), a["bt"], a["stride"], a["new"], a["nstride"], a["kept"], a["n"],
                           a["keep"], w, a["wt"], a["wstride"], a["nwt"],
                           a["nwstride"], None)


@pytest.mark.parametrize("over", [dict(k=None), dict(v=None), dict(k=8), dict(v=24), dict(num_blocks=0),
                                  dict(n_kv_heads=0), dict(head_dim=80), dict(num_blocks=-1),
                                  dict(num_blocks=1 << 27)])
def test_bad_pool_is_refused_by_every_call(L, over):
    assert _shared(L, _pool(**over)) == HB_EINVAL
    assert _shared(L, _pool(**over), n=0, rows=[], pre=[]) == HB_EINVAL
    assert _weigh(L, _pool(**over)) == HB_EINVAL
    assert _move(L, _pool(**over)) == HB_EINVAL


@pytest.mark.parametrize("over", [dict(data=None), dict(data=8), dict(num_blocks=0), dict(n_kv_heads=0),
                                  dict(num_blocks=1 << 27)])
def test_bad_weights_are_refused_by_every_call(L, over):
    assert _weigh(L, w=_weights(**over)) == HB_EINVAL
    assert _select(L, w=_weights(**over)) == HB_EINVAL
    assert _move(L, w=_weights(**over)) == HB_EINVAL


def test_shared_refusals(L):
    for over in (dict(q=None), dict(bt=None), dict(ctx=None), dict(out=None), dict(q=8), dict(out=24), dict(qs=504),
                 dict(os=516), dict(qs=508), dict(n=-1), dict(heads=3), dict(heads=0), dict(max_ctx=-1), dict(ws=None),
                 dict(ws=8), dict(bt=18), dict(ctx=17), dict(rows=None, ng=2), dict(pre=None), dict(rows=[3, 2]),
                 dict(rows=[4, 0]), dict(rows=[5, -1]), dict(pre=[-1, 0]), dict(rows=[], pre=[]), dict(n=0),
                 dict(ng=-1)):
        assert _shared(L, **over) == HB_EINVAL, over
    many = dict(n=65536, rows=[65536], pre=[0])
    for over in (dict(stride=62), dict(wn=0), many, dict(max_ctx=1 << 27, stride=1 << 24), dict(pre=[1002, 0])):
        assert _shared(L, **over) == HB_ERANGE, over
    need = paged.decode_shared_workspace(4, 4, 2, 128, 1000, [3, 1], [100, 0])
    assert need > 0 and _shared(L, wn=need - 1) == HB_ERANGE
    assert _shared(L, n=0, rows=[], pre=[], q=None, out=None, bt=None, ctx=None, ws=None, wn=0) == HB_OK
    assert paged.decode_shared_workspace(0, 4, 2, 64, 10, [], []) == 0
    # the most keys there can be: a few splits of 40000 heads, which are tiles enough
    assert paged.decode_shared_workspace(1, 40000, 40000, 64, (1 << 27) - 1, [1], [(1 << 27) - 1]) < 1 << 30
    for bad, code in (((-1, 4, 2, 128, 10), HB_EINVAL), ((4, 3, 2, 128, 10), HB_EINVAL), ((4, 4, 2, 96, 10), HB_EINVAL),
                      ((4, 4, 2, 64, -1), HB_EINVAL), ((65536, 4, 2, 64, 10), HB_ERANGE),
                      ((4, 4, 2, 64, 1 << 27), HB_ERANGE)):
        with pytest.raises(HbError) as e:
            paged.decode_shared_workspace(*bad, [bad[0]], [0])
        assert e.value.code == code, bad
    with pytest.raises(ValueError):
        paged.decode_shared_workspace(4, 4, 2, 64, 10, [4], [0, 0])
    with pytest.raises(HbError):
        paged.decode_shared_workspace(4, 4, 2, 64, 10, [4 + (1 << 32)], [0])


def test_weigh_refusals(L):
    for over in (dict(q=None), dict(bt=None), dict(ctx=None), dict(out=None), dict(wt=None), dict(q=8), dict(out=24),
                 dict(qs=504), dict(os=516), dict(n=-1), dict(nq=0), dict(heads=3), dict(heads=0), dict(max_ctx=-1),
                 dict(ws=None), dict(ws=8), dict(wt=18), dict(decay=-0.5), dict(decay=1.5), dict(decay=float("nan")),
                 dict(decay=float("inf"))):
        assert _weigh(L, **over) == HB_EINVAL, over
    assert _weigh(L, w=_weights(n_kv_heads=1)) == HB_EINVAL
    for over in (dict(stride=62), dict(wstride=62), dict(wn=0), dict(n=65536), dict(n=100, nq=1000), dict(nq=1025),
                 dict(n=1 << 30, nq=4), dict(max_ctx=1 << 27, stride=1 << 24, wstride=1 << 24)):
        assert _weigh(L, **over) == HB_ERANGE, over
    need = paged.decode_weigh_workspace(2, 2, 4, 2, 128, 1000)
    assert need > 0 and _weigh(L, wn=need - 1) == HB_ERANGE
    assert _weigh(L, n=0, q=None, out=None, bt=None, ctx=None, wt=None, ws=None, wn=0) == HB_OK
    assert paged.decode_weigh_workspace(0, 1, 4, 2, 64, 10) == 0
    # past 32 bits: 4 bytes for each row, head and key
    assert paged.decode_weigh_workspace(16, 1, 64, 8, 128, 4000000) > 16 * 64 * 4000000 * 4
    for bad in ((-1, 1, 4, 2, 64, 10), (1, 0, 4, 2, 64, 10), (1, 1, 3, 2, 64, 10), (1, 1, 4, 2, 80, 10),
                (1, 1, 4, 2, 64, -1), (70000, 1, 4, 2, 64, 10), (1, 1 << 32, 4, 2, 64, 10)):
        with pytest.raises(HbError):
            paged.decode_weigh_workspace(*bad)


def test_select_refusals(L):
    for over in (dict(wt=None), dict(lens=None), dict(kept=None), dict(wt=18), dict(lens=18), dict(kept=18), dict(n=-1),
                 dict(max_len=-1), dict(keep=0), dict(keep=-3), dict(first=-1), dict(recent=-1), dict(first=91),
                 dict(first=1 << 30, recent=1 << 30, keep=(1 << 31) - 1)):
        assert _select(L, **over) == HB_EINVAL, over
    for over in (dict(stride=62), dict(n=65536), dict(max_len=(1 << 27) + 1, stride=1 << 24),
                 dict(keep=(1 << 27) + 1)):
        assert _select(L, **over) == HB_ERANGE, over
    assert _select(L, n=0, wt=None, lens=None, kept=None) == HB_OK


def test_move_refusals(L):
    for over in (dict(bt=None), dict(new=None), dict(kept=None), dict(bt=18), dict(new=18), dict(kept=18), dict(n=-1),
                 dict(keep=0), dict(stride=0)):
        assert _move(L, **over) == HB_EINVAL, over
        assert _move(L, w=_weights(), **over) == HB_EINVAL, over
    for over in (dict(wt=None), dict(nwt=None), dict(wt=18), dict(nwt=18), dict(wstride=0)):
        assert _move(L, w=_weights(), **over) == HB_EINVAL, over
    assert _move(L, w=_weights(n_kv_heads=3)) == HB_EINVAL
    for over in (dict(nstride=6), dict(n=65536), dict(keep=(1 << 27) + 1, nstride=1 << 24)):
        assert _move(L, **over) == HB_ERANGE, over
    assert _move(L, w=_weights(), nwstride=6) == HB_ERANGE
    big = (1 << 27) - 1  # rows of a pool past 32 bits
    assert _move(L, _pool(num_blocks=big, n_kv_heads=3)) == HB_ERANGE
    assert _move(L, _pool(n_kv_heads=3), w=_weights(num_blocks=big, n_kv_heads=3)) == HB_ERANGE
    assert _move(L, n=0, bt=None, new=None, kept=None) == HB_OK


def test_binding_refuses_what_only_tensors_show(L):
    bf, i32 = torch.bfloat16, torch.int32
    k = torch.zeros(4, 2, 16, 64, dtype=bf)
    for bad in ((k[:, :, :8], k[:, :, :8]), (k, k[:2]), (k.float(), k.float()), (k[0], k[0]),
                (k.transpose(0, 1), k.transpose(0, 1))):
        with pytest.raises(ValueError):
            paged.PagedPool(*bad)
    pool = paged.PagedPool(k, k.clone())
    assert (pool.num_blocks, pool.n_kv_heads, pool.head_dim) == (4, 2, 64)
    q, bt, ctx = torch.zeros(3, 4, 64, dtype=bf), torch.zeros(3, 2, dtype=i32), torch.zeros(3, dtype=i32)
    w, kept = torch.zeros(4, 2, 16), torch.zeros(3, 2, 8, dtype=i32)
    for call in (lambda: paged.decode_shared(pool, q, bt, ctx, 20, [3], [0], q.clone()),  # host memory
                 lambda: paged.decode_shared(pool, q[0], bt, ctx, 20, [3], [0], q[0]),
                 lambda: paged.decode_shared(pool, q, bt, ctx, 20, [3], [0, 1], q.clone()),
                 lambda: paged.decode_shared(pool, q, bt, ctx, 20, [3.0], [0], q.clone()),
                 lambda: paged.decode_weigh(pool, q, bt, ctx, 20, w, bt, 1.0, q.clone()),
                 lambda: paged.decode_weigh(pool, q, bt[:2], ctx[:2], 20, w, bt[:2], 1.0, q.clone()),
                 lambda: paged.evict_select(w, bt, ctx, 20, 8, 0, 0, kept),
                 lambda: paged.evict_select(w[0], bt, ctx, 20, 8, 0, 0, kept),
                 lambda: paged.evict_move(pool, bt, bt, kept),
                 lambda: paged.evict_move(pool, bt, bt, kept[:, :1])):
        with pytest.raises(ValueError):
            call()
