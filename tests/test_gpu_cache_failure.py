"""The failure path of the attention over the 4-bit cache, without faulting
the GPU: a hook makes one CTA of a launch leave out one page's copy, so that
the waits for it reach their limit of two seconds.  No address changes and no
copy is left under way.  What the CTA was to compute becomes NaN, everything
else and the calls after it are as ever."""
import pytest

from chunked_prefill_hybrid_gb300 import cache

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def _pool(keys, kv, d):
    pool = cache.Kv4Pool.empty((keys + 15) // 16, kv, d)
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn(keys, kv, d, generator=g, device="cuda").bfloat16() for _ in range(2))
    cache.kv4_append(pool, k, v, torch.arange(keys, dtype=torch.int32, device="cuda"))
    return pool, torch.arange(pool.num_blocks, dtype=torch.int32, device="cuda"), g


def _lose_a_page(call, like):
    """(rows and heads that became NaN, the good result)"""
    good, out = torch.empty_like(like), torch.empty_like(like)
    call(good)
    assert torch.isfinite(good).all()
    cache.kv4_test_lost_page()
    call(out)
    torch.cuda.synchronize()
    nan = torch.isnan(out)
    assert torch.equal(nan.any(-1), nan.all(-1))
    lost = nan.any(-1)
    assert torch.equal(out[~lost], good[~lost])
    for _ in range(2):
        call(out)
        assert torch.equal(out, good)
    return lost


@pytest.mark.parametrize("rows,keys,kv,group,d", [(3, 500, 2, 1, 128), (1, 20000, 2, 1, 128), (3, 700, 2, 12, 64),
                                                  (300, 40, 4, 1, 128)])
def test_decode_that_loses_a_page(rows, keys, kv, group, d):
    pool, table, g = _pool(keys, kv, d)
    q = torch.randn(rows, kv * group, d, generator=g, device="cuda").bfloat16()
    ctx = torch.full((rows,), keys - 1, dtype=torch.int32, device="cuda")
    tables = table.repeat(rows, 1)
    lost = _lose_a_page(lambda out: cache.kv4_decode(pool, q, tables, ctx, keys - 1, out), q)
    want = torch.zeros_like(lost)
    want[0, :min(group, 8)] = True                           # the first CTA's queries
    assert torch.equal(lost, want)


@pytest.mark.parametrize("kv,group,d,offset,n", [(2, 1, 64, 300, 5), (4, 2, 128, 2000, 257), (5, 3, 64, 12001, 301),
                                                 (8, 1, 128, 0, 1500), (8, 1, 128, 16000, 300)])
def test_chunk_that_loses_a_page(kv, group, d, offset, n):
    pool, table, g = _pool(offset + n, kv, d)
    q = torch.randn(n, kv * group, d, generator=g, device="cuda").bfloat16()
    lost = _lose_a_page(lambda out: cache.kv4_chunk(pool, q, table, offset, out), q)
    assert lost[0, 0] and not lost.all()

