"""The failure path of the attention that takes a group's or a window's common
keys at once, without faulting the GPU: a hook makes one CTA of a launch leave
out one copy, so that the waits for it reach their limit of two seconds.  No
address changes and no copy is left under way.  What the CTA was to compute
becomes NaN, everything else and the calls after it are as ever."""
import pytest

from chunked_prefill_hybrid_gb300 import paged

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def _pool(keys, kv, d):
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn(-(-keys // 16), kv, 16, d, generator=g, device="cuda").bfloat16() for _ in range(2))
    return paged.PagedPool(k, v), torch.arange(k.shape[0], dtype=torch.int32, device="cuda"), g


# few rows, and more than one Q tile; one sub-tile and many
@pytest.mark.parametrize("rows,prefix,kv,group,d", [(9, 4000, 2, 2, 128), (60, 3000, 1, 5, 64), (160, 1024, 2, 1, 128),
                                                    (20, 64, 50, 1, 128)])
def test_shared_prefix_that_loses_a_block(rows, prefix, kv, group, d):
    assert (rows - 1) * prefix * kv * 4 * d >= 24 << 20  # enough for one pass over the prefix
    pool, table, g = _pool(prefix + 16, kv, d)
    q = torch.randn(rows, kv * group, d, generator=g, device="cuda").bfloat16()
    ctx = torch.full((rows,), prefix + 5, dtype=torch.int32, device="cuda")
    tables = table.repeat(rows, 1)

    def call(out):
        paged.decode_shared(pool, q, tables, ctx, prefix + 5, [rows], [prefix], out)

    good, out = torch.empty_like(q), torch.empty_like(q)
    call(good)
    assert torch.isfinite(good).all()
    paged.paged_test_lost_block()
    call(out)
    torch.cuda.synchronize()
    want = torch.zeros(rows, kv * group, dtype=torch.bool, device="cuda")
    first = torch.arange(rows * group, device="cuda") < 256  # the first kv head's (row, head) pairs, 256 of them
    want.view(rows, kv, group)[:, 0] = first.view(rows, group)
    nan = torch.isnan(out)
    assert torch.equal(nan.any(-1), nan.all(-1))
    assert torch.equal(nan.all(-1), want)
    assert torch.equal(out[~want], good[~want])
    for _ in range(2):
        call(out)
        assert torch.equal(out, good)


@pytest.mark.parametrize("nq,kv,group,d", [(16, 2, 2, 128), (70, 1, 4, 64)])
def test_window_that_loses_a_block(nq, kv, group, d):
    keys = 1500
    pool, table, g = _pool(keys, kv, d)
    q = torch.randn(nq, kv * group, d, generator=g, device="cuda").bfloat16()
    ctx = torch.tensor([keys - 1], dtype=torch.int32, device="cuda")
    w0 = torch.rand(table.numel(), kv, 16, generator=g, device="cuda")

    def call():
        out, w = torch.empty_like(q), w0.clone()
        paged.decode_weigh(pool, q, table[None], ctx, keys - 1, w, table[None], 1.0, out)
        torch.cuda.synchronize()
        return out, w

    good = call()
    paged.paged_test_lost_block()
    out, w = call()
    lost = torch.isnan(out).all(-1)
    assert torch.equal(torch.isnan(out).any(-1), lost)
    want = torch.zeros(nq, kv, group, dtype=torch.bool, device="cuda")
    want[:, 0] = (torch.arange(nq * group, device="cuda") < 256).view(nq, group)
    assert torch.equal(lost, want.view(nq, -1))
    assert torch.equal(out[~lost], good[0][~lost])
    # the lost rows add nothing: no weight is more than before and the good ones' sum, none is less than before
    old = (torch.arange(keys, device="cuda") < keys - nq)  # the call's own rows start from 0
    flat = lambda x: x.transpose(0, 1).reshape(kv, -1)[:, :keys]  # noqa: E731
    assert torch.isfinite(w).all()
    assert (flat(w) <= flat(good[1]) * (1 + 1e-5)).all() and (flat(w) >= flat(w0) * old * (1 - 1e-6)).all()
    assert torch.equal(flat(w)[1:], flat(good[1])[1:])
    again = call()
    assert torch.equal(again[0], good[0]) and torch.equal(again[1], good[1])
