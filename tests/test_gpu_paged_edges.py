"""The attention calls of include/hb_paged.h on the GPU where workspaces and
numbers are the least usual that they allow, against plain 64-bit forms
(paged_ref.py)."""
import numpy as np
import pytest

from chunked_prefill_hybrid_gb300 import paged
from test_gpu_paged import Case, _dev, _weigh_case

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def _weigh(c, nq, decay, workspace=None, max_ctx=None):
    out, w = torch.full_like(c.q, 7.0), c.w.clone()
    paged.decode_weigh(c.pool, c.q, _dev(c.tables), _dev(c.ctx), int(c.ctx.max()) if max_ctx is None else max_ctx, w,
                       _dev(c.wtables), decay, out, workspace)
    torch.cuda.synchronize()
    return out, w


def _offset_workspace(need, offset):
    """A workspace of exactly `need` bytes at `offset` past a multiple of 256, and the bytes about it, which stay 0x5a."""
    arena = torch.full((need + 512,), 0x5a, dtype=torch.uint8, device="cuda")
    at = -arena.data_ptr() % 256 + offset
    ws, rest = arena[at:at + need], torch.ones_like(arena, dtype=torch.bool)
    rest[at:at + need] = False
    assert ws.data_ptr() % 256 == offset
    return ws, lambda: bool((arena[rest] == 0x5a).all())


@pytest.mark.parametrize("kv,group,d,rows,prefix", [
    (2, 1, 128, [18], [1500]),              # one Q tile
    (1, 20, 64, [30], [3603]),              # several
    (2, 1, 128, [1, 30] * 10, [50, 900] * 10),   # groups in the workspace too
    (2, 3, 64, [2, 3], [0, 37]),            # no prefix in one pass
])
def test_shared_takes_any_workspace_at_sixteen_bytes(kv, group, d, rows, prefix):
    ctx = [p + 9 * (i % 5) for r, p in zip(rows, prefix) for i in range(r)]
    c = Case(71, kv, group, d, rows, prefix, ctx)
    need = paged.decode_shared_workspace(len(ctx), kv * group, kv, d, max(ctx) + 700, rows, prefix)
    want = c.run(max_ctx=max(ctx) + 700)
    for offset in (0, 16, 32, 48):
        ws, whole = _offset_workspace(need, offset)
        assert torch.equal(c.run(max_ctx=max(ctx) + 700, workspace=ws), want), offset
        assert whole(), offset


@pytest.mark.parametrize("kv,group,d,ctx,nq", [
    (1, 4, 128, [1300, 40, 3], 70),         # a window's common keys in one pass
    (2, 2, 64, [700, 1500], 16),
    (1, 8, 64, [9000, 30], 1),              # splits, the join beside the weights
    (1, 8, 64, [400, 17], 1),               # scores of one split in the workspace
])
def test_weigh_takes_any_workspace_at_sixteen_bytes(kv, group, d, ctx, nq):
    c = _weigh_case(72, kv, group, d, ctx, nq)
    need = paged.decode_weigh_workspace(len(ctx), nq, kv * group, kv, d, max(ctx))
    want = _weigh(c, nq, 0.5, None)
    for offset in (0, 16, 32, 48):
        ws, whole = _offset_workspace(need, offset)
        got = _weigh(c, nq, 0.5, ws)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), offset
        assert whole(), offset


def _level_scores(c, rng, scale):
    """K and q so that every score is exact in 32 bits, of magnitude `scale` to twice that, and the keys of a row lie within 24 of one
    another: q . k = q0 k0 + q1 k1 with few bits in each, rising with the position.  V tells where a key lies."""
    n, heads, d = c.q.shape
    for j in range(len(c.ctx)):
        t = np.arange(int(c.ctx[j]) + 1)
        p = c.prefix[int(np.searchsorted(np.cumsum(c.rows), j, side="right"))]
        level = np.where(t < p, 8 * t // max(1, p), 3 + j % 4)
        page, slot = _dev(c.tables[j, t // 16], np.int64), _dev(t % 16, np.int64)
        # the last digit of a token's level goes by its position alone, as rows share the prefix' tokens
        value = torch.from_numpy((level + (t * 7919 % 13) % 5).astype(np.float32)).cuda()
        c.k[page, :, slot, 0] = 2.0 ** 6
        c.k[page, :, slot, 1] = value.to(torch.bfloat16)[:, None]
        c.v[page, :, slot] = (0.25 * torch.randn(c.kv, len(t), d, generator=rng, device="cuda").transpose(0, 1)
                              + torch.where(torch.from_numpy(t % 512 < 256).cuda(), 1.0, -1.0)[:, None, None]).to(torch.bfloat16)
    c.q.zero_()
    at = torch.arange(n * heads, device="cuda").view(n, heads) % 32
    c.q[:, :, 0] = ((1 + at / 64) * scale * 2.0 ** -6 * torch.where(at % 3 == 2, -1.0, 1.0)).to(torch.bfloat16)
    c.q[:, :, 1] = 2.0


def _exact(c, j, row, see):
    """o, p and sum p |v| of one row whose scores are exact."""
    d = c.d
    page = _dev(c.tables[j, :(see + 15) // 16]).long()
    k, v = (pool[page].double().transpose(0, 1).flatten(1, 2)[:, :see] for pool in (c.k, c.v))
    s = torch.einsum("hgd,hkd->hgk", c.q[row].double().view(c.kv, c.group, d), k)
    assert torch.equal(s, s.float().double()) and float((s.amax(-1) - s.amin(-1)).max()) <= 24
    p = torch.softmax(s / d ** 0.5, -1)
    return torch.einsum("hgk,hkd->hgd", p, v), p, torch.einsum("hgk,hkd->hgd", p, v.abs())


# A weight 2^((s - m) log2(e) / sqrt d) of exact scores at most 24 apart: an exponent of at most 24 x 1.45 / 8 < 5 with
# log2(e) / sqrt d off by 2^-23 of it and a product rounded by 2^-24 (together < 2^-20), and four exponentials (its own,
# a rescaled maximum's, the halves' and the join's) of 2^-22 each
EXACT_EPS = 2.0 ** -20 + 4 * 2.0 ** -22


@pytest.mark.parametrize("scale", [2.0 ** 6, 2.0 ** 15, 2.0 ** 20, 2.0 ** 21, 2.0 ** 22, 2.0 ** 23])
@pytest.mark.parametrize("kv,group,d,rows,prefix", [
    (1, 1, 128, 20, 6000),       # one Q tile
    (1, 8, 128, 20, 6000),       # two
    (2, 3, 64, 30, 4001),        # one
])
def test_shared_large_scores_that_are_exact(kv, group, d, rows, prefix, scale):
    """Whatever the scores' magnitude, keys of all parts of a prefix and own keys are weighed by their differences."""
    ctx = [prefix + 30 + 11 * j for j in range(rows)]
    c = Case(81, kv, group, d, [rows], [prefix], ctx, poison=False)
    assert (rows - 1) * (prefix // 16 * 16) * kv * 4 * d >= 24 << 20
    _level_scores(c, torch.Generator(device="cuda").manual_seed(3), scale)
    for max_ctx in (max(ctx), max(ctx) + 3000):
        out = c.run(max_ctx=max_ctx)
        for j in range(rows):
            m = ctx[j] + 1
            o, _, w = _exact(c, j, j, m)
            bound = 2.0 ** -8 * o.abs() + w * (2.0 ** -16 + 2 * EXACT_EPS + (m / 16 + 64) * 2.0 ** -23)
            off = (out[j].double().view_as(o) - o).abs()
            assert (off <= bound).all(), (j, (off / bound).max(), off.max())


@pytest.mark.parametrize("scale", [2.0 ** 6, 2.0 ** 15, 2.0 ** 20, 2.0 ** 21, 2.0 ** 22, 2.0 ** 23])
@pytest.mark.parametrize("kv,group,d,nq", [(1, 4, 128, 32), (2, 2, 64, 70)])
def test_weigh_large_scores_that_are_exact(kv, group, d, nq, scale):
    """The same for a window's rows and their weights."""
    ctx = [4000, 2600]
    c = _weigh_case(82, kv, group, d, ctx, nq, poison=False)
    c.prefix = [x + 1 for x in ctx]
    _level_scores(c, torch.Generator(device="cuda").manual_seed(4), scale)
    out, w = _weigh(c, nq, 0.0)
    for j, x in enumerate(ctx):
        total = torch.zeros(kv, x + 1, dtype=torch.float64, device="cuda")
        for i in range(nq):
            see = x + 1 - (nq - 1) + i
            o, p, mass = _exact(c, j, j * nq + i, see)
            bound = 2.0 ** -8 * o.abs() + mass * (2.0 ** -16 + 2 * EXACT_EPS + (see / 16 + 64) * 2.0 ** -23)
            off = (out[j * nq + i].double().view_as(o) - o).abs()
            assert (off <= bound).all(), (j, i, (off / bound).max())
            total[:, :see] += p.sum(1)
        got = w[_dev(c.wtables[j, :(x + 16) // 16]).long()].double().transpose(0, 1).flatten(1, 2)[:, :x + 1]
        # a weight and the sum that it is divided by are off by EXACT_EPS each, and sums of see and nq x group numbers
        assert ((got - total).abs() <= total * (2 * EXACT_EPS + (x / 16 + 64 + nq * group) * 2.0 ** -23)).all()


INF, NAN = float("inf"), float("nan")


def _plant(c, j, at):
    """Infinities and NaN in V of row j's tokens, of every kv head: channel -> token, value.  Channels 1 to 5 become
    +inf, -inf, +inf of two tokens, NaN of two infinities, NaN."""
    a, b = at
    for t, e, x in ((a, 1, INF), (b, 2, -INF), (a, 3, INF), (b, 3, INF), (a, 4, INF), (b, 4, -INF), (b, 5, NAN)):
        c.v[int(c.tables[j, t // 16]), :, t % 16, e] = x


def _planted(out, was, seen, by_key=False):
    """out against the call without them: rows `seen` have what _plant says, everything else has the same bits.  by_key:
    the channels beside them are summed in another order, each within 2^-8 of itself and 2^-15 of sum p |v| < 1 of the
    formula's."""
    got, want = out.clone(), was.clone()
    want[seen, :, 1], want[seen, :, 2], want[seen, :, 3] = INF, -INF, INF
    want[seen, :, 4:6] = NAN
    bad = torch.isnan(want)
    assert torch.equal(torch.isnan(got), bad)
    if by_key:
        bad |= torch.isinf(want)
        assert torch.equal(got[torch.isinf(want)], want[torch.isinf(want)])
        assert ((got - want).abs() <= 2.0 ** -7 * want.abs() + 2.0 ** -14)[~bad].all()
    else:
        assert torch.equal(got[~bad], want[~bad])


@pytest.mark.parametrize("kv,group,d,ctx,at", [
    (1, 1, 64, [0, 4], (0, 0)),               # one key, whose weight is 1
    (2, 1, 128, [5, 40], (2, 3)),
    (1, 12, 64, [333, 100], (17, 300)),       # four warps, more than eight heads
    (1, 2, 128, [3000, 2100], (5, 2999)),     # splits and their join
    (2, 1, 64, [60000], (100, 59999)),        # many splits
    (4, 1, 64, [100] * 150, (3, 99)),         # a warp a row and head
])
def test_shared_infinities_in_v(kv, group, d, ctx, at):
    """An infinity of V that a row sees is that row's, in its channel alone."""
    c = Case(91, kv, group, d, [1] * len(ctx), [0] * len(ctx), ctx)
    was = c.run()
    if at[0] == at[1]:
        c.v[int(c.tables[0, 0]), :, 0, 1], c.v[int(c.tables[0, 0]), :, 0, 2] = INF, -INF
        out = c.run()
        want = was.clone()
        want[0, :, 1], want[0, :, 2] = INF, -INF
        assert torch.equal(out, want)
        return
    _plant(c, 0, at)
    _planted(c.run(), was, [0])


@pytest.mark.parametrize("kv,group,d,rows,prefix,at", [
    (2, 1, 128, 18, 1500, (3, 1400)),         # one Q tile
    (1, 20, 64, 30, 3603, (64, 65)),          # several, neighbours
    (50, 1, 128, 21, 64, (0, 63)),            # one sub-tile
    (2, 1, 128, 18, 1500, (1501, 1510)),      # a row's own keys
    (1, 8, 128, 20, 6000, (5999, 3000)),
])
def test_shared_prefix_infinities_in_v(kv, group, d, rows, prefix, at):
    assert (rows - 1) * (prefix // 16 * 16) * kv * 4 * d >= 24 << 20
    c = Case(92, kv, group, d, [rows], [prefix], [prefix + 20 + j for j in range(rows)])
    was = c.run()
    _plant(c, 0, at)
    everyone = all(t < prefix // 16 * 16 for t in at)
    _planted(c.run(), was, list(range(rows)) if everyone else [0])


def test_shared_infinity_of_a_key_that_weighs_nothing():
    """A weight that is 0 in 32 bits: its channel is infinite or not a number, and the others have the same bits."""
    for rows, prefix, ctx in (([1], [0], [3000]), ([20], [2000], [2100] * 20), ([3], [0], [200, 180, 150])):
        c = Case(93, 2, 1, 128, rows, prefix, ctx, poison=False)
        t = 77
        c.k[int(c.tables[0, t // 16]), :, t % 16] = 0.0
        c.k[int(c.tables[0, t // 16]), :, t % 16, 0] = -30000.0
        c.q[:, :, 0] = 5.0
        was = c.run()
        c.v[int(c.tables[0, t // 16]), :, t % 16, 7] = INF
        out = c.run()
        seen = slice(0, None if prefix[0] else 1)
        assert (torch.isnan(out) | (out == INF))[seen, :, 7].all()
        out[seen, :, 7] = was[seen, :, 7]
        assert torch.equal(out, was)


@pytest.mark.parametrize("kv,group,d,ctx,nq,at", [
    (1, 3, 64, [60], 6, (10, 20)),            # pages that all queries see, no common keys
    (2, 1, 128, [40, 30], 1, (3, 39)),
    (1, 8, 64, [9000, 40], 1, (100, 8999)),   # splits, the join beside the weights
    (1, 4, 128, [1300, 200], 70, (5, 1000)),  # common keys
    (2, 2, 64, [1500, 70], 16, (700, 1484)),  # common keys and a page that not all of them see in whole
])
def test_weigh_infinities_in_v(kv, group, d, ctx, nq, at):
    """The same, and the weights do not change."""
    c = _weigh_case(94, kv, group, d, ctx, nq)
    was, weights = _weigh(c, nq, 0.5)
    _plant(c, 0, at)
    out, w = _weigh(c, nq, 0.5)
    _planted(out, was, list(range(nq)), by_key=at[1] > ctx[0] - 17 and nq > 1)
    assert torch.equal(w, weights)
