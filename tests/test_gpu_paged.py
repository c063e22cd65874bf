"""Attention over shared prefixes, attention weights and eviction on the GPU,
against plain 64-bit forms (paged_ref.py)."""
import numpy as np
import pytest

import paged_ref as ref
from chunked_prefill_hybrid_gb300 import cache, native, paged
from chunked_prefill_hybrid_gb300.native import HbError

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

NAN = float("nan")


def _f64(t):
    return t.double().cpu().numpy()


def _dev(x, dtype=np.int32):
    return torch.from_numpy(np.ascontiguousarray(x, dtype)).cuda()


def _bf(rng, *shape, scale=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(torch.bfloat16).cuda()


class Case:
    """Rows in groups over one pool: row j's table starts with its group's shared pages."""

    def __init__(self, seed, kv, group, d, rows, prefix, ctx, spare=2, poison=True, scale=1.0):
        rng = np.random.default_rng(seed)
        self.kv, self.group, self.d, self.rows, self.prefix = kv, group, d, list(rows), list(prefix)
        self.ctx = np.array(ctx, np.int64)
        n = len(ctx)
        assert n == sum(rows)
        of = np.repeat(np.arange(len(rows)), rows)
        shared = np.array(prefix)[of] // 16
        width = max(1, int(max(max(self.ctx) // 16 + 1, max(shared))))
        need = np.maximum(self.ctx // 16 + 1 - shared, 0)
        blocks = int(need.sum()) + sum(p // 16 for p in prefix) + spare
        perm = list(rng.permutation(blocks))
        common = [[perm.pop() for _ in range(p // 16)] for p in prefix]
        self.tables = np.full((n, width), -1, np.int64)  # entries that nothing needs are never read
        for j in range(n):
            t = common[of[j]] + [perm.pop() for _ in range(need[j])]
            self.tables[j, :len(t)] = t
        self.k, self.v = _bf(rng, blocks, kv, 16, d, scale=scale), _bf(rng, blocks, kv, 16, d)
        first = np.cumsum(rows) - rows
        for g, p in enumerate(prefix):  # the part-filled page: the same tokens in each row's copy
            if p % 16:
                for j in range(first[g] + 1, first[g] + rows[g]):
                    a, b = self.tables[first[g], p // 16], self.tables[j, p // 16]
                    if a >= 0 and b >= 0:
                        for pool in (self.k, self.v):
                            pool[b, :, :p % 16] = pool[a, :, :p % 16]
        if poison:  # every slot that no row sees
            seen = np.zeros((blocks, 16), bool)
            for g, p in enumerate(prefix):
                for b in common[g]:
                    seen[b] = True
            for j in range(n):
                for t in range(self.ctx[j] + 1):
                    seen[self.tables[j, t // 16], t % 16] = True
            hide = torch.from_numpy(~seen).cuda()
            for pool, bad in ((self.k, NAN), (self.v, float("inf"))):
                pool.transpose(1, 2)[hide] = bad
        self.q = _bf(rng, n, kv * group, d)
        self.pool = paged.PagedPool(self.k, self.v)

    def run(self, q=None, out=None, max_ctx=None, ctx=None, tables=None, workspace=None):
        q = self.q if q is None else q
        out = torch.full_like(self.q, 7.0) if out is None else out
        max_ctx = max(0, int(self.ctx.max())) if max_ctx is None else max_ctx
        tables = self.tables if tables is None else tables
        if tables.shape[1] < max_ctx // 16 + 1:
            tables = np.pad(tables, ((0, 0), (0, max_ctx // 16 + 1 - tables.shape[1])), constant_values=-1)
        paged.decode_shared(self.pool, q, _dev(tables), _dev(self.ctx if ctx is None else ctx), max_ctx, self.rows,
                            self.prefix, out, workspace)
        torch.cuda.synchronize()
        return out

    def check_large(self, out, rows=None):
        """check() on the GPU, in 64 bits as well."""
        n, heads, d = self.q.shape
        for j in range(n) if rows is None else rows:
            m = int(self.ctx[j]) + 1
            page = _dev(self.tables[j, :(m + 15) // 16]).long()
            k, v = (pool[page].double().transpose(0, 1).flatten(1, 2)[:, :m] for pool in (self.k, self.v))
            q = self.q[j].double().view(self.kv, self.group, d)
            p = torch.softmax(torch.einsum("hgd,hkd->hgk", q, k) / d ** 0.5, -1)
            o, w = torch.einsum("hgk,hkd->hgd", p, v), torch.einsum("hgk,hkd->hgd", p, v.abs())
            a = torch.einsum("hgd,hkd->hgk", q.abs(), k.abs()).amax(-1, keepdim=True) / d ** 0.5
            eps = 2.0 ** -21 + (d + 8) * 2.0 ** -23 * a
            bound = 2.0 ** -8 * o.abs() + w * (2.0 ** -16 + 2 * eps + (m / 16 + 64) * 2.0 ** -23) + 1e-37
            off = (out[j].double().view_as(o) - o).abs()
            assert (off <= bound).all(), (j, off.max(), bound.max())

    def check(self, out, rows=None):
        o, b = ref.shared(_f64(self.q), _f64(self.k), _f64(self.v), self.tables, self.ctx, self.group)
        rows = range(len(self.ctx)) if rows is None else rows
        got = _f64(out)
        for j in rows:
            assert (np.abs(got[j] - o[j]) <= b[j]).all(), (j, np.abs(got[j] - o[j]).max(), b[j].max())


# ----------------------------------------------------------- shared prefixes

@pytest.mark.parametrize("kv,group,d,rows,prefix,ctx", [
    (1, 1, 64, [1], [0], [0]),                                          # one row, one key
    (2, 1, 128, [4], [64], [64, 79, 80, 200]),
    (3, 1, 64, [3], [16], [15, 16, 300]),                               # a row whose own keys are none
    (2, 3, 128, [2, 3], [0, 37], [0, 5, 36, 37, 90]),                   # an odd prefix, part-filled pages
    (1, 8, 128, [5], [1000], [1000, 1001, 1015, 1016, 2100]),
    (2, 12, 64, [2, 1], [100, 50], [99, 130, 700]),                     # more than eight heads a kv head
    (1, 20, 128, [3], [333], [333, 500, 340]),
    (1, 5, 64, [2, 2], [15, 17], [14, 15, 16, 17]),                     # prefixes about one page
    (5, 1, 128, [18], [768], [1024] * 18),
    (2, 4, 128, [40], [513], [513 + 7 * j for j in range(40)]),         # more queries than a tile of 128
    (1, 64, 64, [9, 1, 2], [640, 640, 0], [640 + j for j in range(9)] + [700, 3, 650]),
    (1, 1, 128, [150], [2049], [2049 + j for j in range(150)]),
])
def test_shared_matches_the_plain_form(kv, group, d, rows, prefix, ctx):
    c = Case(sum(ctx) + kv, kv, group, d, rows, prefix, ctx)
    out = c.run()
    c.check(out)
    assert torch.equal(out, c.run())  # the same bits again
    wide = c.run(max_ctx=max(ctx) + 4000)  # another split of the keys
    c.check(wide)


SHARE = 24 << 20  # bytes of reads that are saved from which on a prefix is read once


@pytest.mark.parametrize("kv,group,d,rows,prefix,own", [
    (2, 1, 128, [18], [1500], 300),         # one Q tile
    (1, 8, 128, [16], [3500], 40),          # exactly 128 queries, an odd prefix
    (1, 3, 128, [43], [1616], 5),           # 129: a second tile with one row; a last sub-tile of one block
    (4, 2, 128, [128], [112], 20),          # 256: two sub-tiles, the last of three blocks
    (1, 1, 128, [257], [208], 33),          # 257: a CTA with one row
    (40, 1, 64, [130], [64], 17),           # one sub-tile, two Q tiles
    (50, 1, 128, [21], [64], 17),           # one sub-tile, one Q tile: the second half has nothing
    (1, 20, 64, [30], [3603], 100),         # 600 queries
    (1, 5, 64, [30, 1, 60], [5000, 700, 2500], 64),   # two prefixes shared, one not
    (2, 1, 128, [20, 20], [1400, 50], 900),           # one shared, one too short for it
])
def test_shared_prefix_in_one_pass(kv, group, d, rows, prefix, own):
    """Prefixes long enough to be read once for their groups, on the tensor cores."""
    rng = np.random.default_rng(len(rows) + d)
    assert (rows[0] - 1) * (prefix[0] // 16 * 16) * kv * 4 * d >= SHARE
    ctx = [p + int(rng.integers(0, own)) for r, p in zip(rows, prefix) for _ in range(r)]
    ctx[0] = prefix[0] - 1  # a row whose own keys are none but the part-filled block's
    c = Case(sum(rows), kv, group, d, rows, prefix, ctx)
    out = c.run()
    c.check_large(out)
    assert torch.equal(out, c.run())
    c.check_large(c.run(max_ctx=max(ctx) + 3000))


def test_shared_prefix_in_one_pass_of_many_groups():
    """More groups than the kernels' parameters hold, some of them shared."""
    rows, prefix = [1, 30] * 10, [50, 900] * 10
    ctx = [p + 7 * (i % 9) for i, (r, p) in enumerate(zip(rows, prefix)) for _ in range(r)]
    c = Case(44, 2, 1, 128, rows, prefix, ctx)
    assert (30 - 1) * 896 * 2 * 512 >= SHARE
    c.check_large(c.run())


def test_shared_prefix_in_one_pass_padding_and_bad_blocks():
    c = Case(45, 2, 2, 128, [40, 3], [700, 0], [700 + j for j in range(40)] + [9, 40, 3])
    assert 39 * 688 * 2 * 512 >= SHARE
    ctx = c.ctx.copy()
    ctx[[0, 17]], ctx[3], ctx[4] = -1, 698, 100000   # padding, not covering the prefix, past max_ctx
    out = c.run(ctx=ctx, max_ctx=760)
    assert (out[[0, 17]] == 0).all() and torch.isnan(out[[3, 4]]).all()
    c.check_large(out, [j for j in range(43) if j not in (0, 17, 3, 4)])
    bad = c.tables.copy()
    bad[0, 43] = c.k.shape[0]         # the prefix's last whole block would be 42: this is row 0's own
    bad[5, 2] = -9                    # not read: the first row's is
    bad[41, 1] = 1 << 28
    out = c.run(tables=bad)
    assert torch.isnan(out[[0, 41]]).all()
    c.check_large(out, [j for j in range(43) if j not in (0, 41)])
    bad = c.tables.copy()
    bad[0, 30] = -1
    out = c.run(tables=bad)
    assert torch.isnan(out[:40]).all()
    c.check_large(out, [40, 41, 42])


def test_shared_prefix_in_one_pass_large_and_infinite_scores():
    c = Case(46, 1, 2, 64, [60], [4000], [4100 - j for j in range(60)], poison=False, scale=300.0)
    assert 59 * 4000 * 256 >= SHARE
    c.q *= 100.0
    c.check_large(c.run())
    c = Case(47, 2, 1, 128, [40], [700], [760] * 40, poison=False)
    page = c.tables[0, 7]
    c.k[page, 0, 3] = 0.0
    c.k[page, 0, 3, 0] = -float("inf")    # a key that no row looks at
    c.q[:, :, 0] = 1.0
    c.check_large(c.run())
    c.k[page, 0, 3, 0] = 3e38             # one whose score, 9e38, is infinite in 32 bits: inf - inf
    c.q[:, 0, 0] = 3.0
    out = c.run()
    assert torch.isnan(out[:, 0]).all() and torch.isfinite(out[:, 1]).all()
    c.q[:, 0, 0] = 1.0                    # 3e38: it takes all of kv head 0's weight
    out = c.run()
    assert torch.equal(out[:, 0], c.v[page, 0, 3].expand(40, -1)) and torch.isfinite(out).all()
    c.k[page, 0, 3, 0] = NAN
    out = c.run()
    assert torch.isnan(out[:, 0]).all() and torch.isfinite(out[:, 1]).all()
    c = Case(48, 2, 1, 128, [40], [700], [760] * 40, poison=False)
    c.v[c.tables[0, 3], 1, 2, 9] = NAN    # a channel of every row
    out = c.run()
    assert torch.isnan(out[:, 1, 9]).all() and torch.isfinite(out[:, 1, :9]).all() and torch.isfinite(out[:, 0]).all()
    c.k[:] = -float("inf")                # nothing to look at: not a number, as the formula
    c.q[:] = 1.0
    assert torch.isnan(c.run()).all()


def test_shared_with_many_groups():
    """More groups than the kernels' parameters hold, of every kind."""
    rng = np.random.default_rng(5)
    rows = [int(x) for x in rng.integers(1, 4, 45)]
    prefix = [int(x) for x in rng.integers(0, 90, 45)]
    ctx = [prefix[g] + int(rng.integers(0, 70)) for g in range(45) for _ in range(rows[g])]
    c = Case(6, 2, 2, 64, rows, prefix, ctx)
    c.check(c.run())


def test_shared_padding_and_rows_out_of_range():
    c = Case(7, 2, 2, 128, [4, 3], [40, 0], [60, 45, 50, 39, 10, 0, 30])
    ctx = c.ctx.copy()
    ctx[[1, 5]] = -1     # padding
    ctx[2] = 38          # does not cover its prefix
    ctx[4] = 1000        # past max_ctx
    ctx[6] = -2
    out = c.run(ctx=ctx, max_ctx=60)
    assert (out[[1, 5]] == 0).all()
    assert torch.isnan(out[[2, 4, 6]]).all()
    c.check(out, [0, 3])
    alone = Case(8, 1, 1, 64, [1, 1], [0, 0], [5, 9])  # the same without splits
    out = alone.run(ctx=np.array([-1, 400]), max_ctx=16)
    assert (out[0] == 0).all() and torch.isnan(out[1]).all()


def test_shared_blocks_outside_the_pool():
    c = Case(9, 2, 1, 64, [3, 2], [64, 0], [100, 90, 70, 40, 30])
    bad = c.tables.copy()
    bad[1, 5] = c.k.shape[0]         # an own page of row 1
    bad[3, 0] = -7
    out = c.run(tables=bad)
    assert bool(torch.isnan(out[[1, 3]]).all())
    c.check(out, [0, 2, 4])
    bad = c.tables.copy()
    bad[0, 1] = 1 << 30              # the prefix, through the first row's table
    out = c.run(tables=bad)
    assert bool(torch.isnan(out[:3]).all())
    c.check(out, [3, 4])
    bad[0, 1] = c.tables[0, 1]
    bad[1:3, :4] = -1                # the others' entries of the shared pages are not read
    c.check(c.run(tables=bad))


@pytest.mark.parametrize("kv,group,d", [(3, 1, 128), (2, 4, 64)])
def test_shared_takes_strided_rows_and_leaves_the_rest(kv, group, d):
    c = Case(11, kv, group, d, [3, 1], [33, 5], [70, 80, 33, 90])
    heads = kv * group
    big = torch.full((4, heads + 3, d), 5.0, dtype=torch.bfloat16, device="cuda")
    big[:, 1:1 + heads] = c.q
    out = torch.full((4, heads + 2, d), 3.0, dtype=torch.bfloat16, device="cuda")
    c.run(q=big[:, 1:1 + heads], out=out[:, 2:])
    assert torch.equal(out[:, 2:], c.run())
    assert (out[:, :2] == 3.0).all()


def test_shared_large_and_infinite_scores():
    c = Case(12, 1, 2, 64, [3], [100], [150, 100, 130], poison=False, scale=300.0)
    c.q *= 100.0  # scores of 1e5: one key takes all
    c.check(c.run())
    c = Case(13, 1, 1, 64, [2], [32], [70, 80], poison=False)
    c.k[c.tables[0, 0], 0, 3] = 0.0
    c.k[c.tables[0, 0], 0, 3, 0] = -float("inf")  # a key of the prefix that no row with q[0] > 0 looks at
    c.q[:, :, 0] = 1.0
    out = c.run()
    c.check(out)
    c.v[c.tables[0, 1], 0, 2, 9] = NAN  # a NaN in the prefix is every row's
    assert torch.isnan(c.run()[:, 0, 9]).all()


def test_shared_pool_past_four_gigabytes():
    """Pages whose bytes lie beyond 2^32: the last ones of a pool of 2^18 blocks of 8 kv heads."""
    kv, d, blocks = 8, 128, (1 << 18) + 40
    k = torch.empty(blocks, kv, 16, d, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    small = Case(14, kv, 1, d, [2], [48], [100, 60], poison=False)
    m = small.k.shape[0]
    k[-m:], v[-m:] = small.k, small.v
    far = np.where(small.tables >= 0, small.tables + blocks - m, -1)
    out, want = torch.empty_like(small.q), small.run()
    paged.decode_shared(paged.PagedPool(k, v), small.q, _dev(far), _dev(small.ctx), 100, [2], [48], out)
    assert torch.equal(out, want)


# ------------------------------------------------------------------- weights

def _weigh_case(seed, kv, group, d, ctx, nq, poison=True):
    c = Case(seed, kv, group, d, [1] * len(ctx), [0] * len(ctx), ctx, poison=poison)
    rng = np.random.default_rng(seed + 1)
    c.q = _bf(rng, len(ctx) * nq, kv * group, d)
    wb = c.k.shape[0] + 5
    perm = rng.permutation(wb)
    c.wtables = np.full((len(ctx), c.tables.shape[1]), -1, np.int64)
    at = 0
    for j, x in enumerate(ctx):
        m = x // 16 + 1 if x >= 0 else 0
        c.wtables[j, :m] = perm[at:at + m]
        at += m
    c.w = torch.from_numpy(rng.random((wb, kv, 16)).astype(np.float32)).cuda()
    return c


def _weigh(c, nq, decay, **over):
    out = torch.full_like(c.q, 7.0)
    w = c.w.clone()
    max_ctx = over.get("max_ctx", max(0, int(c.ctx.max())))
    pad = max(0, max_ctx // 16 + 1 - c.tables.shape[1])
    tables, wtables = (np.pad(t, ((0, 0), (0, pad)), constant_values=-1) for t in (c.tables, c.wtables))
    paged.decode_weigh(c.pool, c.q, _dev(over.get("tables", tables)), _dev(over.get("ctx", c.ctx)), max_ctx, w,
                       _dev(over.get("wtables", wtables)), decay, out)
    torch.cuda.synchronize()
    return out, w


@pytest.mark.parametrize("kv,group,d,ctx,nq,decay", [
    (1, 1, 64, [0], 1, 1.0),
    (2, 1, 128, [5, -1, 15, 16, 300], 1, 1.0),
    (3, 4, 64, [1000, 31], 1, 0.5),
    (1, 8, 128, [2300], 1, 0.96875),
    (2, 12, 64, [100, 40], 1, 0.0),
    (2, 1, 64, [1, 2, 50], 2, 1.0),
    (1, 3, 128, [6, 300, 40], 7, 0.25),       # more than eight queries, the first row of all at position 0
    (2, 2, 64, [10, 33, 700], 33, 1.0),       # queries before the start of their sequences
    (1, 5, 64, [90], 64, 0.0),                # more queries than the weights' kernel takes at once
    (1, 8, 64, [400, 17], 1, 0.5),                  # one split, more scores than a CTA keeps
    (2, 1, 128, [1500, 1008, 16, 1023], 1, 0.5),    # long enough for the tensor cores' kernel, and not
    (1, 8, 64, [1200, -1, 1030], 20, 1.0),          # 160 queries: two tiles of Q
    (1, 4, 128, [1300, 40, 3], 70, 0.0),            # 280 queries: one CTA more, and sequences shorter than the window
])
def test_weigh_matches_the_plain_form(kv, group, d, ctx, nq, decay):
    c = _weigh_case(sum(ctx) + nq, kv, group, d, ctx, nq)
    old = _f64(c.w)
    if decay == 0:
        c.w.fill_(NAN)  # what is not to count may be anything
    out, w = _weigh(c, nq, decay)
    o, b, want, wb = ref.weigh(_f64(c.q), _f64(c.k), _f64(c.v), c.tables, c.ctx, group, nq, old, c.wtables, decay)
    assert (np.abs(_f64(out) - o) <= b).all()
    touched = wb > 0
    got = _f64(w)
    assert (np.abs(got - want) <= wb)[touched].all(), np.abs(got - want)[touched].max()
    assert np.array_equal(got[~touched], _f64(c.w)[~touched], equal_nan=True)  # other slots stay
    again = _weigh(c, nq, decay)
    assert torch.equal(again[0], out) and torch.equal(again[1][~torch.isnan(w)], w[~torch.isnan(w)])
    far = _weigh(c, nq, decay, max_ctx=max(ctx) + 3000)
    assert (np.abs(_f64(far[0]) - o) <= b).all() and (np.abs(_f64(far[1]) - want) <= wb)[touched].all()


@pytest.mark.parametrize("kv,group,d,ctx,nq,max_ctx", [
    (1, 1, 64, [9000, 3, 700], 1, 9000),                      # one long row has most splits
    (2, 2, 64, [5000, 4999, 64, 63, -1, 0], 2, 20000),        # far below what the call allows
    (1, 4, 128, [2000], 1, 60000),
    (1, 1, 64, [-1, -1], 1, 8000),                            # padding alone
    (1, 1, 64, [12000] + [5] * 99, 1, 12000),                 # the splits of one row are all there are
    (1, 1, 64, [40 + 7 * j for j in range(200)], 1, 4000),
    (1, 1, 64, [900] * 227, 1, 1700),                         # no room for more CTAs than rows
    (1, 1, 64, [900] * 257, 1, 70000),                        # one split: nothing to balance
])
def test_weigh_splits_by_the_lengths_there_are(kv, group, d, ctx, nq, max_ctx):
    c = _weigh_case(len(ctx) + ctx[0] + 7, kv, group, d, ctx, nq)
    o, b, want, wb = ref.weigh(_f64(c.q), _f64(c.k), _f64(c.v), c.tables, c.ctx, group, nq, _f64(c.w), c.wtables, 0.5)
    out, w = _weigh(c, nq, 0.5, max_ctx=max_ctx)
    assert (np.abs(_f64(out) - o) <= b).all()
    assert (np.abs(_f64(w) - want) <= wb)[wb > 0].all()
    assert np.array_equal(_f64(w)[wb == 0], _f64(c.w)[wb == 0])
    beyond = np.where(np.arange(len(ctx)) == 0, max_ctx + 1, c.ctx)  # the first out of its range: NaN, and it counts for nothing
    out2, w2 = _weigh(c, nq, 0.5, max_ctx=max_ctx, ctx=beyond)
    assert torch.isnan(out2[:nq]).all() and (np.abs(_f64(out2) - o) <= b)[nq:].all()
    mine = c.wtables[0][c.wtables[0] >= 0]
    assert torch.equal(w2[mine], c.w[mine])


def test_weigh_new_tokens_start_from_zero():
    c = _weigh_case(3, 2, 2, 64, [40, 20], 3)
    dirty = c.w.clone()
    for j, x in enumerate(c.ctx):
        for t in range(x - 2, x + 1):
            c.w[c.wtables[j, t // 16], :, t % 16] = NAN
    out, w = _weigh(c, 3, 1.0)
    o, b, want, wb = ref.weigh(_f64(c.q), _f64(c.k), _f64(c.v), c.tables, c.ctx, 2, 3, _f64(dirty), c.wtables, 1.0)
    assert (np.abs(_f64(w) - want) <= wb)[wb > 0].all()


def test_weigh_sequences_and_blocks_out_of_range():
    c = _weigh_case(4, 2, 1, 64, [40, 100, 30, 20], 1)
    ctx = c.ctx.copy()
    ctx[0], ctx[1] = -1, 101
    tables, wtables = c.tables.copy(), c.wtables.copy()
    tables[2, 0] = c.k.shape[0]
    wtables[3, 1] = -5
    out, w = _weigh(c, 1, 0.5, ctx=ctx, max_ctx=100, tables=tables, wtables=wtables)
    o, b, want, wb = ref.weigh(_f64(c.q), _f64(c.k), _f64(c.v), c.tables, c.ctx, 1, 1, _f64(c.w), c.wtables, 0.5)
    assert (out[0] == 0).all() and torch.isnan(out[1]).all() and torch.isnan(out[2]).all()
    assert (np.abs(_f64(out[3]) - o[3]) <= b[3]).all()
    got, old = _f64(w), _f64(c.w)
    for j in (0, 1):
        used = [x for x in c.wtables[j] if x >= 0]
        assert np.array_equal(got[used], old[used])
    for t in range(31):  # a bad block: nothing is added, old weights fade all the same
        x = (c.wtables[2, t // 16], slice(None), t % 16)
        assert np.array_equal(got[x], 0.5 * old[x] if t < 30 else 0 * old[x])
    for t in range(21):
        x = (c.wtables[3, t // 16], slice(None), t % 16)
        if t < 16:
            assert (np.abs(got[x] - want[x]) <= wb[x]).all()
        else:
            assert np.array_equal(got[x], old[x])  # the block outside the pool: neither read nor written


def test_weigh_a_head_that_is_not_a_number_adds_nothing():
    c = _weigh_case(5, 1, 2, 64, [50], 1)
    c.q[0, 1, 5] = NAN
    out, w = _weigh(c, 1, 1.0)
    assert torch.isnan(out[0, 1]).all() and torch.isfinite(out[0, 0]).all()
    half = _weigh_case(5, 1, 2, 64, [50], 1)
    half.q[0, 1] = half.q[0, 0]
    _, twice = _weigh(half, 1, 0.0)
    t = 7
    x = (c.wtables[0, t // 16], 0, t % 16)
    assert abs(float(w[x]) - float(c.w[x]) - 0.5 * float(twice[x])) <= 1e-6


def test_weigh_queries_do_not_see_later_infinities():
    """V of a later token of the call's own rows is infinite: rows before it are as ever."""
    c = _weigh_case(6, 1, 3, 64, [40], 6)
    o, b, _, _ = ref.weigh(_f64(c.q), _f64(c.k), _f64(c.v), c.tables, c.ctx, 3, 6, _f64(c.w), c.wtables, 1.0)
    c.v[c.tables[0, 2], 0, 38 % 16] = float("inf")
    c.v[c.tables[0, 2], 0, 40 % 16, 3] = NAN
    out, w = _weigh(c, 6, 1.0)
    got = _f64(out)
    assert (np.abs(got[:3] - o[:3]) <= b[:3]).all()     # positions 35, 36, 37
    assert np.isposinf(got[3:5]).all()                  # 38, 39
    assert np.isnan(got[5, :, 3]).all() and np.isposinf(np.delete(got[5], 3, axis=1)).all()
    assert torch.isfinite(w[c.wtables[0, :3]]).all()


# ------------------------------------------------------------------ eviction

def _weight_pool(rng, lens, kv, spare=3, stride=0):
    need = [(int(m) + 15) // 16 for m in lens]
    blocks = sum(need) + spare
    perm = rng.permutation(blocks)
    tables = np.full((len(lens), max(max(need), stride, 1)), -1, np.int64)
    at = 0
    for j, m in enumerate(need):
        tables[j, :m] = perm[at:at + m]
        at += m
    return np.exp(2 * rng.standard_normal((blocks, kv, 16))).astype(np.float32), tables


def _select(w, tables, lens, keep, first, recent, max_len=None):
    kept = torch.full((len(lens), w.shape[1], keep), 12345, dtype=torch.int32, device="cuda")
    paged.evict_select(_dev(w, np.float32), _dev(tables), _dev(lens), max(lens) if max_len is None else max_len, keep,
                       first, recent, kept)
    torch.cuda.synchronize()
    return kept.cpu().numpy()


@pytest.mark.parametrize("lens,kv,keep,first,recent", [
    ([1], 1, 1, 0, 0), ([5, 1, 0, 17], 2, 1, 0, 0), ([5, 2, 33], 3, 2, 1, 1), ([100, 64, 65, 63], 2, 64, 4, 8),
    ([200, 31, 129], 4, 32, 4, 8), ([300], 1, 299, 0, 0), ([1025, 513], 5, 512, 4, 128), ([4096, 4097], 1, 100, 0, 100),
    ([4095], 2, 50, 50, 0), ([9000, 5000], 2, 4500, 100, 1000), ([70000], 1, 30000, 4, 64),
    ([128, 127, 33, 32, 1, 0, 64, 65, 100], 3, 40, 2, 3), ([128, 96], 1, 127, 0, 0), ([31, 128, 129], 2, 32, 32, 0),
    ([32, 31, 0, 1, 17], 3, 8, 1, 2), ([20, 32], 5, 32, 0, 0), ([64, 33, 63, 0, 48, 2, 32] * 4, 26, 24, 4, 3),
    ([3001, 5900], 3, 1000, 3, 7), ([10000, 100, 7] + [9] * 27, 1, 5000, 0, 5),
    ([500, 60001], 13, 100, 4, 8),
    ([60001], 2, 100, 4, 8), ([51000, 16384, 70], 1, 16384, 0, 1000), ([90000, 55000], 2, 30000, 4, 64),  # clusters of 16
])
def test_select_keeps_the_heaviest(lens, kv, keep, first, recent):
    rng = np.random.default_rng(sum(lens) + keep)
    w, tables = _weight_pool(rng, lens, kv)
    assert np.array_equal(_select(w, tables, lens, keep, first, recent), ref.select(w, tables, lens, keep, first, recent))


@pytest.mark.parametrize("lens,kv", [([500, 90, 70], 2), ([4000, 3500], 1), ([9000], 1), ([12000, 9000, 7000], 30)])
@pytest.mark.parametrize("bits", [0, 1, 8, 12, 22])
def test_select_where_the_first_digits_tell(lens, kv, bits):
    """The heavier tokens, `keep` of them or a few more, differ from the others in their first bits only or in none."""
    rng = np.random.default_rng(bits + kv)
    w, tables = _weight_pool(rng, lens, kv)
    keep = 64
    low = rng.integers(0, 4, w.shape).astype(np.uint32)
    w[:] = (np.uint32(0x3f000000) + low).view(np.float32)
    for extra, m in zip((0, 3, 0), lens):
        j = lens.index(m)
        for h in range(kv):
            at = rng.choice(m, keep + extra, replace=False)
            x = (tables[j, at // 16], h, at % 16)
            w[x] = (np.uint32(0x3f000000) + np.uint32(1 << (31 - bits) if 8 <= bits < 31 else bits << 24) + low[x]).view(np.float32)
    assert np.array_equal(_select(w, tables, lens, keep, 2, 5), ref.select(w, tables, lens, keep, 2, 5))


@pytest.mark.parametrize("seed", range(8))
def test_select_ties_signs_and_numbers_that_are_none(seed):
    """Few distinct values, both zeros, infinities, NaN, denormals and negative ones: the lower position first."""
    rng = np.random.default_rng(seed)
    lens = [int(x) for x in rng.integers(1, 5000 if seed < 4 else 200 if seed < 6 else 32, 3)]
    w, tables = _weight_pool(rng, lens, 2)
    pick = np.array([0.0, -0.0, 1.0, 1.0, np.inf, -np.inf, NAN, -NAN, 1e-45, -1e-45, -3.0, 2.5, 2.5000002], np.float32)
    w[:] = pick[rng.integers(0, len(pick), w.shape)] if seed not in (3, 5) else 0.0
    for j in range(3):
        if lens[j] > 40:
            tables[j, 1] = [-1, w.shape[0], 1 << 30][j]  # weights outside the pool
    for keep in (1, 7, max(1, min(lens) // 2), max(lens) // 2 + 1):
        first, recent = min(2, keep // 3), min(3, keep // 3)
        assert np.array_equal(_select(w, tables, lens, keep, first, recent),
                              ref.select(w, tables, lens, keep, first, recent)), (lens, keep)


@pytest.mark.parametrize("kv,keep,n", [(1, 300000, 450000), (30, 100, 450000), (1, 300000, 900000)])
def test_select_of_more_tokens_than_a_cluster_keeps(kv, keep, n):
    """Longer than the shared memory of eight CTAs, or of sixteen: the weights are read again in every pass.  Whole
    numbers, many of them equal, so that the choice is by position too."""
    tables = np.random.default_rng(2).permutation(n // 16 + 1)[None]
    w = torch.randint(0, 1000 if keep > 1000 else n, (n // 16 + 1, kv, 16), device="cuda").float()
    kept = torch.empty(1, kv, keep, dtype=torch.int32, device="cuda")
    paged.evict_select(w, _dev(tables), _dev([n]), n, keep, 3, 50, kept)
    flat = w[torch.from_numpy(tables[0]).cuda()].transpose(0, 1).reshape(kv, -1)[:, :n].clone()
    flat[:, :3], flat[:, n - 50:] = float("inf"), float("inf")
    want = torch.sort(torch.sort(flat, dim=1, descending=True, stable=True).indices[:, :keep], dim=1).values
    assert torch.equal(kept[0].long(), want)


def test_select_lengths_out_of_range():
    rng = np.random.default_rng(1)
    w, tables = _weight_pool(rng, [50, 50, 50], 2)
    kept = _select(w, tables, [51, -1, 50], 20, 0, 0, max_len=50)
    assert (kept[:2] == -1).all()
    assert np.array_equal(kept[2:], ref.select(w, tables[2:], [50], 20, 0, 0))


def _move_case(seed, d, kv, lens, keep, place):
    """Pools of random bytes, kept as select gives it; place: new pages, the old tables, or every other page new."""
    rng = np.random.default_rng(seed)
    w, tables = _weight_pool(rng, lens, kv, spare=sum((min(m, keep) + 15) // 16 for m in lens) + 2)
    blocks = w.shape[0]
    free = [b for b in range(blocks) if b not in set(tables.ravel())]
    width = (keep + 15) // 16
    new = np.full((len(lens), width), -1, np.int64)
    for j, m in enumerate(lens):
        for i in range((min(m, keep) + 15) // 16):
            fresh = place == "new" or (place == "mixed" and i % 2)
            new[j, i] = free.pop() if fresh else tables[j, i]
    k, v = _bf(rng, blocks, kv, 16, d), _bf(rng, blocks, kv, 16, d)
    kept = ref.select(w, tables, lens, keep, min(2, keep), 0)
    return w, tables, new, k, v, kept


@pytest.mark.parametrize("place", ["new", "old", "mixed"])
@pytest.mark.parametrize("d,kv,lens,keep", [
    (64, 1, [1], 1), (128, 2, [40, 7, 0, 100], 30), (64, 3, [17, 33], 16), (128, 5, [600, 1000], 512),
    (64, 1, [9000], 7000), (128, 1, [6000, 6500], 3001), (128, 3, [100, 33, 20], 32), (64, 2, [70] * 19, 31),
    (128, 5, [30, 1, 0, 90, 33, 32, 17], 32), (64, 33, [15, 40], 3),
    (128, 1, [12000], 11000), (64, 4, [900, 2000, 1500], 800),
    (64, 2, [20000, 17000], 16500), (128, 4, [17000], 16384), (128, 1, [3000], 1999),
])
def test_move_brings_the_kept_tokens_to_the_front(place, d, kv, lens, keep):
    w, tables, new, k, v, kept = _move_case(sum(lens) + keep, d, kv, lens, keep, place)
    dw, dk, dv = _dev(w, np.float32), k.clone(), v.clone()
    old_t, new_t = _dev(tables), _dev(new)
    if place == "old" and tables.shape[1] >= new.shape[1]:
        new_t = old_t  # the same memory
    paged.evict_move(paged.PagedPool(dk, dv), old_t, new_t, _dev(kept), dw, old_t, new_t)
    torch.cuda.synchronize()
    for got, was in ((dk, k), (dv, v)):
        assert np.array_equal(_f64(got), ref.move(_f64(was), tables, new, kept))
    assert np.array_equal(dw.cpu().numpy(), ref.move(w, tables, new, kept))
    dk2 = k.clone()  # K and V alone, the weights' tables left out
    paged.evict_move(paged.PagedPool(dk2, v.clone()), old_t, new_t, _dev(kept))
    assert torch.equal(dk2, dk)


def test_move_skips_what_lies_outside():
    w, tables, new, k, v, kept = _move_case(3, 64, 2, [80, 90], 40, "new")
    tables[0, 1], new[0, 2], new[1, 0] = -1, k.shape[0], -3
    tables[1, 2] = 1 << 30
    kept[1, 0, 39] = 16 * tables.shape[1]  # beyond the table
    dk, dv = k.clone(), v.clone()
    paged.evict_move(paged.PagedPool(dk, dv), _dev(tables), _dev(new), _dev(kept))
    assert np.array_equal(_f64(dk), ref.move(_f64(k), tables, new, kept))
    assert np.array_equal(_f64(dv), ref.move(_f64(v), tables, new, kept))


def test_move_of_few_tokens_skips_what_lies_outside():
    """Many sequences that keep at most 32 tokens: a warp each."""
    w, tables, new, k, v, kept = _move_case(4, 128, 3, [40 + j for j in range(12)], 20, "new")
    tables[0, 1], new[1, 1], new[2, 0] = -1, k.shape[0], -3
    tables[3, 0] = 1 << 30
    kept[4, 0, 19] = 16 * tables.shape[1]  # beyond the table
    dk, dv, dw = k.clone(), v.clone(), _dev(w, np.float32)
    paged.evict_move(paged.PagedPool(dk, dv), _dev(tables), _dev(new), _dev(kept), dw, _dev(tables), _dev(new))
    assert np.array_equal(_f64(dk), ref.move(_f64(k), tables, new, kept))
    assert np.array_equal(_f64(dv), ref.move(_f64(v), tables, new, kept))
    assert np.array_equal(dw.cpu().numpy(), ref.move(w, tables, new, kept))


# ------------------------------------------------------------------ together

def test_fork_decode_weigh_evict_and_decode_again():
    """A prompt forked into three, decoded over the shared prefix; its weights from a window; two forks evicted, one to
    pages of its own; then decoded again.  The page table says where everything lies."""
    kv, group, d, prompt = 2, 2, 64, 150
    heads = kv * group
    rng = np.random.default_rng(21)
    pt = cache.PageTable(64)
    pt.extend(0, prompt)
    k, v = _bf(rng, 64, kv, 16, d), _bf(rng, 64, kv, 16, d)
    pool = paged.PagedPool(k, v)
    w = torch.full((64, kv, 16), NAN, device="cuda")
    # the prompt's last eight rows give the first weights
    table = pt.table(0)
    qw = _bf(rng, 8, heads, d)
    ow = torch.empty_like(qw)
    before = np.zeros((64, kv, 16))
    paged.decode_weigh(pool, qw, _dev(table[None]), _dev([prompt - 1]), prompt - 1, w, _dev(table[None]), 0.0, ow)
    o, b, want, wb = ref.weigh(_f64(qw), _f64(k), _f64(v), table[None], [prompt - 1], group, 8, before, table[None], 0.0)
    assert (np.abs(_f64(ow) - o) <= b).all() and (np.abs(_f64(w) - want) <= wb)[wb > 0].all()
    # three forks of it decode one token each
    for child in (1, 2, 3):
        pt.fork(0, child)
        c = pt.extend(child, prompt + 1)
        if c:
            cache.copy_pages(k[None], [c[0]], [c[1]])
            cache.copy_pages(v[None], [c[0]], [c[1]])
            cache.copy_pages(w[None], [c[0]], [c[1]])
    tables = np.stack([pt.table(s) for s in (1, 2, 3)])
    assert (tables[0, :prompt // 16] == tables[2, :prompt // 16]).all()
    q = _bf(rng, 3, heads, d)
    out = torch.empty_like(q)
    paged.decode_shared(pool, q, _dev(tables), _dev([prompt] * 3), prompt, [3], [prompt], out)
    o, b = ref.shared(_f64(q), _f64(k), _f64(v), tables, [prompt] * 3, group)
    assert (np.abs(_f64(out) - o) <= b).all()
    # the first fork keeps 64 tokens in new pages, as the others still read the shared ones
    pt.extend(9, 64)
    new = pt.table(9)
    kept = torch.empty(1, kv, 64, dtype=torch.int32, device="cuda")
    paged.evict_select(w, _dev(tables[:1]), _dev([prompt]), prompt, 64, 4, 16, kept)
    assert np.array_equal(kept.cpu().numpy(), ref.select(w.cpu().numpy(), tables[:1], [prompt], 64, 4, 16))
    was = [_f64(x) for x in (k, v)]
    paged.evict_move(pool, _dev(tables[:1]), _dev(new[None]), kept, w, _dev(tables[:1]), _dev(new[None]))
    for x, y in zip((k, v), was):
        assert np.array_equal(_f64(x), ref.move(y, tables[:1], new[None], kept.cpu().numpy()))
    pt.release(1)
    # and decodes on over them, its weights with it
    pt.extend(9, 65)
    t9 = pt.table(9)[None]
    q = _bf(rng, 1, heads, d)
    out = torch.empty_like(q)
    old = _f64(w)
    paged.decode_weigh(pool, q, _dev(t9), _dev([64]), 64, w, _dev(t9), 1.0, out)
    o, b, want, wb = ref.weigh(_f64(q), _f64(k), _f64(v), t9, [64], group, 1, old, t9, 1.0)
    assert (np.abs(_f64(out) - o) <= b).all() and (np.abs(_f64(w) - want) <= wb)[wb > 0].all()


def test_captured_calls_replay_with_new_contents():
    c = Case(31, 2, 2, 64, [3, 1], [100, 20], [130, 110, 120, 60], poison=False)
    tables, ctx = _dev(np.where(c.tables < 0, 0, c.tables)), _dev(c.ctx)
    keep = 32
    kept = torch.zeros(4, 2, keep, dtype=torch.int32, device="cuda")
    out, out2 = torch.zeros_like(c.q), torch.zeros_like(c.q)
    ws = torch.empty(16 << 20, dtype=torch.uint8, device="cuda")
    wt = torch.arange(4 * tables.shape[1], device="cuda", dtype=torch.int32).view(4, -1)
    w = torch.zeros(wt.numel(), 2, 16, device="cuda")

    def step():
        paged.decode_shared(c.pool, c.q, tables, ctx, 130, c.rows, c.prefix, out, ws)
        paged.decode_weigh(c.pool, c.q, tables, ctx, 130, w, wt, 0.0, out2, ws)
        paged.evict_select(w, wt, ctx, 130, keep, 2, 4, kept)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    rng = np.random.default_rng(1)
    for _ in range(2):
        c.q.copy_(_bf(rng, *c.q.shape))
        ctx.copy_(_dev(c.ctx - rng.integers(0, 10, 4)))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone(), out2.clone(), kept.clone()
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (out, out2, kept)))


def test_a_stream_of_its_own_wants_a_workspace_of_its_own():
    c = Case(32, 1, 1, 64, [2], [40], [3000, 2000], poison=False)
    want = c.run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = torch.zeros_like(c.q)
    args = (c.pool, c.q, _dev(c.tables), _dev(c.ctx), 3000, c.rows, c.prefix, out)
    with pytest.raises(ValueError):
        paged.decode_shared(*args, None, s)
    need = paged.decode_shared_workspace(2, 1, 1, 64, 3000, c.rows, c.prefix)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    paged.decode_shared(*args, ws, s)
    s.synchronize()
    assert torch.equal(out, want)
    with pytest.raises(HbError):
        paged.decode_shared(*args, ws[:need - 16])


class Chain:
    """A decode behind a shared prefix, a window's weights over keys common to its rows, and an eviction by them."""

    def __init__(self, seed):
        self.c = c = Case(seed, 2, 4, 128, [20], [1500], [1500 + 13 * j for j in range(20)], poison=False)
        assert 19 * 1488 * 2 * 512 >= SHARE
        rng = np.random.default_rng(seed)
        self.tables, self.ctx = _dev(np.where(c.tables < 0, 0, c.tables)), _dev(c.ctx)
        self.lens = _dev([700, 1200])
        self.q = _bf(rng, 32, 8, 128)
        self.wt = torch.arange(2 * self.tables.shape[1], device="cuda", dtype=torch.int32).view(2, -1)
        self.w = torch.zeros(self.wt.numel(), 2, 16, device="cuda")
        self.out, self.out2 = torch.zeros_like(c.q), torch.zeros_like(self.q)
        self.kept = torch.zeros(2, 2, 600, dtype=torch.int32, device="cuda")
        self.ws = torch.empty(max(
            paged.decode_shared_workspace(20, 8, 2, 128, 1747, c.rows, c.prefix),
            paged.decode_weigh_workspace(2, 16, 8, 2, 128, 1200)), dtype=torch.uint8, device="cuda")

    def step(self, stream=None):
        c = self.c
        paged.decode_shared(c.pool, c.q, self.tables, self.ctx, 1747, c.rows, c.prefix, self.out, self.ws, stream)
        paged.decode_weigh(c.pool, self.q, self.tables[:2], self.lens, 1200, self.w, self.wt, 0.5, self.out2, self.ws,
                           stream)
        paged.evict_select(self.w, self.wt, self.lens, 1200, 600, 4, 32, self.kept, stream)

    def results(self):
        return [x.clone() for x in (self.out, self.out2, self.w, self.kept)]


def test_two_streams_and_two_graphs_at_once():
    """Two chains of calls on streams of their own, and as graphs that run side by side, each with its own workspace:
    the bits that each gives alone."""
    chains = [Chain(41), Chain(42)]
    alone = []
    for x in chains:
        for _ in range(5):
            x.step()
        torch.cuda.synchronize()
        alone.append(x.results())
        x.c.check_large(x.out, rows=(0, 7, 19))
    streams = [torch.cuda.Stream() for _ in chains]

    def compare():
        torch.cuda.synchronize()
        for x, want in zip(chains, alone):
            assert all(torch.equal(a, b) for a, b in zip(x.results(), want))
            x.w.zero_()
            for t in (x.out, x.out2, x.kept):
                t.zero_()
        torch.cuda.synchronize()

    compare()
    for _ in range(5):
        for x, s in zip(chains, streams):
            x.step(s)
    compare()
    graphs = []
    for x in chains:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            x.step()
        graphs.append(g)
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    compare()


def test_calls_that_follow_one_another_see_new_contents():
    """Common keys: q, contexts and K are written by a kernel right before the call, again and again."""
    x = Chain(43)
    rng = np.random.default_rng(2)
    qs = [_bf(rng, *x.c.q.shape) for _ in range(6)]
    ctxs = [_dev(np.maximum(x.c.ctx - int(rng.integers(0, 40)), 1499)) for _ in qs]
    ks = [x.c.k * f for f in (1.0, 0.5, 0.25, 2.0, 1.0, 0.5)]
    want = []
    for q, ctx, k in zip(qs, ctxs, ks):
        for to, new in ((x.c.q, q), (x.ctx, ctx), (x.c.k, k)):
            to.copy_(new)
        torch.cuda.synchronize()
        x.step()
        torch.cuda.synchronize()
        want.append(x.results())
    x.w.zero_()
    got = []
    for q, ctx, k in zip(qs, ctxs, ks):
        for to, new in ((x.c.k, k), (x.c.q, q), (x.ctx, ctx)):
            to.copy_(new)
        x.step()
        got.append(x.results())
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for p, r in zip(got, want) for a, b in zip(p, r))
