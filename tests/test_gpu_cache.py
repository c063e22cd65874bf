"""The 4-bit paged cache and the page operations on the GPU, against plain
64-bit forms (cache_ref.py)."""
import numpy as np
import pytest

import cache_ref as ref
from chunked_prefill_hybrid_gb300 import cache, native, synth, workloads
from chunked_prefill_hybrid_gb300.native import HbError

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

NAN16 = 0x7FC0


def _bf(x):
    """float array -> bf16 tensor on the GPU and the same values in float64."""
    t = torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16)
    return t.cuda(), t.double().numpy()


def _f64(t):
    return t.double().cpu().numpy()


# ------------------------------------------------------------ quantisation

def _special_rows(n, kv, d, seed):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((n, kv, d)) * np.exp(rng.standard_normal((1, kv, d)))
    x[0] = 0
    x[1 % n, 0, :16] = 0
    x[1 % n, 0, 16:32] = 1e-6        # a scale that rounds to 0
    x[2 % n, -1, :16] = np.linspace(-6, 6, 16) * 0.8125   # ties
    x[3 % n, 0] = 1e5                # a scale that saturates
    x[4 % n, -1, 3] = np.inf
    x[4 % n, 0, 17] = -np.inf
    x[5 % n, 0, 40] = np.nan
    x[6 % n] *= 1e-3
    return x


@pytest.mark.parametrize("n,kv,d,ks,vs", [(1, 1, 64, 1.0, 1.0), (37, 3, 64, 1.0, 0.3779644668), (19, 5, 128, 0.5, 2.0),
                                          (200, 2, 128, 0.7071067691, 1.0)])
def test_append_stores_the_nearest_codes(n, kv, d, ks, vs):
    """Every byte of the pool: the rows' codes and scales at their slots, everything else as it was; and what
    hb_kv4_read gives is those codes' values, rounded once."""
    ks, vs = float(np.float32(ks)), float(np.float32(vs))
    blocks = n // 16 + 4
    rng = np.random.default_rng(n)
    k, k64 = _bf(_special_rows(n, kv, d, 1))
    v, v64 = _bf(_special_rows(n, kv, d, 2))
    slots = rng.permutation(blocks * 16)[:n].astype(np.int32)
    if n > 8:
        slots[7], slots[8] = -1, blocks * 16        # padding, and past the end
    before = rng.integers(0, 256, (blocks, kv, 18 * d)).astype(np.uint8)
    pool = cache.Kv4Pool(torch.from_numpy(before).cuda(), ks, vs)
    ds = torch.from_numpy(slots).cuda()
    cache.kv4_append(pool, k, v, ds)
    k_out, v_out = torch.full_like(k, 7.0), torch.full_like(v, 7.0)
    cache.kv4_read(pool, ds, k_out, v_out)
    torch.cuda.synchronize()
    want = before.copy()
    for x, which, ps in ((k64, "k", ks), (v64, "v", vs)):
        codes, sb = ref.quantise(x, ps)
        # a NaN's block is NaN by its scale; its codes mean nothing
        ref.store(want, slots, codes, sb, which)
    got = pool.data.cpu().numpy()
    nan_k, nan_v = np.isnan(k64), np.isnan(v64)
    for which, ps, nan, out in (("k", ks, nan_k, k_out), ("v", vs, nan_v, v_out)):
        gv, wv = ref.values(got, which, ps), ref.values(want, which, ps)
        assert np.array_equal(np.isnan(gv), np.isnan(wv))
        assert np.array_equal(np.nan_to_num(gv, nan=0.0), np.nan_to_num(wv, nan=0.0)), which
        rows = gv.reshape(-1, kv, d)
        o = _f64(out)
        for r in range(n):
            if not 0 <= slots[r] < 16 * blocks:
                assert (o[r] == 7.0).all()
                continue
            w = rows[slots[r]].astype(np.float64)
            # the product of three fp32 factors, then bf16
            w32 = torch.from_numpy(w).to(torch.float32).to(torch.bfloat16).double().numpy()
            assert np.array_equal(np.isnan(o[r]), np.isnan(w32))
            ok = np.abs(o[r] - w) <= (2.0 ** -8 + 2.0 ** -22) * np.abs(w)
            assert (ok | np.isnan(w)).all()
    if not nan_k.any() and not nan_v.any():
        assert np.array_equal(got, want)


def test_append_takes_strided_rows_and_leaves_the_rest():
    n, kv, d = 50, 4, 64
    qkv = torch.randn(n, 3, kv, d, device="cuda").to(torch.bfloat16)
    slots = torch.randperm(96, device="cuda")[:n].to(torch.int32)
    a = cache.Kv4Pool.empty(6, kv, d)
    b = cache.Kv4Pool.empty(6, kv, d)
    cache.kv4_append(a, qkv[:, 1], qkv[:, 2], slots)
    cache.kv4_append(b, qkv[:, 1].contiguous(), qkv[:, 2].contiguous(), slots)
    assert torch.equal(a.data, b.data)
    wide = torch.full((n, 5, kv, d), 3.0, device="cuda", dtype=torch.bfloat16)
    cache.kv4_read(a, slots, wide[:, 1], wide[:, 3])
    k, v = torch.empty(n, kv, d, device="cuda", dtype=torch.bfloat16), torch.empty(n, kv, d, device="cuda", dtype=torch.bfloat16)
    cache.kv4_read(a, slots, k, v)
    assert torch.equal(wide[:, 1], k) and torch.equal(wide[:, 3], v)
    assert (wide[:, [0, 2, 4]] == 3.0).all()
    cache.kv4_append(a, qkv[:0, 1], qkv[:0, 2], slots[:0])  # no rows
    assert torch.equal(a.data, b.data)


# --------------------------------------------------------------- attention

class Filled:
    """Sequences of given lengths in a pool whose other slots hold NaN scales."""

    def __init__(self, lens, kv, d, seed, ks=1.0, vs=1.0, spread=1.0):
        rng = np.random.default_rng(seed)
        self.kv, self.d, self.lens = kv, d, list(lens)
        need = [max(1, (n + 15) // 16) for n in lens]
        blocks = sum(need) + 3
        perm = rng.permutation(blocks).astype(np.int32)
        data = np.full((blocks, kv, 18 * d), 0xFF, np.uint8)
        self.k, self.v, tabs, at = [], [], [], 0
        for n, m in zip(lens, need):
            tab = perm[at:at + m]
            at += m
            slots = (tab[np.arange(n) // 16] * 16 + np.arange(n) % 16).astype(np.int32) if n else np.zeros(0, np.int32)
            kq = ref.quantise(rng.standard_normal((n, kv, d)) * spread, ks)
            vq = ref.quantise(rng.standard_normal((n, kv, d)) + 0.5, vs)
            ref.store(data, slots, *kq, "k")
            ref.store(data, slots, *vq, "v")
            tabs.append(tab)
        self.width = max(need)
        self.tables = np.full((len(lens), self.width), -1, np.int32)
        for j, tab in enumerate(tabs):
            self.tables[j, :len(tab)] = tab
        self.host, self.ks, self.vs = data, ks, vs
        self.pool = cache.Kv4Pool(torch.from_numpy(data).cuda(), ks, vs)
        self.dev_tables = torch.from_numpy(self.tables).cuda()

    def kv_of(self, j, n):
        pages = self.host[self.tables[j, :(n + 15) // 16]]
        k = ref.values(pages, "k", self.ks).reshape(-1, self.kv, self.d)[:n]
        v = ref.values(pages, "v", self.vs).reshape(-1, self.kv, self.d)[:n]
        return k, v


CTX = [0, 15, 16, 255, 256, 257, 700, 1100, 63, 64]
HEADS = [(4, 1, 64), (2, 1, 128), (2, 2, 128), (1, 3, 64), (2, 4, 128), (1, 8, 128), (1, 12, 64), (3, 5, 128)]


@pytest.mark.parametrize("kv,group,d", HEADS)
def test_decode(kv, group, d):
    f = Filled([c + 1 for c in CTX], kv, d, 3, ks=0.75, vs=1.5)
    heads, n = kv * group, len(CTX)
    qkv, q64 = _bf(np.random.default_rng(5).standard_normal((n, heads + 2, d)) * 2)
    q = qkv[:, :heads]                                      # rows wider than the heads
    ctx = torch.tensor(CTX, dtype=torch.int32, device="cuda")
    outs = []
    for _ in range(2):
        out = torch.full((n, heads + 1, d), 7.0, dtype=torch.bfloat16, device="cuda")
        cache.kv4_decode(f.pool, q, f.dev_tables, ctx, max(CTX), out[:, :heads])
        outs.append(out)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1])
    assert (outs[0][:, heads] == 7.0).all()                 # past the heads: left alone
    got = _f64(outs[0][:, :heads])
    for j, c in enumerate(CTX):
        o, bound = ref.attention_row(q64[j, :heads], *f.kv_of(j, c + 1))
        assert (np.abs(got[j] - o) <= bound).all(), (j, c, np.max(np.abs(got[j] - o) / bound))

    # max_ctx far above every context changes only the split
    out = torch.empty((n, heads, d), dtype=torch.bfloat16, device="cuda")
    wide = torch.full((n, 20000 // 16 + 1), -1, dtype=torch.int32, device="cuda")
    wide[:, :f.width] = f.dev_tables
    cache.kv4_decode(f.pool, q, wide, ctx, 20000, out)
    for j, c in enumerate(CTX):
        o, bound = ref.attention_row(q64[j, :heads], *f.kv_of(j, c + 1))
        assert (np.abs(_f64(out[j]) - o) <= bound).all(), (j, c)

    # padding rows get zeros, contexts out of range and bad blocks NaN; the other rows stay what they were
    bad_ctx, tables = ctx.clone(), f.dev_tables.clone()
    bad_ctx[1], bad_ctx[3], bad_ctx[4] = -1, -2, max(CTX) + 1
    tables[6, 20], tables[7, 68] = f.pool.num_blocks, -7
    tables[5, 17] = -1                                      # past the row's context (key 257 and on): not read
    out = torch.full((n, heads, d), 7.0, dtype=torch.bfloat16, device="cuda")
    cache.kv4_decode(f.pool, q, tables, bad_ctx, max(CTX), out)
    assert (out[1] == 0).all()
    for j in (3, 4, 6, 7):
        assert torch.isnan(out[j]).all(), j
    for j in (0, 2, 5, 8, 9):
        assert torch.equal(out[j], outs[0][j, :heads]), j


@pytest.mark.parametrize("kv,group,d,ctx", [(1, 1, 128, 20001), (2, 4, 64, 9000), (1, 9, 128, 5000)])
def test_decode_of_one_long_row(kv, group, d, ctx):
    f = Filled([ctx + 1], kv, d, 8)
    q, q64 = _bf(np.random.default_rng(5).standard_normal((1, kv * group, d)))
    out = torch.empty_like(q)
    ws = torch.empty(cache.kv4_decode_workspace(1, kv * group, kv, d, ctx), dtype=torch.uint8, device="cuda")
    assert ws.numel() > 0
    lens = torch.tensor([ctx], dtype=torch.int32, device="cuda")
    cache.kv4_decode(f.pool, q, f.dev_tables, lens, ctx, out, ws)
    o, bound = ref.attention_row(q64[0], *f.kv_of(0, ctx + 1))
    assert (np.abs(_f64(out[0]) - o) <= bound).all()
    # a short row in the same split
    lens[0] = 100
    cache.kv4_decode(f.pool, q, f.dev_tables, lens, ctx, out, ws)
    o, bound = ref.attention_row(q64[0], *f.kv_of(0, 101))
    assert (np.abs(_f64(out[0]) - o) <= bound).all()
    with pytest.raises(HbError):
        cache.kv4_decode(f.pool, q, f.dev_tables, lens, ctx, out, ws[:-16])


@pytest.mark.parametrize("size", [0.0, 1e-30, 3e4, 1e30])
def test_queries_of_any_size(size):
    """A query is scaled by a power of two, so its size costs no precision: 1e30 picks one key."""
    f = Filled([300], 2, 64, 9)
    q, q64 = _bf(np.random.default_rng(6).standard_normal((1, 2, 64)) * size)
    out = torch.empty_like(q)
    cache.kv4_decode(f.pool, q, f.dev_tables, torch.tensor([299], dtype=torch.int32, device="cuda"), 299, out)
    k, v = f.kv_of(0, 300)
    for h in range(2):
        s = k[:, h] @ q64[0, h] / 8.0
        p = np.exp(s - s.max())
        o = (p / p.sum()) @ v[:, h]
        mean_abs = (p / p.sum()) @ np.abs(v[:, h])
        reach = (np.abs(k[:, h]) @ np.abs(q64[0, h])).max() / 8.0 * 1.4427
        if size < 1e20 and 2.0 ** -17 * reach > 0.5:
            continue  # scores rounded by more than the softmax can bear: nothing to compare
        if size >= 1e20:  # the largest score wins by far more than any rounding
            o, mean_abs, reach = v[np.argmax(s), h], np.abs(v[np.argmax(s), h]), 0.0
        assert (np.abs(_f64(out[0, h]) - o) <= 2.0 ** -8 * np.abs(o) + mean_abs * (2.0 ** -10 + 2.0 ** -17 * reach) + 1e-6).all()


def test_nan_is_seen_where_it_counts_and_nowhere_else():
    kv, d, n = 1, 128, 40
    f = Filled([n], kv, d, 10)
    q, _ = _bf(np.random.default_rng(6).standard_normal((1, 2, d)))
    lens = torch.tensor([n - 1], dtype=torch.int32, device="cuda")
    want = torch.empty_like(q)
    cache.kv4_decode(f.pool, q, f.dev_tables, lens, n - 1, want)
    row = torch.full((1, kv, d), 1.0, device="cuda").to(torch.bfloat16)
    nan = row.clone()
    nan[0, 0, 20] = float("nan")                           # block 1 of 8
    slot = torch.tensor([int(f.tables[0, 1]) * 16 + 3], dtype=torch.int32, device="cuda")  # key 19
    cache.kv4_append(f.pool, row, nan, slot)
    out = torch.empty_like(q)
    cache.kv4_decode(f.pool, q, f.dev_tables, lens, n - 1, out)
    assert torch.isnan(out[..., 16:32]).all() and not torch.isnan(out[..., :16]).any() and not torch.isnan(out[..., 32:]).any()
    cache.kv4_append(f.pool, nan, row, slot)
    cache.kv4_decode(f.pool, q, f.dev_tables, lens, n - 1, out)
    assert torch.isnan(out).all()
    # a context that ends before the key does not see it
    lens[0] = 18
    cache.kv4_decode(f.pool, q, f.dev_tables, lens, n - 1, out)
    assert torch.isfinite(out).all()
    # nor do the rows of a chunk before it
    big = torch.randn(n, 2, d, device="cuda").to(torch.bfloat16)
    for k_row, v_row in ((row, nan), (nan, row)):
        cache.kv4_append(f.pool, k_row, v_row, slot)
        o = torch.empty_like(big)
        cache.kv4_chunk(f.pool, big, f.dev_tables[0], 0, o)
        assert torch.isfinite(o[:19]).all()
        assert torch.isnan(o[19:, :, 16:32]).all()


@pytest.mark.parametrize("kv,group,d", HEADS)
@pytest.mark.parametrize("offset,n", [(0, 1), (0, 16), (0, 130), (37, 29), (255, 257), (1000, 65), (3000, 3)])
def test_chunk(kv, group, d, offset, n):
    f = Filled([5, offset + n], kv, d, 11, ks=1.25, vs=0.5)
    heads = kv * group
    wide, q64 = _bf(np.random.default_rng(7).standard_normal((n, heads + 2, d)) * 2)
    q = wide[:, :heads]
    outs = []
    for _ in range(2):
        out = torch.full((n, heads + 1, d), 7.0, dtype=torch.bfloat16, device="cuda")
        cache.kv4_chunk(f.pool, q, f.dev_tables[1], offset, out[:, :heads])
        outs.append(out)
    assert torch.equal(outs[0], outs[1]) and (outs[0][:, heads] == 7.0).all()
    got = _f64(outs[0][:, :heads])
    k, v = f.kv_of(1, offset + n)
    for i in sorted({0, 1, 15, 16, 17, n // 2, n - 2, n - 1} & set(range(n))):
        o, bound = ref.attention_row(q64[i, :heads], k[:offset + i + 1], v[:offset + i + 1])
        assert (np.abs(got[i] - o) <= bound).all(), (i, np.max(np.abs(got[i] - o) / bound))


def test_chunk_whole_rows_against_decode():
    """Every row of a chunk against the decode of the same query, whose bound the first test holds."""
    kv, group, d, offset, n = 2, 4, 128, 517, 150
    f = Filled([offset + n], kv, d, 12)
    heads = kv * group
    q, q64 = _bf(np.random.default_rng(8).standard_normal((n, heads, d)))
    out, dec = torch.empty_like(q), torch.empty_like(q)
    cache.kv4_chunk(f.pool, q, f.dev_tables[0], offset, out)
    lens = torch.arange(offset, offset + n, dtype=torch.int32, device="cuda")
    cache.kv4_decode(f.pool, q, f.dev_tables[0].repeat(n, 1), lens, offset + n - 1, dec)
    k, v = f.kv_of(0, offset + n)
    for i in range(n):
        o, bound = ref.attention_row(q64[i], k[:offset + i + 1], v[:offset + i + 1])
        assert (np.abs(_f64(out[i]) - o) <= bound).all(), i
        assert (np.abs(_f64(dec[i]) - o) <= bound).all(), i


def test_chunk_with_a_bad_block():
    f = Filled([200], 1, 64, 13)
    q, _ = _bf(np.random.default_rng(8).standard_normal((100, 1, 64)))
    out, good = torch.empty_like(q), torch.empty_like(q)
    cache.kv4_chunk(f.pool, q, f.dev_tables[0], 100, good)
    for bad in (f.pool.num_blocks, -1, 2 ** 31 - 1, -2 ** 31):
        tab = f.dev_tables[0].clone()
        tab[2] = bad
        cache.kv4_chunk(f.pool, q, tab, 100, out)
        assert torch.isnan(out).all()
    cache.kv4_chunk(f.pool, q, f.dev_tables[0], 100, out)
    assert torch.equal(out, good)


# kv heads, group, head size, offset, rows: many rows over many keys, a last item of a few columns; between them they
# have each way in which the work is cut (items of 128 and of 256 columns; a CTA for each, several, or several items a
# CTA; evenly, whatever the items)
LARGE = [(40, 1, 128, 1000, 130), (8, 4, 64, 700, 333), (8, 12, 64, 1800, 40), (4, 2, 128, 2000, 257),
         (2, 5, 64, 5000, 129), (1, 8, 128, 20000, 64), (8, 2, 128, 15000, 130), (8, 1, 128, 0, 3000),
         (2, 3, 128, 3000, 1500), (5, 3, 64, 12001, 301), (8, 8, 64, 0, 1000), (40, 1, 128, 0, 1500),
         (8, 8, 64, 0, 3000), (8, 8, 128, 0, 500)]


def _check_rows(got, q64, k, v, offset, rows):
    for i in rows:
        o, bound = ref.attention_row(q64[i], k[:offset + i + 1], v[:offset + i + 1])
        assert (np.abs(got[i] - o) <= bound).all(), (i, np.max(np.abs(got[i] - o) / bound))


@pytest.mark.parametrize("kv,group,d,offset,n", LARGE)
def test_large_chunk(kv, group, d, offset, n):
    f = Filled([5, offset + n], kv, d, 15, ks=1.25, vs=0.5)
    heads = kv * group
    need = cache.kv4_chunk_workspace(offset, n, heads, kv, d)
    wide, q64 = _bf(np.random.default_rng(7).standard_normal((n, heads + 2, d)) * 2)
    q = wide[:, :heads]
    ws = torch.full((need + 16,), 0xFF, dtype=torch.uint8, device="cuda")
    outs = []
    for _ in range(3):
        out = torch.full((n, heads + 1, d), 7.0, dtype=torch.bfloat16, device="cuda")
        cache.kv4_chunk(f.pool, q, f.dev_tables[1], offset, out[:, :heads], ws)
        outs.append(out)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    assert (outs[0][:, heads] == 7.0).all() and (ws[need:] == 0xFF).all()
    k, v = f.kv_of(1, offset + n)
    _check_rows(_f64(outs[0][:, :heads]), q64[:, :heads], k, v, offset,
                sorted({0, 1, 127 // group, 128 // group, 255 // group, 256 // group, n // 2, n - 2, n - 1} & set(range(n))))


@pytest.mark.parametrize("kv,group,d,offset,n", [(40, 1, 128, 1000, 130), (4, 2, 64, 2000, 257), (8, 2, 128, 15000, 130)])
def test_large_chunk_sees_nan_and_bad_blocks_where_they_count(kv, group, d, offset, n):
    f = Filled([offset + n], kv, d, 16)
    heads = kv * group
    q, q64 = _bf(np.random.default_rng(9).standard_normal((n, heads, d)))
    out, good = torch.empty_like(q), torch.empty_like(q)
    cache.kv4_chunk(f.pool, q, f.dev_tables[0], offset, good)
    row = torch.ones(1, kv, d, device="cuda").to(torch.bfloat16)
    nan = row.clone()
    nan[0, kv - 1, 20] = float("nan")                       # block 1 of the last head
    mine = slice((kv - 1) * group, heads)
    held = f.pool.data.clone()
    # keys of both halves' tiles, the first, and ones that only the chunk's later rows see
    for key in (3, 130, offset - 1, offset + n // 2, offset + n - 1):
        first = max(0, key - offset)                        # the first row that sees it
        slot = torch.tensor([int(f.tables[0, key // 16]) * 16 + key % 16], dtype=torch.int32, device="cuda")
        for kr, vr in ((row, nan), (nan, row)):
            f.pool.data.copy_(held)
            cache.kv4_append(f.pool, kr, vr, slot)
            for _ in range(3):
                out.fill_(7.0)
                cache.kv4_chunk(f.pool, q, f.dev_tables[0], offset, out)
                assert torch.isfinite(out[:first]).all()
                assert torch.isnan(out[first:, mine, 16:32]).all(), key
                if vr is nan:
                    assert torch.isfinite(out[:, mine, :16]).all() and torch.isfinite(out[:, mine, 32:]).all()
                else:
                    assert torch.isnan(out[first:, mine]).all()
                assert torch.isfinite(out[:, :mine.start]).all()
        f.pool.data.copy_(held)
        for bad in (f.pool.num_blocks, -1, 2 ** 31 - 1):
            tab = f.dev_tables[0].clone()
            tab[key // 16] = bad
            cache.kv4_chunk(f.pool, q, tab, offset, out)
            seen = max(0, key // 16 * 16 - offset)
            assert torch.isnan(out[seen:]).all() and torch.isfinite(out[:seen]).all(), (key, bad)
    cache.kv4_chunk(f.pool, q, f.dev_tables[0], offset, out)
    assert torch.equal(out, good)


@pytest.mark.parametrize("kv,group,d,offset,n", [(40, 1, 128, 1000, 130), (5, 3, 64, 12001, 301)])
def test_large_chunk_with_queries_of_any_size(kv, group, d, offset, n):
    """Rows of every size side by side: each keeps its own precision, and none spoils another."""
    f = Filled([offset + n], kv, d, 17)
    heads = kv * group
    size = np.array([1.0, 0.0, 1e-30, 1e30, 3e4, 1e-4, 30.0])
    x = np.random.default_rng(10).standard_normal((n, heads, d)) * size[np.arange(n) % 7][:, None, None]
    x[14, 0, 5], x[21, 0, 6] = np.nan, np.inf
    q, q64 = _bf(x)
    out = torch.empty_like(q)
    cache.kv4_chunk(f.pool, q, f.dev_tables[0], offset, out)
    got = _f64(out)
    assert np.isnan(got[14, 0]).all() and np.isnan(got[21, 0]).all()
    k, v = f.kv_of(0, offset + n)
    # 1, 0, 1e-30, 1e-4, 30, beside and between the odd ones; the other heads of the odd rows
    _check_rows(got, q64, k, v, offset, [0, 1, 2, 5, 6, 7, 8, 9, 12, 13, n - n % 7 - 7])
    for i in (14, 21):
        o, bound = ref.attention_row(q64[i, group:], k[:offset + i + 1, 1:], v[:offset + i + 1, 1:])
        assert (np.abs(got[i, group:] - o) <= bound).all()
    for i in (3, 10):  # the largest score wins by far more than any rounding
        for h in range(heads):
            s = k[:offset + i + 1, h // group] @ q64[i, h]
            top = np.sort(s)[-2:]
            if top[1] - top[0] > 2.0 ** -16 * (np.abs(k[:offset + i + 1, h // group]) @ np.abs(q64[i, h])).max():
                o = v[np.argmax(s), h // group]
                good = np.abs(got[i, h] - o) <= (2.0 ** -8 + 2.0 ** -10) * np.abs(o) + 1e-6
                assert good.all(), (i, h)


def _odd_rows(n, width, fill=7.0):
    """n rows of `width` bf16 values that start 16 bytes past a 32-byte border, in turn at one and off one."""
    flat = torch.full((16 + n * (width + 8),), fill, dtype=torch.bfloat16, device="cuda")
    return flat, flat[8:8 + n * (width + 8)].view(n, width + 8)[:, :width]


@pytest.mark.parametrize("kv,group,d,offset,n", [(40, 1, 128, 1000, 130), (8, 4, 64, 700, 333), (2, 1, 64, 40, 9)])
def test_rows_on_sixteen_byte_borders(kv, group, d, offset, n):
    """Every call with rows at the least alignment that it allows: the results of aligned rows, and nothing beside them."""
    heads = kv * group
    f = Filled([offset + n], kv, d, 19)
    k, v = torch.randn(n, kv, d, device="cuda").bfloat16(), torch.randn(n, kv, d, device="cuda").bfloat16()
    q = torch.randn(n, heads, d, device="cuda").bfloat16()
    odd = {}
    for name, t in (("k", k), ("v", v), ("q", q)):
        _, odd[name] = _odd_rows(n, t[0].numel())
        odd[name].copy_(t.reshape(n, -1))
        odd[name] = odd[name].unflatten(1, t.shape[1:])
        assert odd[name].data_ptr() % 32 == 16
    pos = torch.arange(offset, offset + n, device="cuda")
    slots = (f.dev_tables[0].long()[pos // 16] * 16 + pos % 16).to(torch.int32)
    cache.kv4_append(f.pool, k, v, slots)
    held = f.pool.data.clone()
    cache.kv4_append(f.pool, odd["k"], odd["v"], slots)
    assert torch.equal(f.pool.data, held)
    lens = torch.arange(offset, offset + n, dtype=torch.int32, device="cuda")
    tables = f.dev_tables[0].repeat(n, 1)
    for call in (lambda q, o: cache.kv4_chunk(f.pool, q, f.dev_tables[0], offset, o),
                 lambda q, o: cache.kv4_decode(f.pool, q, tables, lens, offset + n - 1, o)):
        want = torch.empty_like(q)
        call(q, want)
        flat, out = _odd_rows(n, heads * d)
        call(odd["q"], out.unflatten(1, (heads, d)))
        assert torch.equal(out, want.reshape(n, -1))
        out.fill_(7.0)
        assert (flat == 7.0).all()
    kw, vw = torch.empty_like(k), torch.empty_like(v)
    cache.kv4_read(f.pool, slots, kw, vw)
    (fk, ko), (fv, vo) = _odd_rows(n, kv * d), _odd_rows(n, kv * d)
    cache.kv4_read(f.pool, slots, ko.unflatten(1, (kv, d)), vo.unflatten(1, (kv, d)))
    assert torch.equal(ko, kw.reshape(n, -1)) and torch.equal(vo, vw.reshape(n, -1))
    ko.fill_(7.0), vo.fill_(7.0)
    assert (fk == 7.0).all() and (fv == 7.0).all()


def test_captured_large_chunks_replay_on_two_streams():
    """Chunks of both item sizes in two graphs with workspaces of their own, replayed at once with new queries and
    another block table; the same answers as calls made one by one."""
    shapes = [(4, 2, 128, 2000, 257), (5, 3, 64, 12001, 301)]
    sets, graphs = [], []
    for kv, group, d, offset, n in shapes:
        f = Filled([offset + n, offset + n], kv, d, 18)
        x = dict(q=torch.randn(n, kv * group, d, device="cuda").to(torch.bfloat16), tab=f.dev_tables[0].clone(), offset=offset)
        x["out"] = torch.empty_like(x["q"])
        x["ws"] = torch.empty(cache.kv4_chunk_workspace(offset, n, kv * group, kv, d), dtype=torch.uint8, device="cuda")
        cache.kv4_chunk(f.pool, x["q"], x["tab"], offset, x["out"], x["ws"])
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(2):
                cache.kv4_chunk(f.pool, x["q"], x["tab"], offset, x["out"], x["ws"])
        sets.append((f, x))
        graphs.append(g)
    for f, x in sets:
        x["q"].copy_(torch.randn_like(x["q"], dtype=torch.float32))
        x["tab"].copy_(f.dev_tables[1])
        x["out"].fill_(7.0)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for f, x in sets:
        want = torch.empty_like(x["out"])
        cache.kv4_chunk(f.pool, x["q"], x["tab"], x["offset"], want, x["ws"])
        assert torch.equal(want, x["out"])


@pytest.mark.parametrize("n,kv,group,d,most", [(65535, 1, 1, 64, 20), (3, 1, 200, 64, 500), (2, 300, 1, 128, 100),
                                               (1000, 2, 9, 64, 40), (300, 4, 1, 128, 256), (400, 3, 4, 128, 128)])
def test_decode_of_many_rows_and_heads(n, kv, group, d, most):
    """Rows that share the pages of a few sequences, up to as many as a call takes; heads far beyond a CTA's eight."""
    lens = [1 + j * (most - 1) // (min(n, 16) - 1) for j in range(min(n, 16))]
    f = Filled(lens, kv, d, 25)
    seq = torch.arange(n, device="cuda") % len(lens)
    ctx = (torch.tensor(lens, dtype=torch.int32, device="cuda") - 1)[seq]
    q, q64 = _bf(np.random.default_rng(26).standard_normal((n, kv * group, d)))
    out = torch.empty_like(q)
    cache.kv4_decode(f.pool, q, f.dev_tables[seq].contiguous(), ctx, most - 1, out)
    got = _f64(out)
    for i in sorted({0, 1, n // 3, n // 2, n - 2, n - 1} & set(range(n))):
        j = i % len(lens)
        o, bound = ref.attention_row(q64[i], *f.kv_of(j, lens[j]))
        assert (np.abs(got[i] - o) <= bound).all(), i
    # padding, contexts out of range and a bad block, among rows that stay what they were
    odd_ctx, odd_tables, other = ctx.clone(), f.dev_tables[seq].contiguous(), torch.full_like(out, 7.0)
    odd_ctx[0], odd_ctx[n // 2] = -1, most
    odd_tables[n - 1, 0] = f.pool.num_blocks
    cache.kv4_decode(f.pool, q, odd_tables, odd_ctx, most - 1, other)
    assert (other[0] == 0).all() and torch.isnan(other[n // 2]).all() and torch.isnan(other[n - 1]).all()
    same = torch.ones(n, dtype=torch.bool, device="cuda")
    same[[0, n // 2, n - 1]] = False
    assert torch.equal(other[same], out[same])
    if n > 65000:
        with pytest.raises(HbError):
            cache.kv4_decode(f.pool, torch.cat([q, q[:1]]), f.dev_tables[torch.cat([seq, seq[:1]])].contiguous(),
                             torch.cat([ctx, ctx[:1]]), most - 1, torch.cat([out, out[:1]]))


@pytest.mark.parametrize("n,kv,group,d,offset", [(20000, 1, 1, 64, 0), (30, 1, 200, 64, 900), (20, 300, 2, 128, 300),
                                                 (1, 1, 500, 128, 2000)])
def test_chunk_of_many_rows_and_heads(n, kv, group, d, offset):
    f = Filled([offset + n], kv, d, 27)
    q, q64 = _bf(np.random.default_rng(28).standard_normal((n, kv * group, d)))
    out = torch.empty_like(q)
    cache.kv4_chunk(f.pool, q, f.dev_tables[0], offset, out)
    k, v = f.kv_of(0, offset + n)
    _check_rows(_f64(out), q64, k, v, offset, sorted({0, 1, 127, 128, 9999, n // 2, n - 2, n - 1} & set(range(n))))


def test_captured_calls_replay_with_new_contents_and_other_streams():
    """A step (append, decode, chunk) in two graphs, each with a workspace of its own, replayed at once on two
    streams with changed inputs; the same answers as calls made one by one."""
    kv, group, d = 2, 4, 128
    heads, ctx = kv * group, 3000
    rng = np.random.default_rng(20)

    def make(seed):
        f = Filled([ctx + 1, 600], kv, d, seed)
        x = dict(q=_bf(rng.standard_normal((1, heads, d)))[0], c=_bf(rng.standard_normal((90, heads, d)))[0],
                 k=_bf(rng.standard_normal((1, kv, d)))[0], v=_bf(rng.standard_normal((1, kv, d)))[0])
        x["lens"] = torch.tensor([ctx], dtype=torch.int32, device="cuda")
        x["slot"] = torch.tensor([int(f.tables[0, ctx // 16]) * 16 + ctx % 16], dtype=torch.int32, device="cuda")
        x["od"], x["oc"] = torch.empty_like(x["q"]), torch.empty_like(x["c"])
        x["wd"] = torch.empty(cache.kv4_decode_workspace(1, heads, kv, d, ctx) + 16, dtype=torch.uint8, device="cuda")
        x["wc"] = torch.empty(cache.kv4_chunk_workspace(510, 90, heads, kv, d) + 16, dtype=torch.uint8, device="cuda")
        return f, x

    def step(f, x, stream=None):
        cache.kv4_append(f.pool, x["k"], x["v"], x["slot"], stream=stream)
        cache.kv4_decode(f.pool, x["q"], f.dev_tables[:1], x["lens"], ctx, x["od"], x["wd"], stream=stream)
        cache.kv4_chunk(f.pool, x["c"], f.dev_tables[1], 510, x["oc"], x["wc"], stream=stream)

    sets = [make(s) for s in (31, 32)]
    graphs = []
    for f, x in sets:
        step(f, x)
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            step(f, x)
        graphs.append(gr)
    for f, x in sets:
        for name in ("q", "c", "k", "v"):
            x[name].copy_(_bf(rng.standard_normal(tuple(x[name].shape)))[0])
        x["lens"].fill_(ctx - 7)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for gr, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                gr.replay()
    torch.cuda.synchronize()
    replayed = [(x["od"].clone(), x["oc"].clone()) for _, x in sets]
    for (f, x), (od, oc), s in zip(sets, replayed, streams):
        x["od"].fill_(0), x["oc"].fill_(0)
        torch.cuda.synchronize()
        step(f, x, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(x["od"], od) and torch.equal(x["oc"], oc)


@pytest.mark.parametrize("kv,d", [(8, 128), (16, 64)])
def test_pages_past_four_gigabytes(kv, d):
    """The same rows in the low pages of one pool and in the last pages of one of 5 GB: the same bytes, the same
    answers, and pages copied from one end to the other."""
    n, heads, blocks = 2200, 2 * kv, 5 * (1 << 30) // (kv * 18 * d)
    need = (n + 15) // 16
    big = torch.empty(blocks, kv, 18 * d, dtype=torch.uint8, device="cuda")
    pools = [cache.Kv4Pool.empty(need, kv, d), cache.Kv4Pool(big)]
    assert big.numel() > 1 << 32
    tabs = [torch.arange(need, dtype=torch.int32, device="cuda")]
    tabs.append(blocks - 1 - tabs[0])
    big[tabs[1].long()] = 0
    k, v = (torch.randn(n, kv, d, device="cuda").to(torch.bfloat16) for _ in range(2))
    q = torch.randn(n, heads, d, device="cuda").to(torch.bfloat16)
    pos = torch.arange(n, device="cuda")
    lens = torch.tensor([n - 1], dtype=torch.int32, device="cuda")
    got = []
    for pool, tab in zip(pools, tabs):
        slots = (tab.long()[pos // 16] * 16 + pos % 16).to(torch.int32)
        cache.kv4_append(pool, k, v, slots)
        o = [torch.empty_like(k), torch.empty_like(v), torch.empty_like(q[:1]), torch.empty_like(q[:3]), torch.empty_like(q[:900])]
        cache.kv4_read(pool, slots, o[0], o[1])
        cache.kv4_decode(pool, q[:1], tab[None], lens, n - 1, o[2])
        for chunk in (3, 900):                              # few rows, and many
            cache.kv4_chunk(pool, q[:chunk], tab, n - chunk, o[3 if chunk == 3 else 4])
        got.append(o)
    for a, b in zip(*got):
        assert torch.equal(a, b)
    assert torch.equal(big[tabs[1].long()], pools[0].data)
    cache.copy_pages(big[None], [blocks - 1, blocks - 2], [0, 1])
    assert torch.equal(big[:2], pools[0].data[:2])


def test_binding_refuses_what_it_cannot_order():
    f = Filled([300], 1, 64, 14)
    q = torch.zeros(1, 1, 64, dtype=torch.bfloat16, device="cuda")
    lens = torch.tensor([299], dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        cache.kv4_decode(f.pool, q, f.dev_tables, lens, 299, torch.empty_like(q), stream=torch.cuda.Stream())
    with pytest.raises(ValueError):
        cache.kv4_decode(f.pool, q, f.dev_tables.cpu(), lens, 299, torch.empty_like(q))
    with pytest.raises(HbError):
        cache.kv4_decode(f.pool, q, f.dev_tables, lens, 16 * f.width, torch.empty_like(q))


# -------------------------------------------------------------------- pages

@pytest.mark.parametrize("shape,dtype", [((1, 40, 16), torch.uint8), ((3, 50, 2, 18 * 64), torch.uint8),
                                         ((2, 33, 4104), torch.float32), ((80, 9, 5, 16, 64), torch.bfloat16),
                                         ((2, 4000, 8), torch.int64)])
def test_copy_pages(shape, dtype):
    rng = np.random.default_rng(3)
    g = torch.Generator(device="cuda").manual_seed(1)
    big = torch.randint(0, 100, (shape[0], shape[1] + 2) + shape[2:], generator=g, device="cuda").to(dtype)
    for pools in (big[:, :shape[1]], big[:, :shape[1]].contiguous()):  # pools further apart than their pages, and dense
        before = big.clone()
        order = rng.permutation(shape[1])
        n = shape[1] // 2
        src, dst = order[:n].astype(np.int32), order[n:2 * n].astype(np.int32)
        src[n // 2:] = src[0]                                # forks of one page
        want = pools.clone()
        want[:, torch.from_numpy(dst).long().cuda()] = want[:, torch.from_numpy(src).long().cuda()]
        cache.copy_pages(pools, src, dst)
        assert torch.equal(pools, want)
        assert torch.equal(big[:, shape[1]:], before[:, shape[1]:])
        cache.copy_pages(pools, [], [])
        cache.copy_pages(pools, src[:1].tolist(), dst[:1].tolist())
        assert torch.equal(pools, want)
    with pytest.raises(HbError):
        cache.copy_pages(big, [0], [shape[1] + 2])
    with pytest.raises(HbError):
        cache.copy_pages(big, [0, 1], [2, 2])


def test_copy_blocks_of_a_context():
    dims = synth.TINY
    cfg = native.model_config(dims, 12, 16, 4, 128, n_layers=3)
    ctx = native.Context(cfg)
    ctx.fill_kv(0x3F80)
    k = torch.randn(40, dims.n_kv_heads, dims.head_dim, device="cuda").to(torch.bfloat16)
    for layer in range(3):
        ctx.append_kv(layer, np.array([3, 7, 1], np.int32), 0, k + layer, k - layer)
    n0 = ctx.launch_count
    cache.copy_blocks(ctx, [3, 7, 1], [0, 2, 9])
    assert ctx.launch_count == n0 + 1
    for layer in range(3):
        for tab in ([0, 2, 9], [3, 7, 1]):
            a, b = torch.empty_like(k), torch.empty_like(k)
            ctx.read_kv(layer, np.array(tab, np.int32), 0, a, b)
            ctx.sync()
            assert torch.equal(a, k + layer) and torch.equal(b, k - layer)
    other = torch.empty_like(k[:16])
    ctx.read_kv(0, np.array([4], np.int32), 0, other, other.clone())
    ctx.sync()
    assert (other == 1.0).all()
    for s, d, code in (([0], [12], native.HB_ERANGE), ([0], [0], native.HB_EINVAL), ([0, 1], [2, 2], native.HB_EINVAL)):
        with pytest.raises(HbError) as e:
            cache.copy_blocks(ctx, s, d)
        assert e.value.code == code and "hb_copy_blocks" in str(e.value)
    ctx.free()


def test_a_conversation_forks_grows_and_is_compacted():
    """The operators together, as a server uses them: a prompt is appended and prefilled in two chunks, forked, each
    branch grows by decodes (the shared part-filled page is copied first), one branch ends, the cache is compacted;
    after each step every live sequence's attention is that of its own keys."""
    kv, group, d, layers = 2, 2, 64, 2
    heads, blocks = kv * group, 24
    rng = np.random.default_rng(40)
    table = cache.PageTable(blocks)
    data = torch.full((layers, blocks, kv, 18 * d), 0xFF, dtype=torch.uint8, device="cuda")
    pools = [cache.Kv4Pool(data[l]) for l in range(layers)]
    keys = {}  # seq -> [layers][tokens] values as the cache holds them

    def grow(seq, n):
        have = table.length(seq) if seq in keys else 0
        move = table.extend(seq, have + n)
        if move:
            cache.copy_pages(data, [move[0]], [move[1]])
        tab = table.table(seq)
        pos = np.arange(have, have + n)
        slots = torch.from_numpy((tab[pos // 16] * 16 + pos % 16).astype(np.int32)).cuda()
        keys.setdefault(seq, [(np.zeros((0, kv, d)), np.zeros((0, kv, d)))] * layers)
        fresh = []
        for l in range(layers):
            k, k64 = _bf(rng.standard_normal((n, kv, d)))
            v, v64 = _bf(rng.standard_normal((n, kv, d)))
            cache.kv4_append(pools[l], k, v, slots)
            held = []
            for x, old in ((k64, keys[seq][l][0]), (v64, keys[seq][l][1])):
                codes, sb = ref.quantise(x, 1.0)
                val = ref.E2M1[codes & 7] * np.where(codes & 8, -1, 1) * np.repeat(ref.E4M3[sb], 16, axis=-1)
                held.append(np.concatenate([old, val]))
            fresh.append(tuple(held))
        keys[seq] = fresh
        return have

    def check():
        seqs = sorted(keys)
        width = max(len(table.table(s)) for s in seqs)
        tabs = np.full((len(seqs), width), -1, np.int32)
        for j, s in enumerate(seqs):
            tabs[j, :len(table.table(s))] = table.table(s)
        ctx = np.array([table.length(s) - 1 for s in seqs], np.int32)
        for l in range(layers):
            q, q64 = _bf(rng.standard_normal((len(seqs), heads, d)))
            out = torch.empty_like(q)
            cache.kv4_decode(pools[l], q, torch.from_numpy(tabs).cuda(), torch.from_numpy(ctx).cuda(), int(ctx.max()), out)
            for j, s in enumerate(seqs):
                o, bound = ref.attention_row(q64[j], *keys[s][l])
                assert (np.abs(_f64(out[j]) - o) <= bound).all(), (l, s)

    def prefill(seq, n):
        offset = grow(seq, n)
        for l in range(layers):
            q, q64 = _bf(rng.standard_normal((n, heads, d)))
            out = torch.empty_like(q)
            cache.kv4_chunk(pools[l], q, torch.from_numpy(table.table(seq)).cuda(), offset, out)
            for i in (0, n // 2, n - 1):
                k, v = keys[seq][l]
                o, bound = ref.attention_row(q64[i], k[:offset + i + 1], v[:offset + i + 1])
                assert (np.abs(_f64(out[i]) - o) <= bound).all(), (l, i)

    grow(9, 30)                      # an older request in the low pages
    prefill(1, 50)
    prefill(1, 23)                   # 73 tokens: the last page part-filled
    check()
    table.fork(1, 2)
    keys[2] = list(keys[1])
    check()
    for _ in range(9):               # past a page's end
        grow(2, 1)
        grow(1, 1)
        check()
    table.fork(2, 3, 40)             # a branch from the middle of a page
    keys[3] = [(k[:40], v[:40]) for k, v in keys[2]]
    grow(3, 5)
    check()
    table.release(9)
    del keys[9]
    table.release(1)
    del keys[1]
    src, dst = table.compact()
    assert len(src)
    cache.copy_pages(data, src, dst)
    held = blocks - table.num_free
    assert max(int(table.table(s).max()) for s in keys) == held - 1
    check()
    grow(2, 20)
    check()
