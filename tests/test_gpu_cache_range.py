"""Attention over the 4-bit cache where a softmax is peaked, where V is small
or of several sizes, and where a NaN has no weight: against the plain 64-bit
forms (cache_ref.py)."""
import numpy as np
import pytest

import cache_ref as ref
from chunked_prefill_hybrid_gb300 import cache
from chunked_prefill_hybrid_gb300.native import HB_ERANGE, HbError

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def _bf(x):
    t = torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16)
    return t.cuda(), t.double().numpy()


class Held:
    """One sequence of keys and values [n][kv][d] in a pool whose other slots hold NaN scales."""

    def __init__(self, k, v, ks=1.0, vs=1.0):
        n, self.kv, self.d = k.shape
        need = (n + 15) // 16
        self.table = np.random.default_rng(1).permutation(need + 3).astype(np.int32)[:need]
        slots = self.table[np.arange(n) // 16] * 16 + np.arange(n) % 16
        self.host = np.full((need + 3, self.kv, 18 * self.d), 0xFF, np.uint8)
        ref.store(self.host, slots, *ref.quantise(k, ks), "k")
        ref.store(self.host, slots, *ref.quantise(v, vs), "v")
        pages = self.host[self.table]
        self.k = ref.values(pages, "k", ks).reshape(-1, self.kv, self.d)[:n]
        self.v = ref.values(pages, "v", vs).reshape(-1, self.kv, self.d)[:n]
        self.pool = cache.Kv4Pool(torch.from_numpy(self.host).cuda(), ks, vs)
        self.dev_table = torch.from_numpy(self.table).cuda()

    def decode(self, q, n):
        """Query j of q at position n[j] - 1."""
        out = torch.empty_like(q)
        lens = torch.tensor([x - 1 for x in n], dtype=torch.int32, device="cuda")
        cache.kv4_decode(self.pool, q, self.dev_table.repeat(len(n), 1), lens, max(n) - 1, out)
        return out

    def chunk(self, q, offset):
        out = torch.empty_like(q)
        cache.kv4_chunk(self.pool, q, self.dev_table, offset, out)
        return out


def _peaked(rng, rows, n, kv, group, d, log2_gap, at):
    """Queries and keys where key `at` of each kv head lies about log2_gap (powers of two of weight) above the others."""
    u = rng.standard_normal((kv, d))
    u *= np.sqrt(d) / np.linalg.norm(u, axis=-1, keepdims=True)
    q = np.repeat(u, group, axis=0)[None] + 0.2 * rng.standard_normal((rows, kv * group, d))
    k = rng.standard_normal((n, kv, d))
    k -= (k * u).sum(-1, keepdims=True) / d * u  # at right angles to the common direction
    k[at] = u * (log2_gap * np.log(2) / np.sqrt(d))
    return q, k


def _near(got, q64, k, v, rows_keys):
    got = got.double().cpu().numpy()
    for i, n in rows_keys:
        o, bound = ref.attention_row(q64[i], k[:n], v[:n])
        assert (np.abs(got[i] - o) <= bound).all(), (i, n, np.max(np.abs(got[i] - o) / bound))


FORMS = [(1, 1, 128), (2, 1, 64), (1, 2, 64), (1, 2, 128), (2, 4, 128), (1, 8, 64), (1, 11, 128)]


@pytest.mark.parametrize("kv,group,d", FORMS)
def test_a_nan_of_v_counts_however_small_its_weight(kv, group, d):
    """A key that a row sees makes its channels NaN wherever it lies: in the last pages, which are masked by position,
    as in an earlier one; also where its weight is 2^-45 of the largest."""
    n = 200
    q, k = _peaked(np.random.default_rng(2), 4, n, kv, group, d, 45, 7)
    v = np.random.default_rng(3).standard_normal((n, kv, d))
    for key in (20, 150, n - 3):
        with_nan = v.copy()
        with_nan[key, :, 20] = np.nan                       # block 1
        h = Held(k, with_nan)
        qd, q64 = _bf(q)
        clean = np.nan_to_num(h.v, nan=0.0)
        for out, lens in ((h.decode(qd[:1], [n]), [n]), (h.decode(qd, [n, key, n, key + 1]), [n, key, n, key + 1]),
                          (h.chunk(qd[:3], key - 1), [key, key + 1, key + 2]), (h.chunk(qd[:1], n - 1), [n])):
            for i, m in enumerate(lens):
                hit = out[i, :, 16:32]
                assert torch.isnan(hit).all() if m > key else torch.isfinite(hit).all(), (key, i, m)
                o, bound = ref.attention_row(q64[i], h.k[:m], clean[:m])
                rest = np.r_[0:16, 32:d]
                assert (np.abs(out[i].double().cpu().numpy() - o) <= bound)[:, rest].all(), (key, i, m)


# V's sizes: small ones, 18 powers of two between blocks of a head, growing and shrinking along the sequence, and a
# token far above the rest
SIZES = {
    "small": lambda n, kv, d, rng: np.full((n, 1, 1), 0.02),
    "large": lambda n, kv, d, rng: np.full((n, 1, 1), 300.0),
    "blocks": lambda n, kv, d, rng: np.repeat(2.0 ** np.linspace(-7, 9, d // 16), 16)[None, None],
    "growing": lambda n, kv, d, rng: 2.0 ** np.linspace(-7, 5, n)[:, None, None],
    "shrinking": lambda n, kv, d, rng: 2.0 ** np.linspace(5, -7, n)[:, None, None],
    "outlier": lambda n, kv, d, rng: np.where(np.arange(n) == n // 3, 4.0, 0.02)[:, None, None],
    "zeros first": lambda n, kv, d, rng: np.where(np.arange(n) < n // 2, 0.0, 0.02)[:, None, None],
}


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("kv,group,d", FORMS)
def test_a_sink_takes_no_bits_from_the_rest(kv, group, d, size):
    """One key 2^18 to 2^24 above each of the others, its V near zero: what the others add is kept, whatever V's size."""
    n = 3000
    rng = np.random.default_rng(4)
    for gap, at in ((18, 0), (24, 5)):
        q, k = _peaked(rng, 4, n, kv, group, d, gap, at)
        v = rng.standard_normal((n, kv, d)) * SIZES[size](n, kv, d, rng)
        v[at] *= 0.001
        h = Held(k, v)
        qd, q64 = _bf(q)
        lens = [n, 1000, n - 5, 70]
        _near(h.decode(qd, lens), q64, h.k, h.v, list(enumerate(lens)))
        _near(h.decode(qd[:1], [n]), q64, h.k, h.v, [(0, n)])                   # split over CTAs
        _near(h.chunk(qd[:1], n - 1), q64, h.k, h.v, [(0, n)])
        _near(h.chunk(qd, n - 4), q64, h.k, h.v, [(i, n - 3 + i) for i in range(4)])


@pytest.mark.parametrize("kv,group,d", [(1, 1, 128), (1, 4, 64), (1, 8, 128)])
def test_a_sink_over_many_keys(kv, group, d):
    n = 40000
    q, k = _peaked(np.random.default_rng(5), 2, n, kv, group, d, 27, 0)
    v = np.random.default_rng(6).standard_normal((n, kv, d)) + 0.3
    v[0] *= 0.001
    h = Held(k, v)
    qd, q64 = _bf(q)
    _near(h.decode(qd[:1], [n]), q64, h.k, h.v, [(0, n)])
    _near(h.decode(qd, [n, n - 100]), q64, h.k, h.v, [(0, n), (1, n - 100)])


@pytest.mark.parametrize("kv,group,d,offset,n", [(40, 1, 128, 1000, 130), (4, 2, 64, 2000, 257), (1, 8, 128, 20000, 64),
                                                 (2, 4, 128, 3000, 600)])
@pytest.mark.parametrize("gap", [20, 27, 31])
def test_a_sink_in_a_large_chunk(kv, group, d, offset, n, gap):
    q, k = _peaked(np.random.default_rng(7), n, offset + n, kv, group, d, gap, 3)
    v = np.random.default_rng(8).standard_normal((offset + n, kv, d)) + 0.3
    v[3] = 0
    h = Held(k, v)
    qd, q64 = _bf(q)
    rows = sorted({0, 1, 127 // group, 128 // group, n // 2, n - 1} & set(range(n)))
    _near(h.chunk(qd, offset), q64, h.k, h.v, [(i, offset + i + 1) for i in rows])


@pytest.mark.parametrize("kv,group,d,offset,n", [(2, 1, 128, 0, 700), (2, 1, 64, 100, 3), (2, 4, 128, 600, 200),
                                                 (1, 8, 64, 2000, 2)])
def test_scores_that_rise_all_along(kv, group, d, offset, n):
    """Each key above the one before it: the running maximum moves in every tile."""
    rng = np.random.default_rng(9)
    m = offset + n
    u = rng.standard_normal((kv, d))
    q = np.repeat(u, group, axis=0)[None] + 0.05 * rng.standard_normal((n, kv * group, d))
    for reach in (30.0, 400.0):                              # of the scores, from the first key to the last
        k = u[None] * np.linspace(0, reach / np.sqrt(d), m)[:, None, None]
        h = Held(k, rng.standard_normal((m, kv, d)) * 0.1 + 0.05)
        qd, q64 = _bf(q)
        rows = sorted({0, 1, n // 2, n - 1} & set(range(n)))
        _near(h.chunk(qd, offset), q64, h.k, h.v, [(i, offset + i + 1) for i in rows])
        _near(h.decode(qd[:3], [m, m // 2, 1][:min(3, n)]), q64, h.k, h.v, list(enumerate([m, m // 2, 1][:min(3, n)])))


def test_shapes_past_32_bits_are_refused_not_cut():
    """2^32 + 1 rows or pools are not one."""
    many = (1 << 32) + 1
    pool = cache.Kv4Pool.empty(2, 1, 64)
    held = pool.data.clone()
    rows = torch.ones(1, 1, 64, dtype=torch.bfloat16, device="cuda").expand(many, 1, 64)
    slots = torch.zeros(many, dtype=torch.int32, device="cuda")
    pages = torch.arange(64, device="cuda").view(1, 2, 32)
    for call in (lambda: cache.kv4_append(pool, rows, rows, slots),
                 lambda: cache.kv4_read(pool, slots, rows, rows),
                 lambda: cache.kv4_decode(pool, rows, slots[:, None], slots, 0, rows),
                 lambda: cache.copy_pages(pages.expand(many, 2, 32), [0], [1])):
        with pytest.raises(HbError) as e:
            call()
        assert e.value.code == HB_ERANGE
    assert torch.equal(pool.data, held) and torch.equal(pages.flatten(), torch.arange(64, device="cuda"))
    assert (rows[0] == 1).all()


@pytest.mark.parametrize("kv,group,d", [(1, 1, 128), (1, 2, 64), (2, 4, 128)])
def test_a_score_of_zero_stays_zero(kv, group, d):
    """Keys of zeros score 0 whatever the query's size and k_scale make of the others' scores."""
    n = 500
    v = np.random.default_rng(11).standard_normal((n, kv, d))
    h = Held(np.zeros((n, kv, d)), v, ks=2.0 ** 60)
    for size in (1e30, 3e38, 1e-38):
        qd, q64 = _bf(np.random.default_rng(12).choice((-1.0, 1.0), (300, kv * group, d)) * size)
        zero = np.zeros_like(q64)
        _near(h.decode(qd[:3], [n, 17, 1]), zero, h.k, h.v, [(0, n), (1, 17), (2, 1)])
        _near(h.chunk(qd[:2], n - 2), zero, h.k, h.v, [(0, n - 1), (1, n)])
        _near(h.chunk(qd, n - 300), zero, h.k, h.v, [(i, n - 299 + i) for i in (0, 1, 130, 299)])


@pytest.mark.parametrize("n,kv,d,ks,vs", [(1, 1, 64, 1.0, 1.0), (37, 3, 64, 1.0, 0.3779644668), (19, 5, 128, 0.5, 2.0),
                                          (200, 2, 128, 0.7071067691, 1.0)])
@pytest.mark.parametrize("with_nan", [False, True])
def test_append_writes_its_own_bytes_and_no_others(n, kv, d, ks, vs, with_nan):
    """Every byte of the pool, among random ones, but for two that mean nothing: the codes of a block that held a NaN,
    and the sign of a code of zero."""
    ks, vs = float(np.float32(ks)), float(np.float32(vs))
    rng = np.random.default_rng(13)
    blocks = n // 16 + 4
    x = rng.standard_normal((2, n, kv, d)) * np.exp(rng.standard_normal((1, 1, kv, d)))
    x[:, 0, 0, :16] = 0
    x[0, n // 2, 0, 16:32] = np.linspace(-6, 6, 16) * 0.8125  # ties
    x[1, n // 3, 0, 32] = 1e5                                 # a scale that saturates
    x[1, n - 1, -1, 3] = np.inf
    if with_nan:
        x[0, n // 2, -1, 40] = x[1, 0, 0, 17] = np.nan
    slots = rng.permutation(blocks * 16)[:n].astype(np.int32)
    if n > 8:
        slots[7], slots[8] = -1, blocks * 16
    before = rng.integers(0, 256, (blocks, kv, 18 * d)).astype(np.uint8)
    pool = cache.Kv4Pool(torch.from_numpy(before).cuda(), ks, vs)
    want, codes_at = before.copy(), ref.addresses(d)
    given = []
    for which, ps, rows in (("k", ks, x[0]), ("v", vs, x[1])):
        t, x64 = _bf(rows)
        given.append(t)
        ref.store(want, slots, *ref.quantise(x64, ps), which)
    cache.kv4_append(pool, *given, torch.from_numpy(slots).cuda())
    got = pool.data.cpu().numpy()
    assert torch.isnan(given[0]).any().item() == with_nan

    def settled(data):
        """The bytes with what means nothing in the written slots made 0."""
        data = data.copy()
        for s in slots[(slots >= 0) & (slots < 16 * blocks)]:
            page, tok = data[s // 16], s % 16
            for which in "kv":
                sb = np.repeat(page[:, codes_at[which + "s"][tok]] & 0x7f, 16, axis=-1)  # [kv][d]
                for nib in (0, 1):
                    sel = codes_at["nib"][tok] == nib
                    at = codes_at[which][tok][sel]
                    code = page[:, at] >> (4 * nib) & 15
                    code = np.where((sb[:, sel] == 0x7f) | (code == 8), 0, code)
                    page[:, at] = (page[:, at] & (0xF0 if nib == 0 else 0x0F)) | (code << (4 * nib))
        return data

    assert np.array_equal(settled(got), settled(want))
    untouched = np.ones(blocks * 16, bool)
    untouched[slots[(slots >= 0) & (slots < 16 * blocks)]] = False
    assert untouched.sum() >= 48 and not np.array_equal(got, before)


@pytest.mark.parametrize("size", [300.0, 3e3, 3e4, 1e30])
@pytest.mark.parametrize("kv,group,d", [(2, 1, 64), (2, 1, 128), (1, 4, 128)])
def test_large_queries_keep_a_tie(kv, group, d, size):
    """Two equal keys far above the rest share a row evenly, in whatever pages they lie, even where a score's last
    place is worth more than one: the same sums of the same numbers."""
    n = 300
    rng = np.random.default_rng(14)
    q, k = _peaked(rng, 150, n, kv, group, d, 0, 5)
    k[101] = k[142] = 3 * q[0, ::group] / np.abs(q[0]).max()
    h = Held(k, rng.standard_normal((n, kv, d)))
    qd, q64 = _bf(q * size)
    for out, rows in ((h.decode(qd[:2], [n, n]), (0, 1)), (h.decode(qd[:1], [n]), (0,)), (h.chunk(qd, n - 150), (0, 149)),
                      (h.chunk(qd[:2], n - 2), (0, 1))):
        for i in rows:
            for head in range(kv * group):
                s = h.k[:, head // group] @ q64[i, head] / np.sqrt(d)
                top = np.sort(s)[-3:]
                assert top[1] == top[2] > top[0] + 100
                pair = h.v[[101, 142], head // group]
                bound = 2.0 ** -8 * np.abs(pair.mean(0)) + 2.0 ** -10 * np.abs(pair).mean(0) + 1e-6
                assert (np.abs(out[i, head].double().cpu().numpy() - pair.mean(0)) <= bound).all(), (i, head)
