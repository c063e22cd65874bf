"""Attention over the 4-bit cache where a softmax is peaked, where V is small
or of several sizes, and where a NaN has no weight: against the plain 64-bit
forms (cache_ref.py)."""
import numpy as np
import pytest

import cache_ref as ref
from chunked_prefill_hybrid_gb300 import cache

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
