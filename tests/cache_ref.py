"""Plain 64-bit forms of the 4-bit paged cache's operators (numpy, no code of
the library): quantisation, the pool's layout, attention over it."""
import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([(1 + m / 8) * 2.0 ** (e - 7) if e else m * 2.0 ** -9 for e in range(16) for m in range(8)][:127])


def nearest(a, grid):
    """Index of the grid value nearest to a >= 0, ties to the even index, beyond the last the last."""
    hi = np.clip(np.searchsorted(grid, a), 1, len(grid) - 1)
    lo = hi - 1
    up, down = grid[hi] - a, a - grid[lo]
    return np.where(up < down, hi, np.where(up > down, lo, np.where(hi % 2 == 0, hi, lo)))


def quantise(x, ps):
    """x [n][kv][d] float64 -> (codes [n][kv][d] 0..15, scale bytes [n][kv][d/16])."""
    n, kv, d = x.shape
    b = x.reshape(n, kv, d // 16, 16)
    amax = np.abs(b).max(-1)
    with np.errstate(invalid="ignore"):
        sb = nearest(np.minimum(np.nan_to_num(amax / (6 * ps), nan=0.0, posinf=1e300), 1e300), E4M3)
        s = E4M3[sb] * ps
        q = np.where(s[..., None] > 0, np.abs(b) / np.where(s > 0, s, 1)[..., None], 0)
        codes = nearest(np.minimum(np.nan_to_num(q, nan=0.0, posinf=1e300), 1e300), E2M1) + 8 * np.signbit(b)
    sb = np.where(np.isnan(b).any(-1), 0x7f, sb)
    return codes.reshape(n, kv, d).astype(np.uint8), sb.astype(np.uint8)


def addresses(d):
    """Byte and nibble of each (token, channel) and byte of each scale (token, block), for K and V."""
    nb = d // 16
    tok, ch = np.meshgrid(np.arange(16), np.arange(d), indexing="ij")
    i, c = ch // 16, ch % 16
    k = (tok * 4 + c // 4) * 2 * nb + 2 * i + (c % 4) // 2
    v = 8 * d + (((tok // 2 % 2) * 8 + c // 2) * 4 + tok // 4) * 2 * nb + (tok % 2) * nb + i
    st, si = np.meshgrid(np.arange(16), np.arange(nb), indexing="ij")
    return dict(k=k, v=v, nib=c % 2, ks=16 * d + st * nb + si, vs=17 * d + si * 16 + st)


def store(pool, slots, codes, sb, which):
    """Put rows into a pool [blocks][kv][18 d] (numpy uint8); slots outside it are skipped."""
    n, kv, d = codes.shape
    a = addresses(d)
    for r in range(n):
        s = int(slots[r])
        if s < 0 or s >= 16 * pool.shape[0]:
            continue
        page, tok = pool[s // 16], s % 16
        at = a[which][tok]
        for nib in (0, 1):
            sel = a["nib"][tok] == nib
            keep = 0xF0 if nib == 0 else 0x0F
            page[:, at[sel]] = (page[:, at[sel]] & keep) | (codes[r][:, sel] << (4 * nib))
        page[:, a[which + "s"][tok]] = sb[r]


def values(pages, which, ps):
    """[m][kv][18 d] bytes -> [m][16][kv][d] values (NaN where a scale is NaN)."""
    d = pages.shape[-1] // 18
    a = addresses(d)
    byte = pages[:, :, a[which]]                     # m kv 16 d
    code = (byte >> (4 * a["nib"])) & 15
    mag = E2M1[code & 7] * np.where(code & 8, -1.0, 1.0)
    sb = pages[:, :, a[which + "s"]]
    table = np.concatenate([E4M3, [np.nan], -E4M3, [np.nan]])
    out = mag * np.repeat(table[sb], 16, axis=-1) * ps
    return out.transpose(0, 2, 1, 3)


def attention_row(q, k, v):
    """q [heads][d], k, v [keys][kv][d] -> (o, bound) with bound the error a correct kernel may make.

    Roundings counted: P to f16 and its product with a V scale (2^-11 each, of
    the weighted mean of |v|); scores as fp32 sums of exact products and one
    exp2 (2^-17 of the largest sum of |q k| in log2 units, numerator and
    denominator together); the result to bf16 (2^-8 of it)."""
    heads, d = q.shape
    kv = k.shape[1]
    g = heads // kv
    o, bound = np.empty((heads, d)), np.empty((heads, d))
    for h in range(heads):
        kk, vv = k[:, h // g], v[:, h // g]
        s = kk @ q[h] / np.sqrt(d)
        p = np.exp(s - s.max())
        p /= p.sum()
        o[h] = p @ vv
        mean_abs = p @ np.abs(vv)
        reach = (np.abs(kk) @ np.abs(q[h])).max() / np.sqrt(d) * 1.4427
        bound[h] = 2.0 ** -8 * np.abs(o[h]) + mean_abs * (2.0 ** -10 + 2.0 ** -17 * reach) + 1e-6
    return o, bound
