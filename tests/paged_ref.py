"""Plain 64-bit forms of the operators of include/hb_paged.h (numpy, no code
of the library), and how far a result may be from them."""
import numpy as np


def keys_of(pool, table, kvh, n):
    """Rows of the first n tokens of one kv head, [n][d], through a block table."""
    pages = pool[np.asarray(table)[:(n + 15) // 16], kvh]
    return pages.reshape(-1, pool.shape[-1])[:n]


def attend(q, k, v):
    """softmax(q k / sqrt d) v of one row and head: (o, p, W, eps).  W = sum p |v|.  eps bounds the relative error of
    a weight: a score is a sum of d exact products, each addition off by 2^-23 of the sum of magnitudes at most (a
    tensor core's chopped addition; fp32's is half of that); the maximum, subtracted and scaled, and the exponential
    add 2^-21 and a few 2^-23 of the score's range."""
    d = q.shape[-1]
    s = k @ q / np.sqrt(d)
    a = (np.abs(k) @ np.abs(q)).max() / np.sqrt(d)
    p = np.exp(s - s.max())
    p /= p.sum()
    return p @ v, p, p @ np.abs(v), 2.0 ** -21 + (d + 8) * 2.0 ** -23 * a


def out_bound(o, w, eps, n):
    """o rounded to bf16 (half a step: 2^-8); weights in two bf16 terms (2^-16), off by eps each and in their sum;
    n terms summed in fp32 (a chopped addition a page and warp, 2^-23 each, and the joins)."""
    return 2.0 ** -8 * np.abs(o) + w * (2.0 ** -16 + 2 * eps + (n / 16 + 64) * 2.0 ** -23) + 1e-37


def shared(q, k_pool, v_pool, tables, ctx, group):
    """Rows [n][heads][d]: (o, bound); a row with ctx -1 is 0."""
    n, heads, d = q.shape
    o, b = np.zeros(q.shape), np.zeros(q.shape)
    for j in range(n):
        if ctx[j] < 0:
            continue
        for h in range(heads):
            k, v = (keys_of(pool, tables[j], h // group, ctx[j] + 1) for pool in (k_pool, v_pool))
            o[j, h], _, w, eps = attend(q[j, h], k, v)
            b[j, h] = out_bound(o[j, h], w, eps, ctx[j] + 1)
    return o, b


def weigh(q, k_pool, v_pool, tables, ctx, group, nq, weights, wtables, decay):
    """(o, bound, weights, their bound) of n sequences of nq rows; weights [blocks][kv][16] are copied first."""
    rows, heads, d = q.shape
    o, b = np.zeros(q.shape), np.zeros(q.shape)
    new, wb = weights.copy(), np.zeros(weights.shape)
    for j in range(len(ctx)):
        c = ctx[j]
        if c < 0:
            continue
        total, slack = np.zeros((heads // group, c + 1)), np.zeros((heads // group, c + 1))
        for i in range(nq):
            see = c + 1 - (nq - 1) + i
            if see <= 0:
                continue
            for h in range(heads):
                k, v = (keys_of(pool, tables[j], h // group, see) for pool in (k_pool, v_pool))
                r = j * nq + i
                o[r, h], p, w, eps = attend(q[r, h], k, v)
                b[r, h] = out_bound(o[r, h], w, eps, see)
                total[h // group, :see] += p
                slack[h // group, :see] += p * (2 * eps + (see / 16 + 64) * 2.0 ** -23)
        for t in range(c + 1):
            blk = wtables[j][t // 16]
            old = np.zeros(heads // group) if t > c - nq or decay == 0 else decay * weights[blk, :, t % 16]
            new[blk, :, t % 16] = old + total[:, t]
            # nq x group weights added in fp32 to what was there; weights below 2^-126 are 0
            wb[blk, :, t % 16] = slack[:, t] + (nq * group + 3) * 2.0 ** -24 * (np.abs(old) + total[:, t]) + nq * group * 2.0 ** -120
    return o, b, new, wb


def select(weights, tables, lens, keep, first, recent):
    """kept [n][kv][keep], by a sort of (weight descending, position ascending)."""
    n, kv = len(lens), weights.shape[1]
    out = np.full((n, kv, keep), -1, np.int64)
    for j in range(n):
        m = int(lens[j])
        for h in range(kv):
            if m <= keep:
                out[j, h, :m] = np.arange(m)
                continue
            w = np.empty(m)
            for t in range(m):
                blk = tables[j][t // 16]
                w[t] = weights[blk, h, t % 16] if 0 <= blk < weights.shape[0] else np.nan
            pos = [t for t in range(m) if t < first or t >= m - recent]
            rest = [t for t in range(m) if first <= t < m - recent]
            # a NaN is below every number, -inf included
            rest.sort(key=lambda t: (np.isnan(w[t]), 0.0 if np.isnan(w[t]) else -w[t], t))
            out[j, h] = sorted(pos + rest[:keep - len(pos)])
    return out


def move(pool, tables, new_tables, kept):
    """pool [blocks][kv][16][..] after the move."""
    out = pool.copy()
    for j in range(kept.shape[0]):
        for h in range(kept.shape[1]):
            for i, t in enumerate(kept[j, h]):
                if t < 0:
                    break
                if t // 16 >= len(tables[j]):
                    continue
                a, b = tables[j][t // 16], new_tables[j][i // 16]
                if 0 <= a < pool.shape[0] and 0 <= b < pool.shape[0]:
                    out[b, h, i % 16] = pool[a, h, t % 16]
    return out
