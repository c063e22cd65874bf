"""What is measured of the attention over shared prefixes and of eviction by accumulated attention weight.

Three operators over the bf16 paged cache (K and V pools [num_blocks][n_kv_heads][16][head_dim], block tables):

shared  decode attention of rows in groups; the rows of a group share their first tokens, whose keys are read once.
weigh   decode attention (or that of a window of several queries a sequence) that also adds every key's softmax
        weight, summed over the queries and the heads of a kv head, to a paged fp32 pool [num_blocks][n_kv_heads][16]:
        w = decay w + sum p.  A key that the call's own rows bring starts from 0.
evict   for each sequence and kv head, the tokens to keep (the first, the most recent and the heaviest of the rest, in
        order) and the move of their K, V and weights to the front of new pages.

``run`` computes each in plain torch operations, or, where ``own`` is set, through the library's calls.
"""
import math

import numpy as np
import torch

own = False

BS = 16  # tokens a block


# ------------------------------------------------------------------- cases
# kv: kv heads, group: heads of each.  shared: rows and prefix of each group, lo..hi further tokens of each row.
# weigh: n sequences of lo..hi cached tokens, nq queries each.  evict: n sequences of lo..hi tokens, keep of them stay.

def listed():
    return [
        # the tiny layer's decodes after a fork: latency alone
        dict(name="shared 4 rows, prefix 64 + 1-136, 4 x 64", op="shared", rows="4", prefix="64", lo=1, hi=136, kv=4,
             group=1, d=64),
        # the decodes of the LLaMA-13B hybrid batch, three quarters of their context a common prompt
        dict(name="shared 18 rows, prefix 768 + 257, 40 x 128", op="shared", rows="18", prefix="768", lo=257, hi=257,
             kv=40, group=1, d=128),
        # the largest decode batch of the 40-layer stack behind one system prompt
        dict(name="shared 128 rows, prefix 2048 + 64-512, 40 x 128", op="shared", rows="128", prefix="2048", lo=64,
             hi=512, kv=40, group=1, d=128),
        # parallel samples over one very long document, grouped heads
        dict(name="shared 16 rows, prefix 130000 + 1-999, 8 x 8 x 128", op="shared", rows="16", prefix="130000", lo=1,
             hi=999, kv=8, group=8, d=128),
        # a request of its own, a few behind an odd prefix and many behind a long one: the products count, not the bytes
        dict(name="shared 1 + 7 + 56 rows, prefix 0, 333, 16389, 8 x 8 x 128", op="shared", rows="1,7,56",
             prefix="0,333,16389", lo=1, hi=1000, kv=8, group=8, d=128),
        # weights along with the tiny layer's decodes
        dict(name="weigh 4 x ctx 32-200, 4 x 64", op="weigh", n=4, nq=1, lo=32, hi=200, kv=4, group=1, d=64, decay=1.0),
        # along with the decodes of the LLaMA-13B hybrid batch
        dict(name="weigh 18 x ctx 1024, 40 x 128", op="weigh", n=18, nq=1, lo=1024, hi=1024, kv=40, group=1, d=128,
             decay=1.0),
        # one request with a very long context, grouped heads, old weights fading
        dict(name="weigh 1 x ctx 130999, 8 x 8 x 128", op="weigh", n=1, nq=1, lo=130999, hi=130999, kv=8, group=8,
             d=128, decay=0.96875),
        # a prompt's first weights: those that its last 32 queries give
        dict(name="weigh 2 x 32 queries, ctx 2047-4001, 8 x 4 x 128", op="weigh", n=2, nq=32, lo=2047, hi=4001, kv=8,
             group=4, d=128, decay=0.0),
        # a small cache halved: latency alone
        dict(name="evict 4 x 33-201 to 32, 4 x 64", op="evict", n=4, lo=33, hi=201, keep=32, first=4, recent=8, kv=4,
             d=64),
        # the LLaMA-13B decodes' caches halved
        dict(name="evict 18 x 1025 to 512, 40 x 128", op="evict", n=18, lo=1025, hi=1025, keep=512, first=4, recent=128,
             kv=40, d=128),
        # one very long cache halved
        dict(name="evict 1 x 131000 to 65536, 8 x 128", op="evict", n=1, lo=131000, hi=131000, keep=65536, first=4,
             recent=1024, kv=8, d=128),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("shared", "weigh", "evict"))
    d = rng.choice((64, 128, 128))
    kv = rng.choice((1, 2, 4, 5, 8, 10, 16, 32, 40, 52))
    group = rng.choice((1, 1, 2, 3, 4, 5, 8, 12)) if kv <= 10 else 1
    heads = kv * group
    if op == "shared":
        groups = rng.choice((1, 1, 1, 2, 3, 6))
        rows = [_log_int(rng, 1, 128 // groups) for _ in range(groups)]
        prefix = [rng.choice((0, 1, 1, 1)) * _log_int(rng, 1, 100000 // groups) for _ in range(groups)]
        hi = _log_int(rng, 1, 1000)
        # bytes of the own keys, scores of the products, and both again where they are padded to the largest group
        while sum(rows) * hi * kv * 4 * d > 3e8:
            hi = (hi + 1) // 2
        while (max(prefix) * kv * 4 * d * groups > 4.5e8 or 4 * d * heads * max(rows) * groups * max(prefix) > 5e10
               or heads * max(rows) * groups * max(prefix) > 4e8):
            prefix = [x // 2 for x in prefix]
        return dict(op=op, rows=",".join(map(str, rows)), prefix=",".join(map(str, prefix)),
                    lo=max(1, hi // rng.choice((1, 2, 16))), hi=hi, kv=kv, group=group, d=d)
    if op == "weigh":
        hi = _log_int(rng, 1, 100000)
        nq = rng.choice((1, 1, 2, 7, 16, 32))
        n = _log_int(rng, 1, 128)
        while n > 1 and (n * hi * kv * 4 * d > 4e8 or n * hi * heads * d > 1e9):
            n = (n + 1) // 2
        while hi > 1 and (hi * n * kv * 4 * d > 4e8 or hi * n * heads * d > 1e9):
            hi = (hi + 1) // 2
        while nq > 1 and (4 * d * heads * n * nq * hi > 3e10 or heads * n * nq * hi > 2e7):
            nq = nq // 2
        return dict(op=op, n=n, nq=nq, lo=max(nq - 1, hi // rng.choice((1, 2, 16)) - 1), hi=max(nq - 1, hi), kv=kv,
                    group=group, d=d, decay=rng.choice((1.0, 1.0, 0.96875, 0.5, 0.0)))
    hi = _log_int(rng, 2, 130000)
    n = _log_int(rng, 1, max(1, min(128, int(4.5e8 / (hi * kv * 4 * d)))))
    while hi > 2 and n * hi * kv * 4 * d > 4.5e8:
        hi = hi // 2
    keep = max(1, int(hi * rng.choice((0.1, 0.25, 0.5, 0.8))))
    first, recent = rng.choice((0, 1, 4, 64)), rng.choice((0, 1, 32, 500))
    first = min(first, keep // 4)
    recent = min(recent, keep // 2)
    return dict(op=op, n=n, lo=max(1, hi // rng.choice((1, 2, 16))), hi=hi, keep=keep, first=first, recent=recent, kv=kv,
                d=d)


def _ints(text):
    return np.array([int(x) for x in text.split(",")], np.int32)


def work(case):
    op, kv, d = case["op"], case["kv"], case["d"]
    if op == "evict":
        lens = _spread(case["n"], case["lo"], case["hi"], 0)
        kept = int(np.minimum(lens, case["keep"]).sum())
        # the weights read and the choice written; K, V and the weights of the kept tokens read and written
        return {"bytes": kv * (4 * int(lens.sum()) + 4 * case["n"] * case["keep"] + 2 * kept * (4 * d + 4)), "flops": 0}
    heads = kv * case["group"]
    if op == "shared":
        rows, prefix = _ints(case["rows"]).astype(np.int64), _ints(case["prefix"]).astype(np.int64)
        mine = int(_spread(int(rows.sum()), case["lo"], case["hi"], 0).sum())
        keys = int(prefix.sum()) + mine
        pairs = int((rows * prefix).sum()) + mine
        return {"bytes": keys * kv * 4 * d + 4 * int(rows.sum()) * heads * d + keys // 4, "flops": 4 * d * heads * pairs}
    n, nq = case["n"], case["nq"]
    keys = int(_spread(n, case["lo"], case["hi"], 0).sum()) + n
    old = 4 if case["decay"] else 0  # old weights that count are read
    return {"bytes": keys * kv * (4 * d + 4 + old) + 4 * n * nq * heads * d + keys // 2,
            "flops": 4 * d * heads * (keys * nq - n * nq * (nq - 1) // 2)}


# ------------------------------------------------------------------- inputs

def _spread(n, lo, hi, seed):
    """n lengths from lo to hi, even over their logarithm: the same sum for every seed, in another order."""
    x = np.round(np.exp(np.linspace(math.log(lo + 1), math.log(hi + 1), n)) - 1).astype(np.int64) if n > 1 else np.array([hi])
    return np.random.RandomState(seed % (1 << 31)).permutation(np.clip(x, lo, hi))


def _pools(g, blocks, kv, d):
    """K and V pools as a model leaves them: normal, a few channels several times larger than the rest."""
    out = []
    for spread in (0.4, 0.2):
        pool = torch.empty((blocks, kv, BS, d), dtype=torch.bfloat16, device="cuda")
        pool.normal_(generator=g)
        pool *= torch.exp(spread * torch.randn((kv, 1, d), generator=g, device="cuda")).to(torch.bfloat16)
        out.append(pool)
    return out


def _tables(need, perm, at=0):
    """Block tables of need[j] pages each, taken from perm in order; unused entries are 0."""
    tables = np.zeros((len(need), max(1, int(max(need)))), np.int32)
    for j, m in enumerate(need):
        tables[j, :m] = perm[at:at + m]
        at += m
    return tables


def prepare(case, seed):
    op, kv, d = case["op"], case["kv"], case["d"]
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rs = np.random.RandomState((seed * 7 + 3) % (1 << 31))
    if op == "evict":
        n, keep = case["n"], case["keep"]
        lens = _spread(n, case["lo"], case["hi"], seed)
        need, need2 = (lens + BS - 1) // BS, (np.minimum(lens, keep) + BS - 1) // BS
        blocks = int(need.sum() + need2.sum()) + 2
        perm = rs.permutation(blocks)
        tables, new = _tables(need, perm), _tables(need2, perm, int(need.sum()))
        k, v = _pools(g, blocks, kv, d)
        # sums of softmax weights: heavy-tailed; some tokens were never looked at
        w = torch.exp(2 * torch.randn((blocks, kv, BS), generator=g, device="cuda") - 4)
        w *= (torch.rand(w.shape, generator=g, device="cuda") > 0.02)
        return dict(case=case, k=k, v=v, w=w, lens=torch.from_numpy(lens.astype(np.int32)).cuda(),
                    max_len=int(lens.max()), tables=torch.from_numpy(tables).cuda(), new=torch.from_numpy(new).cuda(),
                    kept=torch.empty((n, kv, keep), dtype=torch.int32, device="cuda"))
    heads = kv * case["group"]
    if op == "shared":
        rows, prefix = _ints(case["rows"]), _ints(case["prefix"])
        n = int(rows.sum())
        of = np.repeat(np.arange(len(rows)), rows)
        ctx = prefix[of] + _spread(n, case["lo"], case["hi"], seed) - 1
        shared = prefix // BS  # whole pages that a group's rows share; a part-filled one each row has for itself
        need = ctx // BS + 1 - shared[of]
        blocks = int(need.sum() + shared.sum()) + 3
        perm = rs.permutation(blocks)
        mine = _tables(need, perm, int(shared.sum()))
        common = _tables(shared, perm)
        tables = np.zeros((n, int((ctx // BS).max()) + 1), np.int32)
        for j in range(n):
            tables[j, :shared[of[j]]] = common[of[j], :shared[of[j]]]
            tables[j, shared[of[j]]:ctx[j] // BS + 1] = mine[j, :need[j]]
        k, v = _pools(g, blocks, kv, d)
        first = np.cumsum(rows) - rows
        for i, p in enumerate(prefix):
            if p % BS:  # the same tokens in each row's own copy
                own_pages = torch.from_numpy(tables[first[i]:first[i] + rows[i], p // BS].astype(np.int64)).cuda()
                for pool in (k, v):
                    pool[own_pages, :, :p % BS] = pool[own_pages[:1], :, :p % BS]
        q = torch.randn((n, heads, d), generator=g, device="cuda").to(torch.bfloat16)
        return dict(case=case, k=k, v=v, q=q, rows=rows, prefix=prefix, tables=torch.from_numpy(tables).cuda(),
                    ctx=torch.from_numpy(ctx.astype(np.int32)).cuda(), max_ctx=int(ctx.max()), out=torch.empty_like(q),
                    workspace=torch.empty(192 << 20, dtype=torch.uint8, device="cuda"))
    n, nq = case["n"], case["nq"]
    ctx = _spread(n, case["lo"], case["hi"], seed)
    need = ctx // BS + 1
    blocks = int(need.sum()) + 3
    tables = _tables(need, rs.permutation(blocks))
    wtables = _tables(need, rs.permutation(blocks))
    k, v = _pools(g, blocks, kv, d)
    q = torch.randn((n * nq, heads, d), generator=g, device="cuda").to(torch.bfloat16)
    return dict(case=case, k=k, v=v, q=q, tables=torch.from_numpy(tables).cuda(),
                wtables=torch.from_numpy(wtables).cuda(), w=torch.rand((blocks, kv, BS), generator=g, device="cuda"),
                ctx=torch.from_numpy(ctx.astype(np.int32)).cuda(), max_ctx=int(ctx.max()), out=torch.empty_like(q),
                workspace=torch.empty(192 << 20, dtype=torch.uint8, device="cuda"))


# ------------------------------------------------------------------- plain forms

def _keys(pool, tables):
    """Rows of the pages that tables [a, pages] name, in 32 bits: [a, kv, pages x 16, d]."""
    x = pool[tables.long()].float()  # a pages kv 16 d
    a, m, kv, _, d = x.shape
    return x.transpose(1, 2).reshape(a, kv, m * BS, d)


def _plain_shared(st):
    q, k, v = st["q"], st["k"], st["v"]
    n, heads, d = q.shape
    kv = k.shape[1]
    rows = torch.from_numpy(st["rows"]).cuda().long()
    prefix = torch.from_numpy(st["prefix"]).cuda().long()
    first = rows.cumsum(0) - rows
    of = torch.repeat_interleave(torch.arange(len(rows), device="cuda"), rows)
    within = torch.arange(n, device="cuda") - first[of]
    most = int(st["rows"].max())
    scale = 1 / math.sqrt(d)
    qf = q.float().reshape(n, kv, heads // kv, d)
    # the prefixes, padded to the longest and to the most rows: one product for all rows of a group
    pages = max(1, -(-int(st["prefix"].max()) // BS))
    at = torch.arange(pages * BS, device="cuda")
    kp, vp = (_keys(pool, st["tables"][first][:, :pages]) for pool in (k, v))
    padded = torch.zeros((len(rows), most, kv, heads // kv, d), device="cuda")
    padded[of, within] = qf
    x = padded.permute(0, 2, 1, 3, 4).reshape(len(rows), kv, -1, d)
    sp = torch.matmul(x, kp.transpose(-1, -2)) * scale
    sp = sp.masked_fill((at >= prefix[:, None])[:, None, None], -math.inf)
    # each row's own keys: pages from the prefix's last, part-filled one on
    own_pages = int((st["ctx"].long() // BS - prefix[of] // BS).max()) + 1
    page = prefix[of, None] // BS + torch.arange(own_pages, device="cuda")
    table = st["tables"].gather(1, page.clamp_max(st["tables"].shape[1] - 1))
    ks, vs = (_keys(pool, table) for pool in (k, v))
    pos = (page[:, :, None] * BS + torch.arange(BS, device="cuda")).reshape(n, -1)
    ss = torch.matmul(qf, ks.transpose(-1, -2)) * scale
    hidden = (pos < prefix[of, None]) | (pos > st["ctx"][:, None])
    ss = ss.masked_fill(hidden[:, None, None], -math.inf)
    # one softmax over both
    mp = sp.amax(-1).reshape(len(rows), kv, most, -1).transpose(1, 2)[of, within]  # n kv g
    m = torch.maximum(mp, ss.amax(-1))
    mx = torch.zeros((len(rows), most, kv, heads // kv), device="cuda")
    mx[of, within] = m
    ep = torch.exp(sp - mx.transpose(1, 2).reshape(len(rows), kv, -1, 1))
    es = torch.exp(ss - m[..., None])
    op = torch.matmul(ep, vp).reshape(len(rows), kv, most, -1, d).transpose(1, 2)[of, within]
    lp = ep.sum(-1).reshape(len(rows), kv, most, -1).transpose(1, 2)[of, within]
    o = (op + torch.matmul(es, vs)) / (lp + es.sum(-1))[..., None]
    return o.reshape(n, heads, d).to(torch.bfloat16)


def _plain_weigh(st):
    q, case = st["q"], st["case"]
    n, nq, kv = case["n"], case["nq"], case["kv"]
    heads, d = q.shape[1:]
    k, v = _keys(st["k"], st["tables"]), _keys(st["v"], st["tables"])
    keys = k.shape[2]
    x = q.float().reshape(n, nq, kv, heads // kv, d).permute(0, 2, 1, 3, 4).reshape(n, kv, -1, d)
    s = torch.matmul(x, k.transpose(-1, -2)) / math.sqrt(d)
    at = torch.arange(keys, device="cuda")
    pos = st["ctx"][:, None] - (nq - 1) + torch.arange(nq, device="cuda")  # n nq
    hidden = (at > pos[..., None]).repeat_interleave(heads // kv, 1)       # n nq x g keys
    s = s.masked_fill(hidden[:, None], -math.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    out = torch.matmul(p, v).reshape(n, kv, nq, heads // kv, d).transpose(1, 2).reshape(n * nq, heads, d)
    blk, tok = st["wtables"].long()[:, at // BS], at % BS  # n keys
    old = st["w"][blk, :, tok]                             # n keys kv
    fresh = (at > st["ctx"][:, None] - nq)[..., None]
    new = torch.where(fresh, torch.zeros_like(old), old * case["decay"]) + p.sum(2).transpose(1, 2)
    seen = at <= st["ctx"][:, None]
    j, t = torch.nonzero(seen, as_tuple=True)
    st["w"][blk[j, t], :, tok[t]] = new[j, t]
    return out.to(torch.bfloat16), st["w"]


def _plain_evict(st):
    case = st["case"]
    n, kv, keep = case["n"], case["kv"], case["keep"]
    lens = st["lens"].long()
    at = torch.arange(st["tables"].shape[1] * BS, device="cuda")
    w = st["w"][st["tables"].long()].transpose(1, 2).reshape(n, kv, -1)
    held = (at < case["first"]) | (at >= lens[:, None] - case["recent"])
    w = w.masked_fill(held[:, None], math.inf).masked_fill((at >= lens[:, None])[:, None], -math.inf)
    order = torch.sort(w, dim=-1, descending=True, stable=True).indices[..., :keep]
    gone = order >= lens[:, None, None]
    kept = torch.sort(order.masked_fill(gone, 1 << 30), dim=-1).values
    pad = keep - kept.shape[-1]
    if pad:
        kept = torch.nn.functional.pad(kept, (0, pad), value=1 << 30)
    kept = torch.where(kept < (1 << 30), kept, -1)
    j, h, i = torch.nonzero(kept >= 0, as_tuple=True)
    src = kept[j, h, i]
    b, t = st["tables"].long()[j, src // BS], src % BS
    nb, nt = st["new"].long()[j, i // BS], i % BS
    st["k"][nb, h, nt] = st["k"][b, h, t]
    st["v"][nb, h, nt] = st["v"][b, h, t]
    st["w"][nb, h, nt] = st["w"][b, h, t]
    return kept.int(), st["k"], st["v"], st["w"]


# ------------------------------------------------------------------- one pass

def _own(st):
    from chunked_prefill_hybrid_gb300 import paged
    case = st["case"]
    pool = paged.PagedPool(st["k"], st["v"])
    if case["op"] == "shared":
        paged.decode_shared(pool, st["q"], st["tables"], st["ctx"], st["max_ctx"], st["rows"], st["prefix"], st["out"],
                            workspace=st["workspace"])
        return st["out"]
    if case["op"] == "weigh":
        paged.decode_weigh(pool, st["q"], st["tables"], st["ctx"], st["max_ctx"], st["w"], st["wtables"], case["decay"],
                           st["out"], workspace=st["workspace"])
        return st["out"], st["w"]
    paged.evict_select(st["w"], st["tables"], st["lens"], st["max_len"], case["keep"], case["first"], case["recent"],
                       st["kept"])
    paged.evict_move(pool, st["tables"], st["new"], st["kept"], weights=st["w"], weight_tables=st["tables"],
                     new_weight_tables=st["new"])
    return st["kept"], st["k"], st["v"], st["w"]


def run(state):
    if own:
        return _own(state)
    return {"shared": _plain_shared, "weigh": _plain_weigh, "evict": _plain_evict}[state["case"]["op"]](state)


# ------------------------------------------------------------------- 64 bits

def _cached(st, name, j, keys):
    """K or V of sequence j's first `keys` tokens through its own table, in 64 bits: [kv, keys, d]."""
    page = st[name][st["tables"][j, :(keys + BS - 1) // BS].long()].double()
    return page.transpose(0, 1).flatten(1, 2)[:, :keys]


def exact(case, seed):
    st = prepare(case, seed)
    op, kv, d = case["op"], case["kv"], case["d"]
    if op == "evict":
        kept = torch.full((case["n"], kv, case["keep"]), -1, dtype=torch.int64, device="cuda")
        lens = st["lens"].tolist()
        moved = {name: st[name].double() for name in ("k", "v", "w")}
        for j, m in enumerate(lens):
            keep = min(m, case["keep"])
            w = st["w"][st["tables"][j, :(m + BS - 1) // BS].long()].double().transpose(0, 1).flatten(1, 2)[:, :m]
            lo = min(case["first"], keep)
            hi = max(lo, m - min(case["recent"], keep - lo))
            # the heaviest between lo and hi: all that pass the smallest that stays, and the first of those that equal it
            most = keep - lo - (m - hi)
            stays = torch.ones((kv, m), dtype=torch.bool, device="cuda")
            if most < hi - lo:
                mid = w[:, lo:hi]
                if most:
                    edge = torch.topk(mid, most, dim=-1).values[:, -1:]
                    above, equal = mid > edge, mid == edge
                    room = most - above.sum(-1, keepdim=True)
                    stays[:, lo:hi] = above | (equal & (equal.cumsum(-1) <= room))
                else:
                    stays[:, lo:hi] = False
            kept[j, :, :keep] = torch.nonzero(stays)[:, 1].view(kv, keep)
            to, slot = st["new"][j].long(), torch.arange(keep, device="cuda")
            for h in range(kv):
                at = kept[j, h, :keep]
                page = st["tables"][j].long()[at // BS]
                for name in moved:
                    moved[name][to[slot // BS], h, slot % BS] = st[name][page, h, at % BS].double()
        return kept.int(), moved["k"], moved["v"], moved["w"]
    heads = kv * case["group"]
    q = st["q"].double()
    out = torch.empty(q.shape, dtype=torch.float64, device="cuda")
    if op == "shared":
        for j, c in enumerate(st["ctx"].tolist()):
            k, v = _cached(st, "k", j, c + 1), _cached(st, "v", j, c + 1)
            p = torch.softmax(torch.einsum("hgd,hkd->hgk", q[j].view(kv, -1, d), k) / math.sqrt(d), -1)
            out[j] = torch.einsum("hgk,hkd->hgd", p, v).reshape(heads, d)
        return out
    nq, w = case["nq"], st["w"].double()
    for j, c in enumerate(st["ctx"].tolist()):
        k, v = _cached(st, "k", j, c + 1), _cached(st, "v", j, c + 1)
        total = torch.zeros((kv, c + 1), dtype=torch.float64, device="cuda")
        for i in range(nq):
            see = c + 1 - (nq - 1) + i
            p = torch.softmax(torch.einsum("hgd,hkd->hgk", q[j * nq + i].view(kv, -1, d), k[:, :see]) / math.sqrt(d), -1)
            out[j * nq + i] = torch.einsum("hgk,hkd->hgd", p, v[:, :see]).reshape(heads, d)
            total[:, :see] += p.sum(1)
        pos = torch.arange(c + 1, device="cuda")
        page = st["wtables"][j].long()[pos // BS]
        old = w[page, :, pos % BS] * case["decay"]
        old[max(0, c + 1 - nq):] = 0
        w[page, :, pos % BS] = old + total.transpose(0, 1)
    return out, w
