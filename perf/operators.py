"""Cases of the serving operators around the sparse-attention indexer: attention
over a paged key/value cache (chunks of new tokens and single tokens, with an
optional sliding window and first tokens that stay visible), attention over the
tokens the indexer selected, and copying, forking, compacting and freeing the
pages of the caches.

``run`` computes an operator in plain torch when ``own`` is false and through
the package's entry points when it is true; ``exact`` restates the attention
operators in 64 bits. Lengths follow from the case alone (``_lengths``), values
from the seed.
"""
import math
import random

import torch

own = False

PAGE = 64            # tokens of a cache page
INDEX_PAGE = 8448    # bytes of an index-cache page (64 fp8 keys and their scales)
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # the smallest call: one request, one new token, a short context
        dict(name="chunk_one_token", op="attend", reqs=1, q_lo=1, q_hi=1, l_lo=1000, l_hi=1000, empty=0,
             heads=32, kv_heads=8, dim=128, dtype="bf16", window=0, sinks=0, shape=1),
        # the decode batch: 32 requests of one new token each
        dict(name="chunk_decode_batch", op="attend", reqs=32, q_lo=1, q_hi=1, l_lo=2048, l_hi=32768, empty=0,
             heads=64, kv_heads=8, dim=128, dtype="bf16", window=0, sinks=0, shape=2),
        # a mixed step: single tokens beside ragged chunks, padding requests, an odd group of heads
        dict(name="chunk_mixed", op="attend", reqs=24, q_lo=1, q_hi=300, l_lo=300, l_hi=9000, empty=2,
             heads=40, kv_heads=8, dim=128, dtype="fp16", window=0, sinks=0, shape=3),
        # a chunk of a long prompt: few new tokens over a long cache
        dict(name="chunk_long_context", op="attend", reqs=1, q_lo=512, q_hi=512, l_lo=65536, l_hi=65536, empty=0,
             heads=64, kv_heads=8, dim=128, dtype="bf16", window=0, sinks=0, shape=4),
        # the prefill batch: 4 requests of 8192 new tokens, causal over themselves
        dict(name="chunk_prefill", op="attend", reqs=4, q_lo=8192, q_hi=8192, l_lo=8192, l_hi=8192, empty=0,
             heads=16, kv_heads=2, dim=128, dtype="bf16", window=0, sinks=0, shape=5),
        # speculative decode on a windowed layer: two rows a request, long caches of which a window is read
        dict(name="window_decode", op="attend", reqs=64, q_lo=2, q_hi=2, l_lo=4096, l_hi=65536, empty=0,
             heads=32, kv_heads=4, dim=128, dtype="bf16", window=4096, sinks=4, shape=6),
        # a windowed layer's prefill, ragged, with smaller heads
        dict(name="window_prefill", op="attend", reqs=3, q_lo=2000, q_hi=8192, l_lo=8192, l_hi=8192, empty=0,
             heads=24, kv_heads=8, dim=64, dtype="fp16", window=1024, sinks=64, shape=7),
        # sparse decode of a small batch
        dict(name="selected_small", op="selected", reqs=4, q_lo=1, q_hi=1, l_lo=1000, l_hi=4096, topk=512,
             heads=32, kv_heads=8, dim=64, dtype="fp16", shape=8),
        # the decode batch after the indexer's top-2048
        dict(name="selected_decode", op="selected", reqs=32, q_lo=1, q_hi=1, l_lo=2048, l_hi=32768, topk=2048,
             heads=64, kv_heads=8, dim=128, dtype="bf16", shape=9),
        # ragged chunks after the indexer's prefill top-2048 (early rows hold fewer keys than that)
        dict(name="selected_chunk", op="selected", reqs=4, q_lo=100, q_hi=200, l_lo=1000, l_hi=32768, topk=2048,
             heads=32, kv_heads=4, dim=128, dtype="bf16", shape=10),
        # every decode request forked once: shared full pages, copied last pages
        dict(name="pages_fork", op="fork", reqs=32, forks=32, l_lo=2048, l_hi=32768, kv_heads=2, dim=128,
             spare=64, shape=11),
        # half of the requests leave, the pool is compacted
        dict(name="pages_compact", op="compact", reqs=48, leave=24, l_lo=2048, l_hi=32768, kv_heads=2, dim=128,
             spare=64, shape=12),
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm where the range is wide."""
    if hi <= 10 * lo:
        return rng.randint(lo, hi)
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _lengths(case):
    """(new tokens, keys) of every request; `empty` requests of no keys (padding) come last."""
    rng = random.Random(case["shape"])
    ql, kl = [], []
    for _ in range(case["reqs"]):
        q = _spread(rng, case.get("q_lo", 1), case.get("q_hi", 1))
        ql.append(q)
        kl.append(max(q, rng.randint(case["l_lo"], case["l_hi"])))
    for _ in range(case.get("empty", 0)):
        ql.append(1)
        kl.append(0)
    return ql, kl


def draw(rng):
    most, flops = max(_plain_cost(c) for c in listed()), max(work(c)["flops"] for c in listed())
    while True:
        op = rng.choice(["attend", "attend", "attend", "selected", "selected", "fork", "compact"])
        shape = rng.randrange(1 << 30)
        dim, dtype = rng.choice([64, 128]), rng.choice(["bf16", "fp16"])
        kv = rng.choice([1, 2, 3, 4, 8])
        heads = kv * rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
        if op in ("fork", "compact"):
            lo = _spread(rng, 1, 4096)
            c = dict(op=op, reqs=_spread(rng, 1, 64), l_lo=lo, l_hi=max(lo, _spread(rng, 64, 32768)),
                     kv_heads=rng.choice([1, 2]), dim=dim, spare=_spread(rng, 33, 400), shape=shape)
            c["forks" if op == "fork" else "leave"] = rng.randint(1, min(32, c["reqs"]))
        else:
            q = _spread(rng, 1, 8192) if rng.random() < 0.6 else 1
            lo = _spread(rng, 1, 32768)
            c = dict(op=op, reqs=_spread(rng, 1, 64), q_lo=max(1, q // rng.choice([1, 2, 20])), q_hi=q,
                     l_lo=lo, l_hi=max(lo, _spread(rng, 64, 65536)), heads=heads, kv_heads=kv, dim=dim,
                     dtype=dtype, shape=shape)
            if op == "attend":
                c.update(empty=rng.choice([0, 0, 1, 3]), window=0, sinks=0)
                if rng.random() < 0.4:
                    c.update(window=_spread(rng, 1, 8192), sinks=rng.choice([0, 1, 4, 64, 130]))
            else:
                c.update(topk=_spread(rng, 16, 2048))
        if _plain_cost(c) <= most:
            w = work(c)
            if w["bytes"] <= 4e9 and w["flops"] <= flops:
                return c


def _plain_cost(case):
    """What the plain form touches, in values: the padded score matrix and the gathered keys."""
    if case["op"] in ("fork", "compact"):
        return 0
    ql, kl = _lengths(case)
    if case["op"] == "selected":
        return sum(ql) * case["topk"] * (case["heads"] + 2 * case["kv_heads"] * case["dim"])
    keys = -(-max(kl) // PAGE) * PAGE
    return len(ql) * keys * (case["heads"] * max(ql) + 2 * case["kv_heads"] * case["dim"])


def _seen(case, q, n):
    """(query, key) pairs of a request that are visible, and keys that some query sees."""
    w, s = case.get("window", 0), case.get("sinks", 0)
    if w <= 0:
        first = n - q + 1
        return q * (first + n) // 2, n
    pairs = 0
    for p in range(n - q, n):
        pairs += min(p + 1, w) + max(0, min(s, p + 1 - w))
    start = max(0, n - q - w + 1)
    return pairs, n - start + min(s, start)


def work(case):
    if case["op"] in ("fork", "compact"):
        return _page_work(case)
    ql, kl = _lengths(case)
    h, hk, d = case["heads"], case["kv_heads"], case["dim"]
    pairs = keys = 0
    for q, n in zip(ql, kl):
        if not n:
            continue
        if case["op"] == "selected":
            k = case["topk"]
            counts = [min(k, p + 1) for p in range(n - q, n)]
            pairs += sum(counts)
            # tokens that at least one of the rows selects, in the mean
            missed = 1.0
            for p, c in zip(range(n - q, n), counts):
                missed *= 1.0 - c / (p + 1)
            keys += min(sum(counts), n) * (1.0 - missed) if q > 1 else counts[0]
        else:
            a, b = _seen(case, q, n)
            pairs += a
            keys += b
    rows = sum(ql)
    lists = 4 * (rows * case["topk"] if case["op"] == "selected" else sum(-(-n // PAGE) for n in kl))
    return {"bytes": float(rows * h * d * 2 * 2 + rows * h * 4 + keys * hk * d * 2 * 2 + lists), "flops": float(4 * pairs * h * d)}


def _page_bytes(case):
    return INDEX_PAGE + 2 * PAGE * case["kv_heads"] * case["dim"] * 2


def _page_work(case):
    _, kl = _lengths(case)
    pages = [-(-n // PAGE) for n in kl]
    pool = sum(pages) + case["spare"]
    if case["op"] == "fork":
        parents = _parents(case)
        copied = sum(1 for p in parents if kl[p] % PAGE)
        shared = sum(pages[p] for p in parents)
        return {"bytes": float(2 * copied * _page_bytes(case) + 4 * (pool + 2 * shared)), "flops": 0.0}
    perm = _pool_order(case, pool)
    leave, at, live = _leaving(case), 0, []
    for b, n in enumerate(pages):
        if b not in leave:
            live += perm[at:at + n]
        at += n
    moved = sum(1 for p in live if p >= len(live))
    return {"bytes": float(2 * moved * _page_bytes(case) + 4 * (2 * pool + 2 * len(live))), "flops": 0.0}


def _parents(case):
    return [random.Random(case["shape"] + 1 + i).randrange(case["reqs"]) for i in range(case["forks"])]


def _leaving(case):
    return set(random.Random(case["shape"] + 1).sample(range(case["reqs"]), case["leave"]))


def _pool_order(case, pool):
    order = list(range(pool))
    random.Random(case["shape"] + 2).shuffle(order)
    return order


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _table(order, pages, rows, width):
    """Block table whose row b lists the next pages[b] entries of `order`; unused entries are -1."""
    table, at = [[-1] * width for _ in range(rows)], 0
    for b, n in enumerate(pages):
        table[b][:n] = order[at:at + n]
        at += n
    return _ints(table)


def prepare(case, seed):
    g = _gen(seed)
    dev = "cuda"
    if case["op"] in ("fork", "compact"):
        _, kl = _lengths(case)
        pages = [-(-n // PAGE) for n in kl]
        pool = sum(pages) + case["spare"]
        rows = case["reqs"] + case.get("forks", 0)
        # a pool that has served for a while: the requests' pages lie scattered over it
        order = _pool_order(case, pool)
        kv_shape = (pool, PAGE, case["kv_heads"], case["dim"])
        refs = torch.zeros(pool, dtype=torch.int32, device=dev)
        refs[torch.tensor(order[:sum(pages)], device=dev)] = 1
        s = dict(case=case, rows=rows,
                 index=torch.randint(0, 256, (pool, INDEX_PAGE), generator=g, device=dev, dtype=torch.uint8),
                 k=torch.randn(kv_shape, generator=g, device=dev, dtype=torch.bfloat16),
                 v=torch.randn(kv_shape, generator=g, device=dev, dtype=torch.bfloat16),
                 table=_table(order, pages, rows, max(pages)), lens=_ints(kl + [0] * (rows - len(kl))), refs=refs)
        if case["op"] == "fork":
            s.update(parents=_ints(_parents(case)), children=_ints(list(range(case["reqs"], rows))))
        else:
            s.update(leave=_ints(sorted(_leaving(case))))
        return s
    ql, kl = _lengths(case)
    pages = [-(-n // PAGE) for n in kl]
    pool = max(1, sum(pages))
    order = torch.randperm(pool, generator=g, device=dev).tolist()
    dt = TYPES[case["dtype"]]
    rows, kv_shape = sum(ql), (pool, PAGE, case["kv_heads"], case["dim"])
    start = [0]
    for q in ql:
        start.append(start[-1] + q)
    s = dict(case=case, max_q=max(ql),
             q=torch.randn((rows, case["heads"], case["dim"]), generator=g, device=dev, dtype=torch.float32).to(dt),
             k=torch.randn(kv_shape, generator=g, device=dev, dtype=torch.bfloat16).to(dt),
             v=torch.randn(kv_shape, generator=g, device=dev, dtype=torch.bfloat16).to(dt),
             table=_table(order, pages, len(ql), max(1, max(pages))), lens=_ints(kl), start=_ints(start))
    if case["op"] == "selected":
        # what the indexer hands over: k distinct keys in no order, or the whole causal row and -1
        k, lists = case["topk"], []
        seen = torch.tensor([n - q + 1 + i for q, n in zip(ql, kl) for i in range(q)], device=dev)
        for r0 in range(0, rows, 256):
            c = seen[r0:r0 + 256, None]
            pos = torch.arange(max(max(kl), k), device=dev)[None]
            score = torch.rand((c.shape[0], pos.shape[1]), generator=g, device=dev).masked_fill_(pos >= c, -1.0)
            best = score.topk(k, dim=1).indices
            row = torch.where(c <= k, torch.where(pos[:, :k] < c, pos[:, :k], -1), best)
            lists.append(row.to(torch.int32))
        s["indices"] = torch.cat(lists).contiguous()
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------


def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    return _PLAIN[op](state)


def _own_attend(s):
    import sparse_attention_indexer_block_gb300 as saib
    c = s["case"]
    out, lse = saib.indexer_attend_paged(s["q"], s["k"], s["v"], s["table"], s["lens"], s["start"], s["max_q"],
                                         window=c["window"], sinks=c["sinks"])
    return {"out": out, "lse": lse}


def _own_selected(s):
    import sparse_attention_indexer_block_gb300 as saib
    out, lse = saib.indexer_attend_selected(s["q"], s["k"], s["v"], s["table"], s["indices"], s["start"])
    return {"out": out, "lse": lse}


def _own_fork(s):
    import sparse_attention_indexer_block_gb300 as saib
    table, lens, refs = s["table"].clone(), s["lens"].clone(), s["refs"].clone()
    saib.indexer_fork_pages([s["index"], s["k"], s["v"]], table, lens, refs, s["parents"], s["children"])
    return {"table": table, "lens": lens, "refs": refs, "index": s["index"], "k": s["k"], "v": s["v"]}


def _own_compact(s):
    import sparse_attention_indexer_block_gb300 as saib
    table, lens, refs = s["table"].clone(), s["lens"].clone(), s["refs"].clone()
    saib.indexer_free_pages(table, lens, refs, s["leave"])
    remap, live = saib.indexer_compact_pages([s["index"], s["k"], s["v"]], table, lens, refs)
    return {"table": table, "lens": lens, "refs": refs, "remap": remap, "live": live, "index": s["index"],
            "k": s["k"], "v": s["v"]}


def _token_rows(s):
    """(request, place within it) of every token row."""
    t = torch.arange(s["q"].shape[0], device="cuda")
    b = torch.searchsorted(s["start"], t.to(torch.int32), right=True) - 1
    return b, t - s["start"][b]


def _plain_attend(s):
    c = s["case"]
    h, hk, d = c["heads"], c["kv_heads"], c["dim"]
    g, reqs, rows = h // hk, s["lens"].shape[0], s["q"].shape[0]
    start, lens = s["start"].long(), s["lens"].long()
    new = start[1:] - start[:-1]
    j = torch.arange(s["max_q"], device="cuda")
    q = s["q"][(start[:-1, None] + j).clamp(max=rows - 1)].float()
    q = q.view(reqs, -1, hk, g, d).permute(0, 2, 3, 1, 4).reshape(reqs, hk, -1, d)
    table = s["table"].clamp(min=0).long()
    keys = table.shape[1] * PAGE
    k = s["k"][table].float().reshape(reqs, keys, hk, d).permute(0, 2, 3, 1)
    v = s["v"][table].float().reshape(reqs, keys, hk, d).permute(0, 2, 1, 3)
    key = torch.arange(keys, device="cuda")
    v = v.masked_fill((key >= lens[:, None])[:, None, :, None], 0.0)
    score = torch.matmul(q, k).mul_(1.0 / math.sqrt(d)).view(reqs, hk, g, -1, keys)
    at = (lens - new)[:, None, None] + j[:, None]
    hidden = key > at
    if c["window"] > 0:
        hidden = hidden | ((key <= at - c["window"]) & (key >= c["sinks"]))
    score.masked_fill_(hidden[:, None, None], -math.inf)
    m = score.amax(-1, keepdim=True)
    score.sub_(m.clamp(min=-3e38)).exp_()
    l = score.sum(-1, keepdim=True)
    o = torch.matmul(score.view(reqs, hk, -1, keys), v).view(reqs, hk, g, -1, d)
    o = o / torch.where(l == 0, 1.0, l)
    lse = (m + l.log()).squeeze(-1)
    b, at = _token_rows(s)
    out = o.permute(0, 3, 1, 2, 4)[b, at].reshape(rows, h, d)
    return {"out": out.to(s["q"].dtype), "lse": lse.permute(0, 3, 1, 2)[b, at].reshape(rows, h)}


def _plain_selected(s):
    c = s["case"]
    h, hk, d = c["heads"], c["kv_heads"], c["dim"]
    g, rows = h // hk, s["q"].shape[0]
    b, _ = _token_rows(s)
    idx = s["indices"].long()
    none = idx < 0
    at = idx.clamp(min=0)
    slot = s["table"][b[:, None], at // PAGE].clamp(min=0).long() * PAGE + at % PAGE
    k = s["k"].view(-1, hk, d)[slot].float().permute(0, 2, 3, 1)
    v = s["v"].view(-1, hk, d)[slot].float().permute(0, 2, 1, 3)
    score = torch.matmul(s["q"].float().view(rows, hk, g, d), k).mul_(1.0 / math.sqrt(d))
    score.masked_fill_(none[:, None, None], -math.inf)
    m = score.amax(-1, keepdim=True)
    p = score.sub_(m.clamp(min=-3e38)).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(l == 0, 1.0, l)
    lse = (m + l.log()).squeeze(-1)
    return {"out": o.reshape(rows, h, d).to(s["q"].dtype), "lse": lse.reshape(rows, h)}


def _plain_fork(s):
    table, lens, refs = s["table"].clone(), s["lens"].clone(), s["refs"].clone()
    parents, children = s["parents"].long(), s["children"].long()
    length = lens[parents]
    full = length // PAGE
    part = (length % PAGE) != 0
    column = torch.arange(table.shape[1], device="cuda")
    shared = column < full[:, None]
    # fresh pages in the children's order, each the lowest free one left
    free = torch.argsort((refs != 0).to(torch.int32), stable=True)
    nth = torch.cumsum(part, 0) - 1
    fresh = free[nth.clamp(min=0)]
    last = full.clamp(max=table.shape[1] - 1)[:, None].long()
    source = table[parents].gather(1, last)[:, 0].long()
    rows = torch.where(shared, table[parents], table[children])
    rows = rows.scatter(1, last, torch.where(part, fresh.to(torch.int32), rows.gather(1, last)[:, 0])[:, None])
    held = torch.where(shared, table[parents], 0).long().flatten()
    refs.index_add_(0, held, shared.flatten().to(torch.int32))
    refs.index_add_(0, fresh, part.to(torch.int32))
    table[children] = rows
    lens[children] = length
    # a child that shares all its pages copies its own first page onto itself
    own_page = table[children, 0].clamp(min=0).long()
    source, target = torch.where(part, source, own_page), torch.where(part, fresh, own_page)
    s["index"][target] = s["index"][source]
    s["k"][target] = s["k"][source]
    s["v"][target] = s["v"][source]
    return {"table": table, "lens": lens, "refs": refs, "index": s["index"], "k": s["k"], "v": s["v"]}


def _plain_compact(s):
    table, lens, refs = s["table"].clone(), s["lens"].clone(), s["refs"].clone()
    pool = refs.shape[0]
    column = torch.arange(table.shape[1], device="cuda")
    leave = s["leave"].long()
    held = column < (-(-lens[leave] // PAGE))[:, None]
    refs.index_add_(0, torch.where(held, table[leave], 0).long().flatten(), -held.flatten().to(torch.int32))
    lens[leave] = 0
    live = refs > 0
    n = live.sum()
    page = torch.arange(pool, device="cuda")
    # the i-th live page past the first n goes to the i-th free page among them
    mover, hole = live & (page >= n), ~live & (page < n)
    movers = torch.argsort((~mover).to(torch.int32), stable=True)
    holes = torch.argsort((~hole).to(torch.int32), stable=True)
    moved = page < mover.sum()
    place = torch.where(live, page, -1)
    place = place.scatter(0, movers, torch.where(moved, holes, place[movers])).to(torch.int32)
    held = column < (-(-lens // PAGE))[:, None]
    table = torch.where(held, place[table.clamp(min=0).long()], table)
    source = torch.arange(pool + 1, device="cuda")
    source = source.scatter_(0, torch.where(moved, holes, pool), torch.where(moved, movers, pool))[:pool]
    refs = torch.where(page < n, torch.where(hole, refs[source], refs), 0)
    # pages that stay are copied onto themselves: the number of moves is known on the device alone
    take = torch.where(hole, source, page)
    s["index"].copy_(s["index"][take])
    s["k"].copy_(s["k"][take])
    s["v"].copy_(s["v"][take])
    return {"table": table, "lens": lens, "refs": refs, "remap": place, "live": n.to(torch.int32).reshape(1),
            "index": s["index"], "k": s["k"], "v": s["v"]}


_OWN = {"attend": _own_attend, "selected": _own_selected, "fork": _own_fork, "compact": _own_compact}
_PLAIN = {"attend": _plain_attend, "selected": _plain_selected, "fork": _plain_fork, "compact": _plain_compact}


# ---------------------------------------------------------------------------
# in 64 bits
# ---------------------------------------------------------------------------


def exact(case, seed):
    if case["op"] in ("fork", "compact"):
        return None  # pages and whole numbers are moved, not computed
    if work(case)["flops"] > 5e12:
        return None
    s = prepare(case, seed)
    ql, kl = _lengths(case)
    h, hk, d = case["heads"], case["kv_heads"], case["dim"]
    g, rows = h // hk, s["q"].shape[0]
    out = torch.zeros((rows, h, d), dtype=torch.float64, device="cuda")
    lse = torch.full((rows, h), -math.inf, dtype=torch.float64, device="cuda")
    row = 0
    for b, (q, n) in enumerate(zip(ql, kl)):
        if n:
            slots = (s["table"][b, :-(-n // PAGE)].long()[:, None] * PAGE + torch.arange(PAGE, device="cuda")).flatten()[:n]
            for i0 in range(0, q, 2048):
                i1 = min(q, i0 + 2048)
                tokens = torch.arange(i0, i1, device="cuda") + (n - q)
                if case["op"] == "selected":
                    see = torch.zeros((i1 - i0, n + 1), dtype=torch.bool, device="cuda")
                    see.scatter_(1, torch.where(s["indices"][row + i0:row + i1] < 0, n, s["indices"][row + i0:row + i1]).long(), True)
                    see = see[:, :n]
                else:
                    pos = torch.arange(n, device="cuda")
                    see = pos[None] <= tokens[:, None]
                    if case["window"] > 0:
                        see &= (tokens[:, None] - pos[None] < case["window"]) | (pos[None] < case["sinks"])
                # keys outside [first, past) are visible to none of these rows
                used = torch.nonzero(see.any(0)).flatten()
                if not used.numel():
                    continue
                see = see[:, used]
                for kh in range(hk):
                    key = s["k"][slots[used] // PAGE, slots[used] % PAGE, kh].double()
                    val = s["v"][slots[used] // PAGE, slots[used] % PAGE, kh].double()
                    query = s["q"][row + i0:row + i1, kh * g:(kh + 1) * g].double()
                    for hh in range(g):
                        x = torch.where(see, query[:, hh] @ key.T / math.sqrt(d), -math.inf)
                        z = torch.logsumexp(x, 1)
                        p = torch.exp(x - torch.where(z == -math.inf, 0.0, z)[:, None])
                        out[row + i0:row + i1, kh * g + hh] = p @ val
                        lse[row + i0:row + i1, kh * g + hh] = z
        row += q
    return {"out": out, "lse": lse}
