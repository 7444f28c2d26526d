"""Cases of the operators of a speculative decode step on the paged caches: new
tokens' keys and values into the cache with their rotation, index keys into an
MXFP4 cache, the masks of a tree of drafted tokens, the tree's attention, and the
accepted path kept while the other drafts are dropped.

``run`` computes an operator in plain torch when ``own`` is false and through
the package's entry points when it is true; ``exact`` restates the computed
numbers in 64 bits. Lengths and trees follow from the case alone (``_lengths``,
``_parents``), values from the seed.
"""
import math
import random

import torch

own = False

PAGE = 64            # tokens of a cache page
INDEX_PAGE = 8448    # bytes of an fp8 index-cache page: 64 keys of 128 codes, then 64 scales
MX_TOKEN = 68        # bytes of an MXFP4 index-cache entry: 64 of codes, 4 scales
INDEX_DIM = 128
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # the smallest append: one request's next token
        dict(name="append_one", op="append", tokens=1, padding=0, heads=32, kv_heads=8, dim=128, rotary=128,
             interleaved=False, dtype="bf16", far=4096, shape=1),
        # a step of drafted tokens: 32 requests of 17 nodes in a batch padded for a captured graph,
        # neighbouring values rotated as pairs, far positions
        dict(name="append_drafts", op="append", tokens=544, padding=32, heads=64, kv_heads=8, dim=128, rotary=64,
             interleaved=True, dtype="bf16", far=131072, shape=2),
        # a long prompt's chunk of an odd number of tokens, smaller heads
        dict(name="append_prompt", op="append", tokens=16011, padding=0, heads=64, kv_heads=8, dim=64, rotary=64,
             interleaved=False, dtype="fp16", far=65536, shape=3),
        # index keys of a decode batch into an MXFP4 cache, and of a prompt
        dict(name="insert_decode", op="insert", tokens=32, padding=3, shape=4),
        dict(name="insert_prompt", op="insert", tokens=131071, padding=0, shape=5),
        # a decode batch's trees, and many wide ones on a windowed layer
        dict(name="plan_decode", op="plan", reqs=32, q_lo=8, q_hi=33, l_lo=2048, l_hi=32768, path=16, window=0,
             sinks=0, shape=6),
        dict(name="plan_wide", op="plan", reqs=256, q_lo=64, q_hi=160, l_lo=200, l_hi=32768, path=24, window=8,
             sinks=4, shape=7),
        # one request's small tree over a short context: latency
        dict(name="tree_one", op="tree", reqs=1, q_lo=8, q_hi=8, l_lo=1000, l_hi=1000, heads=32, kv_heads=8, dim=128,
             dtype="bf16", window=0, sinks=0, shape=8),
        # the decode batch: 32 requests of 16 to 32 drafted tokens over ragged contexts
        dict(name="tree_decode", op="tree", reqs=32, q_lo=16, q_hi=32, l_lo=2048, l_hi=32768, heads=64, kv_heads=8,
             dim=128, dtype="bf16", window=0, sinks=0, shape=9),
        # a windowed layer's wide trees, smaller heads, an odd group
        dict(name="tree_window", op="tree", reqs=24, q_lo=40, q_hi=130, l_lo=500, l_hi=16384, heads=24, kv_heads=8,
             dim=64, dtype="fp16", window=2048, sinks=4, shape=10),
        # accepted paths of a small batch, one layer with an MXFP4 index cache
        dict(name="commit_small", op="commit", reqs=4, q_lo=8, q_hi=8, l_lo=1000, l_hi=4096, kv_heads=8, dim=128,
             layers=1, mx=True, shape=11),
        # a large batch, the caches of eight layers at once
        dict(name="commit_layers", op="commit", reqs=64, q_lo=16, q_hi=64, l_lo=200, l_hi=2048, kv_heads=8, dim=128,
             layers=8, mx=False, shape=12),
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm where the range is wide."""
    if hi <= 10 * lo:
        return rng.randint(lo, hi)
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _lengths(case):
    """(drafted tokens, keys with them) of every request."""
    rng = random.Random(case["shape"])
    ql, kl = [], []
    for _ in range(case["reqs"]):
        q = _spread(rng, case["q_lo"], case["q_hi"])
        ql.append(q)
        kl.append(max(q, rng.randint(case["l_lo"], case["l_hi"])))
    return ql, kl


def _parents(case):
    """Every request's tree: the parent of each node, -1 for those that follow the last committed token."""
    rng = random.Random(case["shape"] + 1)
    ql, _ = _lengths(case)
    return [[-1 if i == 0 or rng.random() < 0.1 else rng.randrange(max(0, i - 24), i) for i in range(q)] for q in ql]


def _chains(parents):
    """Every node's chain of ancestors, itself first."""
    chains = []
    for i, p in enumerate(parents):
        chains.append([i] + (chains[p] if p >= 0 else []))
    return chains


def _accepted(case):
    """Every request's accepted nodes: a path down its tree, of up to 16 nodes."""
    rng = random.Random(case["shape"] + 2)
    paths = []
    for parents in _parents(case):
        chain = _chains(parents)[rng.randrange(len(parents))][::-1]
        paths.append(chain[:rng.randint(0, min(16, len(chain)))])
    return paths


def draw(rng):
    most, flops, size = max(_plain_cost(c) for c in listed()), max(work(c)["flops"] for c in listed()), 1.2e9
    while True:
        op = rng.choice(["append", "append", "insert", "plan", "tree", "tree", "tree", "commit"])
        c = dict(op=op, shape=rng.randrange(1 << 30))
        dim, dtype = rng.choice([64, 128]), rng.choice(["bf16", "fp16"])
        kv = rng.choice([1, 2, 3, 4, 8])
        heads = kv * rng.choice([1, 2, 3, 4, 5, 8, 12, 16])
        if op == "append":
            n = _spread(rng, 1, 16011)
            c.update(tokens=n, padding=rng.choice([0, 0, 1, min(n - 1, 7)]) if n > 1 else 0, heads=heads, kv_heads=kv,
                     dim=dim, rotary=rng.choice([dim, dim, dim // 2, 32, 16]), interleaved=rng.random() < 0.4,
                     dtype=dtype, far=_spread(rng, 1000, 131072))
        elif op == "insert":
            n = _spread(rng, 1, 131071)
            c.update(tokens=n, padding=rng.choice([0, 0, 1, min(n - 1, 5)]) if n > 1 else 0)
        else:
            q = _spread(rng, 1, 160)
            lo = _spread(rng, 1, 16384)
            c.update(reqs=_spread(rng, 1, 64), q_lo=max(1, q // rng.choice([1, 2, 10])), q_hi=q, l_lo=lo,
                     l_hi=max(lo, _spread(rng, 64, 32768)))
            if op in ("plan", "tree"):
                c.update(window=0, sinks=0)
                if rng.random() < 0.4:
                    c.update(window=_spread(rng, 1, 4096), sinks=rng.choice([0, 1, 4, 64, 130]))
            if op == "plan":
                c.update(path=rng.choice([24, 40, 64]))
            elif op == "tree":
                c.update(heads=heads, kv_heads=kv, dim=dim, dtype=dtype)
            else:
                c.update(l_hi=max(lo, min(c["l_hi"], 4096)), kv_heads=kv, dim=dim, layers=rng.choice([1, 2, 3, 8]),
                         mx=rng.random() < 0.5)
                if _pool_bytes(c) > 3e9:
                    continue
        if op == "plan" and max(len(x) for p in _parents(c) for x in _chains(p)) > c["path"]:
            continue
        w = work(c)
        if _plain_cost(c) <= most and w["bytes"] <= size and w["flops"] <= flops:
            return c


def _plain_cost(case):
    """What the plain form of the attention touches, in values: the padded score matrix and the gathered keys."""
    if case["op"] != "tree":
        return 0
    ql, kl = _lengths(case)
    keys = -(-max(kl) // PAGE) * PAGE
    return len(ql) * keys * (case["heads"] * max(ql) + 2 * case["kv_heads"] * case["dim"])


def _pool_bytes(case):
    _, kl = _lengths(case)
    return sum(-(-n // PAGE) for n in kl) * PAGE * case["layers"] * _token_bytes(case)


def _token_bytes(case):
    """Bytes of a token in one layer's caches."""
    return 2 * case["kv_heads"] * case["dim"] * 2 + (MX_TOKEN if case["mx"] else INDEX_DIM + 4)


def work(case):
    return _WORK[case["op"]](case)


def _work_append(case):
    n, pad, d = case["tokens"], case["padding"], case["dim"]
    values = ((n + pad) * case["heads"] + 2 * n * case["kv_heads"]) * d
    places = len(set(_places(case)))
    flops = 3 * case["rotary"] * ((n + pad) * case["heads"] + n * case["kv_heads"])
    return {"bytes": float(2 * 2 * values + 4 * case["rotary"] * places + 12 * (n + pad)), "flops": float(flops)}


def _work_insert(case):
    n = case["tokens"]
    return {"bytes": float((2 * 2 * INDEX_DIM + MX_TOKEN + 8) * n), "flops": float(4 * INDEX_DIM * n)}


def _work_plan(case):
    ql, _ = _lengths(case)
    rows = sum(ql)
    return {"bytes": float(4 * rows * (2 + -(-max(ql) // 32) + case["path"]) + 8 * len(ql)), "flops": 0.0}


def _work_tree(case):
    ql, kl = _lengths(case)
    h, hk, d, w, sinks = case["heads"], case["kv_heads"], case["dim"], case["window"], case["sinks"]
    pairs = keys = 0
    for q, n, parents in zip(ql, kl, _parents(case)):
        ahead, chains = n - q, _chains(parents)
        first = ahead
        for c in chains:
            p = ahead + len(c) - 1
            start = max(0, min(ahead, p - w + 1)) if w else 0
            pairs += ahead - start + min(sinks if w else 0, start) + _new_seen(case, ahead, c)
            first = min(first, start)
        keys += ahead - first + min(sinks if w else 0, first) + q
    rows, words = sum(ql), -(-max(ql) // 32)
    lists = 4 * (rows * (words + (1 if w else 0)) + sum(-(-n // PAGE) for n in kl))
    return {"bytes": float(rows * h * (d * 2 * 2 + 4) + keys * hk * d * 2 * 2 + lists), "flops": float(4 * pairs * h * d)}


def _work_commit(case):
    ql, kl = _lengths(case)
    moved = sum(sum(1 for i, a in enumerate(p) if a != i) for p in _accepted(case))
    return {"bytes": float(2 * moved * _token_bytes(case) * case["layers"] + 4 * (16 + 4) * len(ql)), "flops": 0.0}


def _new_seen(case, ahead, chain):
    """Nodes of a chain that its first one sees: with a window, those within it or among the first keys."""
    if not case["window"]:
        return len(chain)
    depth = len(chain) - 1
    return sum(1 for i in range(len(chain)) if i < case["window"] or ahead + depth - i < case["sinks"])


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def _places(case):
    """Positions of the appended tokens: runs of neighbours from random beginnings, some of them drafts of
    one place."""
    rng = random.Random(case["shape"])
    out = []
    while len(out) < case["tokens"]:
        n = min(case["tokens"] - len(out), _spread(rng, 1, 4096))
        at = rng.randrange(max(1, case["far"] - n))
        step = rng.choice([1, 1, 2])
        out += [at + i // step for i in range(n)]
    return out


def _order(g, pages):
    return torch.randperm(pages, generator=g, device="cuda").tolist()


def _table(order, pages, width):
    """Block table whose row b lists the next pages[b] entries of `order`; unused entries are -1."""
    table, at = [[-1] * width for _ in pages], 0
    for b, n in enumerate(pages):
        table[b][:n] = order[at:at + n]
        at += n
    return _ints(table)


def _starts(ql):
    start = [0]
    for q in ql:
        start.append(start[-1] + q)
    return start


def _words(bits, n):
    """A whole number's lowest 32 n bits as int32 words."""
    words = [bits >> 32 * i & 0xffffffff for i in range(n)]
    return [w - (1 << 32) if w >> 31 else w for w in words]


def prepare(case, seed):
    return _PREPARE[case["op"]](case, _gen(seed))


def _prepare_append(case, g):
    n, pad, h, hk, d = case["tokens"], case["padding"], case["heads"], case["kv_heads"], case["dim"]
    dt = TYPES[case["dtype"]]
    pages = -(-n // PAGE) + 8
    # q, k and v are parts of one projection's output
    qkv = torch.randn((n + pad, (h + 2 * hk) * d), generator=g, device="cuda").to(dt)
    slots = torch.randperm(pages * PAGE, generator=g, device="cuda")[:n]
    slots = torch.cat([slots, torch.full((pad,), -1, dtype=slots.dtype, device="cuda")])
    half = case["rotary"] // 2
    freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
    angle = torch.arange(case["far"], dtype=torch.float64, device="cuda")[:, None] * freq
    kv_shape = (pages, PAGE, hk, d)
    return dict(case=case, q=qkv[:, :h * d].view(-1, h, d), k=qkv[:, h * d:(h + hk) * d].view(-1, hk, d),
                v=qkv[:, (h + hk) * d:].view(-1, hk, d), slots=slots, positions=_ints(_places(case) + [0] * pad),
                rotary=torch.cat([angle.cos(), angle.sin()], 1).float(),
                k_cache=torch.randn(kv_shape, generator=g, device="cuda").to(dt),
                v_cache=torch.randn(kv_shape, generator=g, device="cuda").to(dt))


def _prepare_insert(case, g):
    n, pad = case["tokens"], case["padding"]
    pages = -(-n // PAGE) + 4
    # keys with a few large channels
    k = torch.randn((n + pad, INDEX_DIM), generator=g, device="cuda")
    k = k * torch.exp(torch.randn(INDEX_DIM, generator=g, device="cuda"))
    slots = torch.randperm(pages * PAGE, generator=g, device="cuda")[:n]
    slots = torch.cat([slots, torch.full((pad,), -1, dtype=slots.dtype, device="cuda")])
    cache = torch.randint(0, 255, (pages, PAGE * MX_TOKEN), generator=g, device="cuda", dtype=torch.uint8)
    return dict(case=case, k=k.to(torch.bfloat16), slots=slots, cache=cache)


def _prepare_plan(case, g):
    # (trees differ from seed to seed in their nodes' parents, within the case's lengths)
    ql, kl = _lengths(case)
    start = _starts(ql)
    flat = [p for parents in _parents(case) for p in parents]
    first = _ints([start[b] for b, q in enumerate(ql) for _ in range(q)])
    parents = _ints(flat)
    # a node in four moves to a parent's place among the first nodes: no deeper than before
    move = torch.rand(parents.shape, generator=g, device="cuda") < 0.25
    grand = torch.where(parents < 0, -1, parents[(first + parents.clamp(min=0)).long()])
    return dict(case=case, parents=torch.where(move, grand, parents).to(torch.int32), lens=_ints(kl),
                start=_ints(start), max_q=max(ql))


def _prepare_tree(case, g):
    ql, kl = _lengths(case)
    pages = [-(-n // PAGE) for n in kl]
    pool = sum(pages)
    dt = TYPES[case["dtype"]]
    rows, kv_shape = sum(ql), (pool, PAGE, case["kv_heads"], case["dim"])
    words = -(-max(ql) // 32)
    masks, positions = [], []
    for q, n, parents in zip(ql, kl, _parents(case)):
        for chain in _chains(parents):
            depth, bits = len(chain) - 1, 0
            for i, node in enumerate(chain):
                if not case["window"] or i < case["window"] or n - q + depth - i < case["sinks"]:
                    bits |= 1 << node
            masks.append(_words(bits, words))
            positions.append(n - q + depth)
    return dict(case=case, max_q=max(ql),
                q=torch.randn((rows, case["heads"], case["dim"]), generator=g, device="cuda").to(dt),
                k=torch.randn(kv_shape, generator=g, device="cuda", dtype=torch.bfloat16).to(dt),
                v=torch.randn(kv_shape, generator=g, device="cuda", dtype=torch.bfloat16).to(dt),
                table=_table(_order(g, pool), pages, max(pages)), lens=_ints(kl), start=_ints(_starts(ql)),
                masks=_ints(masks), positions=_ints(positions))


def _prepare_commit(case, g):
    ql, kl = _lengths(case)
    pages = [-(-n // PAGE) for n in kl]
    pool, layers = sum(pages) + 8, case["layers"]
    index = torch.randint(0, 256, (layers, pool, PAGE * MX_TOKEN if case["mx"] else INDEX_PAGE), generator=g,
                          device="cuda", dtype=torch.uint8)
    shape = (layers, pool, PAGE, case["kv_heads"], case["dim"])
    k = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
    v = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
    paths = _accepted(case)
    most = max(1, max(len(p) for p in paths))
    order = _order(g, pool)
    refs = torch.zeros(pool, dtype=torch.int32, device="cuda")
    refs[_ints(order[:sum(pages)], torch.int64)] = 1
    return dict(case=case, index=index, k=k, v=v, pools=[t[i] for i in range(layers) for t in (index, k, v)],
                table=_table(order, pages, max(pages)), lens=_ints(kl), start=_ints(_starts(ql)), refs=refs,
                accepted=_ints([p + [-1] * (most - len(p)) for p in paths]))


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------


def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    return _PLAIN[op](state)


def _own_append(s):
    import sparse_attention_indexer_block_gb300 as saib
    q = saib.indexer_append_kv(s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"], q=s["q"],
                               positions=s["positions"], rotary=s["rotary"], interleaved=s["case"]["interleaved"])
    return {"q": q, "k": s["k_cache"], "v": s["v_cache"]}


def _own_insert(s):
    import sparse_attention_indexer_block_gb300 as saib
    values = torch.empty_like(s["k"])
    saib.indexer_insert_keys_mxfp4(s["k"], s["slots"], s["cache"], values=values)
    return {"values": values, "cache": s["cache"]}


def _own_plan(s):
    import sparse_attention_indexer_block_gb300 as saib
    c = s["case"]
    masks, positions, paths = saib.indexer_plan_tree(s["parents"], s["lens"], s["start"], s["max_q"],
                                                     window=c["window"], sinks=c["sinks"], max_path=c["path"])
    return {"masks": masks, "positions": positions, "paths": paths}


def _own_tree(s):
    import sparse_attention_indexer_block_gb300 as saib
    c = s["case"]
    out, lse = saib.indexer_attend_tree(s["q"], s["k"], s["v"], s["table"], s["lens"], s["start"], s["masks"],
                                        s["max_q"], positions=s["positions"], window=c["window"], sinks=c["sinks"])
    return {"out": out, "lse": lse}


def _own_commit(s):
    import sparse_attention_indexer_block_gb300 as saib
    lens, refs = s["lens"].clone(), s["refs"].clone()
    saib.indexer_commit_tree(s["pools"], s["table"], lens, s["start"], s["accepted"], ref_counts=refs)
    return {"lens": lens, "refs": refs, "index": s["index"], "k": s["k"], "v": s["v"]}


def _rotate(x, cos, sin, interleaved):
    """x [tokens, heads, dim] in 32 bits with its first 2 * cos.shape[1] values rotated."""
    half = cos.shape[1]
    cos, sin = cos[:, None], sin[:, None]
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., 2 * half:]], -1)


def _plain_append(s):
    c = s["case"]
    n, half = c["tokens"], c["rotary"] // 2
    row = s["rotary"][s["positions"].long()]
    cos, sin = row[:, :half], row[:, half:]
    q = _rotate(s["q"].float(), cos, sin, c["interleaved"]).to(s["q"].dtype)
    k = _rotate(s["k"][:n].float(), cos[:n], sin[:n], c["interleaved"]).to(s["k"].dtype)
    # (the padding is the batch's last rows)
    s["k_cache"].view(-1, c["kv_heads"], c["dim"])[s["slots"][:n]] = k
    s["v_cache"].view(-1, c["kv_heads"], c["dim"])[s["slots"][:n]] = s["v"][:n]
    return {"q": q, "k": s["k_cache"], "v": s["v_cache"]}


def _plain_insert(s):
    n = s["case"]["tokens"]
    x = s["k"].float().view(-1, 4, 32)
    x = torch.where(x.isnan(), 0.0, x)
    # the largest magnitude's exponent less 2 (e2m1 holds up to 6 = 1.5 * 2^2), as the scale's byte
    field = (x.abs().amax(-1).view(torch.int32) >> 23) & 255
    scale = (field - 2).clamp(min=0)
    y = torch.ldexp(x, (127 - scale)[..., None])
    a = y.abs()
    # steps of 0.5 up to 2, of 1 up to 4, of 2 from there; ties to the even step
    step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0))
    a = (torch.round(a / step) * step).clamp(max=6.0)
    # 0, 0.5, 1, 1.5, 2, 3, 4, 6 are codes 0 to 7
    code = torch.where(a < 2.0, a * 2, torch.where(a < 4.0, a + 2, a / 2 + 4)).to(torch.uint8)
    sign = torch.signbit(y) & (x.abs().amax(-1, keepdim=True) > 0)
    code = (code + 8 * sign.to(torch.uint8)).view(-1, 64, 2)
    entry = torch.cat([code[..., 0] | code[..., 1] << 4, scale.to(torch.uint8)], 1)
    s["cache"].view(-1, MX_TOKEN)[s["slots"][:n]] = entry[:n]
    value = torch.ldexp(torch.where(sign, -a, a), (scale - 127)[..., None]).view(-1, INDEX_DIM).to(torch.bfloat16)
    # rows of padding are zeros
    return {"values": torch.where(s["slots"][:, None] >= 0, value, 0.0), "cache": s["cache"]}


def _plain_plan(s):
    c = s["case"]
    reqs, q = s["lens"].shape[0], s["max_q"]
    start = s["start"].long()
    new = start[1:] - start[:-1]
    node = torch.arange(q, device="cuda")
    parent = s["parents"][(start[:-1, None] + node).clamp(max=s["parents"].shape[0] - 1)]
    parent = torch.where(node < new[:, None], parent, -1)
    edge = (parent[..., None] == node).float()
    # ancestors = 1 + edge + edge^2 + ... = (1 - edge)^-1, whose entries are 0 and 1
    one = torch.eye(q, device="cuda").expand(reqs, q, q)
    chain = torch.linalg.solve_triangular(one - edge, one, upper=False, unitriangular=True) > 0.5
    depth = chain.sum(-1) - 1
    at = (s["lens"] - new)[:, None] + depth
    see = chain
    if c["window"] > 0:
        see = chain & ((depth[:, :, None] - depth[:, None] < c["window"]) | (at[:, None] < c["sinks"]))
    words = -(-q // 32)
    bits = torch.nn.functional.pad(see, (0, 32 * words - q)).view(reqs, q, words, 32).long()
    masks = (bits << torch.arange(32, device="cuda")).sum(-1).to(torch.int32)
    slot = (s["lens"] - new)[:, None, None] + node
    paths = torch.where(chain, slot, -1).sort(-1, descending=True).values
    paths = torch.nn.functional.pad(paths, (0, max(0, c["path"] - q)), value=-1)[..., :c["path"]].to(torch.int32)
    t = torch.arange(s["parents"].shape[0], device="cuda")
    b = torch.searchsorted(s["start"], t.to(torch.int32), right=True) - 1
    i = t - start[b]
    return {"masks": masks[b, i], "positions": at[b, i].to(torch.int32), "paths": paths[b, i]}


def _plain_tree(s):
    c = s["case"]
    h, hk, d = c["heads"], c["kv_heads"], c["dim"]
    g, reqs, rows = h // hk, s["lens"].shape[0], s["q"].shape[0]
    start, lens = s["start"].long(), s["lens"].long()
    new = start[1:] - start[:-1]
    j = torch.arange(s["max_q"], device="cuda")
    row = (start[:-1, None] + j).clamp(max=rows - 1)
    q = s["q"][row].float().view(reqs, -1, hk, g, d).permute(0, 2, 3, 1, 4).reshape(reqs, hk, -1, d)
    table = s["table"].clamp(min=0).long()
    keys = table.shape[1] * PAGE
    k = s["k"][table].float().reshape(reqs, keys, hk, d).permute(0, 2, 3, 1)
    v = s["v"][table].float().reshape(reqs, keys, hk, d).permute(0, 2, 1, 3)
    key = torch.arange(keys, device="cuda")
    v = v.masked_fill((key >= lens[:, None])[:, None, :, None], 0.0)
    score = torch.matmul(q, k).mul_(1.0 / math.sqrt(d)).view(reqs, hk, g, -1, keys)
    ahead = (lens - new)[:, None]
    node = (key - ahead).clamp(min=0, max=32 * s["masks"].shape[1] - 1)[:, None].expand(-1, s["max_q"], -1)
    drafted = (s["masks"][row].gather(2, node >> 5) >> (node & 31) & 1) == 1
    committed = (key < ahead)[:, None].expand_as(drafted)
    if c["window"] > 0:
        committed = committed & ((s["positions"][row][..., None] - key < c["window"]) | (key < c["sinks"]))
    drafted = drafted & ((key >= ahead) & (key < lens[:, None]))[:, None]
    score.masked_fill_(~(committed | drafted)[:, None, None], -math.inf)
    m = score.amax(-1, keepdim=True)
    score.sub_(m.clamp(min=-3e38)).exp_()
    l = score.sum(-1, keepdim=True)
    o = torch.matmul(score.view(reqs, hk, -1, keys), v).view(reqs, hk, g, -1, d)
    o = o / torch.where(l == 0, 1.0, l)
    lse = (m + l.log()).squeeze(-1)
    t = torch.arange(rows, device="cuda")
    b = torch.searchsorted(s["start"], t.to(torch.int32), right=True) - 1
    i = t - start[b]
    out = o.permute(0, 3, 1, 2, 4)[b, i].reshape(rows, h, d)
    return {"out": out.to(s["q"].dtype), "lse": lse.permute(0, 3, 1, 2)[b, i].reshape(rows, h)}


def _plain_commit(s):
    c = s["case"]
    new = (s["start"][1:] - s["start"][:-1])[:, None]
    ahead = s["lens"][:, None] - new
    taken = s["accepted"] >= 0
    i = torch.arange(taken.shape[1], device="cuda")
    # entries past the path copy a later draft onto itself
    to = ahead + torch.minimum(i, new - 1)
    at = torch.where(taken, ahead + s["accepted"], to).long()
    to = to.long()
    from_page, to_page = s["table"].gather(1, at // PAGE).long(), s["table"].gather(1, to // PAGE).long()
    a, b = at % PAGE, to % PAGE
    s["k"][:, to_page, b] = s["k"][:, from_page, a]
    s["v"][:, to_page, b] = s["v"][:, from_page, a]
    layers, pool = s["index"].shape[:2]
    if c["mx"]:
        entry = s["index"].view(layers, pool, PAGE, MX_TOKEN)
        entry[:, to_page, b] = entry[:, from_page, a]
    else:
        code = s["index"][..., :PAGE * INDEX_DIM].unflatten(-1, (PAGE, INDEX_DIM))
        scale = s["index"][..., PAGE * INDEX_DIM:].unflatten(-1, (PAGE, 4))
        code[:, to_page, b] = code[:, from_page, a]
        scale[:, to_page, b] = scale[:, from_page, a]
    kept = (ahead + taken.sum(1, keepdim=True)).to(torch.int32)
    column = torch.arange(s["table"].shape[1], device="cuda")
    gone = (column >= (kept + PAGE - 1) // PAGE) & (column < (s["lens"][:, None] + PAGE - 1) // PAGE)
    refs = s["refs"].clone()
    refs.index_add_(0, torch.where(gone, s["table"], 0).long().flatten(), -gone.flatten().to(torch.int32))
    return {"lens": kept[:, 0], "refs": refs, "index": s["index"], "k": s["k"], "v": s["v"]}


# ---------------------------------------------------------------------------
# in 64 bits
# ---------------------------------------------------------------------------


def exact(case, seed):
    if case["op"] in ("plan", "commit"):
        return None  # whole numbers, and values that are moved
    return _EXACT[case["op"]](case, prepare(case, seed))


def _exact_append(case, s):
    n, half = case["tokens"], case["rotary"] // 2
    row = s["rotary"].double()[s["positions"].long()]
    turn = torch.complex(row[:, :half], row[:, half:])[:, None]

    def turned(x):
        x = x.double().clone()
        if case["interleaved"]:
            pair = torch.complex(x[..., 0:2 * half:2], x[..., 1:2 * half:2]) * turn[:x.shape[0]]
            x[..., 0:2 * half:2], x[..., 1:2 * half:2] = pair.real, pair.imag
        else:
            pair = torch.complex(x[..., :half], x[..., half:2 * half]) * turn[:x.shape[0]]
            x[..., :half], x[..., half:2 * half] = pair.real, pair.imag
        return x

    k = s["k_cache"].double()
    k[s["slots"][:n] // PAGE, s["slots"][:n] % PAGE] = turned(s["k"][:n])
    return {"q": turned(s["q"]), "k": k, "v": None}


def _exact_insert(case, s):
    x = s["k"].double().view(-1, 4, 32)
    top = x.abs().amax(-1, keepdim=True)
    _, e = torch.frexp(top)
    unit = torch.pow(torch.full_like(top, 2.0), (e - 3).clamp(min=-127).double())
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device="cuda")
    a = (x / unit).abs()
    # the nearest value of the grid; of two as near, the one with the even code
    far = (a[..., None] - grid).abs()
    code = far.argmin(-1)
    up = (code + 1).clamp(max=7)
    tie = far.gather(-1, up[..., None]) == far.gather(-1, code[..., None])
    code = torch.where(tie[..., 0] & (code % 2 == 1), up, code)
    value = torch.where(x < 0, -grid[code], grid[code]) * unit
    value = torch.where(s["slots"][:, None] >= 0, value.view(-1, INDEX_DIM), 0.0)
    return {"values": value, "cache": None}


def _exact_tree(case, s):
    ql, kl = _lengths(case)
    h, hk, d, w, sinks = case["heads"], case["kv_heads"], case["dim"], case["window"], case["sinks"]
    g, rows = h // hk, s["q"].shape[0]
    out = torch.zeros((rows, h, d), dtype=torch.float64, device="cuda")
    lse = torch.full((rows, h), -math.inf, dtype=torch.float64, device="cuda")
    row = 0
    for b, (q, n, parents) in enumerate(zip(ql, kl, _parents(case))):
        ahead, chains = n - q, _chains(parents)
        position = [ahead + len(c) - 1 for c in chains]
        see = torch.zeros((q, n), dtype=torch.bool)
        see[:, :ahead] = True
        for i, c in enumerate(chains):
            see[i, [ahead + a for a in c]] = True
        if w:
            of_key = torch.tensor(list(range(ahead)) + position)
            see &= (torch.tensor(position)[:, None] - of_key < w) | (of_key < sinks)
        see = see.cuda()
        slots = (s["table"][b, :-(-n // PAGE)].long()[:, None] * PAGE + torch.arange(PAGE, device="cuda")).flatten()[:n]
        for kh in range(hk):
            key = s["k"][slots // PAGE, slots % PAGE, kh].double()
            val = s["v"][slots // PAGE, slots % PAGE, kh].double()
            query = s["q"][row:row + q, kh * g:(kh + 1) * g].double()
            x = torch.einsum("qgd,nd->gqn", query, key) / math.sqrt(d)
            x = torch.where(see, x, -math.inf)
            z = torch.logsumexp(x, -1)
            p = torch.exp(x - torch.where(z == -math.inf, 0.0, z)[..., None])
            out[row:row + q, kh * g:(kh + 1) * g] = torch.einsum("gqn,nd->qgd", p, val)
            lse[row:row + q, kh * g:(kh + 1) * g] = z.T
        row += q
    return {"out": out, "lse": lse}


_WORK = {"append": _work_append, "insert": _work_insert, "plan": _work_plan, "tree": _work_tree, "commit": _work_commit}
_PREPARE = {"append": _prepare_append, "insert": _prepare_insert, "plan": _prepare_plan, "tree": _prepare_tree,
            "commit": _prepare_commit}
_OWN = {"append": _own_append, "insert": _own_insert, "plan": _own_plan, "tree": _own_tree, "commit": _own_commit}
_PLAIN = {"append": _plain_append, "insert": _plain_insert, "plan": _plain_plan, "tree": _plain_tree,
          "commit": _plain_commit}
_EXACT = {"append": _exact_append, "insert": _exact_insert, "tree": _exact_tree}
