"""A serving loop over one paged pool: prompts in chunks, forks, sparse and
windowed decode steps, steps of drafted trees, freed requests and a compacted pool.

Three caches share the block table: the indexer's keys (fp8 with scales), and
the keys and values of attention. Every step writes the new tokens' entries and
then runs, as the layers of a model would,

  every step      indexer_append_kv, indexer_insert_keys
  prompt chunks   indexer_attend_paged (causal)
  decode          indexer_decode_topk, indexer_attend_selected (sparse layer),
                  indexer_attend_paged with a window and sinks (windowed layer)
  drafted trees   indexer_plan_tree, indexer_attend_tree (dense layer),
                  indexer_decode_topk and indexer_attend_selected (sparse layer),
                  indexer_commit_tree

Random projections stand in for the model. Run on a GB300:

    python examples/paged_serving.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sparse_attention_indexer_block_gb300 as saib  # noqa: E402

PAGE = 64
HEADS, KV_HEADS, DIM = 16, 2, 128      # attention
INDEX_HEADS, INDEX_DIM = 64, 128       # indexer
WINDOW, SINKS, TOPK = 256, 4, 512


class Pool:
    """The caches' pages, the requests' block table and the pages' reference counts."""

    def __init__(self, pages, rows, width, device, seed=0):
        self.dev = device
        self.index = torch.zeros((pages, PAGE * (INDEX_DIM + 4)), dtype=torch.uint8, device=device)
        self.k = torch.zeros((pages, PAGE, KV_HEADS, DIM), dtype=torch.bfloat16, device=device)
        self.v = torch.zeros_like(self.k)
        self.table = torch.zeros((rows, width), dtype=torch.int32, device=device)
        self.lens = torch.zeros(rows, dtype=torch.int32, device=device)
        self.refs = torch.zeros(pages, dtype=torch.int32, device=device)
        self.err = torch.zeros(1, dtype=torch.int32, device=device)
        g = torch.Generator(device=device).manual_seed(seed)

        def weight(n, m):
            return (torch.randn((n, m), generator=g, device=device) / n ** 0.5).to(torch.bfloat16)

        self.wq, self.wk = weight(DIM, HEADS * DIM), weight(DIM, KV_HEADS * DIM)
        self.wv, self.wi = weight(DIM, KV_HEADS * DIM), weight(DIM, INDEX_DIM)
        self.wiq = weight(DIM, INDEX_HEADS * INDEX_DIM)
        self.head_w = torch.randn(INDEX_HEADS, generator=g, device=device).abs() / 8

    @property
    def pools(self):
        return [self.index, self.k, self.v]

    def extend(self, row, n):
        """Room for n more tokens of a row: the lowest free pages, at the row's end. Returns the
        new tokens' slots."""
        old = int(self.lens[row])
        held, need = -(-old // PAGE), -(-(old + n) // PAGE)
        if need > held:
            fresh = torch.nonzero(self.refs == 0).flatten()[:need - held]
            self.table[row, held:need] = fresh.to(torch.int32)
            self.refs[fresh] += 1
        self.lens[row] = old + n
        pos = torch.arange(old, old + n, device=self.dev)
        return self.table[row, pos // PAGE].long() * PAGE + pos % PAGE

    def write(self, x, slots):
        """The entries of tokens x [n, DIM] at their slots."""
        saib.indexer_append_kv((x @ self.wk).view(-1, KV_HEADS, DIM), (x @ self.wv).view(-1, KV_HEADS, DIM), self.k,
                               self.v, slots, dev_error=self.err)
        saib.indexer_insert_keys(x @ self.wi, slots, self.index, dev_error=self.err)

    def prefill(self, rows, chunks):
        """Chunks of tokens [n, DIM] of several rows, as one batch. Returns their attention outputs."""
        for row, x in zip(rows, chunks):
            self.write(x, self.extend(row, x.shape[0]))
        at = torch.tensor(rows, device=self.dev)
        start = [0]
        for x in chunks:
            start.append(start[-1] + x.shape[0])
        q = (torch.cat(chunks) @ self.wq).view(-1, HEADS, DIM)
        out, _ = saib.indexer_attend_paged(q, self.k, self.v, self.table[at], self.lens[at],
                                           torch.tensor(start, dtype=torch.int32, device=self.dev),
                                           max(x.shape[0] for x in chunks), dev_error=self.err)
        return out.split([x.shape[0] for x in chunks])

    def decode(self, rows, x):
        """One token [len(rows), DIM] for every row. Returns (sparse, windowed) attention outputs."""
        self.write(x, torch.cat([self.extend(row, 1) for row in rows]))
        at = torch.tensor(rows, device=self.dev)
        table, lens, n = self.table[at], self.lens[at], len(rows)
        start = torch.arange(n + 1, dtype=torch.int32, device=self.dev)
        q = (x @ self.wq).view(n, HEADS, DIM)
        picked = saib.indexer_decode_topk((x @ self.wiq).view(n, INDEX_HEADS, INDEX_DIM),
                                          self.head_w.expand(n, -1).contiguous(), self.index, table, lens,
                                          1, TOPK, dev_error=self.err)
        sparse, _ = saib.indexer_attend_selected(q, self.k, self.v, table, picked, start, dev_error=self.err)
        windowed, _ = saib.indexer_attend_paged(q, self.k, self.v, table, lens, start, 1, window=WINDOW,
                                                sinks=SINKS, dev_error=self.err)
        return sparse, windowed

    def draft(self, rows, trees, x):
        """Trees of drafted tokens x [nodes, DIM], one for every row (lists of parents, -1 for the nodes that
        follow the row's last token). Returns (dense, sparse) attention outputs and the batch that keep()
        takes."""
        self.write(x, torch.cat([self.extend(row, len(t)) for row, t in zip(rows, trees)]))
        i32 = dict(dtype=torch.int32, device=self.dev)
        at = torch.tensor(rows, device=self.dev)
        table, lens, n = self.table[at], self.lens[at], x.shape[0]
        sizes = [len(t) for t in trees]
        start = torch.tensor([sum(sizes[:i]) for i in range(len(sizes) + 1)], **i32)
        masks, _, paths = saib.indexer_plan_tree(torch.tensor([p for t in trees for p in t], **i32), lens, start,
                                                 max(sizes), max_path=max(sizes), dev_error=self.err)
        q = (x @ self.wq).view(n, HEADS, DIM)
        dense, _ = saib.indexer_attend_tree(q, self.k, self.v, table, lens, start, masks, max(sizes),
                                            dev_error=self.err)
        # the sparse layer: the selection among the keys before the tree, and the node's path
        of = torch.repeat_interleave(torch.arange(len(rows), device=self.dev), torch.tensor(sizes, device=self.dev))
        before = (lens - torch.tensor(sizes, **i32))[of].contiguous()
        picked = saib.indexer_decode_topk((x @ self.wiq).view(n, INDEX_HEADS, INDEX_DIM),
                                          self.head_w.expand(n, -1).contiguous(), self.index, table[of].contiguous(),
                                          before, 1, TOPK, dev_error=self.err)
        sparse, _ = saib.indexer_attend_selected(q, self.k, self.v, table, torch.cat([picked, paths], 1), start,
                                                 dev_error=self.err)
        return dense, sparse, (at, table, lens, start)

    def keep(self, batch, accepted):
        """Keeps every row's accepted nodes (ascending lists) of the trees of draft(), drops the others."""
        at, table, lens, start = batch
        most = max(len(a) for a in accepted)
        rows = torch.tensor([a + [-1] * (most - len(a)) for a in accepted], dtype=torch.int32, device=self.dev)
        saib.indexer_commit_tree(self.pools, table, lens, start, rows, ref_counts=self.refs, dev_error=self.err)
        self.lens[at] = lens

    def fork(self, parents, children):
        i32 = dict(dtype=torch.int32, device=self.dev)
        saib.indexer_fork_pages(self.pools, self.table, self.lens, self.refs, torch.tensor(parents, **i32),
                                torch.tensor(children, **i32), dev_error=self.err)

    def free(self, rows):
        saib.indexer_free_pages(self.table, self.lens, self.refs,
                                torch.tensor(rows, dtype=torch.int32, device=self.dev), dev_error=self.err)

    def compact(self):
        """Pages in use, now the pool's first ones."""
        _, live = saib.indexer_compact_pages(self.pools, self.table, self.lens, self.refs, dev_error=self.err)
        return int(live)


def run(device="cuda", seed=0):
    """Two prompts, three forks of them, decode steps, two requests gone, the pool compacted, more
    decode steps. Returns what each part produced."""
    g = torch.Generator(device=device).manual_seed(seed + 1)

    def tokens(n):
        return torch.randn((n, DIM), generator=g, device=device).to(torch.bfloat16)

    pool = Pool(pages=160, rows=8, width=40, device=device, seed=seed)
    a, b = tokens(1500), tokens(333)
    prompt = [pool.prefill([0, 1], [a[:1000], b]), pool.prefill([0], [a[1000:]])]
    pool.fork([0, 1, 1], [2, 3, 4])
    steps = [tokens(1).expand(5, -1).contiguous()] + [tokens(5) for _ in range(3)]
    decoded = [pool.decode([0, 1, 2, 3, 4], x) for x in steps]
    used = int((pool.refs > 0).sum())
    pool.free([0, 3])
    live = pool.compact()
    more = [pool.decode([1, 2, 4], tokens(3)) for _ in range(2)]
    return dict(pool=pool, tokens=(a, b), prompt=prompt, steps=steps, decoded=decoded, used=used, live=live,
                more=more)


def run_drafts(device="cuda", seed=0):
    """Two prompts, then steps of drafted trees of which a path is kept. Returns what each step produced."""
    g = torch.Generator(device=device).manual_seed(seed + 2)

    def tokens(n):
        return torch.randn((n, DIM), generator=g, device=device).to(torch.bfloat16)

    pool = Pool(pages=64, rows=2, width=30, device=device, seed=seed)
    history = [tokens(700), tokens(90)]
    pool.prefill([0, 1], history)
    trees = [[-1, 0, 0, 1, 1, 2, 3, 3], [-1, -1, 0, 1, 1, 3, 5, 5, 6, 6, 6, 7]]
    accepted = [[0, 1, 4], [1, 3, 5, 7, 11]]
    steps = []
    for _ in range(4):
        x = tokens(sum(len(t) for t in trees))
        dense, sparse, batch = pool.draft([0, 1], trees, x)
        pool.keep(batch, accepted)
        at = [0, len(trees[0])]
        steps.append((list(history), x, dense, sparse))
        history = [torch.cat([h, x[[a + i for i in path]]]) for h, a, path in zip(history, at, accepted)]
    return dict(pool=pool, history=history, trees=trees, accepted=accepted, steps=steps)


if __name__ == "__main__":
    r = run()
    torch.cuda.synchronize()
    assert int(r["pool"].err) == 0, f"device error word {int(r['pool'].err)}"
    print(f"prompts of 1500 and 333 tokens, 3 forks, {len(r['decoded'])} steps of 5 requests: {r['used']} pages; "
          f"2 requests freed and the pool compacted: {r['live']} pages")
    r = run_drafts()
    torch.cuda.synchronize()
    assert int(r["pool"].err) == 0, f"device error word {int(r['pool'].err)}"
    print(f"{len(r['steps'])} steps of trees of {[len(t) for t in r['trees']]} nodes, {[len(a) for a in r['accepted']]} "
          f"kept: {[h.shape[0] for h in r['history']]} tokens")
