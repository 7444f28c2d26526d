"""Page copies, forks, freeing and compaction against a restatement on the CPU.
Everything is whole numbers and moved bytes: equal, not near."""
import numpy as np
import pytest
import torch

import sparse_attention_indexer_block_gb300 as saib

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
PAGE = 64


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from sparse_attention_indexer_block_gb300 import build as libbuild
    libbuild.build()
    saib.load()
    torch.cuda.set_device(DEV)


class Pool:
    def __init__(self, lens, spare, seed, rows=None, width=None, pools=3):
        rng = np.random.default_rng(seed)
        n = [-(-x // PAGE) for x in lens]
        self.pages = sum(n) + spare
        rows = len(lens) if rows is None else rows
        width = max(max(n), 1) + 1 if width is None else width
        order = rng.permutation(self.pages)
        self.table = np.full((rows, width), -1, np.int32)
        self.refs = np.zeros(self.pages, np.int32)
        self.lens = np.zeros(rows, np.int32)
        self.lens[:len(lens)] = lens
        at = 0
        for b, k in enumerate(n):
            self.table[b, :k] = order[at:at + k]
            at += k
            self.refs[self.table[b, :k]] += 1
        g = torch.Generator(device=DEV).manual_seed(seed)
        # an index cache, keys in the middle of wider pages, values
        self.pools = [torch.randint(0, 256, (self.pages, 8448), generator=g, device=DEV, dtype=torch.uint8),
                      torch.randn((self.pages, 2, PAGE, 1, 64), generator=g, device=DEV).to(torch.bfloat16)[:, 1],
                      torch.randn((self.pages, 20), generator=g, device=DEV)][:pools]
        self.err = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.up()

    def up(self):
        self.t, self.r, self.l = (torch.from_numpy(x.copy()).to(DEV) for x in (self.table, self.refs, self.lens))

    def same(self):
        torch.cuda.synchronize()
        assert np.array_equal(self.t.cpu().numpy(), self.table)
        assert np.array_equal(self.r.cpu().numpy(), self.refs)
        assert np.array_equal(self.l.cpu().numpy(), self.lens)

    def error(self):
        torch.cuda.synchronize()
        e = int(self.err.item())
        self.err.zero_()
        return e

    # ---- the definition, in numpy

    def fork(self, parents, children):
        free = [p for p in range(self.pages) if self.refs[p] == 0]
        src, dst, short = [], [], False
        for a, c in zip(parents, children):
            L = int(self.lens[a])
            full = L // PAGE
            self.table[c, :full] = self.table[a, :full]
            np.add.at(self.refs, self.table[a, :full], 1)
            self.lens[c] = L
            if L % PAGE:
                if free:
                    p = free.pop(0)
                    src.append(int(self.table[a, full]))
                    dst.append(p)
                    self.table[c, full] = p
                    self.refs[p] = 1
                else:
                    self.lens[c] = full * PAGE
                    short = True
        want = [p.clone() for p in self.pools]
        for w in want:
            if src:
                w[dst] = w[src]
        pad = [-1] * (len(parents) - len(src))
        return src + pad, dst + pad, want, short

    def free(self, rows):
        for r in rows:
            n = -(-int(self.lens[r]) // PAGE)
            np.add.at(self.refs, self.table[r, :n], -1)
            self.lens[r] = 0

    def compact(self):
        live = [p for p in range(self.pages) if self.refs[p] > 0]
        n = len(live)
        holes = [p for p in range(n) if self.refs[p] == 0]
        remap = np.full(self.pages, -1, np.int32)
        want = [p.clone() for p in self.pools]
        refs = np.zeros_like(self.refs)
        for p in live:
            to = p if p < n else holes.pop(0)
            remap[p] = to
            refs[to] = self.refs[p]
            for w, old in zip(want, self.pools):
                if to != p:
                    w[to] = old[p]
        for r in range(len(self.lens)):
            k = -(-int(self.lens[r]) // PAGE)
            self.table[r, :k] = remap[self.table[r, :k]]
        self.refs = refs
        return remap, n, want


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("n,pages", [(1, 2), (3, 50), (700, 2000)])
def test_copy(n, pages):
    p = Pool([], pages, seed=n, rows=1, width=1)
    order = np.random.default_rng(n).permutation(pages)
    src, dst = order[:n].tolist(), order[n:2 * n].tolist()
    if n == 700:
        src[5], dst[9], src[11], dst[13] = -1, -4, pages, pages
    want = [x.clone() for x in p.pools]
    for a, b in zip(src, dst):
        if 0 <= a < pages and 0 <= b < pages:
            for w, old in zip(want, p.pools):
                w[b] = old[a]
    saib.indexer_copy_pages(p.pools, _i32(src), _i32(dst), dev_error=p.err)
    assert p.error() == (1 if n == 700 else 0)
    for got, w in zip(p.pools, want):
        assert torch.equal(got, w)


def test_copy_of_many_pools_and_of_none():
    g = torch.Generator(device=DEV).manual_seed(0)
    pools = [torch.randint(0, 99, (9, 4 * (1 + i % 5)), generator=g, device=DEV, dtype=torch.int32)
             for i in range(150)]
    want = [x.clone() for x in pools]
    for w in want:
        w[[7, 2]] = w[[1, 3]]
    saib.indexer_copy_pages(pools, _i32([1, 3]), _i32([7, 2]))
    saib.indexer_copy_pages(pools, _i32([]), _i32([]))
    torch.cuda.synchronize()
    for got, w in zip(pools, want):
        assert torch.equal(got, w)


@pytest.mark.parametrize("lens,parents,spare", [
    ([100], [0], 1), ([64, 65, 1], [0, 1, 2], 5), ([200, 64, 0, 7], [0, 0, 0, 3, 2, 1], 9),
    ([5000, 333, 90], [2, 1, 0, 0, 1], 40), ([130, 200, 70], [0, 1, 2, 0], 2),   # two free pages for four
])
def test_fork(lens, parents, spare):
    p = Pool(lens, spare, seed=len(lens) + spare, rows=len(lens) + len(parents) + 1)
    children = list(range(len(lens), len(lens) + len(parents)))
    src, dst, want, short = p.fork(parents, children)
    got = saib.indexer_fork_pages(p.pools, p.t, p.l, p.r, _i32(parents), _i32(children), dev_error=p.err)
    assert p.error() == (64 if short else 0)
    p.same()
    assert got[0].tolist() == src and got[1].tolist() == dst
    for a, w in zip(p.pools, want):
        assert torch.equal(a, w)


def test_fork_of_many_rows_and_pages():
    """More forks than a block has threads, free pages far into a large pool."""
    rng = np.random.default_rng(3)
    lens = rng.integers(0, 400, 300).tolist()
    p = Pool(lens, 6000, seed=3, rows=300 + 1500, pools=1)
    parents = rng.integers(0, 300, 1500).tolist()
    children = (300 + rng.permutation(1500)).tolist()
    src, dst, want, short = p.fork(parents, children)
    assert not short
    got = saib.indexer_fork_pages(p.pools, p.t, p.l, p.r, _i32(parents), _i32(children), dev_error=p.err)
    assert p.error() == 0
    p.same()
    assert got[0].tolist() == src and got[1].tolist() == dst
    assert torch.equal(p.pools[0], want[0])


def test_fork_reports_bad_rows():
    p = Pool([100, 100], 5, seed=4, rows=4)
    _, _, want, _ = p.fork([1], [3])
    saib.indexer_fork_pages(p.pools, p.t, p.l, p.r, _i32([0, 1, -1]), _i32([4, 3, 2]), dev_error=p.err)
    assert p.error() == 32
    p.same()
    assert all(torch.equal(a, w) for a, w in zip(p.pools, want))


def test_free_and_double_free():
    p = Pool([100, 5000, 64, 0, 9], 3, seed=5, rows=7)
    p.fork([1, 0], [5, 6])
    p.up()
    p.free([1, 3, 6])
    saib.indexer_free_pages(p.t, p.l, p.r, _i32([1, 3, 6]), dev_error=p.err)
    assert p.error() == 0
    p.same()
    p.l[2] = p.lens[2] = 64
    p.r[p.table[2, 0]] = 0               # a held page whose count was lost
    p.refs[p.table[2, 0]] = 0
    p.lens[2] = 0
    saib.indexer_free_pages(p.t, p.l, p.r, _i32([2, 90]), dev_error=p.err)
    assert p.error() == 128 | 32
    p.same()


@pytest.mark.parametrize("lens,leave,spare", [
    ([100], [], 0), ([100], [], 4), ([100], [0], 4), ([300, 200, 64, 65, 500], [1, 3], 2),
    ([300, 200, 64, 65, 500], [0, 1, 2, 3, 4], 7), ([70] * 900, list(range(0, 900, 2)), 1300),
    ([4000, 90, 20000, 64, 700, 12000], [0, 2], 3000),
])
def test_compact(lens, leave, spare):
    p = Pool(lens, spare, seed=len(lens), rows=len(lens) + 2)
    p.fork([len(lens) - 1], [len(lens)]) if spare else None    # shared pages
    p.free(leave)
    p.up()
    remap, n, want = p.compact()
    got, live = saib.indexer_compact_pages(p.pools, p.t, p.l, p.r, dev_error=p.err)
    assert p.error() == 0
    p.same()
    assert int(live.item()) == n and np.array_equal(got.cpu().numpy(), remap)
    for a, w in zip(p.pools, want):
        assert torch.equal(a[:n], w[:n])


def test_compact_in_a_graph_and_on_a_stream():
    p = Pool([300, 200, 64, 65, 500], 60, seed=9)
    p.free([0, 3])
    p.up()
    keep = [x.clone() for x in (p.t, p.l, p.r)]
    remap, n, want = p.compact()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, live = saib.indexer_compact_pages(p.pools, p.t, p.l, p.r, dev_error=p.err, stream=side)
    side.synchronize()
    p.same()
    out, num = torch.empty_like(got), torch.empty_like(live)
    ws = torch.empty(1 << 16, dtype=torch.uint8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        saib.indexer_compact_pages(p.pools, p.t, p.l, p.r, remap=out, num_live=num, workspace=ws)
    for _ in range(2):
        for x, y in zip((p.t, p.l, p.r), keep):
            x.copy_(y)
        graph.replay()
        p.same()
        assert np.array_equal(out.cpu().numpy(), remap) and int(num.item()) == n
    for a, w in zip(p.pools, want):
        assert torch.equal(a[:n], w[:n])
