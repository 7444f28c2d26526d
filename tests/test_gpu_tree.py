"""Trees of drafted tokens on the GPU: masks, positions and paths; attention against the formula in 64
bits, with the tolerances of test_gpu_attend; the accepted paths in the caches; and a run of them together
with the appends."""
import math
import random

import pytest
import torch

import sparse_attention_indexer_block_gb300 as saib
from test_gpu_attend import BF, DEV, FP, PAGE, SHAPES, Batch, _lib  # noqa: F401

pytestmark = pytest.mark.gpu


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _trees(ql, seed, reach=40):
    rng = random.Random(seed)
    return [[-1 if i == 0 or rng.random() < 0.1 else rng.randrange(max(0, i - reach), i) for i in range(q)]
            for q in ql]


def _chains(parents):
    out = []
    for i, p in enumerate(parents):
        out.append([i] + (out[p] if p >= 0 else []))
    return out


def _words(bits, n):
    w = [bits >> 32 * i & 0xffffffff for i in range(n)]
    return [x - (1 << 32) if x >> 31 else x for x in w]


def _plan(trees, kl, words, width, window=0, sinks=0):
    """Masks, positions and paths, from the definition."""
    masks, positions, paths = [], [], []
    for parents, n in zip(trees, kl):
        ahead = n - len(parents)
        for chain in _chains(parents):
            depth = len(chain) - 1
            see = [j for up, j in enumerate(chain)
                   if not window or up < window or ahead + depth - up < sinks]
            masks.append(_words(sum(1 << j for j in see), words))
            positions.append(ahead + depth)
            places = [max(ahead + j, -1) for j in chain][:width]
            paths.append(places + [-1] * (width - len(places)))
    return masks, positions, paths


# ---------------------------------------------------------------------------
# masks, positions, paths
# ---------------------------------------------------------------------------


@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (2, 0), (3, 60), (100, 4)])
@pytest.mark.parametrize("ql,kl", [([1], [1]), ([8], [1000]), ([0, 33, 1, 64, 31, 0], [5, 40, 1, 64, 900, 0]),
                                   ([130, 200, 65], [130, 5000, 66]), ([3000], [3100])])
def test_plan(ql, kl, window, sinks):
    trees = _trees(ql, len(ql))
    flat = [p for t in trees for p in t]
    start = [0]
    for q in ql:
        start.append(start[-1] + q)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    width = max(len(c) for t in trees for c in _chains(t)) + 2
    masks, positions, paths = saib.indexer_plan_tree(_i32(flat), _i32(kl), _i32(start), max(ql), window=window,
                                                     sinks=sinks, max_path=width, dev_error=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    want = _plan(trees, kl, -(-max(ql) // 32), width, window, sinks)
    assert masks.tolist() == want[0] and positions.tolist() == want[1] and paths.tolist() == want[2]
    again = saib.indexer_plan_tree(_i32(flat), _i32(kl), _i32(start), max(ql), window=window, sinks=sinks)
    assert torch.equal(again[0], masks) and torch.equal(again[1], positions) and again[2] is None


def test_plan_chains_and_stars():
    n = 300
    for parents in ([-1] + list(range(n - 1)), [-1] * n):
        masks, positions, paths = saib.indexer_plan_tree(_i32(parents), _i32([n + 7]), _i32([0, n]), n, max_path=n)
        want = _plan([parents], [n + 7], 10, n)
        assert masks.tolist() == want[0] and positions.tolist() == want[1] and paths.tolist() == want[2]


def test_plan_reports_and_leaves_alone():
    err = torch.zeros(1, dtype=torch.int32, device=DEV)

    def plan(parents, lens, start, most, **kw):
        err.zero_()
        r = saib.indexer_plan_tree(_i32(parents), _i32(lens), _i32(start), most, dev_error=err, **kw)
        torch.cuda.synchronize()
        return int(err), r

    # a node that is its own parent, a later one, or none: roots
    bits, (masks, positions, _) = plan([-1, 1, 2, -5, 0], [50], [0, 5], 5)
    assert bits == 32
    assert [m[0] for m in masks.tolist()] == [1, 2, 4, 8, 17] and positions.tolist() == [45, 45, 45, 45, 46]
    # more nodes than the masks hold: those that there are bits for
    bits, (masks, positions, _) = plan([-1] + list(range(39)), [40], [0, 40], 32)
    assert bits == 8 and masks[39].tolist() == [-1] and positions[39] == 39
    # a path past its width keeps the nearest ancestors
    bits, (_, _, paths) = plan([-1, 0, 1, 2], [10], [0, 4], 4, max_path=3)
    assert bits == 8 and paths.tolist() == [[6, -1, -1], [7, 6, -1], [8, 7, 6], [9, 8, 7]]
    # fewer keys than nodes, offsets past the tokens
    bits, (_, positions, paths) = plan([-1, 0, 1], [2], [0, 3], 3, max_path=3)
    assert bits == 2 and positions.tolist() == [-1, 0, 1] and paths.tolist() == [[-1] * 3, [0, -1, -1], [1, 0, -1]]
    bits, _ = plan([-1, 0, 1], [9], [0, 7], 3)
    assert bits == 2
    # rows of no request
    masks, positions = torch.full((6, 1), 77, dtype=torch.int32, device=DEV), _i32([77] * 6)
    err.zero_()
    saib.indexer_plan_tree(_i32([5, -1, 0, -1, 5, 5]), _i32([9, 3]), _i32([1, 3, 4]), 4, masks=masks,
                           positions=positions, dev_error=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    assert masks.flatten().tolist() == [77, 1, 3, 1, 77, 77] and positions.tolist() == [77, 7, 8, 2, 77, 77]


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------


class TreeBatch(Batch):
    """A Batch whose new tokens see what `named` [request][node] = columns says (trees by default)."""

    def __init__(self, *args, named=None, words=None, tree_seed=0, **kw):
        super().__init__(*args, **kw)
        self.trees = _trees(self.ql, tree_seed)
        self.depth = [[len(c) - 1 for c in _chains(t)] for t in self.trees]
        self.named = named or [_chains(t) for t in self.trees]
        self.words = words or -(-max(1, max(self.ql)) // 32)
        self.masks = _i32([_words(sum(1 << j for j in set(cols)), self.words)
                           for per in self.named for cols in per]).view(-1, self.words)
        self.positions = _i32([n - q + d for q, n, per in zip(self.ql, self.kl, self.depth) for d in per])

    def seen(self, b, window=0, sinks=0):
        """Request b's [nodes, keys] mask, from the definition."""
        nq, n = self.ql[b], self.kl[b]
        ahead = n - nq
        see = torch.zeros((nq, n), dtype=torch.bool)
        key = torch.arange(n)
        for i in range(nq):
            see[i] = key < ahead
            if window:
                p = min(max(ahead + self.depth[b][i], ahead), n - 1)
                see[i] &= (p - key < window) | (key < sinks)
            for j in self.named[b][i]:
                if ahead + j >= 0 and j < nq and j < 32 * self.words:
                    see[i, ahead + j] = True
        return see.to(DEV)

    def reference_tree(self, window=0, sinks=0):
        d, u, scale = self.dim, torch.finfo(self.dtype).eps / 2, self.dim ** -0.5
        group = self.heads // self.kv_heads
        out = torch.zeros((self.rows, self.heads, d), dtype=torch.float64, device=DEV)
        lse = torch.full((self.rows, self.heads), -math.inf, dtype=torch.float64, device=DEV)
        tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
        for b, (nq, n) in enumerate(zip(self.ql, self.kl)):
            if n == 0 or nq == 0:
                continue
            k, v = self.keys(b)
            r0 = self.start_h[b]
            q, see = self.q[r0:r0 + nq].double(), self.seen(b, window, sinks)
            for h in range(self.heads):
                kk, vv = k[:, h // group], v[:, h // group]
                x = torch.where(see, (q[:, h] @ kk.T) * scale, -math.inf)
                size = torch.where(see, (q[:, h].abs() @ kk.abs().T) * scale, 0.0).amax(1)
                z = torch.logsumexp(x, 1)
                p = torch.exp(x - torch.where(z == -math.inf, 0.0, z)[:, None])
                o, a = p @ vv, p @ vv.abs()
                terms = see.sum(1).double()
                off = (d + 2) * 2.0 ** -24 * size + terms * 2.0 ** -23
                out[r0:r0 + nq, h], lse[r0:r0 + nq, h] = o, z
                t = u * (a + o.abs()) + 2 * off[:, None] * a
                if self.dtype == FP:
                    t = t + (terms * 2.0 ** -25)[:, None] * vv.abs().amax()
                tol[r0:r0 + nq, h] = t
                ltol[r0:r0 + nq, h] = off + 2.0 ** -22 * (1 + z.abs().clamp(max=1e30))
        return out, lse, tol, ltol

    def attend_tree(self, bits=0, **kw):
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        kw.setdefault("max_query_len", max(self.ql))
        r = saib.indexer_attend_tree(self.q, self.k, self.v, self.table, self.lens, self.start, self.masks,
                                     positions=self.positions, dev_error=err, **kw)
        torch.cuda.synchronize()
        assert int(err) == bits, f"device error word {int(err)}"
        return r


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_tree(shape, dtype, dim):
    ql, kl, heads, kv = SHAPES[shape]
    b = TreeBatch(ql, kl, heads, kv, dim, dtype, seed=shape, tree_seed=shape)
    b.check(b.attend_tree(), b.reference_tree())


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (63, 0), (64, 4), (65, 64), (100, 130), (300, 70), (5000, 4),
                                          (2 ** 31 - 1, 0)])
@pytest.mark.parametrize("shape,dtype,dim", [(1, BF, 128), (3, FP, 64), (4, BF, 64), (5, FP, 128), (6, FP, 128),
                                             (7, BF, 128), (9, FP, 64), (11, BF, 128)])
def test_tree_window_and_sinks(shape, dtype, dim, window, sinks):
    ql, kl, heads, kv = SHAPES[shape]
    b = TreeBatch(ql, kl, heads, kv, dim, dtype, seed=100 + shape, tree_seed=shape)
    b.check(b.attend_tree(window=window, sinks=sinks), b.reference_tree(window, sinks))


@pytest.mark.parametrize("ql,kl", [([7, 3], [7, 300]), ([40, 90, 1], [40, 600, 1])])
@pytest.mark.parametrize("dim,dtype", [(64, FP), (128, BF)])
def test_tree_masks_of_any_kind(ql, kl, dim, dtype):
    """Rows that see nothing, nodes that do not see themselves, later nodes; bits past the nodes."""
    rng = random.Random(4)
    named = [[[j for j in range(q + 20) if rng.random() < 0.3] if i % 3 else [] for i in range(q)] for q in ql]
    b = TreeBatch(ql, kl, 8, 2, dim, dtype, seed=5, named=named, words=-(-(max(ql) + 20) // 32))
    b.check(b.attend_tree(), b.reference_tree())
    b.check(b.attend_tree(window=20, sinks=3), b.reference_tree(20, 3))


def test_tree_with_fewer_words_than_nodes():
    b = TreeBatch([50, 10], [90, 200], 8, 2, 64, BF, seed=6, words=1)
    b.check(b.attend_tree(), b.reference_tree())


@pytest.mark.parametrize("hint", [0, 1, 100000])
def test_tree_hint_and_strides(hint):
    b = TreeBatch([20, 3, 33], [300, 60, 700], 16, 2, 128, BF, seed=7, layout="joint", q_pad=8)
    wide = torch.full((b.rows, b.words + 3), -1, dtype=torch.int32, device=DEV)
    wide[:, :b.words] = b.masks
    b.masks = wide[:, :b.words]
    b.check(b.attend_tree(max_query_len=hint), b.reference_tree())


def test_tree_of_a_chain_is_causal():
    """Both forms against the causal formula."""
    b = TreeBatch([4, 30], [1000, 77], 8, 2, 128, BF, seed=8, named=[[list(range(i + 1)) for i in range(q)] for q in (4, 30)])
    want = b.reference()
    b.check(b.attend_tree(), want)
    b.check(b.attend(), want)


@pytest.mark.parametrize("ql,kl", [([60, 8], [30000, 9000]), ([5] * 3, [20000, 100, 40000]), ([700], [2000])])
def test_tree_long_rows_split_over_ctas(ql, kl):
    b = TreeBatch(ql, kl, 8, 1, 128, BF, seed=9, tree_seed=3)
    b.check(b.attend_tree(), b.reference_tree())
    b.check(b.attend_tree(window=15000, sinks=100), b.reference_tree(15000, 100))


def test_tree_many_requests():
    rng = random.Random(2)
    ql = [rng.randrange(0, 9) for _ in range(700)]
    kl = [q + rng.randrange(0, 130) for q in ql]
    b = TreeBatch(ql, kl, 4, 2, 64, FP, seed=10)
    b.check(b.attend_tree(), b.reference_tree())


@pytest.mark.parametrize("ql,kl", [([3, 40], [130, 200]), ([60, 140], [260, 400])])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_tree_nonfinite_values_reach_only_rows_that_see_them(ql, kl, dtype):
    b = TreeBatch(ql, kl, 8, 2, 128, dtype, seed=11)
    clean, _ = b.attend_tree(window=70, sinks=2)
    see = b.seen(0, 70, 2)
    for key, value in ((kl[0] - 1, float("nan")), (kl[0] - ql[0] + 1, float("inf")), (kl[0] - ql[0] - 1, float("nan")),
                       (kl[0] - ql[0] - 71, float("-inf"))):
        page, slot = int(b.table[0, key // PAGE]), key % PAGE
        for cache in (b.v, b.k):
            keep = cache[page, slot].clone()
            cache[page, slot] = value
            out, _ = b.attend_tree(window=70, sinks=2)
            cache[page, slot] = keep
            rows = torch.ones(b.rows, dtype=torch.bool, device=DEV)
            rows[:ql[0]] = ~see[:, key]
            assert torch.equal(out[rows], clean[rows])
            if cache is b.v:
                assert not torch.isfinite(out[~rows]).any()


def test_tree_rows_outside_every_request_and_wild_positions():
    b = TreeBatch([2, 30], [70, 80], 4, 2, 64, BF, seed=12)
    # positions are clamped to the new tokens' places
    b.positions[0], b.positions[3] = -(1 << 31), (1 << 31) - 1
    b.depth[0][0], b.depth[1][1] = -70, 1000
    want = b.reference_tree(20, 1)
    pad = 3
    q = torch.zeros((b.rows + 2 * pad, 4, 64), dtype=BF, device=DEV)
    masks = torch.full((b.rows + 2 * pad, b.words), -1, dtype=torch.int32, device=DEV)
    positions = torch.full((b.rows + 2 * pad,), 1 << 30, dtype=torch.int32, device=DEV)
    q[pad:-pad], masks[pad:-pad], positions[pad:-pad] = b.q, b.masks, b.positions
    out, lse = torch.full_like(q, 7.0), torch.full((q.shape[0], 4), 7.0, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    saib.indexer_attend_tree(q, b.k, b.v, b.table, b.lens, b.start + pad, masks, 30, positions=positions, window=20,
                             sinks=1, out=out, lse=lse, dev_error=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    for t in (out, lse):
        assert (t[:pad] == 7).all() and (t[-pad:] == 7).all()
    b.check((out[pad:-pad], lse[pad:-pad]), want)


@pytest.mark.parametrize("ql,kl,window", [([3], [300], 0), ([60], [300], 0), ([3], [900], 200), ([60], [900], 200)])
def test_tree_bad_pages(ql, kl, window):
    """A needed page outside the cache is reported and counts as zeros; one that a window hides is not."""
    b = TreeBatch(ql, kl, 4, 2, 128, BF, seed=13)
    page = int(b.table[0, 3 if not window else (kl[0] - ql[0]) // PAGE])
    column = (b.table[0] == page).nonzero().item()
    b.k[page], b.v[page] = 0.0, 0.0
    want = b.reference_tree(window, 1)
    b.table[0, column] = b.k.shape[0] + 5
    if window:
        b.table[0, 1:(kl[0] - ql[0] - window + 1) // PAGE] = -9
    got = b.attend_tree(bits=1, window=window, sinks=1)
    b.table[0, column] = page
    if window:
        # (the reference reads the keys that no row sees, too)
        b.table[0, 1:(kl[0] - ql[0] - window + 1) // PAGE] = page
        b.attend_tree(window=window, sinks=1)
    b.check(got, want)


def test_tree_bad_lengths():
    b = TreeBatch([4, 4], [100, 100], 4, 2, 64, BF, seed=14)
    lens = b.lens
    for bad in (b.width * PAGE + 1, -3):
        b.lens = _i32([100, bad])
        b.attend_tree(bits=2 if bad < 0 else 3)
    b.lens = lens
    b.check(b.attend_tree(), b.reference_tree())


def test_tree_repeats_bit_for_bit_in_a_graph_and_on_another_stream():
    b = TreeBatch([30] * 6, [3000] * 6, 16, 2, 128, BF, seed=15)
    ws = saib.attend_workspace(b.rows, 6, 16, 2, 128)
    out, lse = torch.empty_like(b.q), torch.empty((b.rows, 16), device=DEV)
    first = b.attend_tree()

    def call(stream=None):
        saib.indexer_attend_tree(b.q, b.k, b.v, b.table, b.lens, b.start, b.masks, 30, out=out, lse=lse, workspace=ws,
                                 stream=stream)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(side)
    side.synchronize()
    assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    b.q.normal_(generator=b.gen)
    graph.replay()
    torch.cuda.synchronize()
    want = b.attend_tree()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1]) and not torch.equal(out, first[0])


# ---------------------------------------------------------------------------
# accepted paths
# ---------------------------------------------------------------------------


class Caches:
    def __init__(self, ql, kl, kv=2, dim=64, seed=0, layout="pages", spare=3):
        g = torch.Generator(device=DEV).manual_seed(seed)
        pages = [-(-n // PAGE) for n in kl]
        total = sum(pages) + spare
        order = torch.randperm(total, generator=g, device=DEV).tolist()
        self.ql, self.kl = ql, kl
        self.table = torch.full((len(kl), max(1, max(pages)) + 1), -1, dtype=torch.int32, device=DEV)
        self.refs = torch.zeros(total, dtype=torch.int32, device=DEV)
        at = 0
        for b, n in enumerate(pages):
            ids = order[at:at + n]
            at += n
            if n:
                self.table[b, :n] = _i32(ids)
                self.refs[torch.tensor(ids, device=DEV)] = 1
        shape = (total, PAGE, kv, dim)
        self.k = torch.randn(shape, generator=g, device=DEV).to(BF)
        self.v = torch.randn(shape, generator=g, device=DEV).to(BF)
        if layout == "heads":
            self.k, self.v = (c.transpose(1, 2).contiguous().transpose(1, 2) for c in (self.k, self.v))
        elif layout == "joint":
            both = torch.stack([self.k, self.v], 1)
            self.k, self.v = both[:, 0], both[:, 1]
        self.index = torch.randint(0, 256, (total, 8448), generator=g, device=DEV, dtype=torch.uint8)
        self.mx = torch.randint(0, 256, (total, 4352), generator=g, device=DEV, dtype=torch.uint8)
        self.lens = _i32(kl)
        start = [0]
        for q in ql:
            start.append(start[-1] + q)
        self.start = _i32(start)
        self.err = torch.zeros(1, dtype=torch.int32, device=DEV)

    @property
    def pools(self):
        return [self.index, self.k, self.v, self.mx]

    def tokens(self):
        """Every cache as [pages, 64, bytes or values]."""
        n = self.index.shape[0]
        return [self.k.reshape(n, PAGE, -1).clone(), self.v.reshape(n, PAGE, -1).clone(),
                self.index[:, :8192].reshape(n, PAGE, 128).clone(), self.index[:, 8192:].reshape(n, PAGE, 4).clone(),
                self.mx.reshape(n, PAGE, 68).clone()]

    def expected(self, paths, report=None):
        caches, refs, lens = self.tokens(), self.refs.tolist(), list(self.kl)
        for b, path in enumerate(paths):
            ahead = self.kl[b] - self.ql[b]
            row = self.table[b].tolist()
            for i, a in enumerate(path):
                (sp, st), (dp, dt) = (divmod(ahead + x, PAGE) for x in (a, i))
                for c in caches:
                    c[row[dp], dt] = c[row[sp], st].clone()
            lens[b] = ahead + len(path)
            for col in range(-(-lens[b] // PAGE), -(-self.kl[b] // PAGE)):
                refs[row[col]] -= 1
        return caches, refs, lens

    def commit(self, paths, bits=0, refs=True, most=None, **kw):
        most = most or max(1, max(len(p) for p in paths))
        accepted = _i32([list(p) + [-1] * (most - len(p)) for p in paths])
        saib.indexer_commit_tree(self.pools, self.table, self.lens, self.start, accepted,
                                 ref_counts=self.refs if refs else None, dev_error=self.err, **kw)
        torch.cuda.synchronize()
        assert int(self.err) == bits, f"device error word {int(self.err)}"

    def check(self, want):
        caches, refs, lens = want
        for got, c in zip(self.tokens(), caches):
            assert torch.equal(got, c)
        assert self.refs.tolist() == refs and self.lens.tolist() == lens


def _paths(ql, seed, most=1 << 30):
    rng = random.Random(seed)
    out = []
    for q in ql:
        n = rng.randint(0, min(q, most))
        out.append(sorted(rng.sample(range(q), n)))
    return out


@pytest.mark.parametrize("layout", ["pages", "heads", "joint"])
@pytest.mark.parametrize("ql,kl", [([8], [1000]), ([1], [1]), ([16, 0, 64, 5, 33], [80, 7, 64, 130, 128]),
                                   ([300, 200], [300, 777]), ([65] * 40, [200 + 7 * i for i in range(40)])])
def test_commit(ql, kl, layout):
    c = Caches(ql, kl, seed=len(ql), layout=layout)
    paths = _paths(ql, 3)
    want = c.expected(paths)
    c.commit(paths)
    c.check(want)


def test_commit_all_none_and_wide_tokens():
    c = Caches([10, 70, 64], [100, 70, 128], kv=8, dim=128, seed=5)
    paths = [list(range(10)), [], [63]]
    want = c.expected(paths)
    c.commit(paths, most=80)
    c.check(want)


def test_commit_without_pools_or_counts():
    c = Caches([10, 70], [100, 133], seed=6)
    paths = [[0, 4], [3]]
    caches, refs, lens = c.expected(paths)
    before = c.refs.clone()
    c.commit(paths, refs=False)
    assert torch.equal(c.refs, before)
    for got, x in zip(c.tokens(), caches):
        assert torch.equal(got, x)
    assert c.lens.tolist() == lens
    c = Caches([10, 70], [100, 133], seed=6)
    old = c.tokens()
    saib.indexer_commit_tree([], c.table, c.lens, c.start, _i32([[0, 4], [3, -1]]), ref_counts=c.refs)
    torch.cuda.synchronize()
    assert c.lens.tolist() == lens and c.refs.tolist() == refs
    assert all(torch.equal(a, b) for a, b in zip(old, c.tokens()))


def test_commit_reports():
    # a list that does not ascend, or names a node that is not there, ends
    c = Caches([10, 10, 10], [100, 100, 100], seed=7)
    want = c.expected([[0, 5], [2], []])
    c.commit([[0, 5, 5, 7], [2, 10], [3, 1]][:2] + [[-1]], bits=32)
    c.check(want)
    # a page outside the pools: its moves are left out
    c = Caches([40, 40], [100, 100], seed=8)
    want = c.expected([[39], [2]])
    row = c.table[1].clone()
    c.table[1, 0] = 1 << 20
    caches, refs, lens = want
    old = c.tokens()
    for new, o in zip(caches, old):
        new[int(row[0]), 60] = o[int(row[0]), 60]
    c.commit([[39], [2]], bits=1)
    c.check((caches, refs, lens))
    # lengths outside the table, or fewer keys than nodes: left as they are
    c = Caches([10, 10, 10], [100, 100, 100], seed=9)
    caches, refs, lens = c.expected([[3], list(range(10)), list(range(10))])
    lens[1], lens[2] = c.table.shape[1] * PAGE + 1, 9
    c.lens[1], c.lens[2] = lens[1], lens[2]
    c.commit([[3], [4], [4]], bits=2)
    c.check((caches, refs, lens))
    # a page that nobody holds
    c = Caches([70], [130], seed=10)
    caches, refs, lens = c.expected([[1]])
    c.refs[c.table[0, 1].long()] = 0
    refs = c.refs.tolist()
    refs[int(c.table[0, 2])] -= 1
    c.commit([[1]], bits=128)
    c.check((caches, refs, lens))


def test_commit_in_a_graph():
    c = Caches([16, 16], [70, 200], seed=11)
    paths = [[0, 3, 9], [15]]
    want = c.expected(paths)
    accepted = _i32([[0, 3, 9], [15, -1, -1]])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        saib.indexer_commit_tree(c.pools, c.table, c.lens, c.start, accepted, ref_counts=c.refs, dev_error=c.err)
    assert c.lens.tolist() == [70, 200]
    graph.replay()
    torch.cuda.synchronize()
    c.check(want)


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------


def test_speculative_steps():
    """Steps of drafting, tree attention and committing leave in the caches, and give, what the accepted
    tokens alone, appended one by one, leave and give."""
    rng = random.Random(1)
    heads, kv, dim, reqs, width = 8, 2, 128, 3, 12
    g = torch.Generator(device=DEV).manual_seed(2)

    def randn(*shape):
        return torch.randn(shape, generator=g, device=DEV).to(BF)

    angle = torch.rand((800, 32), generator=g, device=DEV, dtype=torch.float64) * 6.2832
    rotary = torch.cat([angle.cos(), angle.sin()], 1).float()
    pages = reqs * width
    k, v = torch.zeros((pages, PAGE, kv, dim), dtype=BF, device=DEV), torch.zeros((pages, PAGE, kv, dim), dtype=BF, device=DEV)
    index = torch.zeros((pages, 4352), dtype=torch.uint8, device=DEV)
    table = torch.randperm(pages, generator=g, device=DEV).view(reqs, width).to(torch.int32)
    lens = _i32([0] * reqs)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    history = [[] for _ in range(reqs)]   # per request: (q, k, v, index key) of every kept token, unrotated
    for step in range(6):
        ql = [rng.randint(1, 60) for _ in range(reqs)]
        trees = _trees(ql, 50 + step, reach=8)
        start = [0]
        for q in ql:
            start.append(start[-1] + q)
        n = start[-1]
        begin = lens.tolist()
        x = dict(q=randn(n, heads, dim), k=randn(n, kv, dim), v=randn(n, kv, dim), i=randn(n, 128))
        lens = lens + _i32(ql)
        masks, positions, paths = saib.indexer_plan_tree(_i32([p for t in trees for p in t]), lens, _i32(start), 60,
                                                         max_path=64, dev_error=err)
        slots = torch.tensor([int(table[b, (begin[b] + i) // PAGE]) * PAGE + (begin[b] + i) % PAGE
                              for b, q in enumerate(ql) for i in range(q)], device=DEV)
        q = saib.indexer_append_kv(x["k"], x["v"], k, v, slots, q=x["q"], positions=positions, rotary=rotary, dev_error=err)
        saib.indexer_insert_keys_mxfp4(x["i"], slots, index, dev_error=err)
        out, lse = saib.indexer_attend_tree(q, k, v, table, lens, _i32(start), masks, 60, dev_error=err)
        # a sparse layer whose selection is every key before the tree: the same rows
        most = max(max(begin), 1)
        before = torch.arange(most, dtype=torch.int32, device=DEV).expand(n, -1)
        ahead = _i32([begin[b] for b, m in enumerate(ql) for _ in range(m)])[:, None]
        lists = torch.cat([torch.where(before < ahead, before, -1), paths], 1).to(torch.int32).contiguous()
        picked, picked_lse = saib.indexer_attend_selected(q, k, v, table, lists, _i32(start), dev_error=err)
        torch.cuda.synchronize()
        # two kernels' sums of the same terms: each within u (|p| |v| + |out|) of the exact one, where
        # |v| <= 5.5 for these values and a score is below 40
        assert (picked.double() - out.double()).abs().max() <= 2 * 2.0 ** -8 * 2 * 5.5
        assert (picked_lse - lse).abs().max() <= 1e-3
        accepted = []
        for b, tree in enumerate(trees):
            chain = _chains(tree)[rng.randrange(len(tree))][::-1]
            accepted.append(chain)
            # the last accepted node as a causal row over the kept tokens and its path
            kept = history[b] + [tuple(x[f][start[b] + j] for f in "qkvi") for j in chain]
            pos = torch.arange(len(kept), dtype=torch.int32, device=DEV)
            kk, vv = torch.stack([t[1] for t in kept]), torch.stack([t[2] for t in kept])
            p = -(-len(kept) // PAGE)
            k1 = torch.zeros((p, PAGE, kv, dim), dtype=BF, device=DEV)
            v1 = torch.zeros_like(k1)
            qq = saib.indexer_append_kv(kk, vv, k1, v1, pos.long(), q=torch.stack([t[0] for t in kept]), positions=pos,
                                        rotary=rotary)
            one, one_lse = saib.indexer_attend_paged(qq[-1:], k1, v1, torch.arange(p, dtype=torch.int32, device=DEV)[None],
                                                     _i32([len(kept)]), _i32([0, 1]), 1)
            row = start[b] + chain[-1]
            assert (one[0].double() - out[row].double()).abs().max() <= 2 * 2.0 ** -8 * 2 * 5.5
            assert (one_lse[0] - lse[row]).abs().max() <= 1e-3
            history[b] = kept
        most = max(len(a) for a in accepted)
        saib.indexer_commit_tree([k, v, index], table, lens, _i32(start), _i32([a + [-1] * (most - len(a)) for a in accepted]),
                                 dev_error=err)
        torch.cuda.synchronize()
        assert int(err) == 0
        assert lens.tolist() == [len(h) for h in history]
        for b, h in enumerate(history):
            at = torch.arange(len(h), device=DEV)
            pg = table[b, at // PAGE].long()
            p = -(-len(h) // PAGE)
            k1 = torch.zeros((p, PAGE, kv, dim), dtype=BF, device=DEV)
            v1, i1 = torch.zeros_like(k1), torch.zeros((p, 4352), dtype=torch.uint8, device=DEV)
            saib.indexer_append_kv(torch.stack([t[1] for t in h]), torch.stack([t[2] for t in h]), k1, v1, at,
                                   positions=at.to(torch.int32), rotary=rotary)
            saib.indexer_insert_keys_mxfp4(torch.stack([t[3] for t in h]), at, i1)
            assert torch.equal(k[pg, at % PAGE], k1.view(-1, kv, dim)[:len(h)])
            assert torch.equal(v[pg, at % PAGE], v1.view(-1, kv, dim)[:len(h)])
            assert torch.equal(index.view(pages, PAGE, 68)[pg, at % PAGE], i1.view(-1, 68)[:len(h)])


def test_step_in_a_graph_follows_its_inputs():
    """Plan, append, attention and commit captured once and replayed on other trees, tokens and tables."""
    heads, kv, dim, reqs, q = 8, 2, 64, 3, 24
    g = torch.Generator(device=DEV).manual_seed(3)
    pages = 30
    k = torch.randn((pages, PAGE, kv, dim), generator=g, device=DEV).to(FP)
    v = torch.randn((pages, PAGE, kv, dim), generator=g, device=DEV).to(FP)
    angle = torch.rand((2000, dim // 2), generator=g, device=DEV) * 6.2832
    rotary = torch.cat([angle.cos(), angle.sin()], 1)
    table, lens = torch.zeros((reqs, 10), dtype=torch.int32, device=DEV), _i32([0] * reqs)
    start, refs, err = _i32([0, q, 2 * q, 3 * q]), _i32([0] * pages), _i32([0])
    parents, accepted = _i32([0] * (reqs * q)), torch.full((reqs, 6), -1, dtype=torch.int32, device=DEV)
    slots = torch.zeros(reqs * q, dtype=torch.int64, device=DEV)
    x = [torch.zeros((reqs * q, n, dim), dtype=FP, device=DEV) for n in (heads, kv, kv)]

    def step():
        masks, positions, _ = saib.indexer_plan_tree(parents, lens, start, q, window=70, sinks=2, dev_error=err)
        turned = saib.indexer_append_kv(x[1], x[2], k, v, slots, q=x[0], positions=positions, rotary=rotary,
                                        interleaved=True, dev_error=err)
        out, lse = saib.indexer_attend_tree(turned, k, v, table, lens, start, masks, q, positions=positions, window=70,
                                            sinks=2, dev_error=err)
        saib.indexer_commit_tree([k, v], table, lens, start, accepted, ref_counts=refs, dev_error=err)
        return out, lse

    def fill(seed):
        rng = random.Random(seed)
        kl = [q + rng.randrange(0, 400) for _ in range(reqs)]
        trees = _trees([q] * reqs, seed)
        parents.copy_(_i32([p for t in trees for p in t]))
        table.copy_(torch.randperm(pages, generator=g, device=DEV).view(reqs, 10))
        refs.fill_(1)
        lens.copy_(_i32(kl))
        slots.copy_(torch.cat([table[b].long()[(n - q + torch.arange(q, device=DEV)) // PAGE] * PAGE
                               + (n - q + torch.arange(q, device=DEV)) % PAGE for b, n in enumerate(kl)]))
        for t in x:
            t.copy_(torch.randn(t.shape, generator=g, device=DEV))
        accepted.fill_(-1)
        for b, t in enumerate(trees):
            chain = _chains(t)[-1][::-1][:6]
            accepted[b, :len(chain)] = _i32(chain)

    state = [k, v, lens, refs]
    fill(1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    fill(2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in (3, 4):
        fill(seed)
        before = [t.clone() for t in state]
        graph.replay()
        torch.cuda.synchronize()
        after = [t.clone() for t in state]
        for t, old in zip(state, before):
            t.copy_(old)
        want = step()
        torch.cuda.synchronize()
        assert int(err) == 0
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        for t, a in zip(state, after):
            assert torch.equal(t, a)


def test_streams_as_objects_and_handles():
    c = Caches([8], [100], seed=20)
    want = c.expected([[0, 7]])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    masks = [saib.indexer_plan_tree(_i32([-1] * 8), _i32([100]), c.start, 8, stream=s)[0]
             for s in (None, side, side.cuda_stream, torch.cuda.current_stream().cuda_stream)]
    c.commit([[0, 7]], stream=side.cuda_stream)
    torch.cuda.synchronize()
    assert all(torch.equal(m, masks[0]) for m in masks)
    c.check(want)


def test_tree_of_a_batch_whose_hint_is_smaller_than_its_trees():
    """Units past those the hint asks for, in clusters and without, of a long and a short table."""
    for width in (0, 3000):
        b = TreeBatch([2, 50, 9], [400, 300, 20], 8, 2, 128, BF, seed=21)
        if width:
            wide = torch.full((3, width), -1, dtype=torch.int32, device=DEV)
            wide[:, :b.width] = b.table
            b.table = wide
        for hint in (1, 2, 9, 50):
            b.check(b.attend_tree(max_query_len=hint), b.reference_tree())


def test_trees_on_two_streams_at_once():
    """Two batches side by side, each with its own outputs and what the call allocates: as one after the other."""
    batches = [TreeBatch([20, 40, 9], [6000, 300, 9000], 16, 2, 128, BF, seed=30),
               TreeBatch([8], [3000], 16, 4, 64, FP, seed=31), TreeBatch([60] * 4, [2000] * 4, 12, 4, 64, FP, seed=32)]
    want = [b.attend_tree() for b in batches]
    streams = [torch.cuda.Stream() for _ in batches]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[] for _ in batches]
    for _ in range(20):
        for b, s, g in zip(batches, streams, got):
            g.append(saib.indexer_attend_tree(b.q, b.k, b.v, b.table, b.lens, b.start, b.masks, max(b.ql), stream=s))
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(o, w[0]) and torch.equal(l, w[1]) for o, l in g)


def test_tree_without_lse_through_the_c_entry():
    import ctypes as C

    from sparse_attention_indexer_block_gb300 import binding
    for ql, kl in (([8], [500]), ([50, 3], [20000, 90])):
        b = TreeBatch(ql, kl, 8, 2, 128, BF, seed=33)
        want = b.attend_tree()
        out, ws = torch.empty_like(b.q), saib.attend_workspace(b.rows, len(ql), 8, 2, 128)
        a = binding.Attend(q=b.q.data_ptr(), k=b.k.data_ptr(), v=b.v.data_ptr(), block_table=b.table.data_ptr(),
                           seq_lens=b.lens.data_ptr(), query_start_loc=b.start.data_ptr(), out=out.data_ptr(),
                           workspace=ws.data_ptr(), workspace_bytes=ws.numel(), q_stride_token=b.q.stride(0),
                           q_stride_head=b.q.stride(1), num_pages=b.k.shape[0], bt_stride=b.table.stride(0),
                           bt_width=b.table.shape[1], num_reqs=len(ql), num_tokens=b.rows, num_heads=8, num_kv_heads=2,
                           head_dim=128, dtype=0, max_query_len=max(ql), scale=128 ** -0.5,
                           **{f"{c}_stride_{d}": t.stride(i) for c, t in (("k", b.k), ("v", b.v))
                              for i, d in enumerate(("page", "token", "head"))})
        st = saib.load().indexer_attend_tree(C.byref(a), b.masks.data_ptr(), b.words, b.words, None,
                                             torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        assert st == 0 and torch.equal(out, want[0])


@pytest.mark.parametrize("kl,ql,heads,kv,dim", [([4500], [8], 32, 8, 128), ([9000, 5000], [4, 8], 8, 2, 128),
                                                ([12000], [16], 8, 1, 64), ([7000], [1], 16, 4, 64)])
def test_tree_in_clusters_of_sixteen(kl, ql, heads, kv, dim):
    b = TreeBatch(ql, kl, heads, kv, dim, BF, seed=34)
    b.check(b.attend_tree(), b.reference_tree())
    b.check(b.attend_tree(window=6000, sinks=5), b.reference_tree(6000, 5))
